// embed.h -- arguments of the embedding lookup and its gradient (host and
// device side).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace twell {

constexpr int EMB_WINDOW = 32, EMB_WINDOW_SHORT = 8;  // sorted tokens that one sum takes at most
constexpr int EMB_ONE = 1024, EMB_ONE_WGS = 4096;  // tokens, and slices of them, up to which one launch does all,
constexpr int64_t EMB_ONE_TABLE = (int64_t)1 << 23;  // with a table to be overwritten of up to so many elements
constexpr int EMB_FILL_ROWS = 1024; // rows that a workgroup of that launch writes zeros to at most
constexpr int EMB_FEW = 8192;       // tokens up to which ranks are counted in one launch
constexpr int EMB_DIGIT_BITS = 9;   // of a sorting pass
constexpr int EMB_MOST_BLOCKS = 256;  // workgroups of a sorting pass

struct EmbArgs {
    int T, V, d;
    int id64, bf16_rows, bf16_table;  // types of ids, of out / dout, of table / dtable
    int accumulate;
    float scale;
    const void *ids;
    const void *in;   // forward: table; backward: dout
    void *out;        // forward: out; backward: dtable
    // backward: the workspace
    int32_t *key, *perm;    // [T] the tokens' keys in ascending order (V: no id), and their rows
    int32_t *key2, *perm2;  // [T] the other side of a sorting pass
    int32_t *counts;        // [blocks][2^EMB_DIGIT_BITS]
    float *part;            // [windows][2][emb_pitch(d)] sums of runs that windows cut
};

// Tokens up to which the short windows are taken: where they are too few, or their
// rows too narrow, for the others to give every CU a few waves.
inline int emb_short(int d) { return d <= 256 ? 8192 : 2048; }

// The most windows of any call with up to T tokens.
inline int64_t emb_most_windows(int64_t T, int d)
{
    const int64_t few = T < emb_short(d) ? T : emb_short(d);
    const int64_t shorter = (few + EMB_WINDOW_SHORT - 1) / EMB_WINDOW_SHORT, n = (T + EMB_WINDOW - 1) / EMB_WINDOW;
    return n > shorter ? n : shorter;
}
__host__ __device__ inline int64_t emb_pitch(int d) { return ((int64_t)d + 3) & ~(int64_t)3; }

// Rows of a table of width d that such a workgroup takes: about 16384 elements.
__host__ __device__ inline int64_t emb_fill_rows(int d)
{
    const int64_t n = 16384 / d;
    return n < 1 ? 1 : n < EMB_FILL_ROWS ? n : EMB_FILL_ROWS;
}

// Places the workspace's parts at `base`; returns its bytes (never less for more tokens).
size_t emb_layout(EmbArgs &a, void *base);

hipError_t launch_embed(const EmbArgs &a, hipStream_t s);
hipError_t launch_embed_backward(const EmbArgs &a, hipStream_t s);

}  // namespace twell
