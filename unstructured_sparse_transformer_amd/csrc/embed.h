// embed.h -- arguments of the embedding lookup and its gradient (host and
// device side).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace twell {

constexpr int EMB_WINDOW = 32, EMB_WINDOW_SHORT = 8;  // sorted tokens that one sum takes at most
// Tokens, and slices of 256 columns of them, up to which one launch does all, with a
// table to be overwritten of up to so many elements.  (us in one launch and by sorting,
// tables of 1024 rows: 1024 tokens of 256 6.8 and 12, of 1024 9.9 and 12.3, of 2048, 8192
// slices, 15.2 and 12.3; 512 of 2048 9.9 and 12.2, of 4096, 8192 slices, 15.0 and 12.1.
// Larger tables, 2^25 elements: 256 tokens 20 and 27, 1024 26 and 29; 2^23 and 1024
// tokens 15.0 and 12.9.)
constexpr int EMB_ONE = 1024, EMB_ONE_WGS = 4096;
constexpr int64_t EMB_ONE_TABLE = (int64_t)1 << 23;
constexpr int EMB_FILL_ROWS = 1024; // rows that a workgroup of that launch writes zeros to at most
// Tokens up to which ranks are counted in one launch, whose LDS holds their keys (the
// whole call, added to a table, and with sorting passes instead: 2048 x 64 12.5 and 20.6
// us, 4096 x 64 15.1 and 21.8, 8192 x 64 21.4 and 22.4, 4096 x 2048 23.0 and 28.5, 8192 x
// 2048 39.0 and 39.1).
constexpr int EMB_FEW = 8192;
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
// rows too narrow, for the others to give every CU a few waves (short and long, added to
// a table: 2048 x 2048 15.2 and 17.5 us, 4096 x 2048 29.2 and 22.9, 4096 x 1024 19.0 and
// 20.0, 4096 x 512 16.1 and 19.6, 8192 x 256 22.4 and 25.3, 16384 x 256 29.5 and 28.9).
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
