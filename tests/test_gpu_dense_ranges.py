"""The gated product and the block norms where one choice of tile, split, layout
or row group hands over to the next, against the formulas in 64 bits within the
bounds of dense_ref.py."""

import pytest

import test_gpu_block_norm as norm
import test_gpu_glu as glu
from helpers import say

pytestmark = pytest.mark.gpu

# rows that end inside a tile and d, F that are odd multiples of 64 wherever the choice allows; together: dx and dW in
# one launch, apart: in two, split: K in parts
FORWARD = [
    ("float32", 386, 320, 7104), ("float32", 2000, 512, 4096),  # 128 x 128
    ("bfloat16", 557, 320, 5696),                               # 256 x 256
    ("bfloat16", 267, 320, 5568), ("bfloat16", 264, 3392, 1472),  # 256 x 128, and split
    ("bfloat16", 260, 1984, 704),                               # 128 x 128, split
    ("bfloat16", 257, 448, 192), ("bfloat16", 257, 1472, 192),  # 128 x 64, and split
]
BACKWARD = [
    # fp32: 128 x 128 for dx and dW together, with dW first (dx split), for dx alone, for dW alone and split
    ("float32", 579, 2496, 320), ("float32", 641, 3008, 576), ("float32", 1106, 3008, 320), ("float32", 407, 3904, 448),
    ("float32", 1500, 2048, 2048), ("float32", 2000, 512, 4096), ("float32", 2037, 1728, 320),
    ("float32", 1601, 2240, 3520), ("float32", 7007, 2240, 832),
    # fp32: 64 x 64 apart, dW split
    ("float32", 467, 2240, 448), ("float32", 1390, 1472, 448),
    # bf16 together: 256 x 256 with dx first and dW first, 256 x 128 likewise, 128 x 128 split
    ("bfloat16", 259, 1472, 1728), ("bfloat16", 2701, 1856, 192), ("bfloat16", 4368, 1216, 192),
    ("bfloat16", 257, 448, 2624), ("bfloat16", 2049, 1088, 192), ("bfloat16", 1025, 320, 192),
    # bf16 apart: each tile for dx and for dW, whole and split
    ("bfloat16", 267, 960, 4160), ("bfloat16", 281, 320, 7872), ("bfloat16", 1442, 3904, 320), ("bfloat16", 4448, 1856, 192),
    ("bfloat16", 15915, 320, 192), ("bfloat16", 669, 3776, 704), ("bfloat16", 334, 1472, 3520), ("bfloat16", 3539, 3264, 192),
    ("bfloat16", 4173, 448, 8128), ("bfloat16", 15577, 448, 2112),
]


def _id(c):
    return "%s_T%d_d%d_F%d" % c


@pytest.mark.parametrize("case", FORWARD, ids=_id)
def test_gated_product(gpu_lib, case):
    dtype, *shape = case
    say(f"case glu forward {case}")
    glu._check_forward(gpu_lib, *shape, dtype, "gelu")


@pytest.mark.parametrize("case", BACKWARD, ids=_id)
def test_gated_product_backward(gpu_lib, case):
    dtype, *shape = case
    say(f"case glu backward {case}")
    glu._check_backward(gpu_lib, *shape, dtype, "silu")


# several rows a group in the backward pass, and (but for the first) more rows than the forward pass has workgroups for
ROWS = [(1300, 1001), (4500, 1024), (4500, 1001), (5000, 2048), (2300, 2056), (1500, 4096), (1100, 8192), (1100, 8191)]


@pytest.mark.parametrize("T,d", ROWS)
@pytest.mark.parametrize("kind,bias", [("rms", False), ("rms", True), ("layer", False), ("layer", True)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_wide_rows(gpu_lib, T, d, kind, bias, dtype):
    say(f"case block norm wide {T} x {d} {kind} bias={bias} {dtype}")
    norm._check(gpu_lib, norm._case(T, d, kind=kind, bias=bias, span=7, r=dtype, y=dtype, n=dtype, dn=dtype))


@pytest.mark.parametrize("T,d,span", [
    *[(T, d, span) for T, d in ((4500, 1001), (5000, 2048), (1100, 8192)) for span in (0, 1, 2, 100, T)],
    # more cut gate rows than workgroups that add them: gate rows longer than a group's rows, and shorter ones
    (6400, 2048, 100), (6400, 2041, 100), (2500, 4096, 37), (1100, 8192, 4), (1100, 8191, 5), (5000, 2048, 3)])
def test_wide_gates(gpu_lib, T, d, span):
    say(f"case block norm wide gates {T} x {d} span={span}")
    norm._check(gpu_lib, norm._case(T, d, span=span, r="bfloat16", y="float32"))


@pytest.mark.parametrize("span", [601, (1 << 31) - 1, 1 << 32, (1 << 32) + 1])
def test_one_gate_row(gpu_lib, span):
    """A span past all rows, or past 32 bits, gives the same bits as one of all rows."""
    import torch
    say(f"case block norm one gate row, span={span}")
    c = norm._case(600, 264, span=600)
    want = norm._forward(gpu_lib, c), norm._backward(gpu_lib, c)
    c["span"] = span
    for a, b in zip(want, (norm._forward(gpu_lib, c), norm._backward(gpu_lib, c))):
        for k in a:
            assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("d", [1, 7, 9, 15, 16, 100, 129, 511, 513, 519, 1001, 1025, 1031, 2049, 4100, 8191, 8192])
@pytest.mark.parametrize("kind,dtype", [("rms", "float32"), ("layer", "bfloat16")])
def test_gradient_in_place(gpu_lib, d, kind, dtype):
    """dres may be dout: the same bits as with a tensor of its own."""
    import torch
    say(f"case block norm gradient in place d={d} {kind} {dtype}")
    tw, T, span = gpu_lib, 600, 7
    c = norm._case(T, d, kind=kind, bias=True, span=span, r=dtype, y=dtype, dn=dtype)
    want = norm._backward(tw, c)
    got = {k: torch.full_like(t, float("nan")) for k, t in want.items()}
    got["dres"] = c["dout"].clone()
    tw.twell_block_norm_backward(norm._bn(tw, c), c["res"], c["y"], got["dres"], c["dn"], got["dres"], got["dy"],
                                 tw.block_norm_workspace(T, d), gate=c["gate"], gate_span=span,
                                 **{k: got[k] for k in ("dgate", "dw_post", "db_post", "dw_pre", "db_pre")})
    for k in want:
        assert torch.equal(got[k], want[k]), k
