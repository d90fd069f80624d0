"""Python binding of libtwell (ReLU-sparse gated FFN with TwELL on MI355X).

Argument marshalling only: every step of the path runs in the HIP kernels of
``libtwell.so`` (built from ``csrc/`` by ``_build.py``); PyTorch supplies device
memory and the current HIP stream.  There is no CPU fallback: ``load()``
raises when the library is missing, and every call raises on a non-OK status.

The functions carry the C names (``include/twell.h``):
``twell_ffn_forward``, ``twell_ffn_from_gate``, ``twell_pack_gate``, ``twell_gate_dense``, ``twell_pack_gate_stats``, ``twell_partition_overflow``,
``twell_pack_gate_hybrid``,
``twell_ffn_fused``, ``twell_ffn_overflow``, ``twell_ffn_hybrid``,
``twell_workspace_bytes``, ``twell_ffn_decode``,
``twell_ffn_decode_workspace_bytes``, ``twell_ffn_decode_noalloc``, ``twell_dense_to_hybrid``,
``twell_hybrid_to_dense``, ``twell_compact_min_bytes``, ``twell_compact_hybrid``,
``twell_compact_to_dense``, ``twell_ffn_backward``,
``twell_ffn_backward_workspace_bytes``, ``twell_glu_forward``, ``twell_glu_workspace_bytes``,
``twell_glu_backward``, ``twell_glu_backward_workspace_bytes``, ``twell_block_norm_forward``,
``twell_block_norm_workspace_bytes``, ``twell_block_norm_backward``, ``twell_adamw_step``, ``twell_adamw_unpack``,
``twell_act_pack``, ``twell_act_unpack``, ``twell_glu_forward_packed``, ``twell_glu_packed_workspace_bytes``,
``twell_glu_backward_packed``, ``twell_embed_forward``, ``twell_embed_backward``, ``twell_embed_workspace_bytes``,
``twell_logprob_forward``, ``twell_logprob_workspace_bytes``, ``twell_logprob_backward``.

One layer's forward pass, bf16 (x [T][d], W_g^T and W_u^T [F][d], W_d [F][d],
all contiguous on the GPU; y [T][d] fp32)::

    import unstructured_sparse_transformer_amd as tw
    hy = tw.Hybrid.empty(T, F, tile_w=256, cap=16, dtype=torch.bfloat16, max_ovf=1024)
    ws = tw.hybrid_workspace(hy, d)
    tw.twell_ffn_forward(x, wg_t, wu_t, wd, hy, y, ws)   # on the current stream
    # hy.ell holds the TwELL of ReLU(x W_g); hy.n_ovf counts the overflow rows.
    # Overflow rows past max_ovf are counted but not computed: after
    # synchronising, check n_ovf <= max_ovf and grow max_ovf otherwise.

For T <= 64 tokens, ``twell_ffn_decode`` with ``decode_workspace(T, F, d,
tile_w)`` computes the same in four short kernels.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtwell.so")

TWELL_F32, TWELL_BF16 = 0, 1
STATUS = {0: "TWELL_OK", -1: "TWELL_E_NULL", -2: "TWELL_E_ALIGN", -3: "TWELL_E_SHAPE",
          -4: "TWELL_E_UNSUPPORTED", -5: "TWELL_E_HIP", -6: "TWELL_E_WORKSPACE", -7: "TWELL_E_SCRATCH"}
EXPORTS = ("twell_ffn_forward", "twell_ffn_from_gate", "twell_pack_gate", "twell_gate_dense", "twell_pack_gate_stats", "twell_partition_overflow", "twell_pack_gate_hybrid",
           "twell_ffn_fused", "twell_workspace_bytes", "twell_ffn_overflow", "twell_ffn_hybrid",
           "twell_ffn_decode_workspace_bytes", "twell_ffn_decode", "twell_ffn_decode_noalloc", "twell_dense_to_hybrid", "twell_hybrid_to_dense",
           "twell_compact_min_bytes", "twell_compact_hybrid", "twell_compact_to_dense",
           "twell_ffn_backward_workspace_bytes", "twell_ffn_backward", "twell_glu_workspace_bytes",
           "twell_glu_forward", "twell_glu_backward_workspace_bytes", "twell_glu_backward", "twell_block_norm_forward",
           "twell_block_norm_workspace_bytes", "twell_block_norm_backward", "twell_adamw_step", "twell_adamw_unpack",
           "twell_act_pack", "twell_act_unpack", "twell_glu_forward_packed", "twell_glu_packed_workspace_bytes",
           "twell_glu_backward_packed", "twell_embed_forward", "twell_embed_backward", "twell_embed_workspace_bytes",
           "twell_logprob_forward", "twell_logprob_workspace_bytes", "twell_logprob_backward",
           "twell_status_str", "twell_version")


class TwellT(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("F", ctypes.c_int32), ("tile_w", ctypes.c_int32),
                ("cap", ctypes.c_int32), ("vdtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("val", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("cnt", ctypes.c_void_p)]


class TwellHybridT(ctypes.Structure):
    _fields_ = [("ell", TwellT), ("max_ovf", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("row_ovf", ctypes.c_void_p), ("ovf_rows", ctypes.c_void_p), ("n_ovf", ctypes.c_void_p),
                ("dense", ctypes.c_void_p), ("order", ctypes.c_void_p)]


class TwellBlockNormT(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("kind", ctypes.c_int32), ("post", ctypes.c_int32),
                ("eps", ctypes.c_float), ("alpha", ctypes.c_float), ("gate_span", ctypes.c_int32),
                ("rdtype", ctypes.c_int32), ("ydtype", ctypes.c_int32), ("ndtype", ctypes.c_int32),
                ("wdtype", ctypes.c_int32), ("reserved", ctypes.c_int32), ("gate", ctypes.c_void_p),
                ("w_post", ctypes.c_void_p), ("b_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p),
                ("b_pre", ctypes.c_void_p)]


class TwellPackedT(ctypes.Structure):
    _fields_ = [("code", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class TwellAdamWTensorT(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("p", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("m_values", ctypes.c_void_p), ("v_values", ctypes.c_void_p),
                ("weight_decay", ctypes.c_double), ("pdtype", ctypes.c_int32), ("gdtype", ctypes.c_int32)]


class TwellError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = _lib.twell_status_str(status).decode() if _lib is not None else ""
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({msg})")
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load libtwell.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libtwell.so not found at {path}: build it with "
                           "`python -m unstructured_sparse_transformer_amd._build` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    P, I32 = ctypes.c_void_p, ctypes.c_int32
    lib.twell_pack_gate.argtypes = [P, P, I32, ctypes.POINTER(TwellT), P]
    lib.twell_pack_gate_stats.argtypes = [P, P, I32, ctypes.POINTER(TwellT), P, P, P]
    lib.twell_gate_dense.argtypes = [P, P, I32, I32, I32, I32, P, P]
    lib.twell_partition_overflow.argtypes = [P, P, I32, ctypes.POINTER(TwellHybridT), P]
    lib.twell_pack_gate_hybrid.argtypes = [P, P, I32, ctypes.POINTER(TwellHybridT), P]
    lib.twell_ffn_fused.argtypes = [ctypes.POINTER(TwellT), P, P, P, P, I32, P, P, ctypes.c_size_t, P]
    lib.twell_workspace_bytes.argtypes = [I32, I32, I32, I32, I32, I32, I32]
    lib.twell_workspace_bytes.restype = ctypes.c_size_t
    lib.twell_ffn_hybrid.argtypes = [ctypes.POINTER(TwellHybridT), P, P, P, I32, P, P, ctypes.c_size_t, P]
    lib.twell_ffn_overflow.argtypes = [ctypes.POINTER(TwellHybridT), P, P, P, I32, P, P, ctypes.c_size_t, P]
    lib.twell_ffn_forward.argtypes = [P, P, P, P, I32, ctypes.POINTER(TwellHybridT), P, P, ctypes.c_size_t, P]
    lib.twell_ffn_from_gate.argtypes = [P, P, P, P, I32, ctypes.POINTER(TwellHybridT), P, P, ctypes.c_size_t, P]
    lib.twell_ffn_decode_workspace_bytes.argtypes = [I32, I32, I32, I32]
    lib.twell_ffn_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.twell_ffn_decode.argtypes = [P, P, P, P, I32, ctypes.POINTER(TwellHybridT), P, P, ctypes.c_size_t, P]
    lib.twell_ffn_decode_noalloc.argtypes = [P, P, P, P, I32, ctypes.POINTER(TwellHybridT), P, P]
    lib.twell_dense_to_hybrid.argtypes = [P, ctypes.POINTER(TwellHybridT), P]
    lib.twell_hybrid_to_dense.argtypes = [ctypes.POINTER(TwellHybridT), P, P]
    lib.twell_compact_min_bytes.argtypes = [I32]
    lib.twell_compact_min_bytes.restype = ctypes.c_size_t
    lib.twell_compact_hybrid.argtypes = [ctypes.POINTER(TwellHybridT), P, ctypes.c_size_t, P]
    lib.twell_compact_to_dense.argtypes = [P, I32, I32, I32, P, P]
    lib.twell_ffn_backward_workspace_bytes.argtypes = [I32, I32, I32, I32]
    lib.twell_ffn_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.twell_ffn_backward.argtypes = [ctypes.POINTER(TwellHybridT), P, P, P, P, I32, P, P, P, P, P, I32, P,
                                       ctypes.c_size_t, P]
    for fn in (lib.twell_glu_workspace_bytes, lib.twell_glu_backward_workspace_bytes):
        fn.argtypes = [I32, I32, I32, I32]
        fn.restype = ctypes.c_size_t
    lib.twell_glu_forward.argtypes = [P, P, P, I32, I32, I32, I32, I32, P, P, P, P, ctypes.c_size_t, P]
    lib.twell_glu_backward.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32, P, P, P, P, ctypes.c_size_t, P]
    BN = ctypes.POINTER(TwellBlockNormT)
    lib.twell_block_norm_forward.argtypes = [BN, P, P, P, P, P]
    lib.twell_block_norm_workspace_bytes.argtypes = [I32, I32]
    lib.twell_block_norm_workspace_bytes.restype = ctypes.c_size_t
    lib.twell_block_norm_backward.argtypes = [BN, P, P, P, P, I32, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    F64 = ctypes.c_double
    lib.twell_adamw_step.argtypes = [P, I32, I32, F64, F64, F64, F64, ctypes.c_int64, ctypes.c_uint32, P, P]
    lib.twell_adamw_unpack.argtypes = [P, I32, P]
    F32, I64, SIZE, PK = ctypes.c_float, ctypes.c_int64, ctypes.c_size_t, ctypes.POINTER(TwellPackedT)
    lib.twell_act_pack.argtypes = [P, I32, I32, I32, PK, P]
    lib.twell_act_unpack.argtypes = [PK, I32, I32, I32, P, P]
    lib.twell_glu_forward_packed.argtypes = [P, P, P, I32, I32, I32, I32, P, PK, PK, I32, P, SIZE, P]
    lib.twell_glu_backward_packed.argtypes = [P, P, P, PK, PK, P, I32, I32, I32, I32, P, P, P, P, P, SIZE, P]
    lib.twell_embed_forward.argtypes = [P, I32, I32, P, I32, I32, I32, F32, P, I32, P]
    lib.twell_embed_backward.argtypes = [P, I32, I32, P, I32, I32, I32, F32, I32, P, I32, P, SIZE, P]
    lib.twell_logprob_forward.argtypes = [P, I64, I32, I32, I32, F32, P, I32, P, P, P, P, P, I32, P, SIZE, P]
    lib.twell_logprob_backward.argtypes = [P, I64, I32, I32, I32, F32, P, I32, P, P, P, P, P, I64, P]
    for fn in (lib.twell_glu_packed_workspace_bytes, lib.twell_embed_workspace_bytes, lib.twell_logprob_workspace_bytes):
        fn.argtypes = [I32, I32, I32]
        fn.restype = SIZE
    lib.twell_status_str.argtypes = [ctypes.c_int]
    lib.twell_status_str.restype = ctypes.c_char_p
    lib.twell_version.restype = ctypes.c_int
    for fn in (lib.twell_pack_gate, lib.twell_gate_dense, lib.twell_pack_gate_stats, lib.twell_partition_overflow, lib.twell_pack_gate_hybrid,
               lib.twell_ffn_fused, lib.twell_ffn_hybrid, lib.twell_ffn_overflow, lib.twell_ffn_forward,
               lib.twell_ffn_from_gate, lib.twell_ffn_decode, lib.twell_ffn_decode_noalloc,
               lib.twell_dense_to_hybrid, lib.twell_hybrid_to_dense, lib.twell_compact_hybrid,
               lib.twell_compact_to_dense, lib.twell_ffn_backward, lib.twell_glu_forward,
               lib.twell_glu_backward, lib.twell_block_norm_forward,
               lib.twell_block_norm_backward, lib.twell_adamw_step, lib.twell_adamw_unpack, lib.twell_act_pack,
               lib.twell_act_unpack, lib.twell_glu_forward_packed, lib.twell_glu_backward_packed, lib.twell_embed_forward,
               lib.twell_embed_backward, lib.twell_logprob_forward, lib.twell_logprob_backward):
        fn.restype = ctypes.c_int
    _lib = lib
    return lib


# ---------------------------------------------------------------- marshalling helpers
def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


_raw_stream = None


def _stream(stream, dev=None) -> int | None:
    """A stream's handle; None: the current one, of the current GPU `dev` where the caller knows it."""
    if stream is None:
        global _raw_stream
        if _raw_stream is None or dev is None:
            import torch
            # the handle without a Stream object (2.7 us less)
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
            dev = torch.cuda.current_device() if dev is None else dev
        return _raw_stream(dev)
    return getattr(stream, "cuda_stream", stream)


_VDTYPES: dict = {}  # torch's element types, once torch is there


def vdtype_of(torch_dtype) -> int:
    v = _VDTYPES.get(torch_dtype)
    if v is None:
        import torch
        _VDTYPES.update({torch.bfloat16: TWELL_BF16, torch.float32: TWELL_F32})
        v = _VDTYPES.get(torch_dtype)
        if v is None:
            raise TypeError(f"unsupported element type {torch_dtype}")
    return v


def _check(fn: str, st: int):
    if st != 0:
        raise TwellError(fn, st)


@dataclass
class TwELL:
    """Device buffers of one TwELL (torch tensors) and its C descriptor."""
    T: int
    F: int
    tile_w: int
    cap: int
    dtype: object
    val: object  # [T][n_b][cap] dtype
    idx: object  # [T][n_b][cap] uint8
    cnt: object  # [T][n_b] int32

    @property
    def n_b(self) -> int:
        return self.F // self.tile_w

    @classmethod
    def empty(cls, T, F, tile_w, cap, dtype, device="cuda"):
        import torch
        n_b = F // tile_w
        return cls(T, F, tile_w, cap, dtype,
                   torch.empty((T, n_b, cap), dtype=dtype, device=device),
                   torch.empty((T, n_b, cap), dtype=torch.uint8, device=device),
                   torch.empty((T, n_b), dtype=torch.int32, device=device))

    def desc(self) -> TwellT:
        return TwellT(self.T, self.F, self.tile_w, self.cap, vdtype_of(self.dtype), 0,
                      _ptr(self.val), _ptr(self.idx), _ptr(self.cnt))


@dataclass
class Hybrid:
    """TwELL plus overflow partition and dense backup buffers."""
    ell: TwELL
    max_ovf: int
    row_ovf: object   # [T] int32
    ovf_rows: object  # [max_ovf] int32
    n_ovf: object     # [1] int32
    dense: object     # [max_ovf][F] dtype
    order: object     # [T] int32: the fused step's work order

    @classmethod
    def empty(cls, T, F, tile_w, cap, dtype, max_ovf, device="cuda"):
        import torch
        return cls(TwELL.empty(T, F, tile_w, cap, dtype, device), max_ovf,
                   torch.empty(T, dtype=torch.int32, device=device),
                   torch.empty(max(max_ovf, 1), dtype=torch.int32, device=device),
                   torch.empty(1, dtype=torch.int32, device=device),
                   torch.empty((max(max_ovf, 1), F), dtype=dtype, device=device),
                   torch.empty(T, dtype=torch.int32, device=device))

    def desc(self) -> TwellHybridT:
        return TwellHybridT(self.ell.desc(), self.max_ovf, 0, _ptr(self.row_ovf), _ptr(self.ovf_rows),
                            _ptr(self.n_ovf), _ptr(self.dense), _ptr(self.order))


# ---------------------------------------------------------------- the C entry points
def twell_pack_gate(x, wg_t, tw: TwELL, stream=None):
    lib = load()
    d = ctypes.byref(tw.desc())
    _check("twell_pack_gate", lib.twell_pack_gate(_ptr(x), _ptr(wg_t), int(x.shape[1]), d, _stream(stream)))


def twell_gate_dense(x, wg_t, h, stream=None):
    """h [T][F] (x's dtype) = ReLU(x W_g), the gate with a plain dense store."""
    _check("twell_gate_dense", load().twell_gate_dense(_ptr(x), _ptr(wg_t), int(x.shape[1]), int(x.shape[0]),
                                                       int(wg_t.shape[0]), vdtype_of(x.dtype), _ptr(h),
                                                       _stream(stream)))


def twell_pack_gate_stats(x, wg_t, tw: TwELL, neuron_cnt, l1, stream=None):
    """neuron_cnt: int32 [F] (added to); l1: float32 [T][F // tile_w] (overwritten)."""
    lib = load()
    d = ctypes.byref(tw.desc())
    _check("twell_pack_gate_stats", lib.twell_pack_gate_stats(_ptr(x), _ptr(wg_t), int(x.shape[1]), d,
                                                              _ptr(neuron_cnt), _ptr(l1), _stream(stream)))


def twell_partition_overflow(x, wg_t, hy: Hybrid, stream=None):
    lib = load()
    _check("twell_partition_overflow",
           lib.twell_partition_overflow(_ptr(x), _ptr(wg_t), int(x.shape[1]), ctypes.byref(hy.desc()),
                                        _stream(stream)))


def twell_pack_gate_hybrid(x, wg_t, hy: Hybrid, stream=None):
    lib = load()
    _check("twell_pack_gate_hybrid",
           lib.twell_pack_gate_hybrid(_ptr(x), _ptr(wg_t), int(x.shape[1]), ctypes.byref(hy.desc()),
                                      _stream(stream)))


def twell_ffn_fused(tw: TwELL, x, wu_t, wd, y, workspace, stream=None, order=None):
    lib = load()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("twell_ffn_fused", lib.twell_ffn_fused(ctypes.byref(tw.desc()), _ptr(order), _ptr(x), _ptr(wu_t),
                                                  _ptr(wd), int(x.shape[1]), _ptr(y), _ptr(workspace), nbytes,
                                                  _stream(stream)))


def twell_workspace_bytes(T: int, F: int, tile_w: int, cap: int, max_ovf: int, d: int, dtype) -> int:
    return int(load().twell_workspace_bytes(T, F, tile_w, cap, max_ovf, d, vdtype_of(dtype)))


def twell_ffn_hybrid(hy: Hybrid, x, wu_t, wd, y, workspace, stream=None):
    lib = load()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("twell_ffn_hybrid",
           lib.twell_ffn_hybrid(ctypes.byref(hy.desc()), _ptr(x), _ptr(wu_t), _ptr(wd), int(x.shape[1]),
                                _ptr(y), _ptr(workspace), nbytes, _stream(stream)))


def twell_ffn_forward(x, wg_t, wu_t, wd, hy: Hybrid, y, workspace, stream=None):
    """The whole layer: fills the hybrid `hy` and y [T][d] float in one call."""
    lib = load()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("twell_ffn_forward",
           lib.twell_ffn_forward(_ptr(x), _ptr(wg_t), _ptr(wu_t), _ptr(wd), int(x.shape[1]), ctypes.byref(hy.desc()),
                                 _ptr(y), _ptr(workspace), nbytes, _stream(stream)))


def twell_ffn_from_gate(x, wg_t, wu_t, wd, hy: Hybrid, y, workspace, stream=None):
    """The layer after twell_pack_gate on hy.ell: the rest of the hybrid and y."""
    lib = load()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("twell_ffn_from_gate",
           lib.twell_ffn_from_gate(_ptr(x), _ptr(wg_t), _ptr(wu_t), _ptr(wd), int(x.shape[1]),
                                   ctypes.byref(hy.desc()), _ptr(y), _ptr(workspace), nbytes, _stream(stream)))


def twell_ffn_overflow(hy: Hybrid, x, wu_t, wd, y, workspace, stream=None):
    lib = load()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("twell_ffn_overflow",
           lib.twell_ffn_overflow(ctypes.byref(hy.desc()), _ptr(x), _ptr(wu_t), _ptr(wd), int(x.shape[1]),
                                  _ptr(y), _ptr(workspace), nbytes, _stream(stream)))


def twell_dense_to_hybrid(h, hy: Hybrid, stream=None):
    """h: [T][F] in the hybrid's value dtype."""
    _check("twell_dense_to_hybrid", load().twell_dense_to_hybrid(_ptr(h), ctypes.byref(hy.desc()), _stream(stream)))


def twell_hybrid_to_dense(hy: Hybrid, out, stream=None):
    """out: [T][F] in the hybrid's value dtype (every element written)."""
    _check("twell_hybrid_to_dense", load().twell_hybrid_to_dense(ctypes.byref(hy.desc()), _ptr(out), _stream(stream)))


COMPACT_HEADER = (("T", "i"), ("F", "i"), ("tile_w", "i"), ("vdtype", "i"), ("n_entries", "i"), ("n_ovf", "i"),
                  ("n_dense", "i"), ("fits", "i"), ("off_row_ptr", "q"), ("off_col", "q"), ("off_val", "q"),
                  ("off_ovf", "q"), ("off_dense", "q"), ("bytes", "q"))


def twell_compact_min_bytes(T: int) -> int:
    return int(load().twell_compact_min_bytes(T))


def twell_compact_hybrid(hy: Hybrid, buf, stream=None):
    """buf: a uint8 device tensor (256-byte aligned by the allocator)."""
    _check("twell_compact_hybrid", load().twell_compact_hybrid(ctypes.byref(hy.desc()), _ptr(buf),
                                                               buf.numel() * buf.element_size(), _stream(stream)))


def twell_compact_to_dense(buf, T: int, F: int, dtype, out, stream=None):
    _check("twell_compact_to_dense", load().twell_compact_to_dense(_ptr(buf), T, F, vdtype_of(dtype), _ptr(out),
                                                                   _stream(stream)))


def compact_header(buf) -> dict:
    """The header of a compact buffer, read back to the host (synchronises)."""
    import struct
    fmt = "<" + "".join(f for _, f in COMPACT_HEADER)
    raw = bytes(buf[: struct.calcsize(fmt)].cpu().numpy().tobytes())
    return dict(zip((n for n, _ in COMPACT_HEADER), struct.unpack(fmt, raw)))


def twell_ffn_backward_workspace_bytes(T: int, F: int, d: int, max_entries: int) -> int:
    return int(load().twell_ffn_backward_workspace_bytes(T, F, d, max_entries))


def backward_workspace(T: int, F: int, d: int, max_entries: int, device="cuda"):
    import torch
    n = twell_ffn_backward_workspace_bytes(T, F, d, max_entries)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def twell_ffn_backward(hy: Hybrid, x, wg_t, wu_t, wd, dy, dx, dwg, dwu, dwd, max_entries: int, workspace,
                       stream=None):
    _check("twell_ffn_backward",
           load().twell_ffn_backward(ctypes.byref(hy.desc()), _ptr(x), _ptr(wg_t), _ptr(wu_t), _ptr(wd),
                                     int(wg_t.shape[1]), _ptr(dy), _ptr(dx), _ptr(dwg), _ptr(dwu), _ptr(dwd),
                                     max_entries, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream)))


def backward_status(workspace) -> tuple:
    """(entries, too_many) from a backward workspace (synchronises)."""
    v = workspace[:8].cpu().numpy().view("<i4")
    return int(v[0]), int(v[1])


def twell_ffn_decode_workspace_bytes(T: int, F: int, d: int, tile_w: int) -> int:
    return int(load().twell_ffn_decode_workspace_bytes(T, F, d, tile_w))


def twell_ffn_decode(x, wg_t, wu_t, wd, hy: Hybrid, y, workspace, stream=None):
    lib = load()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("twell_ffn_decode",
           lib.twell_ffn_decode(_ptr(x), _ptr(wg_t), _ptr(wu_t), _ptr(wd), int(x.shape[1]), ctypes.byref(hy.desc()),
                                _ptr(y), _ptr(workspace), nbytes, _stream(stream)))


def twell_ffn_decode_noalloc(x, wg_t, wu_t, wd, hy: Hybrid, y, stream=None):
    """twell_ffn_decode on the library's static scratch (no workspace argument)."""
    _check("twell_ffn_decode_noalloc",
           load().twell_ffn_decode_noalloc(_ptr(x), _ptr(wg_t), _ptr(wu_t), _ptr(wd), int(x.shape[1]),
                                           ctypes.byref(hy.desc()), _ptr(y), _stream(stream)))


def decode_workspace(T: int, F: int, d: int, tile_w: int, device="cuda"):
    """A workspace tensor of the size twell_ffn_decode needs (256-byte aligned by the allocator)."""
    import torch
    n = twell_ffn_decode_workspace_bytes(T, F, d, tile_w)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def workspace(T: int, F: int, tile_w: int, cap: int, max_ovf: int, d: int, dtype, device="cuda"):
    """A workspace tensor of the size twell_workspace_bytes gives (256-byte
    aligned by the allocator); it serves twell_ffn_fused, twell_ffn_overflow,
    twell_ffn_hybrid, twell_ffn_forward and twell_ffn_from_gate."""
    import torch
    n = twell_workspace_bytes(T, F, tile_w, cap, max_ovf, d, dtype)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def hybrid_workspace(hy: "Hybrid", d: int, device="cuda"):
    """The workspace for the calls on hybrid `hy` with model width d."""
    e = hy.ell
    return workspace(e.T, e.F, e.tile_w, e.cap, hy.max_ovf, d, e.dtype, device)


# ---------------------------------------------------------------- the dense gated product
_current_device = None


def _device(fn: str, t) -> int:
    """The GPU a call's tensors have to be on: the current one, whose streams the kernels run on."""
    global _current_device
    dev = t.get_device()
    if dev >= 0 and _current_device is None:
        import torch
        # (torch.cuda.current_device's own look-up: the tensor says that the GPU is in use, 0.4 us less)
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    if dev < 0 or dev != _current_device():
        raise ValueError(f"{fn}: tensors on the current GPU are needed, got one on {t.device}")
    return dev


def _tensor(fn: str, name: str, t, shape, dev: int, dtype=None) -> int:
    """The pointer of an argument: contiguous, on GPU `dev`, of this shape and (if given) element type."""
    if t is None:
        raise ValueError(f"{fn}: {name} is missing")
    if t.shape == shape and t.is_contiguous() and t.get_device() == dev and (dtype is None or t.dtype is dtype):
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {name} is on {t.device}, not on cuda:{dev}")
    raise TypeError(f"{fn}: {name} must be {dtype}, not {t.dtype}")


def _i32(n: int) -> int:
    """A count for a 32-bit argument.  One that does not fit becomes the largest, which is past the bounds that the C
    side checks (ctypes alone would keep its lower 32 bits)."""
    return n if -1 <= n <= 0x7FFFFFFF else -1 if n < 0 else 0x7FFFFFFF


def _workspace(fn: str, t, dev: int) -> tuple:
    """The pointer and the bytes of a workspace (or None)."""
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{fn}: the workspace must be contiguous and on cuda:{dev}")
    return t.data_ptr(), t.numel() * t.element_size()


ACTS = {"relu": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}


def _act(fn: str, act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"{fn}: act {act!r}: one of {', '.join(ACTS)}")
    return ACTS[act]


def twell_glu_workspace_bytes(T: int, d: int, F: int, dtype) -> int:
    return int(load().twell_glu_workspace_bytes(_i32(T), _i32(d), _i32(F), vdtype_of(dtype)))


def glu_workspace(T: int, d: int, F: int, dtype, device="cuda"):
    """A workspace tensor for twell_glu_forward with up to T rows, or None where none of these needs one."""
    import torch
    n = twell_glu_workspace_bytes(T, d, F, dtype)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def twell_glu_forward(x, wg_t, wu_t, act: str, h, workspace=None, g=None, u=None, stream=None):
    """h = act(x W_g) * (x W_u); g and u (optional, h's shape) receive the two products for the backward pass."""
    fn = "twell_glu_forward"
    dev, dt, (T, d), F = _device(fn, x), x.dtype, x.shape, wg_t.shape[0]
    p = (_tensor(fn, "x", x, (T, d), dev), _tensor(fn, "wg_t", wg_t, (F, d), dev, dt),
         _tensor(fn, "wu_t", wu_t, (F, d), dev, dt))
    out = (_tensor(fn, "h", h, (T, F), dev, dt), None if g is None else _tensor(fn, "g", g, (T, F), dev, dt),
           None if u is None else _tensor(fn, "u", u, (T, F), dev, dt))
    _check(fn, load().twell_glu_forward(*p, _i32(T), _i32(d), _i32(F), vdtype_of(dt), _act(fn, act), *out,
                                        *_workspace(fn, workspace, dev), _stream(stream, dev)))


def twell_glu_backward_workspace_bytes(T: int, d: int, F: int, dtype) -> int:
    return int(load().twell_glu_backward_workspace_bytes(_i32(T), _i32(d), _i32(F), vdtype_of(dtype)))


def glu_backward_workspace(T: int, d: int, F: int, dtype, device="cuda"):
    """A workspace tensor for twell_glu_backward with up to T rows."""
    import torch
    return torch.empty(max(twell_glu_backward_workspace_bytes(T, d, F, dtype), 256), dtype=torch.uint8, device=device)


def twell_glu_backward(x, wg_t, wu_t, g, u, dh, act: str, dx, dwg, dwu, workspace, stream=None):
    """dx [T][d], dwg and dwu [F][d] (dx, or both of the others, may be None) from the forward's g and u and dh."""
    fn = "twell_glu_backward"
    dev, dt, (T, d), F = _device(fn, x), x.dtype, x.shape, wg_t.shape[0]
    p = [_tensor(fn, k, t, s, dev, dt) for k, t, s in (("x", x, (T, d)), ("wg_t", wg_t, (F, d)), ("wu_t", wu_t, (F, d)),
                                                       ("g", g, (T, F)), ("u", u, (T, F)), ("dh", dh, (T, F)))]
    o = [None if t is None else _tensor(fn, k, t, s, dev, dt)
         for k, t, s in (("dx", dx, (T, d)), ("dwg", dwg, (F, d)), ("dwu", dwu, (F, d)))]
    _check(fn, load().twell_glu_backward(*p, _i32(T), _i32(d), _i32(F), vdtype_of(dt), _act(fn, act), *o,
                                         *_workspace(fn, workspace, dev), _stream(stream, dev)))


# ---------------------------------------------------------------- activations kept in 8 bits
ACT_BLOCK = 32  # elements of a row that share a scale


@dataclass
class PackedAct:
    """Activations [T][d] in 8 bits: ``code`` int8 [T][d], ``scale`` bfloat16 [T][ceil(d / 32)]."""
    code: object
    scale: object

    @classmethod
    def empty(cls, T, d, device="cuda"):
        import torch
        return cls(torch.empty((T, d), dtype=torch.int8, device=device),
                   torch.empty((T, -(-d // ACT_BLOCK)), dtype=torch.bfloat16, device=device))

    def desc(self, fn: str, name: str, shape, dev: int) -> TwellPackedT:
        T, d = shape
        kinds = _PACKED_TYPES or _packed_types()
        return TwellPackedT(_tensor(fn, name, self.code, shape, dev, kinds[0]),
                            _tensor(fn, name, self.scale, (T, -(-d // ACT_BLOCK)), dev, kinds[1]))


_PACKED_TYPES: tuple = ()  # of the codes and the scales, once torch is there


def _packed_types() -> tuple:
    global _PACKED_TYPES
    import torch
    _PACKED_TYPES = torch.int8, torch.bfloat16
    return _PACKED_TYPES


def _packed(fn: str, name: str, p, shape, dev: int) -> TwellPackedT:
    if not isinstance(p, PackedAct):
        raise TypeError(f"{fn}: {name} must be a PackedAct, not {type(p).__name__}")
    return p.desc(fn, name, shape, dev)


def twell_act_pack(x, packed: PackedAct, stream=None):
    """The codes and scales of x [T][d] (float32 or bfloat16)."""
    fn = "twell_act_pack"
    dev, (T, d) = _device(fn, x), x.shape
    p = _tensor(fn, "x", x, (T, d), dev)
    to = _packed(fn, "packed", packed, (T, d), dev)
    _check(fn, load().twell_act_pack(p, _i32(T), _i32(d), vdtype_of(x.dtype), to, _stream(stream, dev)))


def twell_act_unpack(packed: PackedAct, out, stream=None):
    """The values that the codes stand for, in out's type (float32: as they are, bfloat16: rounded)."""
    fn = "twell_act_unpack"
    dev, (T, d) = _device(fn, out), out.shape
    p = _tensor(fn, "out", out, (T, d), dev)
    source = _packed(fn, "packed", packed, (T, d), dev)
    _check(fn, load().twell_act_unpack(source, _i32(T), _i32(d), vdtype_of(out.dtype), p, _stream(stream, dev)))


def twell_glu_packed_workspace_bytes(T: int, d: int, F: int) -> int:
    return int(load().twell_glu_packed_workspace_bytes(_i32(T), _i32(d), _i32(F)))


def glu_packed_workspace(T: int, d: int, F: int, device="cuda"):
    """A workspace tensor for twell_glu_forward_packed with up to T rows, or None where none of these needs one."""
    import torch
    n = twell_glu_packed_workspace_bytes(T, d, F)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def twell_glu_forward_packed(x, wg_t, wu_t, act: str, h, g: PackedAct, u: PackedAct, workspace=None, keep_sign: bool = False,
                             stream=None):
    """twell_glu_forward in bfloat16, with g and u kept in 8 bits; keep_sign: positive values of g keep at least code 1,
    for relu, whose gradient where g is small is lost otherwise (see include/twell.h)."""
    import torch
    fn = "twell_glu_forward_packed"
    dev, (T, d), F = _device(fn, x), x.shape, wg_t.shape[0]
    p = [_tensor(fn, k, t, s, dev, torch.bfloat16) for k, t, s in (("x", x, (T, d)), ("wg_t", wg_t, (F, d)),
                                                                   ("wu_t", wu_t, (F, d)), ("h", h, (T, F)))]
    kept = [_packed(fn, k, t, (T, F), dev) for k, t in (("g", g), ("u", u))]
    _check(fn, load().twell_glu_forward_packed(*p[:3], _i32(T), _i32(d), _i32(F), _act(fn, act), p[3], *kept, int(bool(keep_sign)),
                                               *_workspace(fn, workspace, dev), _stream(stream, dev)))


def twell_glu_backward_packed(x, wg_t, wu_t, g: PackedAct, u: PackedAct, dh, act: str, dx, dwg, dwu, workspace, h=None,
                              stream=None):
    """twell_glu_backward in bfloat16 from g and u in 8 bits (workspace: glu_backward_workspace); h (optional) receives
    act(g) * u of these.  dx, or both of dwg and dwu, may be None."""
    import torch
    fn = "twell_glu_backward_packed"
    dev, (T, d), F = _device(fn, x), x.shape, wg_t.shape[0]
    p = [_tensor(fn, k, t, s, dev, torch.bfloat16) for k, t, s in (("x", x, (T, d)), ("wg_t", wg_t, (F, d)),
                                                                   ("wu_t", wu_t, (F, d)), ("dh", dh, (T, F)))]
    kept = [_packed(fn, k, t, (T, F), dev) for k, t in (("g", g), ("u", u))]
    o = [None if t is None else _tensor(fn, k, t, s, dev, torch.bfloat16)
         for k, t, s in (("h", h, (T, F)), ("dx", dx, (T, d)), ("dwg", dwg, (F, d)), ("dwu", dwu, (F, d)))]
    _check(fn, load().twell_glu_backward_packed(*p[:3], *kept, p[3], _i32(T), _i32(d), _i32(F), _act(fn, act), *o,
                                                *_workspace(fn, workspace, dev), _stream(stream, dev)))


# ---------------------------------------------------------------- token embedding
_ID_BITS: dict = {}


def _ids(fn: str, name: str, t, T: int, dev: int) -> tuple:
    """The pointer of token ids [T] and their bits."""
    p = _tensor(fn, name, t, (T,), dev)
    bits = _ID_BITS.get(t.dtype)
    if bits is None:
        import torch
        _ID_BITS.update({torch.int64: 64, torch.int32: 32})
        bits = _ID_BITS.get(t.dtype)
        if bits is None:
            raise TypeError(f"{fn}: {name} must be torch.int32 or torch.int64, not {t.dtype}")
    return p, bits


def twell_embed_forward(ids, table, out, scale: float = 1.0, stream=None):
    """out [T][d] = scale * table [V][d] at ids [T] (int32 or int64); zeros where an id is none of 0 .. V-1."""
    fn = "twell_embed_forward"
    dev, (V, d), T = _device(fn, table), table.shape, ids.shape[0]
    p, bits = _ids(fn, "ids", ids, T, dev)
    rows, to = _tensor(fn, "table", table, (V, d), dev), _tensor(fn, "out", out, (T, d), dev)
    _check(fn, load().twell_embed_forward(p, bits, _i32(T), rows, _i32(V), _i32(d), vdtype_of(table.dtype), scale, to,
                                          vdtype_of(out.dtype), _stream(stream, dev)))


def twell_embed_workspace_bytes(T: int, V: int, d: int) -> int:
    return int(load().twell_embed_workspace_bytes(_i32(T), _i32(V), _i32(d)))


def embed_workspace(T: int, V: int, d: int, device="cuda"):
    """A workspace tensor for twell_embed_backward with up to T tokens."""
    import torch
    return torch.empty(max(twell_embed_workspace_bytes(T, V, d), 256), dtype=torch.uint8, device=device)


def twell_embed_backward(ids, dout, dtable, workspace, scale: float = 1.0, accumulate: bool = False, stream=None):
    """dtable [V][d] = scale * the sums of dout's rows [T][d] by id, overwritten, or with accumulate added to."""
    fn = "twell_embed_backward"
    dev, (V, d), T = _device(fn, dtable), dtable.shape, ids.shape[0]
    p, bits = _ids(fn, "ids", ids, T, dev)
    rows, to = _tensor(fn, "dout", dout, (T, d), dev), _tensor(fn, "dtable", dtable, (V, d), dev)
    _check(fn, load().twell_embed_backward(p, bits, _i32(T), rows, vdtype_of(dout.dtype), _i32(V), _i32(d), scale,
                                           int(bool(accumulate)), to, vdtype_of(dtable.dtype),
                                           *_workspace(fn, workspace, dev), _stream(stream, dev)))


# ---------------------------------------------------------------- log probabilities
def _logits(fn: str, name: str, t, dev: int) -> tuple:
    """The pointer of logits [T][V] whose rows are contiguous, and the elements from one row to the next."""
    T, V = t.shape
    if t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr(), V
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {name} is on {t.device}, not on cuda:{dev}")
    ld = t.stride(0) if T > 1 else V
    if (V > 1 and t.stride(1) != 1) or ld < V:
        raise ValueError(f"{fn}: {name} must have contiguous rows that do not overlap")
    return t.data_ptr(), ld


def twell_logprob_workspace_bytes(T: int, V: int, k: int = 0) -> int:
    return int(load().twell_logprob_workspace_bytes(_i32(T), _i32(V), _i32(k)))


def logprob_workspace(T: int, V: int, k: int = 0, device="cuda"):
    """A workspace tensor for twell_logprob_forward with up to T rows, or None where none of these needs one."""
    import torch
    n = twell_logprob_workspace_bytes(T, V, k)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def twell_logprob_forward(logits, targets, logp, norm, workspace=None, scale: float = 1.0, entropy=None, top_logp=None,
                          top_idx=None, stream=None):
    """From logits [T][V] (rows may be strided) times scale: logp [T] of targets [T] (int32 or int64; both may be None),
    norm [T][2] (each row's largest logit, and the logarithm of the sum relative to it), entropy [T], and the k most
    likely tokens top_idx [T][k] (int32) with their top_logp [T][k]; float32, each may be None (see include/twell.h)."""
    import torch
    fn = "twell_logprob_forward"
    dev, (T, V) = _device(fn, logits), logits.shape
    z, ld = _logits(fn, "logits", logits, dev)
    if (logp is None) != (targets is None):
        raise ValueError(f"{fn}: targets and logp go together")
    if (top_logp is None) != (top_idx is None):
        raise ValueError(f"{fn}: top_logp and top_idx go together")
    ids, bits = (None, 32) if targets is None else _ids(fn, "targets", targets, T, dev)
    f32, row = torch.float32, (T,)
    k = 0 if top_idx is None else top_idx.shape[-1]
    a = None if logp is None else _tensor(fn, "logp", logp, row, dev, f32)
    b = None if norm is None else _tensor(fn, "norm", norm, (T, 2), dev, f32)
    c = None if entropy is None else _tensor(fn, "entropy", entropy, row, dev, f32)
    top = None if top_logp is None else _tensor(fn, "top_logp", top_logp, (T, k), dev, f32)
    idx = None if top_idx is None else _tensor(fn, "top_idx", top_idx, (T, k), dev, torch.int32)
    ws, size = _workspace(fn, workspace, dev)
    _check(fn, load().twell_logprob_forward(z, ld, _i32(T), _i32(V), vdtype_of(logits.dtype), scale, ids, bits, a, b, c, top,
                                            idx, _i32(k), ws, size, _stream(stream, dev)))


def twell_logprob_backward(logits, targets, norm, dlogp, dlogits, scale: float = 1.0, entropy=None, dentropy=None,
                           stream=None):
    """dlogits [T][V] (logits' type; may be logits) from the forward's norm, dlogp [T] (with targets) and dentropy [T]
    (with the forward's entropy), float32; one of the two may be None."""
    import torch
    fn = "twell_logprob_backward"
    dev, (T, V) = _device(fn, logits), logits.shape
    z, ld = _logits(fn, "logits", logits, dev)
    if dlogits.shape != logits.shape or dlogits.dtype is not logits.dtype:
        raise ValueError(f"{fn}: dlogits must have the logits' shape and type")
    dz, ldd = _logits(fn, "dlogits", dlogits, dev)
    if dlogp is not None and targets is None:
        raise ValueError(f"{fn}: dlogp without targets")
    if dentropy is not None and entropy is None:
        raise ValueError(f"{fn}: dentropy without the forward's entropy")
    ids, bits = (None, 32) if dlogp is None else _ids(fn, "targets", targets, T, dev)
    f32, row = torch.float32, (T,)
    n = _tensor(fn, "norm", norm, (T, 2), dev, f32)
    a = None if entropy is None else _tensor(fn, "entropy", entropy, row, dev, f32)
    b = None if dlogp is None else _tensor(fn, "dlogp", dlogp, row, dev, f32)
    c = None if dentropy is None else _tensor(fn, "dentropy", dentropy, row, dev, f32)
    _check(fn, load().twell_logprob_backward(z, ld, _i32(T), _i32(V), vdtype_of(logits.dtype), scale, ids, bits, n, a, b, c, dz,
                                             ldd, _stream(stream, dev)))


# ---------------------------------------------------------------- block norms
NORM_KINDS = {"rms": 0, "layer": 1}


class BlockNorm:
    """The norms around a block and their weights ([d] tensors of one type, or None for 1 and 0): the norm after the
    block (``post``; ``w_post``, ``b_post``), the residual scale ``alpha``, the norm before the next (``w_pre``,
    ``b_pre``).  ``kind``: "rms" or "layer"."""

    def __init__(self, kind="rms", eps=1e-6, alpha=1.0, post=False, w_post=None, b_post=None, w_pre=None, b_pre=None):
        if kind not in NORM_KINDS:
            raise ValueError(f"BlockNorm: kind {kind!r}: one of {', '.join(NORM_KINDS)}")
        self.kind, self.eps, self.alpha, self.post = kind, eps, alpha, post
        self.weights = {"w_post": w_post, "b_post": b_post, "w_pre": w_pre, "b_pre": b_pre}
        self._desc = TwellBlockNormT(kind=NORM_KINDS[kind], eps=eps, alpha=alpha, post=int(bool(post)), wdtype=TWELL_F32)
        self.d, self.dev, self._bound = None, None, []
        self._bind()

    def _bind(self):
        """Checks the weights and takes their addresses."""
        given = [(k, w) for k, w in self.weights.items() if w is not None]
        if not given:
            return
        first = given[0][1]
        dev = _device("BlockNorm", first)
        at = {k: _tensor("BlockNorm", k, w, first.shape, dev, first.dtype) for k, w in given}
        self._desc.wdtype = vdtype_of(first.dtype)
        for k, p in at.items():
            setattr(self._desc, k, p)
        self.d, self.dev = first.numel(), dev
        self._bound = [(w, w.data_ptr(), self.d, w.dtype) for _, w in given]

    def desc(self, fn, dev, rows, y, gate, gate_span) -> TwellBlockNormT:
        T, d = rows.shape
        for w, at, n, dtype in self._bound:
            # (its data may have been set anew)
            if w.data_ptr() != at or w.numel() != n or w.dtype is not dtype or not w.is_contiguous():
                self._bind()
                break
        if self.d is not None and (d != self.d or dev != self.dev):
            raise ValueError(f"{fn}: rows of {d} on cuda:{dev}, weights of {self.d} on cuda:{self.dev}")
        o = TwellBlockNormT.from_buffer_copy(self._desc)
        o.T, o.d, o.rdtype = _i32(T), _i32(d), vdtype_of(rows.dtype)
        if y is not None:
            _tensor(fn, "y", y, (T, d), dev)
            o.ydtype = vdtype_of(y.dtype)
        if gate is not None:
            if y is None:
                raise ValueError(f"{fn}: a gate without a block's y")
            if gate_span < 1:
                raise ValueError(f"{fn}: gate_span {gate_span}: a gate row serves at least one row")
            o.gate_span = _i32(gate_span)
            o.gate = _tensor(fn, "gate", gate, (-(-T // gate_span), d), dev, rows.dtype)
        return o


def twell_block_norm_forward(bn: BlockNorm, res, y, out, n, gate=None, gate_span: int = 0, stream=None):
    """out = res + alpha * gate * norm(y), n = norm(out); y, out, n may be None (see include/twell.h)."""
    fn = "twell_block_norm_forward"
    dev, shape = _device(fn, res), res.shape
    o = bn.desc(fn, dev, res, y, gate, gate_span)
    p_res = _tensor(fn, "res", res, shape, dev)
    p_out = None if out is None else _tensor(fn, "out", out, shape, dev, res.dtype)
    p_n = None
    if n is not None:
        p_n = _tensor(fn, "n", n, shape, dev)
        o.ndtype = vdtype_of(n.dtype)
    _check(fn, load().twell_block_norm_forward(o, p_res, _ptr(y), p_out, p_n, _stream(stream, dev)))


def twell_block_norm_workspace_bytes(T: int, d: int) -> int:
    return int(load().twell_block_norm_workspace_bytes(_i32(T), _i32(d)))


def block_norm_workspace(T: int, d: int, device="cuda"):
    """A workspace tensor for twell_block_norm_backward with up to T rows."""
    import torch
    return torch.empty(max(twell_block_norm_workspace_bytes(T, d), 256), dtype=torch.uint8, device=device)


def twell_block_norm_backward(bn: BlockNorm, out, y, dout, dn, dres, dy, workspace, gate=None, gate_span: int = 0,
                              dgate=None, dw_post=None, db_post=None, dw_pre=None, db_pre=None, stream=None):
    """The forward's gradients; out is the forward's out (its res without a block); y, dout, dn, dy and the weight
    gradients (float32 [d]) may be None (see include/twell.h)."""
    import torch
    fn = "twell_block_norm_backward"
    dev, shape, dt = _device(fn, dres), dres.shape, dres.dtype
    o = bn.desc(fn, dev, dres, y, gate, gate_span)
    if dy is not None and y is None:
        raise ValueError(f"{fn}: dy without a block's y")
    want = {"out": (out, dt), "dout": (dout, dt), "dn": (dn, None), "dy": (dy, None if y is None else y.dtype)}
    p = {k: None if t is None else _tensor(fn, k, t, shape, dev, w) for k, (t, w) in want.items()}
    p_dres = _tensor(fn, "dres", dres, shape, dev)
    p_dgate = None if dgate is None else _tensor(fn, "dgate", dgate, gate.shape if gate is not None else (), dev, dt)
    dw = [None if t is None else _tensor(fn, k, t, (shape[1],), dev, torch.float32)
          for k, t in (("dw_post", dw_post), ("db_post", db_post), ("dw_pre", dw_pre), ("db_pre", db_pre))]
    _check(fn, load().twell_block_norm_backward(o, p["out"], _ptr(y), p["dout"], p["dn"],
                                                TWELL_F32 if dn is None else vdtype_of(dn.dtype), p_dres, p["dy"],
                                                p_dgate, *dw, *_workspace(fn, workspace, dev), _stream(stream, dev)))


# ---------------------------------------------------------------- the optimizer
ADAMW_BLOCK = 256  # elements that share a scale of the 8-bit states


class AdamWTensors:
    """The tensors of one AdamW step, with their C descriptors.

    ``tensors`` is a list of dicts: ``p`` (float32 or bfloat16), ``grad``, ``m``,
    ``v``, and as needed ``copy`` (bfloat16, written with the updated p),
    ``weight_decay``, and for 8-bit states (``m``, ``v`` uint8) ``m_scale``,
    ``v_scale`` (float32, one per 256 elements) and, for ``twell_adamw_unpack``,
    ``m_values``, ``v_values`` (float32).  The tensors are contiguous and stay
    where they are while this object is in use (it keeps references to them);
    build another one when a gradient moves.  All have the same state format.
    """

    def __init__(self, tensors):
        import torch
        self.tensors = [dict(t) for t in tensors]
        for i, t in enumerate(self.tensors):
            for k in ("p", "grad", "m", "v"):
                if t.get(k) is None:
                    raise ValueError(f"AdamWTensors: tensor {i} has no {k!r}")
        self.desc = (TwellAdamWTensorT * max(len(self.tensors), 1))()
        self.state_bits = 8 if self.tensors and self.tensors[0]["m"].dtype == torch.uint8 else 32
        self.device = self.tensors[0]["p"].device if self.tensors else None
        if self.tensors:
            _device("AdamWTensors", self.tensors[0]["p"])
        self.can_unpack = self.state_bits == 8 and all(t.get("m_values") is not None and t.get("v_values") is not None
                                                       for t in self.tensors)
        state = torch.uint8 if self.state_bits == 8 else torch.float32
        for i, (o, t) in enumerate(zip(self.desc, self.tensors)):
            n = t["p"].numel()
            blocks = -(-n // ADAMW_BLOCK)
            want = {"p": (None, n), "grad": (None, n), "copy": (torch.bfloat16, n), "m": (state, n), "v": (state, n),
                    "m_scale": (torch.float32, blocks), "v_scale": (torch.float32, blocks),
                    "m_values": (torch.float32, n), "v_values": (torch.float32, n)}
            for k in ("m_scale", "v_scale") if self.state_bits == 8 else ():
                if t.get(k) is None:
                    raise ValueError(f"AdamWTensors: tensor {i} has no {k!r}")
            for k, (dtype, size) in want.items():
                x = t.get(k)
                if x is None:
                    continue
                if x.device != self.device:
                    raise ValueError(f"AdamWTensors: {k!r} of tensor {i} is on {x.device}, not on {self.device}")
                if not x.is_contiguous() or x.numel() != size:
                    raise ValueError(f"AdamWTensors: {k!r} of tensor {i} must be contiguous with {size} elements")
                if dtype is not None and x.dtype != dtype:
                    raise TypeError(f"AdamWTensors: {k!r} of tensor {i} must be {dtype}, not {x.dtype}")
                setattr(o, k, x.data_ptr())
            o.n = n
            o.weight_decay = float(t.get("weight_decay", 0.0))
            o.pdtype, o.gdtype = vdtype_of(t["p"].dtype), vdtype_of(t["grad"].dtype)


def twell_adamw_step(params: AdamWTensors, lr: float, beta1: float, beta2: float, eps: float, step: int, seed: int = 0,
                     grad_scale=None, stream=None):
    """One step; step counts from 1; grad_scale: a float32 tensor of one element on the GPU (0, inf or NaN in it:
    nothing changes); seed: of the 8-bit states' rounding, another one each step."""
    import torch
    fn, scale = "twell_adamw_step", None
    if params.tensors:
        dev = _device(fn, params.tensors[0]["p"])
        if grad_scale is not None:
            scale = _tensor(fn, "grad_scale", grad_scale.reshape(-1), (1,), dev, torch.float32)
    _check(fn, load().twell_adamw_step(params.desc, len(params.tensors), params.state_bits, lr, beta1, beta2, eps, step,
                                       seed & 0xFFFFFFFF, scale, _stream(stream)))


def twell_adamw_unpack(params: AdamWTensors, stream=None):
    """Writes the values of 8-bit states to m_values and v_values."""
    if not params.can_unpack:
        raise ValueError("twell_adamw_unpack: 8-bit states with m_values and v_values are needed")
    if params.tensors:
        _device("twell_adamw_unpack", params.tensors[0]["p"])
    _check("twell_adamw_unpack", load().twell_adamw_unpack(params.desc, len(params.tensors), _stream(stream)))
