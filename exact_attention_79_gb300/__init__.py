"""Exact attention for GB300 (sm_103a): Python binding of the C ABI in
include/fa.h.

This module only marshals arguments: every step of the forward and backward
runs in the CUDA library libfa_gb300.so, built in-tree by
`__graft_entry__.build()`. There is no fallback: if the library is missing or
the device is not sm_103, the calls raise.
"""
import ctypes
import os
from typing import NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_gb300.so")

FA_OK = 0
_STATUS_NAMES = {
    0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_ARCH",
    4: "FA_ERR_CUDA", 5: "FA_ERR_TIMEOUT", 6: "FA_ERR_WORKSPACE", 7: "FA_ERR_DEVICE",
}

# Every symbol include/fa.h declares, with its ctypes signature.
_VP, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_LL = ctypes.c_longlong
SIGNATURES = {
    "fa_fwd": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_fwd_f32": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_fwd_kv": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_fwd_pair": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_bwd_kv": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ,
                       _I, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_fwd_blocksparse": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _LL, _LL, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_bwd_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_bwd": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ,
                    _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_bwd_deterministic": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ,
                                  _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_bwd_blocksparse_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_bwd_blocksparse": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _LL, _LL,
                                _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_bwd_preprocess": (_I, [_VP, _VP, _VP, _VP, _SZ, _I, _I, _I, _I, _I, _VP]),
    "fa_bwd_dkdv": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_bwd_dq": (_I, [_VP, _VP, _SZ, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_bwd_noalloc": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_fp8_row_scales": (_SZ, [_I]),
    "fa_fp8_vt_keys": (_SZ, [_I]),
    "fa_fp8_quantize_rows": (_I, [_VP, _VP, _VP, _I, _I, _I, _VP]),
    "fa_fp8_quantize_v": (_I, [_VP, _VP, _VP, _I, _I, _I, _VP]),
    "fa_fwd_fp8": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_fwd_fp8_kv": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_fwd_packed": (_I, [_VP, _LL, _LL, _VP, _LL, _LL, _VP, _LL, _LL, _VP, _LL, _LL, _VP, _VP,
                           _I, _I, _I, _I, _I, _I, _F, _VP]),
    "fa_cache8_append": (_I, [_VP, _LL, _LL, _VP, _LL, _LL, _VP, _VP, _I, _I, _VP, _VP, _I, _VP]),
    "fa_cache8_append_rope": (_I, [_VP, _LL, _LL, _VP, _LL, _LL, _VP, _VP, _I, _I, _VP, _VP, _I, _VP, _VP, _LL, _VP]),
    "fa_rope": (_I, [_VP, _LL, _LL, _LL, _VP, _LL, _LL, _LL, _I, _VP, _LL, _LL, _LL, _VP, _LL, _LL, _LL, _I, _I, _I, _I, _I,
                     _VP, _VP, _LL, _LL, _I, _VP]),
    "fa_fwd_cache8_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "fa_fwd_cache8": (_I, [_VP, _VP, _VP, _I, _VP, _VP, _VP, _VP, _SZ, _I, _I, _I, _I, _F, _I, _F, _VP]),
    "fa_fwd_cache8_packed_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "fa_fwd_cache8_packed": (_I, [_VP, _LL, _LL, _VP, _VP, _I, _VP, _VP, _VP, _LL, _LL, _VP, _VP, _SZ, _I, _I, _I, _I, _F, _VP]),
    "fa_cache8_evict": (_I, [_VP, _VP, _I, _VP, _I, _I, _I, _VP, _I, _VP, _VP, _VP]),
    "fa_ex2_throughput": (_I, [ctypes.POINTER(ctypes.c_double), _VP]),
    "fa_sm_clock_mhz": (_I, [ctypes.POINTER(ctypes.c_double), _VP]),
    "fa_device_status": (_I, [_VP]),
    "fa_status_string": (ctypes.c_char_p, [_I]),
    "fa_version": (_I, []),
}

_lib = None


class FAError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        msg = _lib.fa_status_string(code).decode() if _lib is not None else ""
        super().__init__(f"{fn} returned {_STATUS_NAMES.get(code, code)}: {msg}")


def load(path=None):
    """Load the compiled library (once) and declare its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library not built: {p} (run __graft_entry__.build())")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(fn, code):
    if code != FA_OK:
        raise FAError(fn, code)


def _stream(t):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _shape(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be 4-D: [B, H, N, d]")
    B, Hq, N, d = q.shape
    return B, Hq, k.shape[1], N, d


def _index(device):
    """The index that tensors on a CUDA `device` report; one that none reports for others."""
    return device.index if device.type == "cuda" else -2


def _require(device, *specs):
    """Refuse, before any launch, a tensor the kernels would read or write past
    its end. specs: (tensor, name, dtype, shape). Every dtype and shape is
    checked before any placement (contiguous, CUDA, on the device of q), so
    the shape rules hold for CPU tensors too."""
    index = _index(device)
    for t, name, dtype, shape in specs:                 # all of it at once where nothing is wrong
        if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
            break
    else:
        return
    for t, name, dtype, shape in specs:
        if t.dtype != dtype or tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: expected {dtype} of shape {tuple(shape)}, "
                             f"got {t.dtype} of shape {tuple(t.shape)}")
    for t, name, _, _ in specs:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.get_device() != index:
            raise ValueError(f"{name} must be a CUDA tensor on {device}")


def _mask_args(block_mask, B, Hq, N, device):
    """Pointer and byte strides of a block mask tensor: uint8 or bool on the
    device, shape [B or 1, Hq or 1, T, T] with T = ceil(N / 128), the last two
    dimensions dense (a size-1 batch or head dimension broadcasts)."""
    import torch
    T = (N + 127) // 128
    if block_mask.dtype not in (torch.uint8, torch.bool) or block_mask.device != device:
        raise ValueError("block_mask must be a uint8 or bool tensor on the device of q")
    if block_mask.dim() != 4 or tuple(block_mask.shape[2:]) != (T, T) or block_mask.shape[0] not in (1, B) or \
            block_mask.shape[1] not in (1, Hq):
        raise ValueError(f"block_mask must be [B or 1, Hq or 1, {T}, {T}]")
    if block_mask.stride(3) != 1 or block_mask.stride(2) != T:
        raise ValueError("the last two dimensions of block_mask must be dense")
    sb = 0 if block_mask.shape[0] == 1 else block_mask.stride(0)
    sh = 0 if block_mask.shape[1] == 1 else block_mask.stride(1)
    return _ptr(block_mask), sb, sh


def fwd(q, k, v, causal=False, scale=None, out=None, lse=None, block_mask=None):
    """O, LSE = attention(q, k, v) on the current stream.

    q: [B, Hq, N, d]; k, v: [B, Hkv, N, d]; bf16 (fa_fwd) or fp32 (fa_fwd_f32)
    contiguous CUDA tensors. block_mask (bf16 only): uint8/bool
    [B or 1, Hq or 1, T, T], T = ceil(N/128), nonzero where query tile i may
    see key tile j (fa_fwd_blocksparse). k and v may hold another number of
    positions Nk than q (bf16, fa_fwd_kv: the queries are the last N of Nk
    positions for the causal rule). Returns (o like q, lse fp32 [B, Hq, N])."""
    import torch
    lib = load()
    B, Hq, Hkv, N, d = _shape(q, k)
    if scale is None:
        scale = d ** -0.5
    Nk = k.shape[2]
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("q, k, v must be bf16 or fp32")
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _require(q.device, (q, "q", q.dtype, (B, Hq, N, d)), (k, "k", q.dtype, (B, Hkv, Nk, d)),
             (v, "v", q.dtype, (B, Hkv, Nk, d)), (o, "out", q.dtype, (B, Hq, N, d)),
             (lse, "lse", torch.float32, (B, Hq, N)))
    if Nk != N:
        if q.dtype != torch.bfloat16 or block_mask is not None:
            raise ValueError("keys of another length need bf16 inputs and no block mask")
        _check("fa_fwd_kv", lib.fa_fwd_kv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, Nk, d,
                                          int(bool(causal)), float(scale), _stream(q)))
        return o, lse
    if block_mask is not None:
        if q.dtype != torch.bfloat16:
            raise ValueError("block masks need bf16 inputs")
        mp, sb, sh = _mask_args(block_mask, B, Hq, N, q.device)
        _check("fa_fwd_blocksparse", lib.fa_fwd_blocksparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), mp, sb, sh,
                                                            B, Hq, Hkv, N, d, int(bool(causal)), float(scale),
                                                            _stream(q)))
        return o, lse
    fn = {torch.bfloat16: "fa_fwd", torch.float32: "fa_fwd_f32"}.get(q.dtype)
    if fn is None:
        raise ValueError("dtype must be bfloat16 or float32")
    _check(fn, getattr(lib, fn)(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                B, Hq, Hkv, N, d, int(bool(causal)), float(scale), _stream(q)))
    return o, lse


def quantize_fp8(q, k, v):
    """Block-scaled e4m3 copies of bf16 q [B, Hq, N, d], k and v [B, Hkv, Nk, d] (fa_fp8_quantize_rows,
    fa_fp8_quantize_v): returns (q8, q_scale, k8, k_scale, vt8, v_scale) with
    q8, k8 uint8 [B, H, N, d], scales fp32 [B, H, ceil(N/64)], vt8 uint8
    [B, Hkv, d, NP] (V transposed, NP = N rounded up to 128) and v_scale
    fp32 [B, Hkv, d]."""
    import torch
    lib = load()
    B, Hq, Hkv, N, d = _shape(q, k)
    Nk = k.shape[2]
    bf16 = torch.bfloat16
    _require(q.device, (q, "q", bf16, (B, Hq, N, d)), (k, "k", bf16, (B, Hkv, Nk, d)), (v, "v", bf16, (B, Hkv, Nk, d)))
    nb, nbk, NP = int(lib.fa_fp8_row_scales(N)), int(lib.fa_fp8_row_scales(Nk)), int(lib.fa_fp8_vt_keys(Nk))
    dev = q.device
    q8 = torch.empty(q.shape, dtype=torch.uint8, device=dev)
    k8 = torch.empty(k.shape, dtype=torch.uint8, device=dev)
    vt8 = torch.empty((B, Hkv, d, NP), dtype=torch.uint8, device=dev)
    qs = torch.empty((B, Hq, nb), dtype=torch.float32, device=dev)
    ks = torch.empty((B, Hkv, nbk), dtype=torch.float32, device=dev)
    vs = torch.empty((B, Hkv, d), dtype=torch.float32, device=dev)
    st = _stream(q)
    _check("fa_fp8_quantize_rows", lib.fa_fp8_quantize_rows(_ptr(q), _ptr(q8), _ptr(qs), B * Hq, N, d, st))
    _check("fa_fp8_quantize_rows", lib.fa_fp8_quantize_rows(_ptr(k), _ptr(k8), _ptr(ks), B * Hkv, Nk, d, st))
    _check("fa_fp8_quantize_v", lib.fa_fp8_quantize_v(_ptr(v), _ptr(vt8), _ptr(vs), B * Hkv, Nk, d, st))
    return q8, qs, k8, ks, vt8, vs


def fwd_fp8(q8, q_scale, k8, k_scale, vt8, v_scale, causal=False, scale=None, out=None, lse=None):
    """O (bf16), LSE = attention of block-scaled e4m3 inputs (fa_fwd_fp8), as
    returned by quantize_fp8."""
    import torch
    lib = load()
    B, Hq, Hkv, N, d = _shape(q8, k8)
    Nk = k8.shape[2]
    dev = q8.device
    if scale is None:
        scale = d ** -0.5
    o = torch.empty((B, Hq, N, d), dtype=torch.bfloat16, device=dev) if out is None else out
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=dev) if lse is None else lse
    f32, u8 = torch.float32, torch.uint8
    _require(dev, (q8, "q8", u8, (B, Hq, N, d)), (q_scale, "q_scale", f32, (B, Hq, int(lib.fa_fp8_row_scales(N)))),
             (k8, "k8", u8, (B, Hkv, Nk, d)), (k_scale, "k_scale", f32, (B, Hkv, int(lib.fa_fp8_row_scales(Nk)))),
             (vt8, "vt8", u8, (B, Hkv, d, int(lib.fa_fp8_vt_keys(Nk)))), (v_scale, "v_scale", f32, (B, Hkv, d)),
             (o, "out", torch.bfloat16, (B, Hq, N, d)), (lse, "lse", f32, (B, Hq, N)))
    if Nk != N:
        # queries are the last N of Nk positions (fa_fwd_fp8_kv)
        _check("fa_fwd_fp8_kv", lib.fa_fwd_fp8_kv(_ptr(q8), _ptr(q_scale), _ptr(k8), _ptr(k_scale), _ptr(vt8),
                                                  _ptr(v_scale), _ptr(o), _ptr(lse), B, Hq, Hkv, N, Nk, d,
                                                  int(bool(causal)), float(scale), _stream(q8)))
        return o, lse
    _check("fa_fwd_fp8", lib.fa_fwd_fp8(_ptr(q8), _ptr(q_scale), _ptr(k8), _ptr(k_scale), _ptr(vt8), _ptr(v_scale),
                                        _ptr(o), _ptr(lse), B, Hq, Hkv, N, d, int(bool(causal)), float(scale),
                                        _stream(q8)))
    return o, lse


def bwd_workspace_bytes(B, Hq, Hkv, N, d):
    return int(load().fa_bwd_workspace_bytes(B, Hq, Hkv, N, d))


def bwd(q, k, v, o, lse, do, causal=False, scale=None, workspace=None, dq=None, dk=None, dv=None,
        deterministic=False, block_mask=None):
    """dQ, dK, dV of <O, dO> on the current stream (bf16 tensors, fp32 lse).

    deterministic=True runs fa_bwd_deterministic (bit-reproducible, slower);
    block_mask (as in fwd) runs fa_bwd_blocksparse."""
    import torch
    lib = load()
    B, Hq, Hkv, N, d = _shape(q, k)
    if scale is None:
        scale = d ** -0.5
    Nk = k.shape[2]
    dev = q.device
    bf16 = torch.bfloat16
    if block_mask is not None and deterministic:
        raise ValueError("the deterministic backward has no block-sparse form")
    if Nk != N and (deterministic or block_mask is not None):
        raise ValueError("keys of another length: only the default backward")
    nbytes = (int(lib.fa_bwd_blocksparse_workspace_bytes(B, Hq, Hkv, N, d)) if block_mask is not None
              else bwd_workspace_bytes(B, Hq, Hkv, N, d))
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    # the workspace's byte count is passed on; the library refuses one that is too small
    _require(dev, (q, "q", bf16, (B, Hq, N, d)), (k, "k", bf16, (B, Hkv, Nk, d)), (v, "v", bf16, (B, Hkv, Nk, d)),
             (o, "o", bf16, (B, Hq, N, d)), (lse, "lse", torch.float32, (B, Hq, N)), (do, "do", bf16, (B, Hq, N, d)),
             (workspace, "workspace", torch.uint8, (workspace.numel(),)), (dq, "dq", bf16, (B, Hq, N, d)),
             (dk, "dk", bf16, (B, Hkv, Nk, d)), (dv, "dv", bf16, (B, Hkv, Nk, d)))
    if Nk != N:
        _check("fa_bwd_kv", lib.fa_bwd_kv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
                                          _ptr(dv), _ptr(workspace), workspace.numel(), B, Hq, Hkv, N, Nk, d,
                                          int(bool(causal)), float(scale), _stream(q)))
        return dq, dk, dv
    if block_mask is not None:
        mp, sb, sh = _mask_args(block_mask, B, Hq, N, q.device)
        _check("fa_bwd_blocksparse", lib.fa_bwd_blocksparse(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
            _ptr(workspace), workspace.numel(), mp, sb, sh, B, Hq, Hkv, N, d, int(bool(causal)), float(scale),
            _stream(q)))
        return dq, dk, dv
    name = "fa_bwd_deterministic" if deterministic else "fa_bwd"
    _check(name, getattr(lib, name)(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                                    _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel(),
                                    B, Hq, Hkv, N, d, int(bool(causal)), float(scale), _stream(q)))
    return dq, dk, dv


class Rope(NamedTuple):
    """A rotation by positions (fa_rope_plan). turns: int64 [pairs], each pair's frequency / 2 pi in units of 2^-64,
    modulo 2^64; axis: int32 [pairs], which row of the positions a pair goes by, or None (the first); interleaved: pair i
    is columns (2 i, 2 i + 1), otherwise (i, i + pairs). CUDA tensors; `new_rope` makes them."""
    turns: "torch.Tensor"       # noqa: F821
    axis: "torch.Tensor" = None     # noqa: F821
    interleaved: bool = False


class _Rope(ctypes.Structure):
    _fields_ = [("turns", _VP), ("axis", _VP), ("pairs", _I), ("axes", _I), ("interleaved", _I)]


def new_rope(freqs, axis=None, interleaved=False, device="cuda"):
    """A Rope of the frequencies `freqs` (radians per position, one per pair, a multiple of 4 of them), pair i going by
    axis[i] of the positions (None: all by one)."""
    from fractions import Fraction
    import torch
    # in whole numbers: a double's 2^-53 of a turn, times a position of 2^31, would show
    two_pi = Fraction(628318530717958647692528676655900576839433879875021, 10 ** 50)
    turns = [round(Fraction(float(f)) / two_pi * 2 ** 64) % 2 ** 64 for f in freqs]
    turns = torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in turns], dtype=torch.int64, device=device)
    if axis is not None:
        axis = torch.tensor([int(a) for a in axis], dtype=torch.int32, device=device)
    return Rope(turns, axis, bool(interleaved))


def _rope_specs(rope, axes):
    """The plan's tensors as _require takes them and its C form."""
    import torch
    turns, axis, interleaved = rope
    pairs = turns.numel()
    specs = [(turns, "rope.turns", torch.int64, (pairs,))]
    if axis is not None:
        specs.append((axis, "rope.axis", torch.int32, (pairs,)))
    return specs, _Rope(turns.data_ptr(), None if axis is None else axis.data_ptr(), pairs, axes, 1 if interleaved else 0)


def _rope_strides(x, name, shape, dtype, unit):
    """Batch, head and token strides of a [B, H, T, d] (or [H, T, d]) tensor whose rows of d values are contiguous and
    16-byte (`unit` values) aligned. A dimension of size 1 gets a stride that nothing reads through."""
    if x.dtype is not dtype or x.shape != shape:
        raise ValueError(f"{name}: expected {dtype} of shape {tuple(shape)}, got {x.dtype} of shape {tuple(x.shape)}")
    if len(shape) == 4:
        sb, sh, st, sd = x.stride()
    else:
        sb, (sh, st, sd) = 0, x.stride()
    if sd == 1 and not (sb | sh | st) & (unit - 1):
        return sb, sh, st
    *outer, H, T, d = shape
    sb = sb if outer and outer[0] > 1 else 0
    sh, st = (sh if H > 1 else d), (st if T > 1 else d)
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if sb % unit or sh % unit or st % unit:
        raise ValueError(f"{name}: strides other than the last must be multiples of {unit}")
    return sb, sh, st


def _rope_positions(positions, B, T, batched, one_axis):
    """Axes and the strides between them and between batches of int32 positions [axes, B, T], with the batch's dimension
    or without it, with the axes' or (one axis) without it."""
    import torch
    shape = positions.shape
    n = len(shape)
    if positions.dtype is not torch.int32 or not 1 <= n <= (3 if batched else 2) or shape[-1] != T or \
            (T > 1 and positions.stride(-1) != 1):
        raise ValueError("positions must be int32 [axes, B, T], [axes, T] or [T], the last dimension contiguous")
    if n == 1:
        return 1, 0, 0
    if n == 3:
        if shape[1] != B:
            raise ValueError("positions must be [axes, B, T]")
        return shape[0], positions.stride(0), positions.stride(1)
    if batched and shape[0] == B and one_axis:
        return 1, 0, positions.stride(0)                            # [B, T]
    return shape[0], positions.stride(0), 0


def rope(q, k, rope, positions, inverse=False, q_out=None, k_out=None):
    """Q and K turned by their positions (fa_rope), on the current stream; inverse=True: turned back, which takes the
    gradients of the results to those of q and k.

    q: [B, Hq, T, d] or [Hq, T, d], bf16 or fp32, any strides that are multiples of 16 bytes (a projection's
    [B, T, H, d].transpose(1, 2) too); k: the same with its own heads, or None. positions: int32, [axes, B, T] (3-D q:
    [axes, T]); the batch may be left out where all share them, and the axes where the Rope names none. q_out, k_out: where
    the results go, in any such layout (q_out may be q itself and k_out k itself, and they are otherwise apart from both);
    without them tensors laid out like q and k. Returns (q_out, k_out), k_out None without k."""
    import torch
    shape, dtype, dev = q.shape, q.dtype, q.device
    batched = len(shape) == 4
    if batched:
        B, Hq, T, d = shape
    elif len(shape) == 3:
        B, (Hq, T, d) = 1, shape
    else:
        raise ValueError("q must be [B, H, T, d] or [H, T, d]")
    if dtype is torch.bfloat16:
        size, unit = 2, 8
    elif dtype is torch.float32:
        size, unit = 4, 4
    else:
        raise ValueError("q and k must be bf16 or fp32")
    axes, sa, sb = _rope_positions(positions, B, T, batched, rope.axis is None)
    specs, plan = _rope_specs(rope, axes)
    placed = [(positions, "positions")]
    q_os = qs = _rope_strides(q, "q", shape, dtype, unit)
    if q_out is not None:
        q_os = _rope_strides(q_out, "q_out", shape, dtype, unit)
        placed.append((q_out, "q_out"))
    if k is not None:
        k_shape = k.shape
        if len(k_shape) != len(shape):
            raise ValueError("k must have as many dimensions as q")
        Hkv = k_shape[-3]
        if k_shape[-1] != d or k_shape[-2] != T or k_shape[0] != (B if batched else Hkv):
            raise ValueError(f"k: expected {(B, Hkv, T, d) if batched else (Hkv, T, d)}, got {tuple(k_shape)}")
        k_os = ks = _rope_strides(k, "k", k_shape, dtype, unit)
        placed.append((k, "k"))
        if k_out is not None:
            k_os = _rope_strides(k_out, "k_out", k_shape, dtype, unit)
            placed.append((k_out, "k_out"))
    elif k_out is not None:
        raise ValueError("k_out without k")
    _require(dev, *specs)
    _placed(dev, *placed)
    if q_out is None:
        q_out = torch.empty_like(q)
        if q_out.stride() != q.stride():                # (what is cut out of something wider is laid out anew)
            q_os = _rope_strides(q_out, "q_out", shape, dtype, unit)
    if k is not None and k_out is None:
        k_out = torch.empty_like(k)
        if k_out.stride() != k.stride():
            k_os = _rope_strides(k_out, "k_out", k_shape, dtype, unit)
    if T == 0 or B == 0:
        return q_out, k_out
    k_args = (None, 0, 0, 0, None, 0, 0, 0, 0) if k is None else (k.data_ptr(), *ks, k_out.data_ptr(), *k_os, Hkv)
    _call_on(dev, "fa_rope", q.data_ptr(), *qs, q_out.data_ptr(), *q_os, Hq, *k_args, B, T, d, size, ctypes.byref(plan),
             positions.data_ptr(), sa, sb, 1 if inverse else 0)
    return q_out, k_out


CACHE8_BLOCK = 64       # tokens per cache block (FA_CACHE8_BLOCK)


class Cache8(NamedTuple):
    """An 8-bit cache of keys and values (fa_cache8): a pool of blocks of 64 tokens, shared by sequences whose block
    tables (int32 [B, max_blocks]) say which blocks they have. k, v: uint8 e4m3 codes [num_blocks, Hkv, 64, d];
    k_scale, v_scale: fp32 [num_blocks, Hkv]; weight: fp32 [num_blocks, Hkv, 64] accumulated attention weight, or
    None. Contiguous CUDA tensors on one device; nothing else is kept."""
    k: "torch.Tensor"           # noqa: F821
    v: "torch.Tensor"           # noqa: F821
    k_scale: "torch.Tensor"     # noqa: F821
    v_scale: "torch.Tensor"     # noqa: F821
    weight: "torch.Tensor" = None   # noqa: F821


class _Cache8(ctypes.Structure):
    _fields_ = [("k", _VP), ("v", _VP), ("k_scale", _VP), ("v_scale", _VP), ("weight", _VP),
                ("num_blocks", _I), ("Hkv", _I), ("d", _I)]


def new_cache8(num_blocks, Hkv, d, device="cuda", weight=False):
    """An empty Cache8 on `device`, with accumulated weights or without."""
    import torch
    codes = [torch.zeros(num_blocks, Hkv, CACHE8_BLOCK, d, dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.ones(num_blocks, Hkv, dtype=torch.float32, device=device) for _ in range(2)]
    w = torch.zeros(num_blocks, Hkv, CACHE8_BLOCK, dtype=torch.float32, device=device) if weight else None
    return Cache8(*codes, *scales, w)


def _cache8_specs(cache):
    """The cache's tensors as _require takes them, its C form and (num_blocks, Hkv, d)."""
    import torch
    k, v, k_scale, v_scale, weight = cache
    shape = k.shape
    if len(shape) != 4 or shape[2] != CACHE8_BLOCK:
        raise ValueError(f"cache.k must be [num_blocks, Hkv, {CACHE8_BLOCK}, d]")
    nb, Hkv, _, d = shape
    f32, u8 = torch.float32, torch.uint8
    specs = [(k, "cache.k", u8, shape), (v, "cache.v", u8, shape), (k_scale, "cache.k_scale", f32, (nb, Hkv)),
             (v_scale, "cache.v_scale", f32, (nb, Hkv))]
    if weight is not None:
        specs.append((weight, "cache.weight", f32, (nb, Hkv, CACHE8_BLOCK)))
    c = _Cache8(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                None if weight is None else weight.data_ptr(), nb, Hkv, d)
    return specs, c, (nb, Hkv, d)


def _table_spec(block_table, name="block_table", B=None):
    import torch
    if block_table.dim() != 2 or (B is not None and block_table.shape[0] != B):
        raise ValueError(f"{name} must be [B, max_blocks]")
    return block_table, name, torch.int32, block_table.shape


def _call_on(device, name, *args):
    """A library call on `device`'s current stream, with that device current."""
    import torch
    fn = getattr(load(), name)
    stream = torch._C._cuda_getCurrentRawStream(device.index)      # current_stream() without its Stream object
    if device.index == torch._C._cuda_getDevice():
        code = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, stream)
    if code:
        _check(name, code)


def _heads_strides(t, name, H, T, d):
    """Strides (between heads, between tokens) of a bf16 [H, T, d] tensor whose rows of d values are contiguous
    and 16-byte aligned: [H, T, d] itself, or [T, H, d].transpose(0, 1). A dimension of size 1 gets a stride that
    nothing reads through."""
    import torch
    if t.dtype != torch.bfloat16 or t.shape != (H, T, d):
        raise ValueError(f"{name}: expected {torch.bfloat16} of shape {(H, T, d)}, got {t.dtype} of shape {tuple(t.shape)}")
    sh, st, sd = t.stride()
    sh, st = (sh if H > 1 else d), (st if T > 1 else d)
    if (sd != 1 and d > 1) or sh % 8 or st % 8:
        raise ValueError(f"{name}: the last dimension must be contiguous and the other strides multiples of 8")
    return sh, st


def _placed(device, *named):
    index = _index(device)
    for t, name in named:
        if t.get_device() != index:
            raise ValueError(f"{name} must be a CUDA tensor on {device}")


def fwd_packed(q, k, v, cu_seqlens, causal=True, scale=None, out=None, lse=None):
    """O, LSE of S packed sequences of different lengths, each attending to itself (fa_fwd_packed), on the current
    stream.

    q: bf16 [Hq, T, d]; k, v: [Hkv, T, d]; each [H, T, d] or a [T, H, d] tensor's .transpose(0, 1). cu_seqlens: int32
    [S + 1] on the device; sequence s has rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1. Returns (o with q's layout, lse
    fp32 [Hq, T]); rows of no sequence are left as they were (unset in new tensors)."""
    import torch
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be 3-D: [H, T, d]")
    Hq, T, d = q.shape
    Hkv, dev = k.shape[0], q.device
    if scale is None:
        scale = d ** -0.5
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [S + 1]")
    S = cu_seqlens.shape[0] - 1
    specs = [(cu_seqlens, "cu_seqlens", torch.int32, (S + 1,))]
    strides = [*_heads_strides(q, "q", Hq, T, d), *_heads_strides(k, "k", Hkv, T, d), *_heads_strides(v, "v", Hkv, T, d)]
    placed = [(k, "k"), (v, "v")]
    if out is not None:
        _heads_strides(out, "out", Hq, T, d)
        placed.append((out, "out"))
    if lse is not None:
        specs.append((lse, "lse", torch.float32, (Hq, T)))
    _require(dev, *specs)
    _placed(dev, *placed)
    o = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
    if T == 0 or S == 0:
        return o, lse
    q_h, q_t, k_h, k_t, v_h, v_t = strides
    _call_on(dev, "fa_fwd_packed", q.data_ptr(), q_h, q_t, k.data_ptr(), k_h, k_t, v.data_ptr(), v_h, v_t, o.data_ptr(),
             *_heads_strides(o, "out", Hq, T, d), lse.data_ptr(), cu_seqlens.data_ptr(), S, T, Hq, Hkv, d, int(bool(causal)),
             float(scale))
    return o, lse


def cache8_append(cache, k, v, cu_seqlens, block_table, start, rope=None, positions=None):
    """Append tokens to the sequences of an 8-bit cache (fa_cache8_append), in place on the current stream.

    k, v: bf16 [Hkv, T, d] (strided: [T, Hkv, d].transpose(0, 1) as well), the new tokens of all sequences one behind
    the other; sequence b's are cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (int32 [B + 1]) and become its positions from
    start[b] (int32 [B]) on. One token each: cu_seqlens = 0, 1, ..., B.
    rope (a Rope): K is turned by its positions on the way (fa_cache8_append_rope); positions: int32 [axes, T] or [T], None:
    each token's position in its sequence."""
    import torch
    specs, c, (_, Hkv, d) = _cache8_specs(cache)
    if k.dim() != 3:
        raise ValueError("k must be [Hkv, T, d]")
    T, dev = k.shape[1], k.device
    B = block_table.shape[0]
    i32 = torch.int32
    ks, vs = _heads_strides(k, "k", Hkv, T, d), _heads_strides(v, "v", Hkv, T, d)
    if positions is not None:
        if rope is None:
            raise ValueError("positions without rope")
        n = positions.dim()
        if positions.dtype != i32 or n not in (1, 2) or positions.shape[-1] != T or (T > 1 and positions.stride(-1) != 1):
            raise ValueError("positions must be int32 [axes, T] or [T], the last dimension contiguous")
        axes, sa = (positions.shape[0], positions.stride(0)) if n == 2 else (1, 0)
    else:
        axes, sa = 1, 0
    if rope is not None:
        more, plan = _rope_specs(rope, axes)
        specs += more
    _require(dev, *specs, (cu_seqlens, "cu_seqlens", i32, (B + 1,)), _table_spec(block_table), (start, "start", i32, (B,)))
    _placed(dev, (k, "k"), (v, "v"), *([] if positions is None else [(positions, "positions")]))
    if T == 0:
        return
    args = (k.data_ptr(), *ks, v.data_ptr(), *vs, cu_seqlens.data_ptr(), start.data_ptr(), B, T, ctypes.byref(c),
            block_table.data_ptr(), block_table.shape[1])
    if rope is None:
        _call_on(dev, "fa_cache8_append", *args)
    else:
        _call_on(dev, "fa_cache8_append_rope", *args, ctypes.byref(plan), None if positions is None else positions.data_ptr(), sa)


def fwd_cache8(q, cache, block_table, lengths, causal=True, scale=None, out=None, lse=None, workspace=None,
               weight_decay=None):
    """O, LSE of the last Nq positions of each sequence over an 8-bit cache (fa_fwd_cache8), on the current stream.

    q: bf16 [B, Hq, Nq, d]; lengths: int32 [B], tokens held with the Nq new ones among them; (Hq / Hkv) * Nq <= 128.
    weight_decay (a number): cache.weight = weight_decay * cache.weight + each token's summed probabilities as well.
    Returns (o like q, lse fp32 [B, Hq, Nq])."""
    import torch
    lib = load()
    if q.dim() != 4:
        raise ValueError("q must be [B, Hq, Nq, d]")
    specs, c, (_, Hkv, d) = _cache8_specs(cache)
    B, Hq, Nq, _ = q.shape
    dev, bf16 = q.device, torch.bfloat16
    if weight_decay is not None and cache.weight is None:
        raise ValueError("weight_decay needs a cache with weights")
    if scale is None:
        scale = d ** -0.5
    specs += [(q, "q", bf16, (B, Hq, Nq, d)), _table_spec(block_table, B=B), (lengths, "lengths", torch.int32, (B,))]
    if out is not None:
        specs.append((out, "out", bf16, (B, Hq, Nq, d)))
    if lse is not None:
        specs.append((lse, "lse", torch.float32, (B, Hq, Nq)))
    if workspace is not None:
        specs.append((workspace, "workspace", torch.uint8, (workspace.numel(),)))
    _require(dev, *specs)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev)
    max_blocks, weigh = block_table.shape[1], int(weight_decay is not None)
    n = lib.fa_fwd_cache8_workspace_bytes(B, Hq, Hkv, Nq, d, max_blocks, weigh) if workspace is None else workspace.numel()
    if workspace is None and n > 256:                   # 256: none is needed
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    _call_on(dev, "fa_fwd_cache8", q.data_ptr(), ctypes.byref(c), block_table.data_ptr(), max_blocks, lengths.data_ptr(),
             out.data_ptr(), lse.data_ptr(), None if workspace is None else workspace.data_ptr(), n, B, Hq, Nq,
             int(bool(causal)), float(scale), weigh, float(weight_decay or 0.0))
    return out, lse


def fwd_cache8_packed(q, cache, cu_seqlens, block_table, lengths, causal=True, scale=None, out=None, lse=None, workspace=None):
    """O, LSE of chunks of new tokens of B sequences over an 8-bit cache that holds them already (fa_fwd_cache8_packed), on
    the current stream.

    q: bf16 [Hq, T, d] or a [T, Hq, d] tensor's .transpose(0, 1), the chunks one behind the other; sequence b's are rows
    cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (int32 [B + 1]) and the last of its lengths[b] tokens (int32 [B]). Returns (o with
    q's layout, lse fp32 [Hq, T]); rows of no sequence are left as they were (unset in new tensors). workspace: uint8, of
    fa_fwd_cache8_packed_workspace_bytes (about 40 MB); made by the call otherwise. Adds no attention weights: cache8_evict
    ranks tokens that only this call has looked at as equals."""
    import torch
    lib = load()
    if q.dim() != 3:
        raise ValueError("q must be [Hq, T, d]")
    specs, c, (_, Hkv, d) = _cache8_specs(cache)
    Hq, T, _ = q.shape
    B, dev = block_table.shape[0], q.device
    if scale is None:
        scale = d ** -0.5
    qs = _heads_strides(q, "q", Hq, T, d)
    i32 = torch.int32
    specs += [_table_spec(block_table), (cu_seqlens, "cu_seqlens", i32, (B + 1,)), (lengths, "lengths", i32, (B,))]
    os = qs
    if out is not None:
        os = _heads_strides(out, "out", Hq, T, d)
    if lse is not None:
        specs.append((lse, "lse", torch.float32, (Hq, T)))
    if workspace is not None:
        specs.append((workspace, "workspace", torch.uint8, (workspace.numel(),)))
    _require(dev, *specs)
    if out is not None:
        _placed(dev, (out, "out"))
    else:
        out = torch.empty_like(q)
        if out.stride() != q.stride():                  # (what is cut out of something wider is laid out anew)
            os = _heads_strides(out, "out", Hq, T, d)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
    if T == 0 or B == 0:
        return out, lse
    max_blocks = block_table.shape[1]
    n = lib.fa_fwd_cache8_packed_workspace_bytes(B, T, Hq, Hkv, d, max_blocks) if workspace is None else workspace.numel()
    if workspace is None and n > 256:                   # 256: none is needed
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    _call_on(dev, "fa_fwd_cache8_packed", q.data_ptr(), *qs, ctypes.byref(c), block_table.data_ptr(), max_blocks,
             cu_seqlens.data_ptr(), lengths.data_ptr(), out.data_ptr(), *os, lse.data_ptr(),
             None if workspace is None else workspace.data_ptr(), n, B, T, Hq, int(bool(causal)), float(scale))
    return out, lse


def cache8_evict(cache, block_table, lengths, keep, recent, to_table, new_lengths=None, kept=None):
    """Cut sequences of an 8-bit cache to at most `keep` tokens per KV head (fa_cache8_evict), on the current stream:
    the last `recent` and, of the others, those with the largest accumulated weight. They go, in their order, to the
    blocks of to_table (int32 [B, to_blocks], 64 * to_blocks >= keep), none of which the sequences may hold already.
    Returns (new_lengths int32 [B], kept int32 [B, Hkv, keep]: positions before, -1 past the new length)."""
    import torch
    specs, c, (_, Hkv, d) = _cache8_specs(cache)
    if cache.weight is None:
        raise ValueError("eviction needs a cache with weights")
    B, dev, i32 = block_table.shape[0], cache.k.device, torch.int32
    specs += [_table_spec(block_table), _table_spec(to_table, "to_table", B), (lengths, "lengths", i32, (B,))]
    if new_lengths is not None:
        specs.append((new_lengths, "new_lengths", i32, (B,)))
    if kept is not None:
        specs.append((kept, "kept", i32, (B, Hkv, keep)))
    _require(dev, *specs)
    if new_lengths is None:
        new_lengths = torch.empty(B, dtype=i32, device=dev)
    if kept is None:
        kept = torch.empty((B, Hkv, max(keep, 0)), dtype=i32, device=dev)
    _call_on(dev, "fa_cache8_evict", ctypes.byref(c), block_table.data_ptr(), block_table.shape[1], lengths.data_ptr(), B,
             keep, recent, to_table.data_ptr(), to_table.shape[1], kept.data_ptr(), new_lengths.data_ptr())
    return new_lengths, kept


def ex2_throughput(stream=None):
    """ex2 results per SM clock cycle on the current device (fa_ex2_throughput):
    the rate behind the forward's exponential ceiling."""
    import torch
    s = ctypes.c_void_p(stream if stream is not None else torch.cuda.current_stream().cuda_stream)
    out = ctypes.c_double(0.0)
    _check("fa_ex2_throughput", load().fa_ex2_throughput(ctypes.byref(out), s))
    return out.value


def sm_clock_mhz(stream=None):
    """Mean SM clock (MHz) of the forward and dK/dV kernels since the last
    call, measured by the kernels (fa_sm_clock_mhz); 0.0 if none ran."""
    import torch
    s = ctypes.c_void_p(stream if stream is not None else torch.cuda.current_stream().cuda_stream)
    out = ctypes.c_double(0.0)
    _check("fa_sm_clock_mhz", load().fa_sm_clock_mhz(ctypes.byref(out), s))
    return out.value


def check_device_status(stream=None):
    """Synchronise the stream and raise if a kernel's bounded wait ran out."""
    import torch
    s = ctypes.c_void_p(stream if stream is not None else torch.cuda.current_stream().cuda_stream)
    _check("fa_device_status", load().fa_device_status(s))
