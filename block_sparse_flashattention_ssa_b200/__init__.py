"""BLASST skip-softmax attention for B200 (sm_100a): Python binding.

Argument marshalling over the C ABI declared in ``include/ssa.h`` and
implemented in ``libssa.so`` (built in-tree by ``build.py``). Every step of
the computation runs in the library's CUDA kernels; torch only provides
device memory and streams. There is no CPU fallback: importing this package
fails loudly when the library is missing.

Entry points (same names as the C ABI, without the ``ssa_`` prefix):
  fwd          skip-softmax attention forward (optionally with per-tile
               diagnostics, the ``ssa_fwd_ex`` call)
  fwd_fp8      the forward with E4M3 Q and K, or Q, K and V (per-tensor
               descales; ssa_fwd_fp8 / ssa_fwd_fp8_qkv)
  quantize_fp8 bf16 -> E4M3 per-tensor quantisation for fwd_fp8
  calibrate    dense attention + skip counts at N thresholds at once
               (optionally with the per-tile statistic, ``ssa_calibrate_ex``)
  calibrate_fp8  the same with E4M3 Q and K
  resolve      threshold_scale_factor = a * exp(b * target_sparsity)
  fit_logspace log-space least-squares fit of (a, b)
  num_qblocks  number of 128-row query blocks of a batch
  get_error    synchronise and read/clear the device status word
The training step around the forward (module ``training`` has it as autograd
functions):
  fwd_lse      the forward, also writing each row's log-sum-exp; K and V may
               have fewer heads than Q
  bwd          its gradients, dense or on the tiles the forward kept
  save_fp8, restore_fp8   activations in 8 bits, a scale per 128 tokens and head
  bwd_fp8      bwd on Q, K and V saved in 8 bits
  rotary       rotary positions on Q and K, or their adjoint
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
_SO = os.path.join(_PKG, "libssa.so")
TILE = 128
MAX_THRESHOLDS = 32

SSA_OK = 0
SSA_ERR_INVALID_ARG = -1
SSA_ERR_UNSUPPORTED = -2
SSA_ERR_CUDA = -3
SSA_ERR_TIMEOUT = -4
SSA_ERR_DEVICE_ARG = -5


class SSAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = ""
        if status == SSA_ERR_CUDA:
            detail = f": {_lib.ssa_last_cuda_error().decode()}"
        super().__init__(f"{what}: {status} ({_lib.ssa_status_string(status).decode()}{detail})")


def _load():
    if not os.path.exists(_SO):
        raise ImportError(f"libssa.so is not built ({_SO}); run block_sparse_flashattention_ssa_b200/build.py")
    L = ctypes.CDLL(_SO)
    vp, i32, f32, f64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_double
    L.ssa_fwd.restype = i32
    L.ssa_fwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, f32, vp, vp, i32, vp]
    L.ssa_fwd_ex.restype = i32
    L.ssa_fwd_ex.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, f32, vp, vp, i32, vp, vp, vp]
    L.ssa_fwd_fp8.restype = i32
    L.ssa_fwd_fp8.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, f32, f32, f32, vp, vp, i32, vp, vp, vp]
    L.ssa_calibrate_fp8.restype = i32
    L.ssa_calibrate_fp8.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, f32, f32, vp, i32, vp, vp, i32,
                                    vp]
    L.ssa_fwd_fp8_qkv.restype = i32
    L.ssa_fwd_fp8_qkv.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, f32, f32, f32, f32, vp, vp, i32,
                                  vp, vp, vp]
    L.ssa_calibrate_fp8_qkv.restype = i32
    L.ssa_calibrate_fp8_qkv.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, f32, f32, f32, vp, i32, vp,
                                        vp, i32, vp]
    L.ssa_quantize_fp8.restype = i32
    L.ssa_quantize_fp8.argtypes = [vp, vp, ctypes.c_int64, f32, vp]
    L.ssa_calibrate.restype = i32
    L.ssa_calibrate.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, i32, vp, vp, i32, vp]
    L.ssa_calibrate_ex.restype = i32
    L.ssa_calibrate_ex.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, i32, vp, vp, i32, vp, vp]
    i64 = ctypes.c_int64
    L.ssa_fwd_lse.restype = i32
    L.ssa_fwd_lse.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, f32, vp, vp, vp, i32, vp, vp]
    L.ssa_bwd_workspace_bytes.restype = i64
    L.ssa_bwd_workspace_bytes.argtypes = [i32, i32, i32]
    L.ssa_bwd.restype = i32
    L.ssa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, i32, vp, vp, vp, vp, i64,
                          vp]
    L.ssa_save_fp8.restype = i32
    L.ssa_save_fp8.argtypes = [vp, vp, vp, i32, i32, i32, vp]
    L.ssa_restore_fp8.restype = i32
    L.ssa_restore_fp8.argtypes = [vp, vp, vp, i32, i32, i32, vp]
    L.ssa_bwd_fp8_workspace_bytes.restype = i64
    L.ssa_bwd_fp8_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.ssa_bwd_fp8.restype = i32
    L.ssa_bwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, i32, vp,
                              vp, vp, vp, i64, vp]
    L.ssa_rotary.restype = i32
    L.ssa_rotary.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, i32, i32, vp, i32, vp, vp, i32, i32, f32,
                             i32, vp]
    L.ssa_resolve.restype = f64
    L.ssa_resolve.argtypes = [f64, f64, f64]
    L.ssa_fit_logspace.restype = i32
    L.ssa_fit_logspace.argtypes = [vp, vp, i32, vp, vp, vp, vp]
    L.ssa_num_qblocks.restype = i32
    L.ssa_num_qblocks.argtypes = [vp, i32]
    L.ssa_get_error.restype = i32
    L.ssa_get_error.argtypes = [vp]
    L.ssa_status_string.restype = ctypes.c_char_p
    L.ssa_status_string.argtypes = [i32]
    L.ssa_last_cuda_error.restype = ctypes.c_char_p
    L.ssa_last_cuda_error.argtypes = []
    L.ssa_wait_timeout_check.restype = i32
    L.ssa_wait_timeout_check.argtypes = [vp, ctypes.c_int64, vp]
    return L


_lib = _load()


def lib():
    """The loaded ctypes library (for callers that marshal raw pointers)."""
    return _lib


def library_path() -> str:
    return _SO


def _check(rc: int, what: str):
    if rc != SSA_OK:
        raise SSAError(rc, what)


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _shape(q):
    if q.dim() != 3:
        raise ValueError("q, k, v must be [total_tokens, H, D]")
    return q.shape[0], q.shape[1], q.shape[2]


def _require(t, name, dtype, device, shape=None, allow_none=False):
    """Host-side check of a tensor argument: on the device of q, contiguous,
    of the expected dtype (and shape). A host tensor handed to the kernels
    would fault the GPU, so this is checked before the library is called."""
    import torch

    if t is None:
        if allow_none:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_attention_args(q, k, v, cu_seqlens, out, qk_dtype, v_dtype=None):
    import torch

    if not (isinstance(q, torch.Tensor) and q.is_cuda):
        raise ValueError("q must be a CUDA tensor")
    dev = q.device
    shape = tuple(q.shape)
    _require(q, "q", qk_dtype, dev)
    _require(k, "k", qk_dtype, dev, shape)
    _require(v, "v", v_dtype or torch.bfloat16, dev, shape)
    _require(cu_seqlens, "cu_seqlens", torch.int32, dev)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D tensor of batch + 1 offsets")
    _require(out, "out", torch.bfloat16, dev, shape, allow_none=True)
    return dev


def _per_unit_qblocks(dev, H, total, batch, outputs) -> int:
    """Check the per-unit outputs ``(tensor, name, dtypes, inner_shape)``:
    each must be [H, Q, *inner_shape] on ``dev``, all with the same Q, and Q
    no larger than any batch of ``total`` tokens can have. Returns that Q
    (-1 when every output is None). The library counts the q-blocks again
    from the device copy of cu_seqlens and writes nothing when they differ,
    so a wrong Q cannot overrun a buffer either way."""
    q_dim = None
    for t, name, dtype, inner in outputs:
        _require(t, name, dtype, dev, allow_none=True)
        if t is None:
            continue
        if t.dim() != 2 + len(inner) or t.shape[0] != H or tuple(t.shape[2:]) != tuple(inner):
            want = ", ".join([str(H), "num_qblocks"] + [str(i) for i in inner])
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{want}]")
        if q_dim is None:
            q_dim = int(t.shape[1])
        elif int(t.shape[1]) != q_dim:
            raise ValueError(f"{name} has {t.shape[1]} q-blocks, another per-unit output {q_dim}")
    if q_dim is None:
        return -1
    if q_dim > (total + TILE - 1) // TILE + batch:
        raise ValueError(f"{q_dim} q-blocks is more than {total} tokens in {batch} sequences can have")
    return q_dim


def num_qblocks(cu_seqlens) -> int:
    """Total 128-row query blocks over the batch (from a host copy of cu_seqlens)."""
    cu = np.ascontiguousarray(np.asarray(cu_seqlens if not hasattr(cu_seqlens, "cpu") else cu_seqlens.cpu()),
                              dtype=np.int32)
    n = _lib.ssa_num_qblocks(cu.ctypes.data, len(cu) - 1)
    if n < 0:
        raise SSAError(n, "ssa_num_qblocks")
    return n


def fwd(q, k, v, cu_seqlens, max_seqlen: int, threshold_scale_factor: float = 0.0, softmax_scale: float = 0.0,
        out=None, skip_counter=None, decision_bitmap=None, tile_stat=None, stream=None):
    """Skip-softmax attention forward. q, k, v: CUDA bf16 [total_tokens, H, D];
    cu_seqlens: CUDA int32 [B+1]. Returns ``out`` (allocated when None).
    ``skip_counter`` (int32 [H, Q]), ``decision_bitmap`` (int32/uint32
    [H, Q, ceil(T/32)]) and ``tile_stat`` (float32 [H, Q, T]) are optional
    caller-allocated outputs; passing either of the last two selects the
    diagnostic call ``ssa_fwd_ex``."""
    import torch

    total, H, D = _shape(q)
    dev = _check_attention_args(q, k, v, cu_seqlens, out, torch.bfloat16)
    batch = cu_seqlens.numel() - 1
    nq = _per_unit_qblocks(dev, H, total, batch, _forward_outputs(skip_counter, decision_bitmap, tile_stat,
                                                                  max_seqlen))
    if out is None:
        out = torch.empty_like(q)
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), batch, total, int(max_seqlen), H, D,
            float(softmax_scale), float(threshold_scale_factor), _ptr(out), _ptr(skip_counter), nq]
    if decision_bitmap is not None or tile_stat is not None:
        rc = _lib.ssa_fwd_ex(*args, _ptr(decision_bitmap), _ptr(tile_stat), _stream_handle(stream))
        _check(rc, "ssa_fwd_ex")
    else:
        _check(_lib.ssa_fwd(*args, _stream_handle(stream)), "ssa_fwd")
    return out


def fwd_fp8(q8, k8, v, cu_seqlens, max_seqlen: int, q_descale: float, k_descale: float,
            threshold_scale_factor: float = 0.0, softmax_scale: float = 0.0, out=None, skip_counter=None,
            decision_bitmap=None, tile_stat=None, v_descale=None, stream=None):
    """Forward with E4M3 Q and K (CUDA uint8 [total_tokens, H, 128], values
    q_descale * decode(q8)); returns bf16 ``out``. V is bf16 (ssa_fwd_fp8) or,
    with ``v_descale``, E4M3 codes as well, P then rounded to E4M3 for the
    P.V product (ssa_fwd_fp8_qkv)."""
    import torch

    total, H, D = _shape(q8)
    qkv = v_descale is not None
    dev = _check_attention_args(q8, k8, v, cu_seqlens, out, torch.uint8, torch.uint8 if qkv else None)
    batch = cu_seqlens.numel() - 1
    nq = _per_unit_qblocks(dev, H, total, batch, _forward_outputs(skip_counter, decision_bitmap, tile_stat,
                                                                  max_seqlen))
    if out is None:
        out = torch.empty(v.shape, dtype=torch.bfloat16, device=v.device)
    head = [_ptr(q8), _ptr(k8), _ptr(v), _ptr(cu_seqlens), batch, total, int(max_seqlen), H, D,
            float(softmax_scale), float(q_descale), float(k_descale)]
    tail = [float(threshold_scale_factor), _ptr(out), _ptr(skip_counter), nq, _ptr(decision_bitmap),
            _ptr(tile_stat), _stream_handle(stream)]
    if qkv:
        _check(_lib.ssa_fwd_fp8_qkv(*head, float(v_descale), *tail), "ssa_fwd_fp8_qkv")
    else:
        _check(_lib.ssa_fwd_fp8(*head, *tail), "ssa_fwd_fp8")
    return out


def quantize_fp8(x, inv_scale: float, out=None, stream=None):
    """E4M3 codes (uint8, same shape) of fp32(x * inv_scale), nearest even, saturating."""
    import torch

    if not (isinstance(x, torch.Tensor) and x.is_cuda):
        raise ValueError("x must be a CUDA tensor")
    _require(x, "x", torch.bfloat16, x.device)
    _require(out, "out", torch.uint8, x.device, tuple(x.shape), allow_none=True)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(_lib.ssa_quantize_fp8(_ptr(x), _ptr(out), x.numel(), float(inv_scale), _stream_handle(stream)),
           "ssa_quantize_fp8")
    return out


def calibrate(q, k, v, cu_seqlens, max_seqlen: int, thresholds, softmax_scale: float = 0.0, out=None, counts=None,
              tile_stat=None, stream=None):
    """Dense attention plus, per (head, q-block) unit, the number of KV tiles
    that would be skipped at each raw lambda in ``thresholds``. Returns
    (out, counts[H, Q, N]). Passing ``tile_stat`` (float32 [H, Q, T],
    caller-allocated) selects ``ssa_calibrate_ex``, which also writes every
    tile's statistic d_j. Without ``counts`` the q-block count is read from a
    host copy of cu_seqlens (a synchronisation)."""
    import torch

    total, H, D = _shape(q)
    dev = _check_attention_args(q, k, v, cu_seqlens, out, torch.bfloat16)
    th = np.ascontiguousarray(thresholds, dtype=np.float32)
    batch = cu_seqlens.numel() - 1
    if counts is None:
        counts = torch.empty((H, num_qblocks(cu_seqlens), len(th)), dtype=torch.int32, device=dev)
    nq = _per_unit_qblocks(dev, H, total, batch, [(counts, "counts", torch.int32, (len(th),)),
                                                   (tile_stat, "tile_stat", torch.float32, (max_tiles(max_seqlen),))])
    if out is None:
        out = torch.empty_like(q)
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), batch, total, int(max_seqlen), H, D, float(softmax_scale),
            th.ctypes.data, len(th), _ptr(out), _ptr(counts), nq]
    if tile_stat is not None:
        _check(_lib.ssa_calibrate_ex(*args, _ptr(tile_stat), _stream_handle(stream)), "ssa_calibrate_ex")
    else:
        _check(_lib.ssa_calibrate(*args, _stream_handle(stream)), "ssa_calibrate")
    return out, counts


def calibrate_fp8(q8, k8, v, cu_seqlens, max_seqlen: int, q_descale: float, k_descale: float, thresholds,
                  softmax_scale: float = 0.0, out=None, counts=None, v_descale=None, stream=None):
    """calibrate() on the E4M3 scores of fwd_fp8 (V bf16, or E4M3 codes with
    ``v_descale``: ssa_calibrate_fp8_qkv). Returns (out, counts[H, Q, N])."""
    import torch

    total, H, D = _shape(q8)
    qkv = v_descale is not None
    dev = _check_attention_args(q8, k8, v, cu_seqlens, out, torch.uint8, torch.uint8 if qkv else None)
    th = np.ascontiguousarray(thresholds, dtype=np.float32)
    batch = cu_seqlens.numel() - 1
    if counts is None:
        counts = torch.empty((H, num_qblocks(cu_seqlens), len(th)), dtype=torch.int32, device=dev)
    nq = _per_unit_qblocks(dev, H, total, batch, [(counts, "counts", torch.int32, (len(th),))])
    if out is None:
        out = torch.empty(v.shape, dtype=torch.bfloat16, device=v.device)
    head = [_ptr(q8), _ptr(k8), _ptr(v), _ptr(cu_seqlens), batch, total, int(max_seqlen), H, D,
            float(softmax_scale), float(q_descale), float(k_descale)]
    tail = [th.ctypes.data, len(th), _ptr(out), _ptr(counts), nq, _stream_handle(stream)]
    if qkv:
        _check(_lib.ssa_calibrate_fp8_qkv(*head, float(v_descale), *tail), "ssa_calibrate_fp8_qkv")
    else:
        _check(_lib.ssa_calibrate_fp8(*head, *tail), "ssa_calibrate_fp8")
    return out, counts


def _at(t):
    """Device address of a tensor or None, as ctypes takes it."""
    return None if t is None else t.data_ptr()


def _all_are(dev, wanted) -> bool:
    """Whether every (tensor, name, dtype, shape) passes _require(), in few
    steps: the calls of a training step are short on the GPU for small batches."""
    index = dev.index
    try:
        for t, _, dtype, shape in wanted:
            if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
                return False
    except AttributeError:
        return False
    return True


def _need(dev, wanted):
    """_require() of the arguments that must be there."""
    if not _all_are(dev, wanted):
        for t, name, dtype, shape in wanted:
            _require(t, name, dtype, dev, shape)


def _may(dev, wanted):
    """_require() of the optional outputs among ``wanted``."""
    given = [w for w in wanted if w[0] is not None]
    if given:
        _need(dev, given)


def _current_handle(torch, dev):
    """The current stream's cudaStream_t, without a Stream object where torch can."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev.index) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _run(dev, stream, tensors, body):
    """``body(stream handle)`` with ``dev`` current and on ``stream`` (default:
    the device's current one), so that what it allocates belongs to the stream
    its kernels run on. ``tensors`` and the tensors it returns are kept from
    reuse until both that stream and the caller's are done with them."""
    import torch

    here = torch.cuda.current_device() == dev.index
    if stream is None and here:
        return body(_current_handle(torch, dev))
    current = torch.cuda.current_stream(dev)
    if stream is None or stream == current:
        stream = current
    elif stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        result = body(stream.cuda_stream)
    if stream != current:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        for t in result:
            if t is not None:
                t.record_stream(current)
    return result


def _no_overlap(outputs, inputs):
    """Refuse an output that shares memory with an input or another output
    (all contiguous): the kernels read and write them in no fixed order.
    Outputs that are None are allocated later and share nothing."""
    given = [(t, name) for t, name in outputs if t is not None]
    if not given:
        return
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), name)
             for t, name in inputs + given if t is not None]
    for i in range(len(spans) - len(given), len(spans)):
        lo, hi, name = spans[i]
        for other in spans[:i]:
            if lo < other[1] and other[0] < hi:
                raise ValueError(f"{name} overlaps {other[2]}")


def _check_shared_heads(torch, q, k, v, cu_seqlens, qkv_dtype):
    """Checks of fwd_lse and the backward passes: K and V may have fewer heads."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda):
        raise ValueError("q must be a CUDA tensor")
    total, H, D = _shape(q)
    dev = q.device
    for t, name in ((k, "k"), (cu_seqlens, "cu_seqlens")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    k_shape, cu_shape = k.shape, cu_seqlens.shape
    _need(dev, ((q, "q", qkv_dtype, q.shape), (k, "k", qkv_dtype, k_shape), (v, "v", qkv_dtype, k_shape),
                (cu_seqlens, "cu_seqlens", torch.int32, cu_shape)))
    if len(k_shape) != 3 or k_shape[0] != total or k_shape[2] != D or k_shape[1] < 1 or H % k_shape[1] != 0:
        raise ValueError(f"k has shape {tuple(k_shape)}, expected [{total}, a divisor of {H}, {D}]")
    if len(cu_shape) != 1 or cu_shape[0] < 2:
        raise ValueError("cu_seqlens must be a 1-D tensor of batch + 1 offsets")
    return dev, total, H, k_shape[1], D, cu_shape[0] - 1


def fwd_lse(q, k, v, cu_seqlens, max_seqlen: int, threshold_scale_factor: float = 0.0, softmax_scale: float = 0.0,
            out=None, lse=None, skip_counter=None, decision_bitmap=None, stream=None):
    """The forward of a training step: fwd() plus the rows' log-sum-exp over
    the kept tiles (natural logarithm of the scaled scores), which bwd() needs.
    q: CUDA bf16 [total_tokens, H, D]; k, v: [total_tokens, Hkv, D] with Hkv a
    divisor of H (query head h reads head h // (H // Hkv)). Returns (out,
    lse[H, total_tokens] float32). With a threshold, pass ``decision_bitmap``
    (as in fwd) to keep the decisions for bwd()."""
    import torch

    dev, total, H, Hkv, D, batch = _check_shared_heads(torch, q, k, v, cu_seqlens, torch.bfloat16)
    _may(dev, ((out, "out", torch.bfloat16, q.shape), (lse, "lse", torch.float32, (H, total))))
    nq = -1
    if skip_counter is not None or decision_bitmap is not None:
        nq = _per_unit_qblocks(dev, H, total, batch, _forward_outputs(skip_counter, decision_bitmap, None, max_seqlen))
    _no_overlap([(out, "out"), (lse, "lse"), (skip_counter, "skip_counter"), (decision_bitmap, "decision_bitmap")],
                [(q, "q"), (k, "k"), (v, "v"), (cu_seqlens, "cu_seqlens")])

    def body(handle):
        o = torch.empty_like(q) if out is None else out
        r = torch.empty((H, total), dtype=torch.float32, device=dev) if lse is None else lse
        _check(_lib.ssa_fwd_lse(_at(q), _at(k), _at(v), _at(cu_seqlens), batch, total, max_seqlen, H, Hkv, D,
                                float(softmax_scale), float(threshold_scale_factor), _at(o), _at(r),
                                _at(skip_counter), nq,
                                _at(decision_bitmap), handle), "ssa_fwd_lse")
        return o, r

    max_seqlen = int(max_seqlen)
    return _run(dev, stream, (q, k, v, cu_seqlens, out, lse, skip_counter, decision_bitmap), body)


@functools.lru_cache(maxsize=256)
def _bwd_workspace(total, batch, H, Hkv, D):
    return _lib.ssa_bwd_workspace_bytes(total, batch, H)


@functools.lru_cache(maxsize=256)
def _bwd_fp8_workspace(total, batch, H, Hkv, D):
    return _lib.ssa_bwd_fp8_workspace_bytes(total, batch, H, Hkv, D)


def _backward(what, dout, q, k, v, extra, out, lse, cu_seqlens, max_seqlen, softmax_scale, decision_bitmap, dq, dk, dv,
              workspace, stream, qkv_dtype, workspace_bytes, call):
    import torch

    dev, total, H, Hkv, D, batch = _check_shared_heads(torch, q, k, v, cu_seqlens, qkv_dtype)
    bf16, q_shape, k_shape = torch.bfloat16, q.shape, k.shape
    _need(dev, ((dout, "dout", bf16, q_shape), (out, "out", bf16, q_shape), (lse, "lse", torch.float32, (H, total)))
          + tuple((t, name, torch.float32, ((total + TILE - 1) // TILE, heads)) for t, name, heads in extra))
    _may(dev, ((dq, "dq", bf16, q_shape), (dk, "dk", bf16, k_shape), (dv, "dv", bf16, k_shape)))
    if workspace is not None:
        _require(workspace, "workspace", None, dev)
    nq, max_seqlen = -1, int(max_seqlen)
    if decision_bitmap is not None:
        nq = _per_unit_qblocks(dev, H, total, batch, [(decision_bitmap, "decision_bitmap", (torch.int32, torch.uint32),
                                                        (bitmap_words(max_seqlen),))])
    if not (dq is None and dk is None and dv is None and workspace is None):
        _no_overlap([(dq, "dq"), (dk, "dk"), (dv, "dv"), (workspace, "workspace")],
                    [(dout, "dout"), (q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse"),
                     (cu_seqlens, "cu_seqlens"), (decision_bitmap, "decision_bitmap")]
                    + [(t, name) for t, name, _ in extra])
    need = workspace_bytes(total, batch, H, Hkv, D)
    if need < 0:
        raise SSAError(int(need), what)

    def body(handle):
        if workspace is None:
            ws, size = torch.empty(need, dtype=torch.uint8, device=dev), need
        else:
            ws, size = workspace, workspace.numel() * workspace.element_size()
        gq = torch.empty_like(out) if dq is None else dq
        gk = torch.empty_like(k, dtype=bf16) if dk is None else dk
        gv = torch.empty_like(gk) if dv is None else dv
        _check(call(_at(dout), _at(out), _at(lse), _at(cu_seqlens), batch, total, max_seqlen, H, Hkv, D,
                    float(softmax_scale), _at(decision_bitmap), nq, _at(gq), _at(gk), _at(gv), _at(ws), size, handle), what)
        return gq, gk, gv

    return _run(dev, stream, (dout, q, k, v, out, lse, cu_seqlens, decision_bitmap, dq, dk, dv, workspace)
                + tuple(t for t, _, _ in extra), body)


def bwd(dout, q, k, v, out, lse, cu_seqlens, max_seqlen: int, softmax_scale: float = 0.0, decision_bitmap=None,
        dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of fwd_lse(): returns (dq, dk, dv) in bf16 for the output
    gradient ``dout``. ``out``, ``lse`` and, when the forward skipped tiles,
    ``decision_bitmap`` are what it wrote (the decisions count as constants); a
    row whose lse is -inf takes no part, whatever stands in it elsewhere.
    Rows outside every sequence are left as they were in dq, dk and dv (when
    they are allocated here, undefined). ``workspace``: a device buffer of at
    least bwd_workspace_bytes() that no other call uses meanwhile."""
    import torch

    return _backward(
        "ssa_bwd", dout, q, k, v, [], out, lse, cu_seqlens, max_seqlen, softmax_scale, decision_bitmap, dq, dk, dv,
        workspace, stream, torch.bfloat16, _bwd_workspace,
        lambda g, *rest: _lib.ssa_bwd(g, _at(q), _at(k), _at(v), *rest))


def bwd_fp8(dout, q_saved, k_saved, v_saved, out, lse, cu_seqlens, max_seqlen: int, softmax_scale: float = 0.0,
            decision_bitmap=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """bwd() on Q, K and V saved in 8 bits: each ``*_saved`` is save_fp8()'s
    (codes, scales), and the gradients are those at the restored values."""
    import torch

    (q, qs), (k, ks), (v, vs) = q_saved, k_saved, v_saved
    heads = lambda t: t.shape[1] if t.dim() == 3 else -1
    return _backward(
        "ssa_bwd_fp8", dout, q, k, v, [(qs, "q_scales", heads(q)), (ks, "k_scales", heads(k)), (vs, "v_scales", heads(v))],
        out, lse, cu_seqlens, max_seqlen, softmax_scale, decision_bitmap, dq, dk, dv, workspace, stream, torch.uint8,
        _bwd_fp8_workspace,
        lambda g, *rest: _lib.ssa_bwd_fp8(g, _at(q), _at(qs), _at(k), _at(ks), _at(v), _at(vs), *rest))


def bwd_workspace_bytes(total_tokens: int, batch: int, num_heads: int) -> int:
    """Size of bwd()'s workspace."""
    n = int(_lib.ssa_bwd_workspace_bytes(int(total_tokens), int(batch), int(num_heads)))
    if n < 0:
        raise SSAError(n, "ssa_bwd_workspace_bytes")
    return n


def bwd_fp8_workspace_bytes(total_tokens: int, batch: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    """Size of bwd_fp8()'s workspace."""
    n = int(_lib.ssa_bwd_fp8_workspace_bytes(int(total_tokens), int(batch), int(num_heads), int(num_kv_heads),
                                             int(head_dim)))
    if n < 0:
        raise SSAError(n, "ssa_bwd_fp8_workspace_bytes")
    return n


def save_fp8(x, codes=None, scales=None, stream=None):
    """Save activations in 8 bits: x is CUDA bf16 [total_tokens, H, D] (D 64 or
    128). Returns (codes uint8 [total_tokens, H, D], scales float32
    [ceil(total_tokens / 128), H]): E4M3 codes of x / scale, the scale of each
    128 tokens and head the smallest power of two that keeps them in range."""
    import torch

    if not (isinstance(x, torch.Tensor) and x.is_cuda):
        raise ValueError("x must be a CUDA tensor")
    total, H, D = _shape(x)
    dev, s_shape = x.device, ((total + TILE - 1) // TILE, H)
    _need(dev, ((x, "x", torch.bfloat16, x.shape),))
    _may(dev, ((codes, "codes", torch.uint8, x.shape), (scales, "scales", torch.float32, s_shape)))
    _no_overlap([(codes, "codes"), (scales, "scales")], [(x, "x")])

    def body(handle):
        c = torch.empty_like(x, dtype=torch.uint8) if codes is None else codes
        s = torch.empty(s_shape, dtype=torch.float32, device=dev) if scales is None else scales
        _check(_lib.ssa_save_fp8(_at(x), _at(c), _at(s), total, H, D, handle), "ssa_save_fp8")
        return c, s

    return _run(dev, stream, (x, codes, scales), body)


def restore_fp8(codes, scales, out=None, stream=None):
    """What save_fp8() kept: bf16 scale * decode(code), exactly."""
    import torch

    if not (isinstance(codes, torch.Tensor) and codes.is_cuda):
        raise ValueError("codes must be a CUDA tensor")
    total, H, D = _shape(codes)
    dev = codes.device
    _need(dev, ((codes, "codes", torch.uint8, codes.shape),
                (scales, "scales", torch.float32, ((total + TILE - 1) // TILE, H))))
    _may(dev, ((out, "out", torch.bfloat16, codes.shape),))
    _no_overlap([(out, "out")], [(codes, "codes"), (scales, "scales")])

    def body(handle):
        x = torch.empty_like(codes, dtype=torch.bfloat16) if out is None else out
        _check(_lib.ssa_restore_fp8(_at(codes), _at(scales), _at(x), total, H, D, handle), "ssa_restore_fp8")
        return (x,)

    return _run(dev, stream, (codes, scales, out), body)[0]


@functools.lru_cache(maxsize=None)
def _sections_type(axes):
    return ctypes.c_int32 * axes


def _rows(t, name, dev, total, dim):
    """Check a rotary operand [total, H, dim] whose tokens may lie apart (a
    slice of a fused projection, say); returns its token stride."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16 or t.device != dev:
        raise ValueError(f"{name} is {t.dtype} on {t.device}, expected torch.bfloat16 on {dev}")
    shape = t.shape
    if len(shape) != 3 or shape[0] != total or shape[2] != dim:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [{total}, heads, {dim}]")
    row = shape[1] * dim
    if t.is_contiguous():
        return row
    s0, s1, s2 = t.stride()
    if (dim > 1 and s2 != 1) or (shape[1] > 1 and s1 != dim) or (total > 1 and s0 < row):
        raise ValueError(f"{name}: the heads of a token must be contiguous and tokens must not overlap")
    return s0 if total > 1 else row


def _rows_overlap(a, a_stride, b, b_stride):
    """Whether two operands of _rows() share an element."""
    size, n = a.element_size(), a.shape[0]
    wa, wb = a.shape[1] * a.shape[2] * size, b.shape[1] * b.shape[2] * size
    pa, pb, sa, sb = a.data_ptr(), b.data_ptr(), a_stride * size, b_stride * size
    if n == 0 or pa + (n - 1) * sa + wa <= pb or pb + (n - 1) * sb + wb <= pa:
        return False
    if sa != sb:
        return True
    d = (pb - pa) % sa  # the same stride: b's rows start d bytes into a's
    return d < wa or d + wb > sa


def _check_rotary_outputs(dev, total, dim, inputs, xs, outputs, ys, tables):
    """Checks of rotary's given outputs; fills in their token strides.
    ``tables``: the contiguous (tensor, name) that the kernel reads besides."""
    written = []
    for i, (o, x, name) in enumerate(zip(outputs, inputs, ("out_q", "out_k"))):
        if o is None:
            continue
        if x is None:
            raise ValueError("out_k without k")
        ys[i] = _rows(o, name, dev, total, dim)
        if o.shape != x.shape:
            raise ValueError(f"{name} has shape {tuple(o.shape)}, expected {tuple(x.shape)}")
        written.append((o, ys[i]))
        for y, stride, other in zip(inputs, xs, ("q", "k")):
            if y is None or (y is x and o.data_ptr() == x.data_ptr() and ys[i] == stride):
                continue  # in place: a pair is read and written by one thread
            if _rows_overlap(o, ys[i], y, stride):
                raise ValueError(f"{name} overlaps {other}")
        start, size = o.data_ptr(), ((total - 1) * ys[i] + o.shape[1] * dim) * o.element_size() if total else 0
        for t, other in tables:
            if start < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < start + size:
                raise ValueError(f"{name} overlaps {other}")
    if len(written) == 2 and _rows_overlap(*written[0], *written[1]):
        raise ValueError("out_q overlaps out_k")


def rotary(q, k, positions, inv_freq, sections=None, interleaved: bool = False, scale: float = 1.0,
           transpose: bool = False, out_q=None, out_k=None, stream=None):
    """Rotary positions on Q and, unless it is None, on K, in one launch.
    q, k: CUDA bf16 [total_tokens, heads, D], each token's heads contiguous;
    positions: int32 [total_tokens] or [total_tokens, axes]; inv_freq: float64
    [pairs], radians per position (module ``positions`` makes them). The first
    2 * pairs elements of a head are rotated, pair i being (2i, 2i + 1) when
    ``interleaved``, else (i, i + pairs); ``sections`` gives the number of
    consecutive pairs that turn with each axis. ``transpose`` applies the
    adjoint: it turns output gradients into input gradients. ``out_q`` may be
    q itself, ``out_k`` k itself. Returns (q', k')."""
    import torch

    if not (isinstance(q, torch.Tensor) and q.is_cuda):
        raise ValueError("q must be a CUDA tensor")
    total, H, D = _shape(q)
    dev = q.device
    for t, name in ((positions, "positions"), (inv_freq, "inv_freq")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    _need(dev, ((positions, "positions", torch.int32, positions.shape), (inv_freq, "inv_freq", torch.float64, inv_freq.shape)))
    axes = 1 if positions.dim() == 1 else positions.shape[-1]
    if positions.shape != ((total,) if positions.dim() == 1 else (total, axes)):
        raise ValueError(f"positions has shape {tuple(positions.shape)}, expected [{total}] or [{total}, axes]")
    pairs = inv_freq.numel()
    if inv_freq.dim() != 1 or 2 * pairs > D:
        raise ValueError(f"inv_freq must be 1-D with at most {D // 2} frequencies")
    if sections is None and axes > 1:
        raise ValueError("sections must say how many pairs turn with each of the position axes")
    counts = [pairs] if sections is None else [int(n) for n in sections]
    if len(counts) != axes or min(counts) < 0 or sum(counts) != pairs:
        raise ValueError(f"sections must be {axes} counts adding up to {pairs}")
    xs = [_rows(q, "q", dev, total, D), 0 if k is None else _rows(k, "k", dev, total, D)]
    Hk = 0 if k is None else k.shape[1]
    ys = [H * D, Hk * D]
    if out_q is not None or out_k is not None:
        _check_rotary_outputs(dev, total, D, (q, k), xs, (out_q, out_k), ys,
                              ((positions, "positions"), (inv_freq, "inv_freq")))
    n_pairs = _sections_type(axes)(*counts)

    def body(handle):
        oq = torch.empty_like(q, memory_format=torch.contiguous_format) if out_q is None else out_q
        ok = torch.empty_like(k, memory_format=torch.contiguous_format) if out_k is None and k is not None else out_k
        _check(_lib.ssa_rotary(_at(q), _at(k), _at(oq), _at(ok), xs[0], xs[1], ys[0], ys[1], total, H, Hk, D,
                               _at(positions), axes, n_pairs, _at(inv_freq), 2 * pairs, 1 if interleaved else 0,
                               float(scale), 1 if transpose else 0, handle), "ssa_rotary")
        return oq, ok

    return _run(dev, stream, (q, k, positions, inv_freq, out_q, out_k), body)


def resolve(a: float, b: float, target_sparsity: float) -> float:
    return float(_lib.ssa_resolve(a, b, target_sparsity))


def fit_logspace(sparsity, scale_factor):
    """Returns (a, b, s_min, s_max)."""
    s = np.ascontiguousarray(sparsity, dtype=np.float64)
    sf = np.ascontiguousarray(scale_factor, dtype=np.float64)
    if s.shape != sf.shape:
        raise ValueError("sparsity and scale_factor differ in length")
    out = [ctypes.c_double() for _ in range(4)]
    _check(_lib.ssa_fit_logspace(s.ctypes.data, sf.ctypes.data, len(s), *[ctypes.byref(o) for o in out]),
           "ssa_fit_logspace")
    return tuple(o.value for o in out)


def wait_timeout_check(limit_ns: int = 20_000_000, stream=None):
    """Diagnostic: run the kernels' bounded wait on a barrier nothing arrives
    on. Returns (completed, abort_flag, microseconds_waited) from the device;
    the device status then holds SSA_ERR_TIMEOUT (read it with get_error)."""
    import torch

    res = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    _check(_lib.ssa_wait_timeout_check(_ptr(res), int(limit_ns), _stream_handle(stream)), "ssa_wait_timeout_check")
    torch.cuda.synchronize()
    return tuple(int(x) for x in res.cpu().tolist())


def get_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status."""
    return int(_lib.ssa_get_error(_stream_handle(stream)))


def check_device(stream=None):
    """Raise SSAError when a kernel recorded an error on this device."""
    _check(get_error(stream), "device status")


def max_tiles(max_seqlen: int) -> int:
    return (int(max_seqlen) + TILE - 1) // TILE


def bitmap_words(max_seqlen: int) -> int:
    return (max_tiles(max_seqlen) + 31) // 32


def _forward_outputs(skip_counter, decision_bitmap, tile_stat, max_seqlen):
    import torch

    return [(skip_counter, "skip_counter", torch.int32, ()),
            (decision_bitmap, "decision_bitmap", (torch.int32, torch.uint32), (bitmap_words(max_seqlen),)),
            (tile_stat, "tile_stat", torch.float32, (max_tiles(max_seqlen),))]
