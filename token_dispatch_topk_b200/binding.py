"""Thin ctypes binding of libmoe_route.so (include/moe_route.h), same names as the C ABI.

Argument marshalling only: every step of the routing path runs in the library's
CUDA kernels.  torch tensors supply device memory and the stream
(``torch.cuda.current_stream().cuda_stream`` unless one is given).  There is no
CPU fallback: a missing library, a CPU tensor or a non-OK status raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_route.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_TIMEOUT = 5
MOE_ERR_BAD_EXPERT_ID = 6
MOE_ERR_BAD_ROW = 7

MOE_DTYPE_F32 = 0
MOE_DTYPE_BF16 = 1
MOE_RENORMALIZE = 1
MOE_GATHER_ZERO_PAD = 2
MOE_GATHER_HIDDEN_READY = 4
MOE_DISPATCH_GIVEN_IDS = 8
MOE_SCORING_SIGMOID = 16
MOE_MX4_SWIGLU = 32

# Every symbol include/moe_route.h declares, with (restype, argtypes).
_P, _I32, _I64, _U32, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
SIGNATURES = {
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_version": (_I32, []),
    "moe_topk_softmax": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I32, _I32, _U32, _P, _P, _P]),
    "moe_align_capacity": (_I64, [_I64, _I32, _I32, _I32]),
    "moe_align_num_blocks": (_I64, [_I64, _I32, _I32, _I32]),
    "moe_align_workspace_bytes": (_SZ, [_I64, _I32, _I32]),
    "moe_workspace_init": (ctypes.c_int, [_P, _SZ, _P]),
    "moe_align_permute": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_align_permute_noalloc": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                                  _P]),
    "moe_gather": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P, _P, _I64, _U32, _P, _P, _P]),
    "moe_combine": (ctypes.c_int, [_P, _P, _P, _I64, _I32, _I32, _I64, _P, _P, _P]),
    "moe_read_status": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_int)]),
    "moe_route_dispatch_workspace_bytes": (_SZ, [_I64, _I32, _I32]),
    "moe_route_dispatch": (ctypes.c_int, [_P, ctypes.c_int, _P, _I64, _I32, _I32, _I32, _U32, _P, _I32, _I32, _P, _P,
                                          _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_reduce_partials": (ctypes.c_int, [_P, _I32, _I64, _I32, _P, _P]),
    "moe_combine_backward": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I64, _U32, _P, _P, _P, _P]),
    "moe_gather_backward": (ctypes.c_int, [_P, _P, _I64, _I32, _I32, _I64, _P, _P, _P]),
    "moe_topk_softmax_backward": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, _P, _I64, _I32, _I32, _U32, _P, _P, _P]),
    "moe_quantize_mx4": (ctypes.c_int, [_P, _I64, _I32, _P, _P, _P, _P]),
    "moe_dequantize_mx4": (ctypes.c_int, [_P, _P, _I64, _I32, _P, _P]),
    "moe_gather_mx4": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _I64, _P, _P, _P, _P]),
    "moe_grouped_gemm_mx4": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _I64, _I32, _I32, _U32, _P, _P, _P]),
}

_lib: Optional[ctypes.CDLL] = None


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoe_route.so (built by token_dispatch_topk_b200.build); raises if it is missing."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m token_dispatch_topk_b200.build` "
                           "(the routing path has no CPU fallback)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().moe_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, where)


def _dev(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the routing path runs only on the GPU)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


# ----------------------------------------------------------------- host-only queries --
def moe_version() -> int:
    return int(load_library().moe_version())


def moe_align_capacity(T: int, k: int, E_local: int, block_size: int) -> int:
    return int(load_library().moe_align_capacity(T, k, E_local, block_size))


def moe_align_num_blocks(T: int, k: int, E_local: int, block_size: int) -> int:
    return int(load_library().moe_align_num_blocks(T, k, E_local, block_size))


def moe_align_workspace_bytes(T: int, k: int, E_local: int) -> int:
    return int(load_library().moe_align_workspace_bytes(T, k, E_local))


# --------------------------------------------------------------------------- stages --
def moe_workspace_init(workspace: torch.Tensor, stream=None) -> None:
    _check(load_library().moe_workspace_init(_dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                                             _stream(stream)), "moe_workspace_init")


def alloc_workspace(T: int, k: int, E_local: int, device) -> torch.Tensor:
    """A zeroed align workspace (int32 words; word 0 is the device status word)."""
    nbytes = moe_align_workspace_bytes(T, k, E_local)
    return torch.zeros((nbytes + 3) // 4, dtype=torch.int32, device=device)


def _scoring_flag(scoring: str) -> int:
    if scoring == "softmax":
        return 0
    if scoring == "sigmoid":
        return MOE_SCORING_SIGMOID
    raise ValueError(f"scoring must be 'softmax' or 'sigmoid', got {scoring!r}")


def moe_topk_softmax(logits: torch.Tensor, k: int, renormalize: bool, topk_weights: Optional[torch.Tensor] = None,
                     topk_ids: Optional[torch.Tensor] = None, stream=None, scoring: str = "softmax"):
    """logits [T, E] bf16/fp32 -> (topk_weights [T, k] fp32, topk_ids [T, k] int32).

    ``scoring``: "softmax" (default) or "sigmoid" (each selected expert weighs 1/(1+exp(-x)))."""
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    if logits.dtype == torch.bfloat16:
        dt = MOE_DTYPE_BF16
    elif logits.dtype == torch.float32:
        dt = MOE_DTYPE_F32
    else:
        raise ValueError(f"logits dtype {logits.dtype} unsupported (bf16 or fp32)")
    if topk_weights is None:
        topk_weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    assert topk_weights.dtype == torch.float32 and topk_ids.dtype == torch.int32
    assert topk_weights.numel() == T * k and topk_ids.numel() == T * k
    st = load_library().moe_topk_softmax(_dev(logits, "logits"), dt, T, E, k,
                                         (MOE_RENORMALIZE if renormalize else 0) | _scoring_flag(scoring),
                                         _dev(topk_weights, "topk_weights"), _dev(topk_ids, "topk_ids"),
                                         _stream(stream))
    _check(st, "moe_topk_softmax")
    return topk_weights, topk_ids


class AlignResult(NamedTuple):
    counts: torch.Tensor
    offsets: torch.Tensor
    sorted_token_ids: torch.Tensor
    expert_ids: torch.Tensor
    num_tokens_post_pad: torch.Tensor
    inv_perm: torch.Tensor
    capacity: int


def alloc_align_outputs(T: int, k: int, E_local: int, block_size: int, device) -> AlignResult:
    C = moe_align_capacity(T, k, E_local, block_size)
    NB = moe_align_num_blocks(T, k, E_local, block_size)
    if C < 0:
        raise ValueError("invalid align sizes")
    z = dict(dtype=torch.int32, device=device)
    return AlignResult(torch.empty(E_local, **z), torch.empty(E_local + 1, **z), torch.empty(C, **z),
                       torch.empty(NB, **z), torch.empty(1, **z), torch.empty(T * k, **z), C)


def moe_align_permute(topk_ids: torch.Tensor, E_global: int, block_size: int,
                      expert_map: Optional[torch.Tensor] = None, E_local: Optional[int] = None,
                      out: Optional[AlignResult] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> AlignResult:
    """topk_ids [T, k] int32 (+ optional expert_map [E_global] int32) -> AlignResult on the device."""
    T, k = topk_ids.shape
    if E_local is None:
        E_local = E_global
    if out is None:
        out = alloc_align_outputs(T, k, E_local, block_size, topk_ids.device)
    if workspace is None:
        workspace = alloc_workspace(T, k, E_local, topk_ids.device)
    assert topk_ids.dtype == torch.int32 and (expert_map is None or expert_map.dtype == torch.int32)
    st = load_library().moe_align_permute(
        _dev(topk_ids, "topk_ids"), T, k, E_global, _dev(expert_map, "expert_map"), E_local, block_size,
        _dev(out.counts, "counts"), _dev(out.offsets, "offsets"), _dev(out.sorted_token_ids, "sorted_token_ids"),
        _dev(out.expert_ids, "expert_ids"), _dev(out.num_tokens_post_pad, "num_tokens_post_pad"),
        _dev(out.inv_perm, "inv_perm"), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "moe_align_permute")
    return out


def moe_align_permute_noalloc(topk_ids: torch.Tensor, E_global: int, block_size: int,
                              expert_map: Optional[torch.Tensor] = None, E_local: Optional[int] = None,
                              out: Optional[AlignResult] = None, device_status: Optional[torch.Tensor] = None,
                              stream=None) -> AlignResult:
    """moe_align_permute without a workspace: the library's fixed per-device scratch is used instead
    (for callers that cannot allocate; calls must not overlap on the GPU).  ``out`` may be preallocated."""
    T, k = topk_ids.shape
    if E_local is None:
        E_local = E_global
    if out is None:
        out = alloc_align_outputs(T, k, E_local, block_size, topk_ids.device)
    assert topk_ids.dtype == torch.int32 and (expert_map is None or expert_map.dtype == torch.int32)
    st = load_library().moe_align_permute_noalloc(
        _dev(topk_ids, "topk_ids"), T, k, E_global, _dev(expert_map, "expert_map"), E_local, block_size,
        _dev(out.counts, "counts"), _dev(out.offsets, "offsets"), _dev(out.sorted_token_ids, "sorted_token_ids"),
        _dev(out.expert_ids, "expert_ids"), _dev(out.num_tokens_post_pad, "num_tokens_post_pad"),
        _dev(out.inv_perm, "inv_perm"), _dev(device_status, "device_status"), _stream(stream))
    _check(st, "moe_align_permute_noalloc")
    return out


def moe_gather(hidden: torch.Tensor, k: int, inv_perm: torch.Tensor, capacity: int,
               sorted_token_ids: Optional[torch.Tensor] = None, num_tokens_post_pad: Optional[torch.Tensor] = None,
               zero_pad: bool = False, permuted: Optional[torch.Tensor] = None,
               device_status: Optional[torch.Tensor] = None, stream=None, hidden_ready: bool = False) -> torch.Tensor:
    """hidden [T, H] bf16 -> permuted [capacity, H] bf16 (expert-grouped rows).

    hidden_ready: hidden was complete before the previous kernel in the stream was launched
    (MOE_GATHER_HIDDEN_READY), so the kernel may start loading it before that kernel finishes."""
    T, H = hidden.shape
    assert hidden.dtype == torch.bfloat16
    if permuted is None:
        permuted = torch.empty((capacity, H), dtype=torch.bfloat16, device=hidden.device)
    st = load_library().moe_gather(_dev(hidden, "hidden"), T, H, k, _dev(inv_perm, "inv_perm"),
                                   _dev(sorted_token_ids, "sorted_token_ids"),
                                   _dev(num_tokens_post_pad, "num_tokens_post_pad"), capacity,
                                   (MOE_GATHER_ZERO_PAD if zero_pad else 0) |
                                   (MOE_GATHER_HIDDEN_READY if hidden_ready else 0), _dev(permuted, "permuted"),
                                   _dev(device_status, "device_status"), _stream(stream))
    _check(st, "moe_gather")
    return permuted


def moe_combine(expert_out: torch.Tensor, topk_weights: torch.Tensor, inv_perm: torch.Tensor,
                out: Optional[torch.Tensor] = None, device_status: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """expert_out [capacity, H] bf16, topk_weights [T, k] fp32, inv_perm [T*k] -> out [T, H] bf16."""
    T, k = topk_weights.shape
    capacity, H = expert_out.shape
    assert expert_out.dtype == torch.bfloat16
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=expert_out.device)
    st = load_library().moe_combine(_dev(expert_out, "expert_out"), _dev(topk_weights, "topk_weights"),
                                    _dev(inv_perm, "inv_perm"), T, k, H, capacity, _dev(out, "out"),
                                    _dev(device_status, "device_status"), _stream(stream))
    _check(st, "moe_combine")
    return out


def moe_reduce_partials(partials, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """partials: the ranks' bf16 partial combines [rows, H] in rank order (tensors on this GPU or,
    with peer access, on others) -> out [rows, H] bf16: their fp32 sum in rank order, rounded once."""
    partials = list(partials)
    if not partials:
        raise ValueError("moe_reduce_partials needs at least one partial")
    rows, H = partials[0].shape
    for p in partials:
        assert p.dtype == torch.bfloat16 and tuple(p.shape) == (rows, H), "partials must all be bf16 [rows, H]"
    if out is None:
        out = torch.empty((rows, H), dtype=torch.bfloat16, device=partials[0].device)
    ptrs = (ctypes.c_void_p * len(partials))(*[_dev(p, "partial") for p in partials])
    st = load_library().moe_reduce_partials(ctypes.cast(ptrs, ctypes.c_void_p), len(partials), rows, H,
                                            _dev(out, "out"), _stream(stream))
    _check(st, "moe_reduce_partials")
    return out


def moe_route_dispatch_workspace_bytes(T: int, k: int, E_local: int) -> int:
    return int(load_library().moe_route_dispatch_workspace_bytes(T, k, E_local))


def alloc_dispatch_workspace(T: int, k: int, E_local: int, device) -> torch.Tensor:
    """A zeroed workspace for moe_route_dispatch (int32 words; word 0 is the device status word)."""
    nbytes = moe_route_dispatch_workspace_bytes(T, k, E_local)
    return torch.zeros((nbytes + 3) // 4, dtype=torch.int32, device=device)


def moe_route_dispatch(logits: Optional[torch.Tensor], hidden: torch.Tensor, k: int, renormalize: bool,
                       block_size: int, expert_map: Optional[torch.Tensor] = None, E_local: Optional[int] = None,
                       topk_weights: Optional[torch.Tensor] = None, topk_ids: Optional[torch.Tensor] = None,
                       align: Optional[AlignResult] = None, permuted: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None, given_ids: bool = False,
                       E: Optional[int] = None, scoring: str = "softmax"):
    """Gating + align + permute-gather in one call.  Returns (topk_weights, topk_ids, AlignResult, permuted).

    With ``given_ids`` the routes in ``topk_ids`` are the input (no gating): ``logits`` may be None (then
    ``E`` gives the number of global experts) and ``topk_weights`` is neither read nor written."""
    T, H = hidden.shape
    if logits is not None:
        assert logits.shape[0] == T
        E = logits.shape[1]
    if E is None:
        raise ValueError("E is needed when logits is None")
    if logits is None or logits.dtype == torch.bfloat16:
        dt = MOE_DTYPE_BF16
    elif logits.dtype == torch.float32:
        dt = MOE_DTYPE_F32
    else:
        raise ValueError(f"logits dtype {logits.dtype} unsupported (bf16 or fp32)")
    if logits is None and not given_ids:
        raise ValueError("logits are needed unless the routes are given")
    assert hidden.dtype == torch.bfloat16
    if E_local is None:
        E_local = E
    dev = hidden.device
    if topk_weights is None and not given_ids:
        topk_weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    if topk_ids is None:
        if given_ids:
            raise ValueError("given_ids needs topk_ids")
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if align is None:
        align = alloc_align_outputs(T, k, E_local, block_size, dev)
    if permuted is None:
        permuted = torch.empty((align.capacity, H), dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = alloc_dispatch_workspace(T, k, E_local, dev)
    assert expert_map is None or expert_map.dtype == torch.int32
    flags = (MOE_RENORMALIZE if renormalize else 0) | (MOE_DISPATCH_GIVEN_IDS if given_ids else 0) | \
        _scoring_flag(scoring)
    st = load_library().moe_route_dispatch(
        _dev(logits, "logits"), dt, _dev(hidden, "hidden"), T, E, k, H, flags,
        _dev(expert_map, "expert_map"), E_local, block_size, _dev(topk_weights, "topk_weights"),
        _dev(topk_ids, "topk_ids"), _dev(align.counts, "counts"), _dev(align.offsets, "offsets"),
        _dev(align.sorted_token_ids, "sorted_token_ids"), _dev(align.expert_ids, "expert_ids"),
        _dev(align.num_tokens_post_pad, "num_tokens_post_pad"), _dev(align.inv_perm, "inv_perm"),
        _dev(permuted, "permuted"), _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(st, "moe_route_dispatch")
    return topk_weights, topk_ids, align, permuted


def moe_read_status(device_status_word: torch.Tensor, stream=None) -> int:
    """Read (and reset) a device status word; returns the recorded moe_status_t (0 = none)."""
    v = ctypes.c_int(0)
    _check(load_library().moe_read_status(_dev(device_status_word, "device_status_word"), _stream(stream),
                                          ctypes.byref(v)), "moe_read_status")
    return int(v.value)


# ------------------------------------------------------------ gradients and 4-bit products --
# A decode-sized kernel runs in a few microseconds, so what these wrappers do before the launch counts: one test of a
# good tensor, reasons only for a bad one; the raw current stream (0.1 us) instead of a Stream object (3 us).
def _arg(t, name: str, dtype, shape, index: int) -> int:
    """Address of a contiguous CUDA tensor of this dtype and shape on device `index` (ValueError otherwise)."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t is None:
        raise ValueError(f"{name} is missing")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the routing path runs only on the GPU)")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{index}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """A new tensor on `like`'s device, from the memory of the stream that will write it: memory freed on another stream
    may still be in use there."""
    if stream is None or not like.is_cuda:
        return like.new_empty(shape, dtype=dtype)
    if not isinstance(stream, torch.cuda.Stream):
        # (ExternalStream takes handle 0, the default stream's, for "no handle": it would be some stream of torch's pool)
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=like.device) if handle else torch.cuda.default_stream(like.device)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _out(t, name: str, dtype, shape, like: torch.Tensor, stream):
    """An output and its address: t, checked, or a new tensor."""
    if t is None:
        t = _new(like, shape, dtype, stream)
        return t, t.data_ptr()
    return t, _arg(t, name, dtype, shape, like.get_device())


def _matrix(t, name: str):
    if t is None or t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    return t.shape


def _call(name: str, index: int, stream, *args) -> None:
    """Run an entry point with device `index` current, on `stream` or that device's current stream (the last argument)."""
    if index < 0:
        raise ValueError(f"{name} needs CUDA tensors (the routing path runs only on the GPU)")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device.index != index:
            raise ValueError(f"{name}: the stream belongs to {stream.device}, the tensors to cuda:{index}")
        stream = stream.cuda_stream
    fn = getattr(_lib or load_library(), name)
    if torch.cuda.current_device() == index:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            st = fn(*args, stream)
    if st != MOE_OK:
        raise MoeError(st, name)


def _status_arg(device_status, index: int):
    """The status word: the first element of an int32 tensor (a workspace, or a word of its own), or None."""
    if device_status is None:
        return None
    if device_status.numel() < 1:
        raise ValueError("device_status must hold a word")
    return _arg(device_status, "device_status", torch.int32, device_status.shape, index)


def moe_combine_backward(grad_out: torch.Tensor, expert_out: torch.Tensor, topk_weights: torch.Tensor,
                         inv_perm: torch.Tensor, grad_expert_out: Optional[torch.Tensor] = None,
                         grad_topk_weights: Optional[torch.Tensor] = None,
                         sorted_token_ids: Optional[torch.Tensor] = None,
                         num_tokens_post_pad: Optional[torch.Tensor] = None, zero_pad: bool = False,
                         device_status: Optional[torch.Tensor] = None, stream=None):
    """Gradient of moe_combine: grad_out [T, H] bf16, expert_out [capacity, H] bf16 and topk_weights [T, k] fp32 ->
    (grad_expert_out [capacity, H] bf16, grad_topk_weights [T, k] fp32).

    zero_pad writes +0 into the pad rows below N_pad (needs sorted_token_ids and num_tokens_post_pad); other rows of
    no slot are left as they were.  grad_expert_out may be expert_out itself."""
    T, H = _matrix(grad_out, "grad_out")
    k = _matrix(topk_weights, "topk_weights")[1]
    capacity = _matrix(expert_out, "expert_out")[0]
    dev, bf16 = grad_out.get_device(), torch.bfloat16
    grad_expert_out, gy = _out(grad_expert_out, "grad_expert_out", bf16, (capacity, H), grad_out, stream)
    grad_topk_weights, gw = _out(grad_topk_weights, "grad_topk_weights", torch.float32, (T, k), grad_out, stream)
    pads = (None, None)
    if zero_pad:
        pads = (_arg(sorted_token_ids, "sorted_token_ids", torch.int32, (capacity,), dev),
                _arg(num_tokens_post_pad, "num_tokens_post_pad", torch.int32, (1,), dev))
    _call("moe_combine_backward", dev, stream, _arg(grad_out, "grad_out", bf16, (T, H), dev),
          _arg(expert_out, "expert_out", bf16, (capacity, H), dev),
          _arg(topk_weights, "topk_weights", torch.float32, (T, k), dev),
          _arg(inv_perm, "inv_perm", torch.int32, (T * k,), dev), *pads, T, k, H, capacity,
          MOE_GATHER_ZERO_PAD if zero_pad else 0, gy, gw, _status_arg(device_status, dev))
    return grad_expert_out, grad_topk_weights


def moe_gather_backward(grad_permuted: torch.Tensor, inv_perm: torch.Tensor, k: int,
                        grad_hidden: Optional[torch.Tensor] = None, device_status: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Gradient of moe_gather: grad_permuted [capacity, H] bf16 -> grad_hidden [T, H] bf16, each token's local rows
    summed in fp32 (inv_perm holds T*k slots)."""
    capacity, H = _matrix(grad_permuted, "grad_permuted")
    if k < 1 or inv_perm.numel() % k != 0:
        raise ValueError(f"inv_perm must hold T * k slots, got {inv_perm.numel()} with k = {k}")
    T, dev = inv_perm.numel() // k, grad_permuted.get_device()
    grad_hidden, gx = _out(grad_hidden, "grad_hidden", torch.bfloat16, (T, H), grad_permuted, stream)
    _call("moe_gather_backward", dev, stream,
          _arg(grad_permuted, "grad_permuted", torch.bfloat16, (capacity, H), dev),
          _arg(inv_perm, "inv_perm", torch.int32, (T * k,), dev), T, k, H, capacity, gx, _status_arg(device_status, dev))
    return grad_hidden


def moe_topk_softmax_backward(grad_topk_weights: torch.Tensor, logits: torch.Tensor, topk_weights: torch.Tensor,
                              topk_ids: torch.Tensor, renormalize: bool, grad_logits: Optional[torch.Tensor] = None,
                              device_status: Optional[torch.Tensor] = None, stream=None,
                              scoring: str = "softmax") -> torch.Tensor:
    """Gradient of moe_topk_softmax: grad_topk_weights [T, k] fp32 -> grad_logits [T, E] of the logits' dtype.
    topk_weights and topk_ids are what moe_topk_softmax returned with the same renormalize and scoring."""
    T, E = _matrix(logits, "logits")
    k = _matrix(topk_weights, "topk_weights")[1]
    dev, dtype = logits.get_device(), logits.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"logits dtype {dtype} unsupported (bf16 or fp32)")
    grad_logits, gx = _out(grad_logits, "grad_logits", dtype, (T, E), logits, stream)
    f32 = torch.float32
    _call("moe_topk_softmax_backward", dev, stream, _arg(grad_topk_weights, "grad_topk_weights", f32, (T, k), dev),
          _arg(logits, "logits", dtype, (T, E), dev), MOE_DTYPE_BF16 if dtype == torch.bfloat16 else MOE_DTYPE_F32,
          _arg(topk_weights, "topk_weights", f32, (T, k), dev), _arg(topk_ids, "topk_ids", torch.int32, (T, k), dev), T,
          E, k, (MOE_RENORMALIZE if renormalize else 0) | _scoring_flag(scoring),
          gx, _status_arg(device_status, dev))
    return grad_logits


class Mx4Tensor(NamedTuple):
    """A matrix [rows, K] in microscaled 4-bit floating point (layout: moe_route.h)."""
    codes: torch.Tensor   # uint8 [rows, K/2]
    scales: torch.Tensor  # uint8 [ceil(K/128), rows, 4]

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def K(self) -> int:
        return self.codes.shape[1] * 2


def alloc_mx4(rows: int, K: int, device) -> Mx4Tensor:
    if K < 32 or K % 32 != 0:
        raise ValueError(f"a row holds whole blocks of 32 elements, got K = {K}")
    return Mx4Tensor(torch.empty((rows, K // 2), dtype=torch.uint8, device=device),
                     torch.empty((-(-K // 128), rows, 4), dtype=torch.uint8, device=device))


def _mx4_out(out: Optional[Mx4Tensor], rows: int, K: int, like: torch.Tensor, stream):
    """An output in the format and its addresses: `out`, checked, or a new one."""
    if out is None:
        if K < 32 or K % 32 != 0:
            raise ValueError(f"a row holds whole blocks of 32 elements, got K = {K}")
        out = Mx4Tensor(_new(like, (rows, K // 2), torch.uint8, stream),
                        _new(like, (-(-K // 128), rows, 4), torch.uint8, stream))
        return out, out.codes.data_ptr(), out.scales.data_ptr()
    index = like.get_device()
    return (out, _arg(out[0], "out.codes", torch.uint8, (rows, K // 2), index),
            _arg(out[1], "out.scales", torch.uint8, ((K + 127) // 128, rows, 4), index))


def moe_quantize_mx4(x: torch.Tensor, out: Optional[Mx4Tensor] = None, num_rows: Optional[torch.Tensor] = None,
                     stream=None) -> Mx4Tensor:
    """x [rows, K] bf16 -> microscaled 4-bit floating point (K a multiple of 32).  num_rows (int32 [1] on the device):
    rows from there on are neither read nor written."""
    rows, K = _matrix(x, "x")
    out, codes, scales = _mx4_out(out, rows, K, x, stream)
    dev = x.get_device()
    _call("moe_quantize_mx4", dev, stream, _arg(x, "x", torch.bfloat16, (rows, K), dev), rows, K,
          None if num_rows is None else _arg(num_rows, "num_rows", torch.int32, (1,), dev), codes, scales)
    return out


def moe_dequantize_mx4(q: Mx4Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values of q as bf16 [rows, K]."""
    codes, scales = q
    dev, (rows, half) = codes.get_device(), _matrix(codes, "q.codes")
    out, p = _out(out, "out", torch.bfloat16, (rows, 2 * half), codes, stream)
    _call("moe_dequantize_mx4", dev, stream, _arg(codes, "q.codes", torch.uint8, (rows, half), dev),
          _arg(scales, "q.scales", torch.uint8, ((half + 63) // 64, rows, 4), dev), rows, 2 * half, p)
    return out


def moe_gather_mx4(hidden: torch.Tensor, k: int, inv_perm: torch.Tensor, capacity: int,
                   out: Optional[Mx4Tensor] = None, device_status: Optional[torch.Tensor] = None,
                   stream=None) -> Mx4Tensor:
    """moe_gather in microscaled 4-bit floating point: hidden [T, H] bf16 -> expert-grouped rows [capacity, H].
    Rows of no slot are left as they were."""
    T, H = _matrix(hidden, "hidden")
    dev = hidden.get_device()
    out, codes, scales = _mx4_out(out, capacity, H, hidden, stream)
    _call("moe_gather_mx4", dev, stream, _arg(hidden, "hidden", torch.bfloat16, (T, H), dev), T, H, k,
          _arg(inv_perm, "inv_perm", torch.int32, (T * k,), dev), capacity,
          codes, scales, _status_arg(device_status, dev))
    return out


def moe_grouped_gemm_mx4(x: Mx4Tensor, w: Mx4Tensor, counts: torch.Tensor, offsets: torch.Tensor,
                         out: Optional[torch.Tensor] = None, swiglu: bool = False,
                         device_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The experts' product on expert-grouped rows: x [capacity, K], w [E_local * N, K] (expert e's feature n in row
    e * N + n), counts [E_local] and offsets [E_local + 1] as from moe_align_permute -> out [capacity, N] bf16, or
    [capacity, N/2] = silu(first half) * second half with swiglu.  Rows of no expert are left as they were."""
    (xc, xs), (wc, ws), u8 = x, w, torch.uint8
    dev, E = xc.get_device(), counts.numel()
    (capacity, half), (w_rows, w_half) = _matrix(xc, "x.codes"), _matrix(wc, "w.codes")
    if E < 1 or w_rows % E != 0:
        raise ValueError(f"w must hold E_local * N rows, got {w_rows} for {E} experts")
    if w_half != half:
        raise ValueError(f"x has rows of {2 * half}, w of {2 * w_half}")
    N, chunks = w_rows // E, (half + 63) // 64
    if swiglu and N % 2 != 0:
        raise ValueError(f"swiglu needs an even number of features, got {N}")
    out, p = _out(out, "out", torch.bfloat16, (capacity, N // 2 if swiglu else N), xc, stream)
    _call("moe_grouped_gemm_mx4", dev, stream, _arg(xc, "x.codes", u8, (capacity, half), dev),
          _arg(xs, "x.scales", u8, (chunks, capacity, 4), dev), _arg(wc, "w.codes", u8, (w_rows, half), dev),
          _arg(ws, "w.scales", u8, (chunks, w_rows, 4), dev), _arg(counts, "counts", torch.int32, (E,), dev),
          _arg(offsets, "offsets", torch.int32, (E + 1,), dev), E, capacity, N, 2 * half,
          MOE_MX4_SWIGLU if swiglu else 0, p, _status_arg(device_status, dev))
    return out
