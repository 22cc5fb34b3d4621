"""Python binding of libhr (``include/hr.h``): argument marshalling only.

Every function named ``hr_*`` here calls the C entry point of the same name
with the same arguments; every step of the combine runs in libhr's HIP
kernels.  The torch helpers at the bottom only turn tensors and streams into
the device pointers and ``hipStream_t`` handles those entry points take:
PyTorch is used for device memory and streams, nothing else.

The library is loaded from this package's directory on first use.  If it is
missing, loading raises ``ImportError``: there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhr.so")

HR_OK = 0
HR_ERR_INVALID_ARG = 1
HR_ERR_ALIGNMENT = 2
HR_ERR_TOO_LARGE = 3
HR_ERR_UNSUPPORTED = 4
HR_ERR_HIP = 5
HR_ERR_TIMEOUT = 6
HR_ERR_ABORTED = 7

HR_MAX_G = 16
HR_MAX_WORLD = 8
HR_DEFAULT_MAX_NUMEL = 131072
HR_MAX_NUMEL_LIMIT = 1 << 29
HR_NOALLOC_MAX_NUMEL = 131072
HR_NOALLOC_SCRATCH_BYTES = 8 << 20
HR_DEFAULT_TIMEOUT_US = 1_000_000
HR_DEFAULT_LINK_MBPS = 50_000
HR_LINK_UNPACED = 0xFFFFFFFF
HR_LINK_CALIBRATE = 0xFFFFFFFE
HR_MIN_LINK_MBPS = 100
HR_ALGO_AUTO = 0
HR_ALGO_ONE_SHOT = 1
HR_ALGO_TWO_SHOT = 2
HR_ALGO_LL = 3

# Every symbol include/hr.h declares.
EXPORTS = ("hr_create_channel", "hr_allreduce_f16", "hr_reduce_f16", "hr_channel_status",
           "hr_channel_abort", "hr_channel_get_info", "hr_destroy", "hr_status_str",
           "hr_loopback_stream_create", "hr_loopback_stream_destroy",
           "hr_reduce_bf16", "hr_allreduce_bf16", "hr_admit", "hr_route_str", "hr_decode_numel",
           "hr_workspace_stride", "hr_exchange_algorithm", "hr_allreduce_group_f16",
           "hr_allreduce_group_bf16", "hr_allreduce_group_noalloc_f16", "hr_channel_timeout_info",
           "hr_reduce_rmsnorm_f16", "hr_reduce_rmsnorm_bf16", "hr_rmsnorm_grad_f16", "hr_rmsnorm_grad_bf16",
           "hr_rmsnorm_grad_workspace", "hr_router_topk", "hr_router_topk_grad", "hr_experts_rows",
           "hr_experts_sort_workspace", "hr_experts_sort", "hr_experts_gather", "hr_experts_combine_f16",
           "hr_experts_combine_bf16", "hr_experts_combine_grad_f16", "hr_experts_combine_grad_bf16")

HR_ROUTE_HOST = 0
HR_DECLINE_DISABLED = 1
HR_DECLINE_DTYPE = 2
HR_DECLINE_WORLD_SIZE = 3
HR_DECLINE_PEER_ACCESS = 4
HR_DECLINE_TOO_LARGE = 5
HR_DTYPE_F16 = 0
HR_DTYPE_BF16 = 1
HR_DTYPE_OTHER = 2
HR_DTYPE_F32 = 3

HR_RMSNORM_MAX_HIDDEN = 32768
HR_RMSNORM_GRAD_FEW_ROWS = 256
HR_ROUTER_MAX_EXPERTS = 1024
HR_ROUTER_MAX_K = 32
HR_ROUTER_MAX_TOKENS = (1 << 26) - 4
HR_EXPERTS_MAX = 1024
HR_EXPERTS_MAX_K = 32
HR_EXPERTS_SORT_FEW = 8192


class hr_channel_config(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int),
                ("world_size", ctypes.c_int),
                ("max_numel", ctypes.c_size_t),
                ("num_blocks", ctypes.c_int),
                ("timeout_us", ctypes.c_uint32),
                ("algorithm", ctypes.c_int),
                ("link_mbps", ctypes.c_uint32)]


class hr_admit_policy(ctypes.Structure):
    _fields_ = [("enabled", ctypes.c_int),
                ("max_bytes", ctypes.c_size_t),
                ("allow_bf16", ctypes.c_int),
                ("max_world", ctypes.c_int)]


class hr_channel_info(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int),
                ("world_size", ctypes.c_int),
                ("max_numel", ctypes.c_size_t),
                ("num_blocks", ctypes.c_int),
                ("block_threads", ctypes.c_int),
                ("timeout_us", ctypes.c_uint32),
                ("host_slots", ctypes.c_void_p),
                ("slot_stride", ctypes.c_size_t),
                ("host_flags", ctypes.POINTER(ctypes.c_uint64)),
                ("flag_stride", ctypes.c_size_t),
                ("host_error", ctypes.POINTER(ctypes.c_uint32)),
                ("host_abort", ctypes.POINTER(ctypes.c_uint32)),
                ("algorithm", ctypes.c_int),
                ("host_reduced", ctypes.c_void_p),
                ("host_flags2", ctypes.POINTER(ctypes.c_uint64)),
                ("host_ll", ctypes.c_void_p),
                ("ll_stride", ctypes.c_size_t),
                ("link_mbps", ctypes.c_uint32),
                ("dev_epochs", ctypes.c_void_p)]


class hr_rmsnorm_args(ctypes.Structure):
    _fields_ = [("inputs", ctypes.c_void_p * HR_MAX_G),
                *((n, ctypes.c_void_p) for n in ("residual", "weight", "residual_out", "out", "codes", "scales",
                                                 "rstd")),
                *((n, ctypes.c_size_t) for n in ("rows", "hidden", "input_stride", "residual_stride",
                                                 "residual_out_stride", "out_stride", "codes_stride",
                                                 "scales_stride")),
                ("G", ctypes.c_int),
                ("weight_f32", ctypes.c_int),
                ("group", ctypes.c_int),
                ("eps", ctypes.c_float)]


class hr_rmsnorm_grad_args(ctypes.Structure):
    _fields_ = [*((n, ctypes.c_void_p) for n in ("dy", "h", "rstd", "weight", "dresidual", "dx", "dweight",
                                                 "workspace")),
                *((n, ctypes.c_size_t) for n in ("workspace_bytes", "rows", "hidden", "dy_stride", "h_stride",
                                                 "dresidual_stride", "dx_stride")),
                ("weight_f32", ctypes.c_int)]


class hr_experts_gather_args(ctypes.Structure):
    _fields_ = [*((n, ctypes.c_void_p) for n in ("in_", "scales", "out", "scales_out", "pos", "order", "offsets")),
                *((n, ctypes.c_size_t) for n in ("tokens", "rows", "row_bytes", "in_stride", "out_stride",
                                                 "scales_width", "scales_stride", "scales_out_stride")),
                ("k", ctypes.c_int),
                ("experts", ctypes.c_int)]


class hr_experts_combine_args(ctypes.Structure):
    _fields_ = [*((n, ctypes.c_void_p) for n in ("z", "addend", "out", "pos", "weights")),
                *((n, ctypes.c_size_t) for n in ("tokens", "rows", "hidden", "z_stride", "addend_stride",
                                                 "out_stride")),
                ("k", ctypes.c_int)]


class hr_experts_combine_grad_args(ctypes.Structure):
    _fields_ = [*((n, ctypes.c_void_p) for n in ("dy", "z", "dz", "pos", "weights", "dweights", "order",
                                                 "offsets")),
                *((n, ctypes.c_size_t) for n in ("tokens", "rows", "hidden", "dy_stride", "z_stride", "dz_stride")),
                ("k", ctypes.c_int),
                ("experts", ctypes.c_int)]


class HrError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {hr_status_str(status)} ({status})")


_lib = None


def load() -> ctypes.CDLL:
    """Load libhr.so from this package (raises ImportError if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run python -m message_fp16_all_amd.build")
    # torch ships its own HIP runtime under the same soname as the system one;
    # whichever loads first serves the process.  Load torch's first (when
    # torch is installed), so that the library and torch share one runtime.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(LIB_PATH)
    vp = ctypes.c_void_p
    lib.hr_create_channel.argtypes = [ctypes.POINTER(hr_channel_config), ctypes.POINTER(vp)]
    lib.hr_allreduce_f16.argtypes = [vp, ctypes.c_int, vp, vp, ctypes.c_size_t, vp]
    lib.hr_reduce_f16.argtypes = [ctypes.POINTER(vp), ctypes.c_int, vp, ctypes.c_size_t, vp]
    lib.hr_allreduce_bf16.argtypes = [vp, ctypes.c_int, vp, vp, ctypes.c_size_t, vp]
    lib.hr_allreduce_group_f16.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.c_size_t, vp]
    lib.hr_allreduce_group_bf16.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.c_size_t, vp]
    lib.hr_allreduce_group_noalloc_f16.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.c_int,
                                                   ctypes.c_size_t, vp, vp]
    lib.hr_reduce_bf16.argtypes = [ctypes.POINTER(vp), ctypes.c_int, vp, ctypes.c_size_t, vp]
    lib.hr_channel_status.argtypes = [vp]
    lib.hr_exchange_algorithm.argtypes = [vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int)]
    lib.hr_channel_abort.argtypes = [vp]
    lib.hr_channel_timeout_info.argtypes = [vp, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_uint32),
                                            ctypes.POINTER(ctypes.c_uint64)]
    lib.hr_channel_get_info.argtypes = [vp, ctypes.POINTER(hr_channel_info)]
    lib.hr_destroy.argtypes = [vp]
    lib.hr_loopback_stream_create.argtypes = [ctypes.c_int, ctypes.POINTER(vp)]
    lib.hr_loopback_stream_destroy.argtypes = [vp]
    lib.hr_status_str.argtypes = [ctypes.c_int]
    lib.hr_status_str.restype = ctypes.c_char_p
    lib.hr_admit.argtypes = [ctypes.POINTER(hr_admit_policy), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                             ctypes.c_size_t]
    lib.hr_route_str.argtypes = [ctypes.c_int]
    lib.hr_route_str.restype = ctypes.c_char_p
    lib.hr_decode_numel.argtypes = [ctypes.c_size_t, ctypes.c_size_t, ctypes.c_size_t]
    lib.hr_workspace_stride.argtypes = [ctypes.c_size_t]
    # argument structs: byref of the ctypes struct, or its bytes
    for name in ("hr_reduce_rmsnorm_f16", "hr_reduce_rmsnorm_bf16", "hr_rmsnorm_grad_f16", "hr_rmsnorm_grad_bf16",
                 "hr_experts_gather", "hr_experts_combine_f16", "hr_experts_combine_bf16",
                 "hr_experts_combine_grad_f16", "hr_experts_combine_grad_bf16"):
        getattr(lib, name).argtypes = [vp, vp]
    lib.hr_rmsnorm_grad_workspace.argtypes = [ctypes.c_size_t, ctypes.c_size_t]
    lib.hr_router_topk.argtypes = [vp, ctypes.c_int, ctypes.c_size_t, ctypes.c_int, ctypes.c_size_t, ctypes.c_int,
                                   ctypes.c_int, vp, vp, vp]
    lib.hr_router_topk_grad.argtypes = [vp, vp, vp, vp, ctypes.c_int, ctypes.c_size_t, ctypes.c_int, ctypes.c_size_t,
                                        ctypes.c_int, ctypes.c_int, vp, ctypes.c_size_t, vp]
    lib.hr_experts_rows.argtypes = [ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    lib.hr_experts_sort_workspace.argtypes = [ctypes.c_size_t, ctypes.c_int, ctypes.c_int]
    lib.hr_experts_sort.argtypes = [vp, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, vp,
                                    vp, ctypes.c_size_t, vp, vp, ctypes.c_size_t, vp]
    sizes = ("hr_decode_numel", "hr_workspace_stride", "hr_rmsnorm_grad_workspace", "hr_experts_rows",
             "hr_experts_sort_workspace")
    for name in sizes:
        getattr(lib, name).restype = ctypes.c_size_t
    for name in EXPORTS:
        if name not in ("hr_status_str", "hr_route_str", *sizes):
            getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


# ------------------------------------------------------- the C entry points

def hr_status_str(status: int) -> str:
    return load().hr_status_str(int(status)).decode()


def hr_create_channel(device: int = 0, world_size: int = 2, max_numel: int = 0,
                      num_blocks: int = 0, timeout_us: int = 0, algorithm: int = 0,
                      link_mbps: int = 0) -> int:
    """Returns the channel handle (an integer address) or raises HrError."""
    cfg = hr_channel_config(device, world_size, max_numel, num_blocks, timeout_us, algorithm, link_mbps)
    h = ctypes.c_void_p()
    st = load().hr_create_channel(ctypes.byref(cfg), ctypes.byref(h))
    if st != HR_OK:
        raise HrError(st, "hr_create_channel")
    return h.value


def hr_allreduce_f16(ch: int, rank: int, in_ptr: int, out_ptr: int, numel: int,
                     stream: int) -> int:
    """Raw call; returns the hr_status code."""
    return load().hr_allreduce_f16(ch, rank, in_ptr, out_ptr, numel, stream)


def hr_reduce_f16(ptrs, G: int, out_ptr: int, numel: int, stream: int) -> int:
    """Raw call; ``ptrs`` is a sequence of G device addresses.  Returns hr_status."""
    arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
    return load().hr_reduce_f16(arr, G, out_ptr, numel, stream)


def hr_allreduce_bf16(ch: int, rank: int, in_ptr: int, out_ptr: int, numel: int,
                      stream: int) -> int:
    """Raw call; returns the hr_status code."""
    return load().hr_allreduce_bf16(ch, rank, in_ptr, out_ptr, numel, stream)


def hr_allreduce_group_f16(ch: int, in_ptrs, out_ptrs, numel: int, stream: int) -> int:
    """Raw call; ``in_ptrs``/``out_ptrs`` are sequences of world_size device
    addresses (None for a null pointer).  Returns the hr_status code."""
    ins = (ctypes.c_void_p * max(1, len(in_ptrs)))(*in_ptrs)
    outs = (ctypes.c_void_p * max(1, len(out_ptrs)))(*out_ptrs)
    return load().hr_allreduce_group_f16(ch, ins, outs, numel, stream)


def hr_allreduce_group_bf16(ch: int, in_ptrs, out_ptrs, numel: int, stream: int) -> int:
    """As hr_allreduce_group_f16 for bfloat16 buffers."""
    ins = (ctypes.c_void_p * max(1, len(in_ptrs)))(*in_ptrs)
    outs = (ctypes.c_void_p * max(1, len(out_ptrs)))(*out_ptrs)
    return load().hr_allreduce_group_bf16(ch, ins, outs, numel, stream)


def hr_allreduce_group_noalloc_f16(in_ptrs, out_ptrs, world_size: int, numel: int, status_ptr,
                                   stream: int) -> int:
    """Raw call of the channel-free group all-reduce; ``status_ptr`` is a
    device address or None.  Returns the hr_status code."""
    ins = (ctypes.c_void_p * max(1, len(in_ptrs)))(*in_ptrs)
    outs = (ctypes.c_void_p * max(1, len(out_ptrs)))(*out_ptrs)
    return load().hr_allreduce_group_noalloc_f16(ins, outs, world_size, numel, status_ptr, stream)


def hr_reduce_bf16(ptrs, G: int, out_ptr: int, numel: int, stream: int) -> int:
    """Raw call; ``ptrs`` is a sequence of G device addresses.  Returns hr_status."""
    arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
    return load().hr_reduce_bf16(arr, G, out_ptr, numel, stream)


def hr_channel_status(ch: int) -> int:
    return load().hr_channel_status(ch)


def hr_exchange_algorithm(ch: int, numel: int) -> int:
    """The HR_ALGO_* a call of numel values takes (raises HrError)."""
    algo = ctypes.c_int(-1)
    st = load().hr_exchange_algorithm(ch, numel, ctypes.byref(algo))
    if st != HR_OK:
        raise HrError(st, "hr_exchange_algorithm")
    return algo.value


def hr_channel_abort(ch: int) -> int:
    return load().hr_channel_abort(ch)


def hr_channel_timeout_info(ch: int):
    """(rank, peer_mask, call) of the channel's timeout record; rank is -1
    when nothing is recorded (raises HrError)."""
    rank, mask, call = ctypes.c_int(-1), ctypes.c_uint32(0), ctypes.c_uint64(0)
    st = load().hr_channel_timeout_info(ch, ctypes.byref(rank), ctypes.byref(mask), ctypes.byref(call))
    if st != HR_OK:
        raise HrError(st, "hr_channel_timeout_info")
    return rank.value, mask.value, call.value


def hr_channel_get_info(ch: int) -> hr_channel_info:
    info = hr_channel_info()
    st = load().hr_channel_get_info(ch, ctypes.byref(info))
    if st != HR_OK:
        raise HrError(st, "hr_channel_get_info")
    return info


def hr_destroy(ch: int) -> int:
    return load().hr_destroy(ch)


def hr_loopback_stream_create(device: int = 0) -> int:
    """Returns a hipStream_t (integer) that owns its hardware queue."""
    h = ctypes.c_void_p()
    st = load().hr_loopback_stream_create(device, ctypes.byref(h))
    if st != HR_OK:
        raise HrError(st, "hr_loopback_stream_create")
    return h.value


def hr_loopback_stream_destroy(stream: int) -> int:
    return load().hr_loopback_stream_destroy(stream)


def hr_admit(policy, dtype: int, world_size: int, peer_access: bool, numel: int) -> int:
    """Route code for one reduction; ``policy`` is an hr_admit_policy or None."""
    ref = ctypes.byref(policy) if policy is not None else None
    return load().hr_admit(ref, dtype, world_size, int(bool(peer_access)), numel)


def hr_route_str(route: int) -> str:
    return load().hr_route_str(int(route)).decode()


def hr_decode_numel(max_batch: int, tokens_per_request: int, hidden: int) -> int:
    return load().hr_decode_numel(max_batch, tokens_per_request, hidden)


def hr_workspace_stride(numel: int) -> int:
    """Values between consecutive contributions in one fold workspace."""
    return load().hr_workspace_stride(numel)


def hr_reduce_rmsnorm_f16(args, stream: int) -> int:
    """Raw call; ``args`` is an hr_rmsnorm_args.  Returns the hr_status code."""
    return load().hr_reduce_rmsnorm_f16(ctypes.byref(args), stream)


def hr_reduce_rmsnorm_bf16(args, stream: int) -> int:
    """As hr_reduce_rmsnorm_f16 for bfloat16 buffers."""
    return load().hr_reduce_rmsnorm_bf16(ctypes.byref(args), stream)


def hr_rmsnorm_grad_f16(args, stream: int) -> int:
    """Raw call; ``args`` is an hr_rmsnorm_grad_args.  Returns the hr_status code."""
    return load().hr_rmsnorm_grad_f16(ctypes.byref(args), stream)


def hr_rmsnorm_grad_bf16(args, stream: int) -> int:
    """As hr_rmsnorm_grad_f16 for bfloat16 buffers."""
    return load().hr_rmsnorm_grad_bf16(ctypes.byref(args), stream)


def hr_rmsnorm_grad_workspace(rows: int, hidden: int) -> int:
    """Bytes of workspace that a gradient call with dweight needs."""
    return load().hr_rmsnorm_grad_workspace(rows, hidden)


def hr_router_topk(logits_ptr, dtype: int, tokens: int, experts: int, logits_stride: int, k: int, renormalize: int,
                   weights_ptr, ids_ptr, stream: int) -> int:
    """Raw call; returns the hr_status code."""
    return load().hr_router_topk(logits_ptr, dtype, tokens, experts, logits_stride, k, renormalize, weights_ptr,
                                 ids_ptr, stream)


def hr_router_topk_grad(dweights_ptr, weights_ptr, ids_ptr, logits_ptr, dtype: int, tokens: int, experts: int,
                        logits_stride: int, k: int, renormalize: int, dlogits_ptr, dlogits_stride: int,
                        stream: int) -> int:
    """Raw call; returns the hr_status code."""
    return load().hr_router_topk_grad(dweights_ptr, weights_ptr, ids_ptr, logits_ptr, dtype, tokens, experts,
                                      logits_stride, k, renormalize, dlogits_ptr, dlogits_stride, stream)


def hr_experts_rows(tokens: int, k: int, experts: int, pad: int = 1) -> int:
    """Rows that sorted tokens take at most (0 for arguments out of range)."""
    return load().hr_experts_rows(tokens, k, experts, pad)


def hr_experts_sort_workspace(tokens: int, k: int, experts: int) -> int:
    """Bytes of workspace that a sort needs."""
    return load().hr_experts_sort_workspace(tokens, k, experts)


def hr_experts_sort(ids_ptr, tokens: int, k: int, first: int, experts: int, pad: int, offsets_ptr, order_ptr, rows: int,
                    pos_ptr, workspace_ptr, workspace_bytes: int, stream: int) -> int:
    """Raw call; returns the hr_status code."""
    return load().hr_experts_sort(ids_ptr, tokens, k, first, experts, pad, offsets_ptr, order_ptr, rows, pos_ptr,
                                  workspace_ptr, workspace_bytes, stream)


def hr_experts_gather(args, stream: int) -> int:
    """Raw call; ``args`` is an hr_experts_gather_args.  Returns the hr_status code."""
    return load().hr_experts_gather(ctypes.byref(args), stream)


def hr_experts_combine_f16(args, stream: int) -> int:
    """Raw call; ``args`` is an hr_experts_combine_args.  Returns the hr_status code."""
    return load().hr_experts_combine_f16(ctypes.byref(args), stream)


def hr_experts_combine_bf16(args, stream: int) -> int:
    """As hr_experts_combine_f16 for bfloat16 buffers."""
    return load().hr_experts_combine_bf16(ctypes.byref(args), stream)


def hr_experts_combine_grad_f16(args, stream: int) -> int:
    """Raw call; ``args`` is an hr_experts_combine_grad_args.  Returns the hr_status code."""
    return load().hr_experts_combine_grad_f16(ctypes.byref(args), stream)


def hr_experts_combine_grad_bf16(args, stream: int) -> int:
    """As hr_experts_combine_grad_f16 for bfloat16 buffers."""
    return load().hr_experts_combine_grad_bf16(ctypes.byref(args), stream)


def workspace(G: int, numel: int, dtype=None, device=0):
    """A device buffer holding G contributions in the hr_workspace_stride
    layout; returns (buffer, [view of contribution g])."""
    import torch
    dtype = torch.float16 if dtype is None else dtype
    stride = hr_workspace_stride(numel)
    buf = torch.empty(G * stride, dtype=dtype, device=torch.device("cuda", device))
    return buf, [buf[g * stride:g * stride + numel] for g in range(G)]


# ----------------------------------------------------- torch marshalling
#
# An eager call's host time is HIP's kernel launch (about 3 us) plus this
# marshalling, so the per-call helpers keep to attribute reads: torch and its
# two element types are looked up once, dtypes are compared by identity
# (torch dtypes are singletons), and a Channel binds its entry points once.
# Measured on MI355X, host time per enqueued Channel.allreduce: 4.62-4.76 us
# with an import and equality compares per call, 4.22-4.33 us as here, and
# 3.28-3.76 us for the bare ctypes call.

_torch = None
_F16 = None
_BF16 = None


def _tm():
    """The torch module, imported on first use (with its two dtypes)."""
    global _torch, _F16, _BF16
    if _torch is None:
        import torch
        _F16, _BF16 = torch.float16, torch.bfloat16
        _torch = torch
    return _torch


def _check(st: int, where: str):
    if st != HR_OK:
        raise HrError(st, where)


def _f16_ptr(t, name: str, dtype=None) -> int:
    if _torch is None:
        _tm()
    want = _F16 if dtype is None else dtype
    if t.dtype is not want:
        raise TypeError(f"{name}: expected {want}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name}: expected a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _stream_handle(stream, tensor=None) -> int:
    """The hipStream_t of ``stream``; for None, torch's current stream on the
    device of ``tensor`` (or the current device).  torch's raw query returns
    the handle without building a Stream object, which costs more than the
    library call itself; the public call is the fallback."""
    if stream is not None:
        return stream.cuda_stream
    torch = _tm()
    dev = tensor.get_device() if tensor is not None else torch.cuda.current_device()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return int(raw(dev))
    return int(torch.cuda.current_stream(dev).cuda_stream)


def reduce(tensors, out, stream=None):
    """out = left fold of ``tensors`` (all torch.float16, or all
    torch.bfloat16, same numel) on ``stream``."""
    _tm()
    n = out.numel()
    bf = out.dtype is _BF16
    dt = _BF16 if bf else _F16
    ptrs = []
    for i, t in enumerate(tensors):
        if t.numel() != n:
            raise ValueError(f"tensors[{i}] has {t.numel()} values, out has {n}")
        ptrs.append(_f16_ptr(t, f"tensors[{i}]", dt))
    fn, name = (hr_reduce_bf16, "hr_reduce_bf16") if bf else (hr_reduce_f16, "hr_reduce_f16")
    _check(fn(ptrs, len(ptrs), _f16_ptr(out, "out", dt), n, _stream_handle(stream, out)), name)
    return out


def allreduce_group_noalloc(ins, outs, status=None, stream=None):
    """Every rank's call in one launch without a channel
    (hr_allreduce_group_noalloc_f16): ``ins[r]``/``outs[r]`` are rank r's
    torch.float16 tensors; ``status``, if given, a one-element torch.int32
    (or uint32) device tensor that receives the call's status."""
    W = len(ins)
    if len(outs) != W:
        raise ValueError("ins and outs differ in length")
    n = ins[0].numel()
    for r in range(W):
        if ins[r].numel() != n or outs[r].numel() != n:
            raise ValueError(f"rank {r}: every input and output must hold {n} values")
    ip = [_f16_ptr(t, f"ins[{r}]") for r, t in enumerate(ins)]
    op = [_f16_ptr(t, f"outs[{r}]") for r, t in enumerate(outs)]
    sp = None
    if status is not None:
        if status.numel() < 1 or status.element_size() != 4 or not status.is_cuda:
            raise TypeError("status: expected a 4-byte device tensor")
        sp = status.data_ptr()
    _check(hr_allreduce_group_noalloc_f16(ip, op, W, n, sp, _stream_handle(stream, outs[0])),
           "hr_allreduce_group_noalloc_f16")
    return outs


# ------------------------------------------------------- around the combine
#
# The argument structs go over as packed bytes: a struct.pack of the norm's 35
# fields takes 0.4 us, where filling a ctypes.Structure goes field by field.  A
# small call is as long as its host time (MI355X host: the norm 7.2 us, of
# which HIP's launch is 2.9), so the checks below keep to attribute reads and
# take a short way for contiguous tensors.

_NORM = struct.Struct("@23P8N3if")
_NORM_GRAD = struct.Struct("@8P7Ni4x")
_GATHER = struct.Struct("@7P8N2i")
_COMBINE = struct.Struct("@5P6Ni4x")
_COMBINE_GRAD = struct.Struct("@8P6N2i")
_NULLS = [0] * HR_MAX_G
_entries = {}


def _entry(name: str, dtype):
    """(function, its name) of an entry point's variant for torch.float16 or
    torch.bfloat16, bound once."""
    got = _entries.get((name, dtype))
    if got is None:
        _tm()
        if dtype is not _F16 and dtype is not _BF16:
            raise TypeError(f"{name}: expected torch.float16 or torch.bfloat16, got {dtype}")
        full = f"{name}_{'bf16' if dtype is _BF16 else 'f16'}"
        got = _entries[(name, dtype)] = (getattr(load(), full), full)
    return got


_raw_stream = None


def _stream_of(stream, tensor) -> int:
    """_stream_handle with torch's raw query looked up once."""
    global _raw_stream
    if stream is None and _raw_stream is not None:
        return _raw_stream(tensor.get_device())
    _raw_stream = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
    return _stream_handle(stream, tensor)


def _row_view(t, name: str, dtype, rows=None, width=None):
    """(address, rows, row length, row stride) of a device tensor whose last
    dimension is a row: two dimensions with any row stride, or contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name}: expected a device tensor")
    shape = t.shape
    if len(shape) == 2:
        r, w = shape
        sr, sc = t.stride()
        if (sc != 1 and w > 1) or (r > 1 and sr < w):
            raise ValueError(f"{name}: expected rows of adjacent values that do not overlap")
        if r <= 1:
            sr = 0
    else:
        if not shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected two dimensions or a contiguous tensor")
        w, sr = shape[-1], 0
        r = t.numel() // w if w else 0
    if rows is not None and (r != rows or w != width):
        raise ValueError(f"{name}: {r} rows of {w} values, expected {rows} of {width}")
    return t.data_ptr(), r, w, sr


def _rows_like(t, name: str, dtype, shape, rows: int, width: int):
    """(address, row stride) of a device tensor of rows x width values; a
    contiguous one of ``shape`` takes the short way."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr(), 0
    p, _, _, s = _row_view(t, name, dtype, rows, width)
    return p, s


def _flat_ptr(t, name: str, dtype, numel: int) -> int:
    """Address of a contiguous device tensor of ``numel`` values."""
    if t.dtype is dtype and t.is_cuda and t.numel() == numel and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name}: expected a device tensor")
    raise ValueError(f"{name}: expected a contiguous tensor of {numel} values")


def _weight_ptr(t, dtype, hidden: int):
    """(address, is binary32) of a norm's weight, or of none."""
    if t is None:
        return 0, 0
    f32 = t.dtype is _torch.float32
    return _flat_ptr(t, "weight", _torch.float32 if f32 else dtype, hidden), int(f32)


def _scratch(nbytes: int, like, stream):
    """A workspace for one call on ``stream``.  It comes from that stream's
    pool, so what reuses its memory afterwards is ordered behind the call."""
    if stream is None:
        return _torch.empty(nbytes, dtype=_torch.uint8, device=like.device)
    with _torch.cuda.stream(stream):
        return _torch.empty(nbytes, dtype=_torch.uint8, device=like.device)


def reduce_rmsnorm(tensors, out=None, *, residual=None, residual_out=None, weight=None, eps: float = 1e-6,
                   out8=None, scales=None, group: int = 0, rstd=None, stream=None):
    """The fold of ``tensors`` with ``residual`` as its last operand (into
    ``residual_out``), its root-mean-square norm times ``weight`` (into
    ``out``), and the norm in e4m3 with scales (into ``out8`` and ``scales``),
    in one kernel (hr_reduce_rmsnorm).

    ``tensors`` are torch.float16 or torch.bfloat16, all of one shape and row
    stride; the last dimension is the row.  ``weight`` has their type or
    torch.float32.  ``out8`` is torch.float8_e4m3fn and ``scales``
    torch.float32, one per row (``group`` 0) or per 32, 64 or 128 values of
    it.  ``rstd`` (torch.float32, one per row) is what rmsnorm_grad takes.
    Whatever is None is not computed or not written; ``residual_out`` and
    ``out`` may be an input."""
    first = tensors[0]
    dt = first.dtype
    fn, name = _entry("hr_reduce_rmsnorm", dt)
    if len(tensors) > HR_MAX_G:
        raise ValueError(f"{len(tensors)} contributions, at most {HR_MAX_G}")
    p0, rows, hidden, stride = _row_view(first, "tensors[0]", dt)
    shape = first.shape
    ptrs = [p0]
    packed = (stride or hidden) == hidden
    for i in range(1, len(tensors)):
        t = tensors[i]
        if packed and t.dtype is dt and t.shape == shape and t.is_cuda and t.is_contiguous():
            ptrs.append(t.data_ptr())
            continue
        p, s = _rows_like(t, f"tensors[{i}]", dt, shape, rows, hidden)
        if (s or hidden) != (stride or hidden):
            raise ValueError(f"tensors[{i}]: row stride {s}, tensors[0] has {stride}")
        ptrs.append(p)
    ptrs += _NULLS[len(ptrs):]
    rp = hp = op = cp = sp = tp = 0
    rs = hs = os_ = cs = ss = 0
    if residual is not None:
        rp, rs = _rows_like(residual, "residual", dt, shape, rows, hidden)
    if residual_out is not None:
        hp, hs = _rows_like(residual_out, "residual_out", dt, shape, rows, hidden)
    if out is not None:
        op, os_ = _rows_like(out, "out", dt, shape, rows, hidden)
    if out8 is not None:
        cp, cs = _rows_like(out8, "out8", _torch.float8_e4m3fn, shape, rows, hidden)
    if scales is not None:
        groups = -(-hidden // group) if group else 1
        if scales.dim() == 1 and groups == 1:
            scales = scales.unsqueeze(1)
        sp, _, _, ss = _row_view(scales, "scales", _torch.float32, rows, groups)
    if rstd is not None:
        tp = _flat_ptr(rstd, "rstd", _torch.float32, rows)
    wp, wf = _weight_ptr(weight, dt, hidden)
    args = _NORM.pack(*ptrs, rp, wp, hp, op, cp, sp, tp, rows, hidden, stride, rs, hs, os_, cs, ss,
                      len(tensors), wf, group, eps)
    st = fn(args, _stream_of(stream, first))
    if st != HR_OK:
        raise HrError(st, name)
    return out


def rmsnorm_grad(dy, h, rstd, dx, *, weight=None, dresidual=None, dweight=None, workspace=None, stream=None):
    """The gradient of reduce_rmsnorm's ``out``: ``dx`` of its sum ``h`` (the
    forward call's residual_out), ``dresidual`` added, and ``dweight``
    (torch.float32) if given (hr_rmsnorm_grad).  ``workspace``: a device
    tensor of hr_rmsnorm_grad_workspace(rows, hidden) bytes or more; None
    takes one from torch's allocator when the call needs one."""
    dt = h.dtype
    fn, name = _entry("hr_rmsnorm_grad", dt)
    hp, rows, hidden, hs = _row_view(h, "h", dt)
    shape = h.shape
    yp, ys = _rows_like(dy, "dy", dt, shape, rows, hidden)
    xp, xs = _rows_like(dx, "dx", dt, shape, rows, hidden)
    tp = _flat_ptr(rstd, "rstd", _torch.float32, rows)
    rp = rs = gp = kp = kb = 0
    if dresidual is not None:
        rp, rs = _rows_like(dresidual, "dresidual", dt, shape, rows, hidden)
    wp, wf = _weight_ptr(weight, dt, hidden)
    if dweight is not None:
        gp = _flat_ptr(dweight, "dweight", _torch.float32, hidden)
        if workspace is None and (rows > HR_RMSNORM_GRAD_FEW_ROWS or xp == yp or xp == hp):
            need = load().hr_rmsnorm_grad_workspace(rows, hidden)
            if need:
                workspace = _scratch(need, h, stream)
        if workspace is not None:
            kb = workspace.numel() * workspace.element_size()
            kp = _flat_ptr(workspace, "workspace", workspace.dtype, workspace.numel())
    args = _NORM_GRAD.pack(yp, hp, tp, wp, rp, xp, gp, kp, kb, rows, hidden, ys, hs, rs, xs, wf)
    st = fn(args, _stream_of(stream, h))
    if st != HR_OK:
        raise HrError(st, name)
    return dx


def _dtype_code(dtype, name: str) -> int:
    """The hr_dtype of router logits."""
    _tm()
    if dtype is _torch.float32:
        return HR_DTYPE_F32
    if dtype is _F16:
        return HR_DTYPE_F16
    if dtype is _BF16:
        return HR_DTYPE_BF16
    raise TypeError(f"{name}: expected torch.float32, torch.float16 or torch.bfloat16, got {dtype}")


def _picks(weights, ids, tokens: int):
    """(addresses of weights and ids, k) of a token's picks."""
    k = ids.shape[-1]
    return (_flat_ptr(weights, "weights", _torch.float32, tokens * k),
            _flat_ptr(ids, "ids", _torch.int32, tokens * k), k)


def router_topk(logits, weights, ids, *, renormalize: bool = False, stream=None):
    """The k largest logits of every token, by value downward and equal ones
    by index upward, into ``ids`` (torch.int32, tokens x k), and their softmax
    weights into ``weights`` (torch.float32); ``renormalize`` divides them by
    their sum (hr_router_topk).  NaN and -inf logits are never picked: id -1,
    weight 0 where nothing is left."""
    code = _dtype_code(logits.dtype, "logits")
    lp, tokens, experts, ls = _row_view(logits, "logits", logits.dtype)
    wp, ip, k = _picks(weights, ids, tokens)
    st = load().hr_router_topk(lp, code, tokens, experts, ls, k, 1 if renormalize else 0, wp, ip,
                               _stream_of(stream, logits))
    if st != HR_OK:
        raise HrError(st, "hr_router_topk")
    return weights, ids


def router_topk_grad(dweights, weights, ids, dlogits, *, logits=None, renormalize: bool = False, stream=None):
    """The gradient of router_topk's weights with respect to the logits, into
    ``dlogits`` (hr_router_topk_grad).  ``logits`` are needed unless
    ``renormalize``; ``dlogits`` may be ``logits``."""
    dt = dlogits.dtype
    code = _dtype_code(dt, "dlogits")
    dp, tokens, experts, ds = _row_view(dlogits, "dlogits", dt)
    wp, ip, k = _picks(weights, ids, tokens)
    gp = _flat_ptr(dweights, "dweights", _torch.float32, tokens * k)
    lp = ls = 0
    if logits is not None and not renormalize:
        lp, _, _, ls = _row_view(logits, "logits", dt, tokens, experts)
    st = load().hr_router_topk_grad(gp, wp, ip, lp, code, tokens, experts, ls, k, 1 if renormalize else 0, dp, ds,
                                    _stream_of(stream, dlogits))
    if st != HR_OK:
        raise HrError(st, "hr_router_topk_grad")
    return dlogits


def experts_buffers(tokens: int, k: int, experts: int, pad: int = 1, device=0):
    """Device tensors (offsets, order, pos) for experts_sort; order's length is
    the rows that a gathered buffer needs."""
    import torch
    dev = torch.device("cuda", device) if isinstance(device, int) else device
    rows = hr_experts_rows(tokens, k, experts, pad)
    return tuple(torch.empty(shape, dtype=torch.int32, device=dev) for shape in ((experts + 1,), (rows,), (tokens, k)))


def experts_sort(ids, offsets, order, pos, *, first: int = 0, pad: int = 1, workspace=None, stream=None):
    """Where every pick goes (hr_experts_sort): ``ids`` (torch.int32, tokens x
    k) sorted stably by expert, for the experts first .. first + n - 1 with n =
    offsets.numel() - 1, every segment rounded up to ``pad`` rows.
    ``workspace``: a device tensor of hr_experts_sort_workspace bytes; None
    takes one from torch's allocator when the call needs one."""
    if _torch is None:
        _tm()
    shape = ids.shape
    if len(shape) != 2:
        raise ValueError("ids: expected tokens x k")
    tokens, k = shape
    i32 = _torch.int32
    ip = _flat_ptr(ids, "ids", i32, tokens * k)
    experts = offsets.numel() - 1
    op = _flat_ptr(offsets, "offsets", i32, experts + 1)
    rows = order.numel()
    rp = _flat_ptr(order, "order", i32, rows)
    pp = _flat_ptr(pos, "pos", i32, tokens * k)
    lib = load()
    kp = kb = 0
    if workspace is None and tokens * k > HR_EXPERTS_SORT_FEW:
        need = lib.hr_experts_sort_workspace(tokens, k, experts)
        if need:
            workspace = _scratch(need, ids, stream)
    if workspace is not None:
        kb = workspace.numel() * workspace.element_size()
        kp = _flat_ptr(workspace, "workspace", workspace.dtype, workspace.numel())
    st = lib.hr_experts_sort(ip, tokens, k, first, experts, pad, op, rp, rows, pp, kp, kb,
                             _stream_of(stream, ids))
    if st != HR_OK:
        raise HrError(st, "hr_experts_sort")
    return offsets, order, pos


def _pos_ptr(pos, tokens: int):
    """(address, k) of a sort's pos."""
    shape = pos.shape
    if len(shape) != 2 or shape[0] != tokens:
        raise ValueError(f"pos: expected {tokens} x k")
    k = shape[1]
    return _flat_ptr(pos, "pos", _torch.int32, tokens * k), k


def _padding_ptrs(order, offsets, rows: int):
    """(addresses of order and offsets, experts) of a sort, or of none."""
    if order is None:
        return 0, 0, 0
    if offsets is None:
        raise ValueError("order is given without offsets")
    experts = offsets.numel() - 1
    return (_flat_ptr(order, "order", _torch.int32, rows), _flat_ptr(offsets, "offsets", _torch.int32, experts + 1),
            experts)


def experts_gather(x, pos, out, *, offsets=None, order=None, scales=None, scales_out=None, stream=None):
    """Every token's row to its sorted rows, and its scales with it
    (hr_experts_gather): ``x`` and ``out`` of any one type, ``scales``
    torch.float32 (as reduce_rmsnorm writes them).  With ``order`` and
    ``offsets`` the padding rows inside the segments become zeros; rows past the
    last segment are not written.  ``out`` and ``order`` may be the first rows
    of a sort's, down to those in use."""
    if _torch is None:
        _tm()
    dt = x.dtype
    xp, tokens, width, xs = _row_view(x, "x", dt)
    op, rows, w, os_ = _row_view(out, "out", dt)
    if w != width:
        raise ValueError(f"out: rows of {w} values, x has {width}")
    pp, k = _pos_ptr(pos, tokens)
    rp, fp, experts = _padding_ptrs(order, offsets, rows)
    sp = tp = sw = ss = ts = 0
    if scales is not None or scales_out is not None:
        if scales is None or scales_out is None:
            raise ValueError("scales and scales_out go together")
        f32 = _torch.float32
        # one scale per row may come in one dimension
        if scales.dim() == 1 and scales.shape[0] == tokens:
            scales = scales.unsqueeze(1)
        sw = scales.shape[-1]
        if scales_out.dim() == 1 and sw == 1:
            scales_out = scales_out.unsqueeze(1)
        sp, _, _, ss = _row_view(scales, "scales", f32, tokens, sw)
        tp, _, _, ts = _row_view(scales_out, "scales_out", f32, rows, sw)
    size = x.element_size()
    args = _GATHER.pack(xp, sp, op, tp, pp, rp, fp, tokens, rows, width * size, xs * size, os_ * size, sw, ss, ts, k,
                        experts)
    st = load().hr_experts_gather(args, _stream_of(stream, x))
    if st != HR_OK:
        raise HrError(st, "hr_experts_gather")
    return out


def experts_combine(z, pos, out, *, weights=None, addend=None, stream=None):
    """out[t] = addend[t] + sum over j of weights[t, j] * z[pos[t, j]]
    (hr_experts_combine); ``z`` holds sorted rows, torch.float16 or
    torch.bfloat16.  Without weights, the gradient of experts_gather."""
    dt = out.dtype
    fn, name = _entry("hr_experts_combine", dt)
    op, tokens, hidden, os_ = _row_view(out, "out", dt)
    zp, rows, w, zs = _row_view(z, "z", dt)
    if w != hidden:
        raise ValueError(f"z: rows of {w} values, out has {hidden}")
    pp, k = _pos_ptr(pos, tokens)
    wp = ap = as_ = 0
    if weights is not None:
        wp = _flat_ptr(weights, "weights", _torch.float32, tokens * k)
    if addend is not None:
        ap, _, _, as_ = _row_view(addend, "addend", dt, tokens, hidden)
    args = _COMBINE.pack(zp, ap, op, pp, wp, tokens, rows, hidden, zs, as_, os_, k)
    st = fn(args, _stream_of(stream, out))
    if st != HR_OK:
        raise HrError(st, name)
    return out


def experts_combine_grad(dy, z, pos, weights=None, dz=None, dweights=None, *, offsets=None, order=None, stream=None):
    """The gradient of experts_combine (hr_experts_combine_grad): ``dz`` of the
    sorted rows and ``dweights`` (torch.float32, tokens x k), either of which
    may be None.  With ``order`` and ``offsets`` the padding rows of dz become
    zeros; rows past the last segment are not written."""
    dt = dy.dtype
    fn, name = _entry("hr_experts_combine_grad", dt)
    yp, tokens, hidden, ys = _row_view(dy, "dy", dt)
    zp, rows, w, zs = _row_view(z, "z", dt)
    if w != hidden:
        raise ValueError(f"z: rows of {w} values, dy has {hidden}")
    pp, k = _pos_ptr(pos, tokens)
    dp = ds = wp = gp = 0
    if dz is not None:
        dp, _, _, ds = _row_view(dz, "dz", dt, rows, hidden)
    if weights is not None:
        wp = _flat_ptr(weights, "weights", _torch.float32, tokens * k)
    if dweights is not None:
        gp = _flat_ptr(dweights, "dweights", _torch.float32, tokens * k)
    rp, fp, experts = _padding_ptrs(order, offsets, rows)
    args = _COMBINE_GRAD.pack(yp, zp, dp, pp, wp, gp, rp, fp, tokens, rows, hidden, ys, zs, ds, k, experts)
    st = fn(args, _stream_of(stream, dy))
    if st != HR_OK:
        raise HrError(st, name)
    return dz, dweights


class Channel:
    """An owned channel of ``world_size`` ranks; ``allreduce`` enqueues one
    rank's call."""

    def __init__(self, device: int = 0, max_numel: int = 0, num_blocks: int = 0,
                 timeout_us: int = 0, world_size: int = 2, algorithm: int = 0, link_mbps: int = 0):
        self.world_size = world_size
        self.handle = hr_create_channel(device, world_size, max_numel, num_blocks, timeout_us,
                                        algorithm, link_mbps)
        lib = load()
        _tm()
        # the per-rank entry point of each element type, bound once
        self._per_rank = {_F16: (lib.hr_allreduce_f16, "hr_allreduce_f16"),
                          _BF16: (lib.hr_allreduce_bf16, "hr_allreduce_bf16")}

    def allreduce(self, rank: int, inp, out, stream=None):
        """One rank's call; torch.float16 or torch.bfloat16 tensors.

        In loopback every rank's call must be in flight at once, on streams
        from ``LoopbackStreams``.  Those streams are ordered with the null
        stream (they are not non-blocking), so work on the null stream --
        torch's default stream included -- enqueued between the ranks'
        calls of one all-reduce holds back the ranks launched after it while
        the others spin: the call ends at the channel's watchdog with the
        sticky HR_ERR_TIMEOUT.  Enqueue nothing on the null stream between
        the ranks' calls, or use ``allreduce_group``."""
        n = inp.numel()
        if out.numel() != n:
            raise ValueError("in and out differ in numel")
        dt = inp.dtype
        fn, name = self._per_rank.get(dt, self._per_rank[_F16])
        if dt is not _BF16:
            dt = _F16                     # anything else is refused as not float16
        st = fn(self.handle, rank, _f16_ptr(inp, "in", dt), _f16_ptr(out, "out", dt), n,
                _stream_handle(stream, out))
        if st != HR_OK:
            raise HrError(st, self._where(name, st))
        return out

    def _where(self, name: str, st: int) -> str:
        """The call's name, with the timeout record when the channel holds one."""
        if st != HR_ERR_TIMEOUT:
            return name
        info = self.timeout_info()
        if info is None:
            return name
        rank, missing, call = info
        return f"{name} (rank {rank} waited at call {call} for ranks {missing})"

    def allreduce_group(self, ins, outs, stream=None):
        """Every rank's call in one launch (loopback): ``ins[r]``/``outs[r]``
        are rank r's torch.float16 or torch.bfloat16 tensors."""
        if len(ins) != self.world_size or len(outs) != self.world_size:
            raise ValueError(f"expected {self.world_size} inputs and outputs")
        n = ins[0].numel()
        bf = ins[0].dtype is _BF16
        dt = _BF16 if bf else _F16
        for r in range(self.world_size):
            if ins[r].numel() != n or outs[r].numel() != n:
                raise ValueError(f"rank {r}: every input and output must hold {n} values")
        ip = [_f16_ptr(t, f"ins[{r}]", dt) for r, t in enumerate(ins)]
        op = [_f16_ptr(t, f"outs[{r}]", dt) for r, t in enumerate(outs)]
        fn, name = ((hr_allreduce_group_bf16, "hr_allreduce_group_bf16") if bf
                    else (hr_allreduce_group_f16, "hr_allreduce_group_f16"))
        st = fn(self.handle, ip, op, n, _stream_handle(stream, outs[0]))
        if st != HR_OK:
            raise HrError(st, self._where(name, st))
        return outs

    def status(self) -> int:
        return hr_channel_status(self.handle)

    def abort(self):
        _check(hr_channel_abort(self.handle), "hr_channel_abort")

    def timeout_info(self):
        """After HR_ERR_TIMEOUT: (rank whose wait expired, [ranks whose
        publish never arrived], call number), or None if nothing is
        recorded."""
        rank, mask, call = hr_channel_timeout_info(self.handle)
        if rank < 0:
            return None
        return rank, [q for q in range(self.world_size) if (mask >> q) & 1], call

    def info(self) -> hr_channel_info:
        return hr_channel_get_info(self.handle)

    def algorithm_for(self, numel: int) -> int:
        """The HR_ALGO_* a call of numel values on this channel takes."""
        return hr_exchange_algorithm(self.handle, numel)

    def destroy(self):
        if self.handle:
            st = hr_destroy(self.handle)
            self.handle = None
            _check(st, "hr_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.destroy()


class LoopbackStreams:
    """One stream per rank of a loopback channel, each owning its hardware
    queue (see hr_loopback_stream_create), wrapped as torch streams."""

    def __init__(self, device: int = 0, n: int = 2):
        import torch
        self.handles = [hr_loopback_stream_create(device) for _ in range(n)]
        self.streams = tuple(torch.cuda.ExternalStream(h, device=torch.device("cuda", device))
                             for h in self.handles)

    def __getitem__(self, i):
        return self.streams[i]

    def __iter__(self):
        return iter(self.streams)

    def __len__(self):
        return len(self.streams)

    def destroy(self):
        for s in self.streams:
            s.synchronize()
        for h in self.handles:
            _check(hr_loopback_stream_destroy(h), "hr_loopback_stream_destroy")
        self.handles = []
