"""Thin ctypes binding of liblk.so (the C ABI declared in include/lk.h and,
for the attention step, include/lk_attn.h, for a mixture of experts
include/lk_moe.h, for the drawn token include/lk_sample.h).

Each ``lk_*`` function here has the name and argument order of the C entry
point; it only checks and marshals torch tensors (dtype, device, contiguity,
sizes) into pointers and the current CUDA stream.  All arithmetic runs in the
library's sm_103a kernels.  If liblk.so is missing the first call raises: there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblk.so")

LK_DEQUANT, LK_INT8ACT, LK_TWOPASS = 0, 1, 2
MODES = {"dequant": LK_DEQUANT, "int8act": LK_INT8ACT, "twopass": LK_TWOPASS}
LK_MAX_M = 8
LK_MAX_BATCH = 64
LK_MAX_SPLITK = 64
LK_TRACE_REC = 8  # entries of one launch record of option "trace" 3
LK_TRACE_MAX_RECORDS = 4096 // LK_TRACE_REC  # records the timeline keeps before wrapping

STATUS = {0: "LK_OK", -1: "LK_ERR_ARG", -2: "LK_ERR_ALIGN", -3: "LK_ERR_SHAPE",
          -4: "LK_ERR_WORKSPACE", -5: "LK_ERR_CUDA", -6: "LK_ERR_DEVICE_TIMEOUT"}


class LkChainOp(ctypes.Structure):
    """One step of lk_gemv_chain (the C struct lk_chain_op)."""
    _fields_ = [("wq", ctypes.c_void_p), ("ws", ctypes.c_void_p), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("x", ctypes.c_void_p), ("gain", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("argmax_parts", ctypes.c_void_p), ("argmax_idx", ctypes.c_void_p), ("wait", ctypes.c_int),
                ("reserved", ctypes.c_int)]


class LkGemvTarget(ctypes.Structure):
    """One matrix of lk_gemv_q8_group (the C struct lk_gemv_target)."""
    _fields_ = [("wq", ctypes.c_void_p), ("ws", ctypes.c_void_p), ("N", ctypes.c_int), ("reserved", ctypes.c_int),
                ("y", ctypes.c_void_p)]


CFG_FIELDS = ("pdl", "prefill", "path", "grid_ctas", "ring_tk", "mma_min_m", "mma_tk", "mma_warps", "mma_depth",
              "mma_i8", "mma_group", "mma_act16")
PATHS = {"auto": 0, "direct": 1, "ring": 2, "mma": 3}


class LkLaunchCfg(ctypes.Structure):
    """Per-call launch settings (the C struct lk_launch_cfg; see include/lk.h)."""
    _fields_ = [(f, ctypes.c_int) for f in CFG_FIELDS]


def launch_cfg(**kw) -> LkLaunchCfg:
    """lk_launch_cfg from keyword fields (every other field 0, the default):
    pdl, prefill, path (0..3 or "auto"/"direct"/"ring"/"mma"), grid_ctas,
    ring_tk, mma_min_m, mma_tk, mma_warps, mma_depth, mma_i8, mma_group,
    mma_act16."""
    bad = set(kw) - set(CFG_FIELDS)
    if bad:
        raise TypeError(f"launch_cfg: unknown fields {sorted(bad)}")
    if isinstance(kw.get("path"), str):
        kw["path"] = PATHS[kw["path"]]
    return LkLaunchCfg(*[int(kw.get(f, 0)) for f in CFG_FIELDS])


def _cfg(cfg):
    return None if cfg is None else ctypes.byref(cfg)


class LkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_load().lk_status_string(status).decode()})")


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built: run q8_quantized_gemv_gb300.build.build() "
                           "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, L, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_float, ctypes.c_size_t
    sig = {
        "lk_status_string": ([I], ctypes.c_char_p),
        "lk_version": ([], I),
        "lk_rmsnorm_quant": ([P, P, I, I, F, I, P, P, P, P, P, P], I),
        "lk_quantize_act": ([P, I, I, I, P, P, P, P, P], I),
        "lk_gemv_q8": ([P, P, I, I, I, P, P, P, P, I, P, P, P, P, P], I),
        "lk_splitk_workspace_bytes": ([I, I, I, I], S),
        "lk_gemv_q8_splitk": ([P, P, I, I, I, P, P, P, P, I, I, P, S, P, P], I),
        "lk_splitk_combine": ([I, P, I, I, I, P, P, P], I),
        "lk_splitk_chunks_for": ([I, I, I, I], I),
        "lk_format_row_bytes": ([I, I], S),
        "lk_gemv_blk": ([I, P, I, I, I, P, P, P, P, I, P, P, P], I),
        "lk_dequant_blk": ([I, P, I, I, P, P], I),
        "lk_argmax_parts_max": ([I], I),
        "lk_argmax_scratch_entries": ([I], I),
        "lk_argmax": ([P, P, I, I, I, P, P, P], I),
        "lk_q8_block_dots": ([P, I, I, P, P, P, P, P], I),
        "lk_set_option": ([ctypes.c_char_p, L], I),
        "lk_get_option": ([ctypes.c_char_p], L),
        "lk_device_error": ([I, ctypes.POINTER(I)], I),
        "lk_selftest_wait_timeout": ([ctypes.c_uint, P], I),
        "lk_gemv_kernel_for": ([I, I, I, I, I, P], I),
        "lk_rmsnorm_quant_gemv_q8": ([P, P, I, I, I, P, P, F, I, P, P, P, P, P], I),
        "lk_chain_sync_bytes": ([], S),
        "lk_trace_read": ([P, I], I),
        "lk_argmax_noalloc": ([P, I, I, P, P], I),
        "lk_gemv_chain": ([P, P, I, I, I, F, P, P, P], I),
        "lk_gemv_q8_group": ([P, I, I, I, P, P, P, P, I, P, P], I),
        "lk_add_rmsnorm_quant": ([P, P, P, I, I, F, I, P, P, P, P, P, P, P], I),
        "lk_swiglu_quant": ([P, P, I, I, L, I, P, P, P, P, P, P], I),
        "lk_gemv_q8_glu": ([P, P, P, P, I, I, I, P, P, P, P, I, P, P, P, P, P, P, P, P], I),
        "lk_kv_append": ([P, P, P, P, L, I, P, I, P, I, I, I, P, P, I, I, I, P, P, F, P, P, P], I),
        "lk_attn": ([P, P, I, P, I, P, I, I, F, I, P, P, P, P, P, S, P, P], I),
        "lk_attn_shared": ([P, P, I, P, I, I, P, I, P, I, I, F, I, P, P, P, P, P, S, P, P], I),
        "lk_attn_workspace_bytes": ([I, I, I, I, I, I], S),
        "lk_attn_launches": ([I, I, I, I, I, I, I, I], I),
        "lk_moe_route": ([P, P, I, I, I, I, I, I, I, I, F, P, P, P, P], I),
        "lk_moe_glu_q8": ([P, P, P, P, I, I, I, I, P, P, P, P, I, P, I, P, P, P, P, P, P, P], I),
        "lk_moe_down_q8": ([P, P, I, I, I, I, P, P, P, P, I, P, P, I, P, P, P], I),
        "lk_sample": ([P, I, I, P, P, P, P, P, P, P, P, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def exported_symbols():
    return ["lk_status_string", "lk_version", "lk_rmsnorm_quant", "lk_quantize_act", "lk_gemv_q8",
            "lk_splitk_workspace_bytes", "lk_gemv_q8_splitk", "lk_splitk_combine",
            "lk_argmax_parts_max", "lk_argmax_scratch_entries", "lk_argmax", "lk_q8_block_dots",
            "lk_set_option", "lk_get_option", "lk_device_error", "lk_selftest_wait_timeout", "lk_gemv_kernel_for",
            "lk_rmsnorm_quant_gemv_q8", "lk_chain_sync_bytes", "lk_gemv_chain", "lk_trace_read",
            "lk_argmax_noalloc", "lk_gemv_q8_group", "lk_add_rmsnorm_quant", "lk_swiglu_quant",
            "lk_gemv_q8_glu", "lk_splitk_chunks_for", "lk_format_row_bytes", "lk_gemv_blk", "lk_dequant_blk"]


def attn_symbols():
    """The entry points of include/lk_attn.h."""
    return ["lk_kv_append", "lk_attn", "lk_attn_shared", "lk_attn_workspace_bytes", "lk_attn_launches"]


def moe_symbols():
    """The entry points of include/lk_moe.h."""
    return ["lk_moe_route", "lk_moe_glu_q8", "lk_moe_down_q8"]


def sample_symbols():
    """The entry points of include/lk_sample.h."""
    return ["lk_sample"]


def _ok(st, where):
    if st != 0:
        raise LkError(st, where)


def _mode(mode):
    return MODES[mode] if isinstance(mode, str) else int(mode)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


_I8 = torch.int8
_F32 = torch.float32
_WS = (torch.int16, torch.float16)


def lk_status_string(status: int) -> str:
    return _load().lk_status_string(status).decode()


def lk_version() -> int:
    return _load().lk_version()


def lk_rmsnorm_quant(x, gain, mode, eps=1e-6, xn=None, xq=None, xl=None, xs=None, stream=None, cfg=None):
    M, K = x.shape
    _ok(_load().lk_rmsnorm_quant(_ptr(x, _F32, "x"), _ptr(gain, _F32, "gain"), M, K, eps, _mode(mode),
                                 _ptr(xn, _F32, "xn"), _ptr(xq, _I8, "xq"), _ptr(xl, _I8, "xl"),
                                 _ptr(xs, _F32, "xs"), _cfg(cfg), _stream(stream)), "lk_rmsnorm_quant")


def lk_add_rmsnorm_quant(x, r, gain, mode, eps=1e-6, s=None, xn=None, xq=None, xl=None, xs=None, stream=None,
                         cfg=None):
    """s = x + r (optional output), then lk_rmsnorm_quant of the sum."""
    M, K = x.shape
    if tuple(r.shape) != (M, K):
        raise ValueError("r must have the shape of x")
    _ok(_load().lk_add_rmsnorm_quant(_ptr(x, _F32, "x"), _ptr(r, _F32, "r"), _ptr(gain, _F32, "gain"), M, K, eps,
                                     _mode(mode), _ptr(s, _F32, "s"), _ptr(xn, _F32, "xn"), _ptr(xq, _I8, "xq"),
                                     _ptr(xl, _I8, "xl"), _ptr(xs, _F32, "xs"), _cfg(cfg), _stream(stream)),
        "lk_add_rmsnorm_quant")


def _pitched_rows(t, name):
    """Pointer and row pitch (elements) of a 2-D f32 CUDA tensor whose rows
    are contiguous (a column slice of a wider row-major tensor is fine)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != _F32 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D float32 CUDA tensor")
    if t.stride(1) != 1:
        raise ValueError(f"{name} rows must be contiguous")
    return ctypes.c_void_p(t.data_ptr()), t.stride(0)


def lk_swiglu_quant(gate, up, mode, h=None, hq=None, hl=None, hs=None, stream=None, cfg=None):
    """h = silu(gate) * up, quantized for the next GEMV.  gate and up are
    [M, F] f32 with contiguous rows and the same row pitch (e.g. the two
    halves gu[:, :F], gu[:, F:] of a fused gate/up output)."""
    M, F = gate.shape
    if tuple(up.shape) != (M, F):
        raise ValueError("up must have the shape of gate")
    pg, ldg = _pitched_rows(gate, "gate")
    pu, ldu = _pitched_rows(up, "up")
    if ldg != ldu:
        raise ValueError("gate and up must have the same row pitch")
    _ok(_load().lk_swiglu_quant(pg, pu, M, F, ldg, _mode(mode), _ptr(h, _F32, "h"), _ptr(hq, _I8, "hq"),
                                _ptr(hl, _I8, "hl"), _ptr(hs, _F32, "hs"), _cfg(cfg), _stream(stream)),
        "lk_swiglu_quant")


def lk_quantize_act(x, mode, xq, xl, xs, stream=None, cfg=None):
    M, K = x.shape
    _ok(_load().lk_quantize_act(_ptr(x, _F32, "x"), M, K, _mode(mode), _ptr(xq, _I8, "xq"),
                                _ptr(xl, _I8, "xl"), _ptr(xs, _F32, "xs"), _cfg(cfg), _stream(stream)),
        "lk_quantize_act")


def lk_gemv_q8(wq, ws, mode, y, x=None, xq=None, xl=None, xs=None, argmax_parts=None, M=None,
               stream=None, cfg=None) -> int:
    """y[M, N] = W x.  Returns the number of argmax partial keys written per
    activation row (0 when argmax_parts is None).  cfg: launch_cfg(...) or
    None (the defaults)."""
    N, K = wq.shape
    if M is None:
        M = (x if x is not None else xq).shape[0]
    n = ctypes.c_int(0)
    args = [_ptr(wq, _I8, "wq"), _ptr(ws, _WS, "ws"), N, K, _mode(mode), _ptr(x, _F32, "x"), _ptr(xq, _I8, "xq"),
            _ptr(xl, _I8, "xl"), _ptr(xs, _F32, "xs"), M, _ptr(y, _F32, "y"),
            _ptr(argmax_parts, torch.int64, "argmax_parts"), ctypes.byref(n) if argmax_parts is not None else None]
    _ok(_load().lk_gemv_q8(*args, _cfg(cfg), _stream(stream)), "lk_gemv_q8")
    return n.value


def lk_gemv_q8_group(mats, mode, x=None, xq=None, xl=None, xs=None, M=None, stream=None, cfg=None):
    """mats: [(wq, ws, y), ...] sharing K and the activation: y = W x for
    each, with the bits of one lk_gemv_q8 call per matrix; one launch where
    the tensor-core kernel (2..8 rows) or, for two or more matrices, the
    chain kernel's ring arrangement (one row) takes the shapes."""
    K = mats[0][0].shape[1]
    if M is None:
        M = (x if x is not None else xq).shape[0]
    arr = (LkGemvTarget * len(mats))(*[LkGemvTarget(_ptr(wq, _I8, "wq"), _ptr(ws, _WS, "ws"), wq.shape[0], 0,
                                                    _ptr(y, _F32, "y")) for wq, ws, y in mats])
    for wq, _, _ in mats:
        if wq.shape[1] != K:
            raise ValueError("lk_gemv_q8_group: matrices of one group share K")
    args = [ctypes.cast(arr, ctypes.c_void_p), len(mats), K, _mode(mode), _ptr(x, _F32, "x"), _ptr(xq, _I8, "xq"),
            _ptr(xl, _I8, "xl"), _ptr(xs, _F32, "xs"), M]
    _ok(_load().lk_gemv_q8_group(*args, _cfg(cfg), _stream(stream)), "lk_gemv_q8_group")


def lk_gemv_q8_glu(wg, wsg, wu, wsu, mode, gu, x=None, xq=None, xl=None, xs=None, h=None, hq=None, hl=None,
                   hs=None, cnt=None, M=None, stream=None, cfg=None):
    """g = Wg x, u = Wu x into gu [2, M, F]; h = silu(g) * u (optional f32
    [M, F]) and its quantized words hq/hl/hs for the next GEMV.  cnt: int32
    [F/32] zeroed counters (enables the one-launch kernel at M = 1)."""
    F, K = wg.shape
    if tuple(wu.shape) != (F, K):
        raise ValueError("the gate and up matrices must have the same shape")
    if M is None:
        M = (x if x is not None else xq).shape[0]
    if tuple(gu.shape) != (2, M, F):
        raise ValueError("gu must be [2, M, F]")
    args = [_ptr(wg, _I8, "wg"), _ptr(wsg, _WS, "wsg"), _ptr(wu, _I8, "wu"), _ptr(wsu, _WS, "wsu"), F, K,
            _mode(mode), _ptr(x, _F32, "x"), _ptr(xq, _I8, "xq"), _ptr(xl, _I8, "xl"), _ptr(xs, _F32, "xs"), M,
            _ptr(gu, _F32, "gu"), _ptr(h, _F32, "h"), _ptr(hq, _I8, "hq"), _ptr(hl, _I8, "hl"), _ptr(hs, _F32, "hs"),
            _ptr(cnt, torch.int32, "cnt")]
    _ok(_load().lk_gemv_q8_glu(*args, _cfg(cfg), _stream(stream)), "lk_gemv_q8_glu")


def lk_gemv_kernel_for(N, K, mode, M, S=0, cfg=None) -> int:
    """1 direct kernel, 2 bulk-copy ring kernel, 3 tensor-core kernel, 0 none
    (see include/lk.h)."""
    return _load().lk_gemv_kernel_for(N, K, _mode(mode), M, S, _cfg(cfg))


def lk_rmsnorm_quant_gemv_q8(wq, ws, mode, x, y, gain=None, eps=1e-6, argmax_parts=None,
                             stream=None, cfg=None) -> int:
    """RMSNorm (gain given) or quantize only (gain None) -> GEMV in one launch.
    Returns the number of argmax partial keys per activation row."""
    N, K = wq.shape
    M = x.shape[0]
    n = ctypes.c_int(0)
    _ok(_load().lk_rmsnorm_quant_gemv_q8(_ptr(wq, _I8, "wq"), _ptr(ws, _WS, "ws"), N, K, _mode(mode),
                                         _ptr(x, _F32, "x"), _ptr(gain, _F32, "gain"), eps, M,
                                         _ptr(y, _F32, "y"),
                                         _ptr(argmax_parts, torch.int64, "argmax_parts"),
                                         ctypes.byref(n) if argmax_parts is not None else None,
                                         _cfg(cfg), _stream(stream)), "lk_rmsnorm_quant_gemv_q8")
    return n.value


def lk_splitk_workspace_bytes(mode, S, M, N) -> int:
    return _load().lk_splitk_workspace_bytes(_mode(mode), S, M, N)


def lk_gemv_q8_splitk(wq, ws, mode, S, part, x=None, xq=None, xl=None, xs=None, M=None, stream=None, cfg=None):
    N, K = wq.shape
    if M is None:
        M = (x if x is not None else xq).shape[0]
    _ok(_load().lk_gemv_q8_splitk(_ptr(wq, _I8, "wq"), _ptr(ws, _WS, "ws"), N, K, _mode(mode),
                                  _ptr(x, _F32, "x"), _ptr(xq, _I8, "xq"), _ptr(xl, _I8, "xl"),
                                  _ptr(xs, _F32, "xs"), M, S, _ptr(part, None, "part"),
                                  part.numel() * part.element_size(), _cfg(cfg), _stream(stream)),
        "lk_gemv_q8_splitk")


def lk_splitk_combine(mode, part, S, M, N, y, stream=None, cfg=None):
    _ok(_load().lk_splitk_combine(_mode(mode), _ptr(part, None, "part"), S, M, N, _ptr(y, _F32, "y"),
                                  _cfg(cfg), _stream(stream)), "lk_splitk_combine")


def lk_splitk_chunks_for(N, K, mode, M) -> int:
    """The split-K chunk count the library favours for this shape (1: the
    plain GEMV; see include/lk.h)."""
    return _load().lk_splitk_chunks_for(N, K, _mode(mode), M)


def lk_argmax_parts_max(N) -> int:
    return _load().lk_argmax_parts_max(N)


def lk_argmax_scratch_entries(N) -> int:
    return _load().lk_argmax_scratch_entries(N)


def lk_argmax(idx, M, N, logits=None, parts=None, n_parts=0, scratch=None, stream=None):
    _ok(_load().lk_argmax(_ptr(logits, _F32, "logits"), _ptr(parts, torch.int64, "parts"), n_parts, M,
                          N, _ptr(idx, torch.int32, "idx"), _ptr(scratch, torch.int64, "scratch"),
                          _stream(stream)), "lk_argmax")


def lk_q8_block_dots(wq, xq, d, xl=None, e=None, stream=None):
    N, K = wq.shape
    _ok(_load().lk_q8_block_dots(_ptr(wq, _I8, "wq"), N, K, _ptr(xq, _I8, "xq"), _ptr(xl, _I8, "xl"),
                                 _ptr(d, torch.int32, "d"), _ptr(e, torch.int32, "e"), _stream(stream)),
        "lk_q8_block_dots")


def lk_set_option(name: str, value: int):
    _ok(_load().lk_set_option(name.encode(), int(value)), f"lk_set_option({name})")


def lk_get_option(name: str) -> int:
    return _load().lk_get_option(name.encode())


def lk_device_error(reset: bool = True) -> int:
    code = ctypes.c_int(0)
    st = _load().lk_device_error(1 if reset else 0, ctypes.byref(code))
    if st not in (0, -6):
        raise LkError(st, "lk_device_error")
    return code.value


def lk_selftest_wait_timeout(limit_us: int, stream=None):
    _ok(_load().lk_selftest_wait_timeout(int(limit_us), _stream(stream)), "lk_selftest_wait_timeout")


def lk_chain_sync_bytes() -> int:
    return _load().lk_chain_sync_bytes()


def chain_op(wq, ws, x, y, gain=None, argmax_parts=None, argmax_idx=None, wait=False) -> LkChainOp:
    """Marshal one lk_chain_op from device tensors (they must outlive the chain)."""
    N, K = wq.shape
    return LkChainOp(_ptr(wq, _I8, "wq"), _ptr(ws, _WS, "ws"), N, K, _ptr(x, _F32, "x"),
                     _ptr(gain, _F32, "gain"), _ptr(y, _F32, "y"),
                     _ptr(argmax_parts, torch.int64, "argmax_parts"), _ptr(argmax_idx, torch.int32, "argmax_idx"),
                     1 if wait else 0, 0)


class Chain:
    """A host array of lk_chain_op, its device copy and a zeroed sync buffer."""

    def __init__(self, ops, device):
        self.n = len(ops)
        self.host = (LkChainOp * self.n)(*ops)
        raw = bytes(self.host)
        self.dev = torch.frombuffer(bytearray(raw), dtype=torch.uint8).to(device)
        self.sync = torch.zeros((lk_chain_sync_bytes() // 4,), dtype=torch.int32, device=device)


def lk_gemv_chain(chain: "Chain", mode, M, eps=1e-6, stream=None, cfg=None):
    _ok(_load().lk_gemv_chain(ctypes.cast(chain.host, ctypes.c_void_p), _ptr(chain.dev, None, "ops_dev"),
                              chain.n, _mode(mode), M, eps, _ptr(chain.sync, None, "sync"), _cfg(cfg),
                              _stream(stream)), "lk_gemv_chain")


def lk_trace_read(n: int):
    """Block 0's timestamps of the last traced launch (ns), as a list."""
    buf = (ctypes.c_uint64 * n)()
    _ok(_load().lk_trace_read(ctypes.cast(buf, ctypes.c_void_p), n), "lk_trace_read")
    return list(buf)


def lk_argmax_noalloc(logits, idx, stream=None):
    """Argmax of logits [M, N] into idx [M] with no caller scratch (see lk.h)."""
    M, N = logits.shape
    _ok(_load().lk_argmax_noalloc(_ptr(logits, _F32, "logits"), M, N, _ptr(idx, torch.int32, "idx"),
                                  _stream(stream)), "lk_argmax_noalloc")


# ---- the GGUF block formats other than Q8_0 ------------------------------------------

FORMATS = {"q4_0": 2, "q4_1": 3, "q5_0": 6, "q5_1": 7, "q2_k": 10, "q3_k": 11, "q4_k": 12, "q5_k": 13,
           "q6_k": 14, "iq4_nl": 20, "iq4_xs": 23, "mxfp4": 39}


def _fmt(fmt):
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def lk_format_row_bytes(fmt, K) -> int:
    return int(_load().lk_format_row_bytes(_fmt(fmt), K))


def lk_gemv_blk(fmt, w, K, mode, y, x=None, xq=None, xl=None, xs=None, M=None, stream=None, cfg=None):
    """y[M, N] = W x for a block-format matrix w (uint8 [N, row_bytes])."""
    N = w.shape[0]
    if M is None:
        M = (x if x is not None else xq).shape[0]
    if w.shape[1] != lk_format_row_bytes(fmt, K):
        raise ValueError("w rows must be lk_format_row_bytes(fmt, K) bytes")
    _ok(_load().lk_gemv_blk(_fmt(fmt), _ptr(w, torch.uint8, "w"), N, K, _mode(mode), _ptr(x, _F32, "x"),
                            _ptr(xq, _I8, "xq"), _ptr(xl, _I8, "xl"), _ptr(xs, _F32, "xs"), M, _ptr(y, _F32, "y"),
                            _cfg(cfg), _stream(stream)), "lk_gemv_blk")


def lk_dequant_blk(fmt, w, K, out, stream=None):
    """The decoded weights f32 [N, K] of a block-format matrix (test hook)."""
    _ok(_load().lk_dequant_blk(_fmt(fmt), _ptr(w, torch.uint8, "w"), w.shape[0], K, _ptr(out, _F32, "out"),
                               _stream(stream)), "lk_dequant_blk")


# ---- the attention step: paged cache, append, attention (include/lk_attn.h) ----------

LK_KV_F16, LK_KV_BF16, LK_KV_Q8 = 0, 1, 2
_KV_TYPES = {torch.float16: LK_KV_F16, torch.bfloat16: LK_KV_BF16, torch.int8: LK_KV_Q8}
_I32 = torch.int32


class LkKvCache(ctypes.Structure):
    """The C struct lk_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", ctypes.c_void_p), ("vs", ctypes.c_void_p),
                ("type", ctypes.c_int), ("n_kv", ctypes.c_int), ("head_dim", ctypes.c_int), ("page", ctypes.c_int),
                ("n_pages", ctypes.c_int), ("reserved", ctypes.c_int)]


class KvCache:
    """A paged key/value cache over the caller's tensors: k, v [n_pages, n_kv,
    page, head_dim] in float16, bfloat16, or int8 levels with their float16
    scales ks, vs [n_pages, n_kv, page, head_dim / 32].  Marshalled once; the
    tensors are kept alive with it."""

    def __init__(self, k, v, ks=None, vs=None):
        self.k, self.v, self.ks, self.vs = k, v, ks, vs
        if not isinstance(k, torch.Tensor) or k.dtype not in _KV_TYPES:
            raise TypeError("k must be a float16, bfloat16 or int8 tensor")
        if k.dim() != 4:
            raise ValueError("k must be [n_pages, n_kv, page, head_dim]")
        kp, vp = _ptr(k, k.dtype, "k"), _ptr(v, k.dtype, "v")
        if v.shape != k.shape or v.device != k.device:
            raise ValueError("v must have the shape and device of k")
        if (k.dtype == torch.int8) != (ks is not None) or (ks is None) != (vs is None):
            raise ValueError("ks and vs go with int8 levels")
        self.device, self.dev, self.n_kv, self.head_dim = k.device, k.get_device(), k.shape[1], k.shape[3]
        if ks is not None:
            for name, t in (("ks", ks), ("vs", vs)):
                if tuple(t.shape) != (*k.shape[:3], k.shape[3] // 32) or t.device != k.device:
                    raise ValueError(f"{name} must be [n_pages, n_kv, page, head_dim / 32] on the device of k")
        self.c = LkKvCache(kp, vp, _ptr(ks, torch.float16, "ks"), _ptr(vs, torch.float16, "vs"), _KV_TYPES[k.dtype],
                           k.shape[1], k.shape[3], k.shape[2], k.shape[0], 0)
        self.ref = ctypes.byref(self.c)


def _on(dev, t, dtype, name, shape=None):
    """Pointer of a contiguous tensor of that dtype (and shape) on device
    number dev."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _kv_rows(cache, table, lens, R):
    """Checks of the arguments every call on a cache takes: (device number,
    table pointer, table width, lens pointer, B)."""
    dev = cache.dev
    if torch.cuda.current_device() != dev:
        raise ValueError(f"the cache is on cuda:{dev}, which is not the current device")
    if table.dim() != 2:
        raise ValueError("table must be [B, pages]")
    B, w = table.shape
    if R < 0:
        raise ValueError("R must not be negative")
    return dev, _on(dev, table, _I32, "table") if w else None, w, _on(dev, lens, _I32, "lens", (B,)), B


def _on_stream(stream, dev):
    """The raw stream: the device's current one without the object around it."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def lk_kv_append(cache: KvCache, q, k, v, table, lens, cosines, sines, qr, R=1, p0=0, paired=False, q_gain=None,
                 k_gain=None, eps=1e-6, stream=None, cfg=None):
    """Append the rows' keys and values to the cache, rotated, and write the
    rotated queries to qr [M, n_q * head_dim] (see include/lk_attn.h).  q, k, v: f32
    rows of one pitch (column ranges of one fused projection output, say);
    table int32 [B, pages], lens int32 [B] with the R new tokens of each
    sequence counted; cosines, sines f32 [positions, rot / 2] or None (no
    rotation)."""
    dev, tp, tw, lp, B = _kv_rows(cache, table, lens, R)
    D, M, N = cache.head_dim, B * R, q.shape[-1]
    ld = q.stride(0) if M > 1 else N
    for name, t, n in (("q", q, N), ("k", k, cache.n_kv * D), ("v", v, cache.n_kv * D)):
        if not isinstance(t, torch.Tensor) or t.dtype is not _F32 or t.dim() != 2:
            raise TypeError(f"{name} must be a 2-D float32 tensor")
        if t.get_device() != dev or t.shape != (M, n) or t.stride(1) != 1:
            raise ValueError(f"{name} must be [{M}, {n}] with contiguous rows on cuda:{dev}")
        if M > 1 and t.stride(0) != ld:
            raise ValueError("q, k and v must have the same row pitch")
    if N % D:
        raise ValueError("q rows must be heads of head_dim values")
    rot = n_pos = 0
    if cosines is not None:
        if cosines.dim() != 2:
            raise ValueError("cosines must be [positions, rot / 2]")
        n_pos, rot = cosines.shape[0], 2 * cosines.shape[1]
    elif sines is not None:
        raise ValueError("cosines and sines go together")
    for name, t in (("q_gain", q_gain), ("k_gain", k_gain)):
        if t is not None and t.shape != (D,):
            raise ValueError(f"{name} must be [head_dim]")
    _ok(_load().lk_kv_append(cache.ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), ld, N // D, tp, tw, lp, B, R, p0,
                             _on(dev, cosines, _F32, "cosines"),
                             _on(dev, sines, _F32, "sines", cosines.shape) if cosines is not None else None, n_pos,
                             rot, 1 if paired else 0, _on(dev, q_gain, _F32, "q_gain"),
                             _on(dev, k_gain, _F32, "k_gain"), eps, _on(dev, qr, _F32, "qr", (M, N)), _cfg(cfg),
                             _on_stream(stream, dev)), "lk_kv_append")


def lk_attn_workspace_bytes(n_q, n_kv, head_dim, B, R=1, shared=False) -> int:
    return _load().lk_attn_workspace_bytes(n_q, n_kv, head_dim, B, R, 1 if shared else 0)


def lk_attn_launches(cache, n_q, B, table_w, R=1, prefix_len=0) -> int:
    """Kernels that lk_attn (lk_attn_shared) on this cache launches, with tables
    of table_w pages."""
    return _load().lk_attn_launches(cache.c.type, n_q, cache.n_kv, cache.head_dim, B, R, prefix_len,
                                    table_w * cache.c.page)


def _attn_tail(cache, q, M, scale, mode, out, hq, hl, hs, ws):
    dev, N = cache.dev, q.shape[-1]
    qp = _on(dev, q, _F32, "q", (M, N))
    if N % cache.head_dim:
        raise ValueError("q rows must be heads of head_dim values")
    if scale is None:
        scale = cache.head_dim ** -0.5
    return qp, N // cache.head_dim, (
        scale, _mode(mode), _on(dev, out, _F32, "out", (M, N)), _on(dev, hq, _I8, "hq", (M, N)),
        _on(dev, hl, _I8, "hl", (M, N)), _on(dev, hs, _F32, "hs", (M, N // 32)), _on(dev, ws, torch.uint8, "ws"),
        ws.numel())


def lk_attn(cache: KvCache, q, table, lens, ws, R=1, scale=None, mode=LK_DEQUANT, out=None, hq=None, hl=None, hs=None,
            stream=None, cfg=None):
    """Attention of the rows q [B * R, n_q * head_dim] over their sequences'
    cached tokens (see include/lk_attn.h): f32 rows in out and / or, by mode, the
    next projection's words hq, hl and scales hs.  ws: uint8 workspace of
    lk_attn_workspace_bytes.  scale None: 1 / sqrt(head_dim)."""
    dev, tp, tw, lp, B = _kv_rows(cache, table, lens, R)
    qp, n_q, tail = _attn_tail(cache, q, B * R, scale, mode, out, hq, hl, hs, ws)
    _ok(_load().lk_attn(cache.ref, qp, n_q, tp, tw, lp, B, R, *tail, _cfg(cfg),
                        _on_stream(stream, dev)), "lk_attn")


def lk_attn_shared(cache: KvCache, q, prefix_table, prefix_len, table, lens, ws, R=1, scale=None, mode=LK_DEQUANT,
                   out=None, hq=None, hl=None, hs=None, stream=None, cfg=None):
    """lk_attn for sequences that continue one prefix of prefix_len tokens in
    the pages prefix_table (int32); table and lens are the sequences' own."""
    dev, tp, tw, lp, B = _kv_rows(cache, table, lens, R)
    qp, n_q, tail = _attn_tail(cache, q, B * R, scale, mode, out, hq, hl, hs, ws)
    _ok(_load().lk_attn_shared(cache.ref, qp, n_q, _on(dev, prefix_table, _I32, "prefix_table"),
                               0 if prefix_table is None else prefix_table.numel(), prefix_len, tp, tw, lp, B, R,
                               *tail, _cfg(cfg), _on_stream(stream, dev)), "lk_attn_shared")


# ---- a mixture of experts: routing, the experts' products (include/lk_moe.h) ----------

LK_MOE_MAX_E, LK_MOE_MAX_K, LK_MOE_MAX_GROUPS = 1024, 32, 32
SCORES = {"softmax": 0, "sigmoid": 1}


def _here(t, name):
    """The device number of tensor t, which has to be the current device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    dev = t.get_device()
    if dev < 0 or torch.cuda.current_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    return dev


def lk_moe_route(logits, ids, weights, bias=None, score="softmax", n_group=1, top_group=1, group_sum=1, renorm=True,
                 scale=1.0, stream=None, cfg=None):
    """The experts ids int32 [M, k] of each row of router logits f32 [M, E] and
    their weights f32 [M, k] (see include/lk_moe.h).  score "softmax" or
    "sigmoid"; bias f32 [E] is added for the choice alone; of n_group groups
    of experts the top_group best stay, by the sum of their group_sum largest;
    renorm: weights over their sum, times scale."""
    dev = _here(logits, "logits")
    if logits.dim() != 2 or ids.dim() != 2:
        raise ValueError("logits must be [M, E], ids [M, k]")
    M, E = logits.shape
    k = ids.shape[1]
    _ok(_load().lk_moe_route(_on(dev, logits, _F32, "logits"), _on(dev, bias, _F32, "bias", (E,)), M, E,
                             SCORES[score] if isinstance(score, str) else int(score), n_group, top_group, group_sum,
                             k, 1 if renorm else 0, scale, _on(dev, ids, _I32, "ids", (M, k)),
                             _on(dev, weights, _F32, "weights", (M, k)), _cfg(cfg), _on_stream(stream, dev)),
        "lk_moe_route")


class Experts:
    """Q8_0 matrices of E experts over the caller's tensors: gate and up
    (levels int8 [E, F, K], scales float16 [E, F, K / 32]) and / or down
    ([E, K, F], [E, K, F / 32]).  Marshalled once; the tensors are kept alive
    with it."""

    def __init__(self, gate=None, up=None, down=None):
        if (gate is None) != (up is None) or (gate is None and down is None):
            raise ValueError("gate and up go together; at least they or down")
        self.gate, self.up, self.down = gate, up, down
        first = gate or down
        self.dev = first[0].get_device()
        self.E = first[0].shape[0]
        for name, pair in (("gate", gate), ("up", up), ("down", down)):
            if pair is None:
                continue
            q, s = pair
            if not isinstance(q, torch.Tensor) or q.dtype != _I8 or q.dim() != 3 or s.dtype not in _WS:
                raise TypeError(f"{name} must be int8 levels [E, rows, K] and their float16 scales")
            if q.shape[0] != self.E or tuple(s.shape) != (*q.shape[:2], q.shape[2] // 32):
                raise ValueError(f"{name}'s scales must be [E, rows, K / 32], E the same for all")
            if q.get_device() != self.dev or s.get_device() != self.dev or self.dev < 0:
                raise ValueError("the experts' tensors must be on one CUDA device")
            if not q.is_contiguous() or not s.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if gate is not None and gate[0].shape != up[0].shape:
            raise ValueError("gate and up must have the same shape")
        if gate is not None and down is not None and down[0].shape[2] != gate[0].shape[1]:
            raise ValueError("down's rows must be as long as gate has rows")
        self._gu = None if gate is None else (*(t.data_ptr() for t in (*gate, *up)), *gate[0].shape)
        self._down = None if down is None else (*(t.data_ptr() for t in down), *down[0].shape)


def _pairs(experts, ids):
    if torch.cuda.current_device() != experts.dev:
        raise ValueError(f"the experts are on cuda:{experts.dev}, which is not the current device")
    if ids.dim() != 2:
        raise ValueError("ids must be [M, k]")
    return (experts.dev, *ids.shape)


def lk_moe_glu_q8(experts: Experts, mode, ids, h, x=None, xq=None, xl=None, xs=None, hq=None, hl=None, hs=None, cnt=None,
                  stream=None, cfg=None):
    """h[t * k + j] = silu(gate x_t) * (up x_t) with the matrices of expert
    ids[t, j] (see include/lk_moe.h): h f32 [M * k, F] and, with hq, its words hq,
    hl and scales hs for the down products (cnt: zeroed int32, M * k * F / 32 of
    them at least).  The rows x or xq, xl, xs [M, K] by mode, as lk_gemv_q8's."""
    dev, M, k = _pairs(experts, ids)
    if experts._gu is None:
        raise ValueError("these experts have no gate and up matrices")
    *w, E, F, K = experts._gu
    n = M * k
    if cnt is not None and cnt.numel() < n * F // 32:
        raise ValueError("cnt must have M * k * F / 32 entries")
    _ok(_load().lk_moe_glu_q8(*w, E, F, K, _mode(mode), _on(dev, x, _F32, "x", (M, K)), _on(dev, xq, _I8, "xq", (M, K)),
                              _on(dev, xl, _I8, "xl", (M, K)), _on(dev, xs, _F32, "xs", (M, K // 32)), M,
                              _on(dev, ids, _I32, "ids"), k, _on(dev, h, _F32, "h", (n, F)),
                              _on(dev, hq, _I8, "hq", (n, F)), _on(dev, hl, _I8, "hl", (n, F)),
                              _on(dev, hs, _F32, "hs", (n, F // 32)), _on(dev, cnt, _I32, "cnt"), _cfg(cfg),
                              _on_stream(stream, dev)), "lk_moe_glu_q8")


def lk_moe_down_q8(experts: Experts, mode, ids, weights, y, h=None, hq=None, hl=None, hs=None, stream=None, cfg=None):
    """y[t] = sum over j of weights[t, j] * (down h[t * k + j]) with the matrix
    of expert ids[t, j] (see include/lk_moe.h); h, or hq, hl, hs by mode, as
    lk_moe_glu_q8 gives them."""
    dev, M, k = _pairs(experts, ids)
    if experts._down is None:
        raise ValueError("these experts have no down matrices")
    *w, E, N, F = experts._down
    n = M * k
    _ok(_load().lk_moe_down_q8(*w, E, N, F, _mode(mode), _on(dev, h, _F32, "h", (n, F)), _on(dev, hq, _I8, "hq", (n, F)),
                               _on(dev, hl, _I8, "hl", (n, F)), _on(dev, hs, _F32, "hs", (n, F // 32)), M,
                               _on(dev, ids, _I32, "ids"), _on(dev, weights, _F32, "weights", (M, k)), k,
                               _on(dev, y, _F32, "y", (M, N)), _cfg(cfg), _on_stream(stream, dev)), "lk_moe_down_q8")


# ---- the next token drawn from the logits (include/lk_sample.h) -------------------------

def lk_sample(logits, u, idx, prob=None, temperature=None, top_k=None, top_p=None, min_p=None, stream=None, cfg=None):
    """One token idx int32 [M] for each row of logits f32 [M, N], drawn by the
    numbers u f32 [M] in [0, 1) from what temperature, top_k, top_p and min_p
    ([M] tensors, None: off) leave, and its probability prob f32 [M] (see
    include/lk_sample.h)."""
    dev = _here(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [M, N]")
    M, N = logits.shape
    _ok(_load().lk_sample(_on(dev, logits, _F32, "logits"), M, N, _on(dev, temperature, _F32, "temperature", (M,)),
                          _on(dev, top_k, _I32, "top_k", (M,)), _on(dev, top_p, _F32, "top_p", (M,)),
                          _on(dev, min_p, _F32, "min_p", (M,)), _on(dev, u, _F32, "u", (M,)),
                          _on(dev, idx, _I32, "idx", (M,)), _on(dev, prob, _F32, "prob", (M,)), _cfg(cfg),
                          _on_stream(stream, dev)), "lk_sample")
