"""ctypes binding of libace (``include/ace.h``), with the C names.

Argument marshalling only: torch tensors provide device memory and the
current CUDA stream; every step of the computation runs in libace's kernels.
There is no fallback: if ``libace.so`` is missing or fails to load, importing
this module raises.
"""
import ctypes
import functools
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libace.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libace.so not built: run `python -m token_dynamic_expert_b200.build` "
                      "(expected at %s)" % LIB_PATH)
_lib = ctypes.CDLL(LIB_PATH)

# ------------------------------------------------------------------ C types
ACE_OK, ACE_ERR_INVALID_ARG, ACE_ERR_WORKSPACE, ACE_ERR_CUDA, ACE_ERR_UNSUPPORTED, \
    ACE_ERR_DEVICE_FAULT, ACE_ERR_TIMEOUT, ACE_ERR_IO = range(8)
ACE_BF16, ACE_F32 = 0, 1
ACE_GSP_FRO, ACE_GSP_SPECTRAL = 0, 1
ACE_FUSE_MAX, ACE_FUSE_MIN, ACE_FUSE_MEAN, ACE_FUSE_GSP, ACE_FUSE_RCR = 0, 1, 2, 3, 4
FUSIONS = {"max": ACE_FUSE_MAX, "min": ACE_FUSE_MIN, "mean": ACE_FUSE_MEAN, "gsp": ACE_FUSE_GSP,
           "rcr": ACE_FUSE_RCR}
ACE_SCORE_SOFTMAX, ACE_SCORE_SIGMOID = 0, 1
SCORES = {"softmax": ACE_SCORE_SOFTMAX, "sigmoid": ACE_SCORE_SIGMOID}
ACE_GROUP_MAX, ACE_GROUP_TOP2 = 0, 1
GROUP_SCORES = {"max": ACE_GROUP_MAX, "top2": ACE_GROUP_TOP2}
MAX_COUNT = 2 ** 31 - 256  # most rows, tokens or slots of one 8-bit operator
ACE_FLAG_BAD_INDEX, ACE_FLAG_TIMEOUT, ACE_FLAG_OVERFLOW = 0x1, 0x2, 0x4

_vp = ctypes.c_void_p


class ace_layer(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("E", ctypes.c_int), ("m", ctypes.c_int), ("k", ctypes.c_int),
                ("dtype", ctypes.c_int), ("gamma", _vp), ("w_router", _vp), ("router_bias", _vp),
                ("w_gate", _vp), ("w_up", _vp), ("w_down", _vp), ("amax", _vp), ("a_gsp", _vp),
                ("a_rcr", _vp)]


class ace_fwd_opts(ctypes.Structure):
    _fields_ = [("tau", ctypes.c_float), ("renorm_topk", ctypes.c_int), ("fusion", ctypes.c_int),
                ("eps_rms", ctypes.c_float)]


class ace_debug_out(ctypes.Structure):
    _fields_ = [("topk_idx", _vp), ("gate", _vp), ("score", _vp), ("keep", _vp),
                ("expert_offsets", _vp), ("slot_token", _vp), ("slot_rank", _vp),
                ("n_kept", _vp), ("logits", _vp), ("ev_experts_begin", _vp),
                ("ev_experts_mid", _vp), ("ev_experts_end", _vp), ("trace", _vp)]


class ace_gate_opts(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int), ("n_groups", ctypes.c_int), ("topk_groups", ctypes.c_int),
                ("group_score", ctypes.c_int), ("renorm_topk", ctypes.c_int),
                ("scale", ctypes.c_float), ("tau", ctypes.c_float)]


class ace_i8_product(ctypes.Structure):
    _fields_ = [("xq", _vp), ("ldx", ctypes.c_int64), ("n_rows", ctypes.c_int), ("x_scale", _vp),
                ("wq", _vp), ("w_scale", _vp), ("E", ctypes.c_int), ("N", ctypes.c_int),
                ("K", ctypes.c_int), ("offsets", _vp), ("row_of", _vp), ("slot_scale", _vp)]


class ace_table_opts(ctypes.Structure):
    _fields_ = [("gsp_norm", ctypes.c_int), ("eps", ctypes.c_float), ("rho", ctypes.c_float),
                ("power_iters", ctypes.c_int)]


_P = ctypes.POINTER
_lib.ace_workspace_size.argtypes = [_P(ace_layer), ctypes.c_int]
_lib.ace_workspace_size.restype = ctypes.c_size_t
_lib.ace_moe_forward.argtypes = [_P(ace_layer), _vp, ctypes.c_int, _P(ace_fwd_opts), _vp, _vp,
                                 ctypes.c_size_t, _P(ace_debug_out), _vp]
_lib.ace_moe_forward.restype = ctypes.c_int
_lib.ace_moe_scores.argtypes = [_P(ace_layer), _vp, ctypes.c_int, _P(ace_fwd_opts), _vp, _vp, _vp,
                                ctypes.c_size_t, _vp]
_lib.ace_moe_scores.restype = ctypes.c_int
_lib.ace_moe_route.argtypes = [_P(ace_layer), _vp, ctypes.c_int, _P(ace_fwd_opts), _vp, _vp, _vp,
                               _vp, _vp, ctypes.c_size_t, _vp]
_lib.ace_moe_route.restype = ctypes.c_int
_lib.ace_experts_workspace_size.argtypes = [_P(ace_layer), ctypes.c_int]
_lib.ace_experts_workspace_size.restype = ctypes.c_size_t
_lib.ace_moe_experts.argtypes = [_P(ace_layer), _vp, ctypes.c_int, _vp, _vp, _vp, _vp,
                                 ctypes.c_size_t, _vp]
_lib.ace_moe_experts.restype = ctypes.c_int
_lib.ace_moe_combine.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _vp,
                                 ctypes.c_int, _vp, _vp, ctypes.c_size_t, _vp]
_lib.ace_moe_combine.restype = ctypes.c_int
_lib.ace_tables_save.argtypes = [ctypes.c_char_p, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp]
_lib.ace_tables_save.restype = ctypes.c_int
_lib.ace_tables_info.argtypes = [ctypes.c_char_p, _P(ctypes.c_int), _P(ctypes.c_int),
                                 _P(ctypes.c_int)]
_lib.ace_tables_info.restype = ctypes.c_int
_lib.ace_tables_load.argtypes = [ctypes.c_char_p, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp]
_lib.ace_tables_load.restype = ctypes.c_int
_lib.ace_moe_decode_noalloc.argtypes = [_P(ace_layer), _vp, ctypes.c_int, _P(ace_fwd_opts), _vp,
                                        _vp]
_lib.ace_moe_decode_noalloc.restype = ctypes.c_int
_lib.ace_tables_workspace_size.argtypes = [_P(ace_layer)]
_lib.ace_tables_workspace_size.restype = ctypes.c_size_t
_lib.ace_build_tables.argtypes = [_P(ace_layer), ctypes.c_int, _P(ace_table_opts), _vp, _vp, _vp,
                                  _vp, _vp, ctypes.c_size_t, _vp]
_lib.ace_build_tables.restype = ctypes.c_int
_lib.ace_stack_workspace_size.argtypes = [_P(ace_layer), ctypes.c_int, ctypes.c_int]
_lib.ace_stack_workspace_size.restype = ctypes.c_size_t
_lib.ace_moe_stack_forward.argtypes = [_P(ace_layer), ctypes.c_int, _vp, ctypes.c_int,
                                       _P(ace_fwd_opts), _vp, _vp, ctypes.c_size_t, _vp]
_lib.ace_moe_stack_forward.restype = ctypes.c_int
_lib.ace_tau_workspace_size.argtypes = []
_lib.ace_tau_workspace_size.restype = ctypes.c_size_t
_lib.ace_tau_quantile.argtypes = [_vp, ctypes.c_int, ctypes.c_int, ctypes.c_int64, _vp, _vp,
                                  ctypes.c_size_t, _vp]
_lib.ace_tau_quantile.restype = ctypes.c_int
_lib.ace_logits_workspace_size.argtypes = [_P(ace_layer), ctypes.c_int]
_lib.ace_logits_workspace_size.restype = ctypes.c_size_t
_lib.ace_moe_logits.argtypes = [_P(ace_layer), _vp, ctypes.c_int, ctypes.c_float, _vp, _vp,
                                ctypes.c_size_t, _vp]
_lib.ace_moe_logits.restype = ctypes.c_int
_i64 = ctypes.c_int64
_lib.ace_add_rmsnorm.argtypes = [_vp, _i64, _vp, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                 _vp, ctypes.c_float, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp]
_lib.ace_add_rmsnorm.restype = ctypes.c_int
_lib.ace_gate_topk.argtypes = [_vp, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                               _vp, _P(ace_gate_opts), _vp, _vp, _vp, _vp, _vp]
_lib.ace_gate_topk.restype = ctypes.c_int
_lib.ace_moe_group.argtypes = [_vp, _vp, _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _vp,
                               _vp, _vp, _vp]
_lib.ace_moe_group.restype = ctypes.c_int
_lib.ace_matmul_i8.argtypes = [_vp, ctypes.c_int,  # ace_i8_product *
                                _vp, _i64, ctypes.c_int, _vp,
                               ctypes.c_size_t, _vp]
_lib.ace_matmul_i8.restype = ctypes.c_int
_lib.ace_swiglu.argtypes = [_vp, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _vp, _i64,
                            _vp, _i64, _vp, _vp]
_lib.ace_swiglu.restype = ctypes.c_int
_lib.ace_noalloc_read_status.argtypes = [_P(ctypes.c_uint32), _vp]
_lib.ace_noalloc_read_status.restype = ctypes.c_int
_lib.ace_set_peer_wait_limit_ns.argtypes = [ctypes.c_uint64]
_lib.ace_set_peer_wait_limit_ns.restype = ctypes.c_uint64
_lib.ace_read_status.argtypes = [_vp, ctypes.c_size_t, _P(ctypes.c_uint32), _vp]
_lib.ace_read_status.restype = ctypes.c_int
_lib.ace_status_str.argtypes = [ctypes.c_int]
_lib.ace_status_str.restype = ctypes.c_char_p
_lib.ace_version.restype = ctypes.c_char_p
_lib.ace_last_cuda_error.restype = ctypes.c_char_p


class AceError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        msg = "%s: %s" % (where, ace_status_str(code))
        if code == ACE_ERR_CUDA:
            msg += " (%s)" % _lib.ace_last_cuda_error().decode()
        super().__init__(msg)


def _check(code, where):
    if code != ACE_OK:
        raise AceError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def lib():
    return _lib


def ace_status_str(code):
    return _lib.ace_status_str(int(code)).decode()


def ace_version():
    return _lib.ace_version().decode()


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return ACE_BF16
    if t.dtype == torch.float32:
        return ACE_F32
    raise TypeError("unsupported dtype %s" % t.dtype)


def make_layer(gamma, w_router, w_gate, w_up, w_down, k, amax=None, router_bias=None,
               a_gsp=None, a_rcr=None):
    """Pack device tensors into an ``ace_layer``.  The caller keeps the tensors
    alive while the struct is in use."""
    E, d = w_router.shape
    m = w_gate.shape[1]
    for t in (gamma, w_router, w_gate, w_up, w_down, amax, router_bias, a_gsp, a_rcr):
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    return ace_layer(d=d, E=E, m=m, k=k, dtype=_dtype_code(w_router), gamma=_ptr(gamma),
                     w_router=_ptr(w_router), router_bias=_ptr(router_bias), w_gate=_ptr(w_gate),
                     w_up=_ptr(w_up), w_down=_ptr(w_down), amax=_ptr(amax), a_gsp=_ptr(a_gsp),
                     a_rcr=_ptr(a_rcr))


def _fusion(f):
    return FUSIONS[f] if isinstance(f, str) else int(f)


def ace_workspace_size(layer, max_tokens):
    return int(_lib.ace_workspace_size(ctypes.byref(layer), int(max_tokens)))


def alloc_workspace(nbytes, device="cuda"):
    """A byte tensor usable as workspace (torch allocations are 256-B aligned)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def ace_moe_forward(layer, u, tau, y, ws, renorm=True, eps_rms=1e-6, dbg=None, stream=None,
                    fusion="max"):
    opts = ace_fwd_opts(tau=float(tau), renorm_topk=int(bool(renorm)), fusion=_fusion(fusion),
                        eps_rms=float(eps_rms))
    code = _lib.ace_moe_forward(ctypes.byref(layer), _ptr(u), int(u.shape[0]), ctypes.byref(opts),
                                _ptr(y), _ptr(ws), ws.numel(),
                                ctypes.byref(dbg) if dbg is not None else None, _stream(stream))
    _check(code, "ace_moe_forward")
    return y


def ace_moe_scores(layer, u, score, ws, topk_idx=None, renorm=True, eps_rms=1e-6, stream=None,
                   fusion="max"):
    opts = ace_fwd_opts(tau=0.0, renorm_topk=int(bool(renorm)), fusion=_fusion(fusion),
                        eps_rms=float(eps_rms))
    code = _lib.ace_moe_scores(ctypes.byref(layer), _ptr(u), int(u.shape[0]), ctypes.byref(opts),
                               _ptr(score), _ptr(topk_idx), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "ace_moe_scores")
    return score


def ace_moe_route(layer, u, tau, x, idx, gate, keep, ws, renorm=True, eps_rms=1e-6, stream=None,
                  fusion="max"):
    """Routing with its decisions (see include/ace.h): x [T][d] the experts'
    input rows, idx / gate [T][k], keep [T][k] uint8."""
    opts = ace_fwd_opts(tau=float(tau), renorm_topk=int(bool(renorm)), fusion=_fusion(fusion),
                        eps_rms=float(eps_rms))
    code = _lib.ace_moe_route(ctypes.byref(layer), _ptr(u), int(u.shape[0]), ctypes.byref(opts),
                              _ptr(x), _ptr(idx), _ptr(gate), _ptr(keep), _ptr(ws), ws.numel(),
                              _stream(stream))
    _check(code, "ace_moe_route")
    return x, idx, gate, keep


def make_expert_layer(w_gate, w_up, w_down):
    """An ``ace_layer`` holding only experts (for ace_moe_experts): E, m, d
    from the weight shapes [E][m][d] and [E][d][m]."""
    for t in (w_gate, w_up, w_down):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    E, m, d = w_gate.shape
    return ace_layer(d=d, E=E, m=m, k=1, dtype=_dtype_code(w_gate), gamma=None, w_router=None,
                     router_bias=None, w_gate=_ptr(w_gate), w_up=_ptr(w_up), w_down=_ptr(w_down),
                     amax=None, a_gsp=None, a_rcr=None)


def ace_experts_workspace_size(layer, max_slots):
    return int(_lib.ace_experts_workspace_size(ctypes.byref(layer), int(max_slots)))


def ace_moe_experts(layer, xp, offsets, slot_gate, yslot, ws, stream=None):
    """yslot[s] = slot_gate[s] * f_e(xp[s]) for the slots of expert e,
    offsets[e] <= s < offsets[e + 1] (see include/ace.h); yslot [S][d] in
    xp's dtype."""
    if yslot.dtype != xp.dtype:
        raise ValueError("yslot must have xp's dtype")
    code = _lib.ace_moe_experts(ctypes.byref(layer), _ptr(xp), int(xp.shape[0]), _ptr(offsets),
                                _ptr(slot_gate), _ptr(yslot), _ptr(ws), ws.numel(),
                                _stream(stream))
    _check(code, "ace_moe_experts")
    return yslot


def ace_moe_combine(slot_of, yslot, y, ws, stream=None):
    """y[t] = sum over i of yslot[slot_of[t, i]] for slot_of >= 0, in i order
    (see include/ace.h); slot_of [T][k] int32, yslot [n][d] in y's dtype."""
    if yslot.dtype != y.dtype:
        raise ValueError("yslot must have y's dtype")
    T, k = slot_of.shape
    code = _lib.ace_moe_combine(int(T), int(k), int(y.shape[1]), _dtype_code(y), _ptr(slot_of),
                                _ptr(yslot), int(yslot.shape[0]), _ptr(y), _ptr(ws), ws.numel(),
                                _stream(stream))
    _check(code, "ace_moe_combine")
    return y


# The 8-bit layer's operators are called once per step of a decode loop, where
# the host's time a call counts: their checks read each property of a tensor
# once and pass plain addresses.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda dev: torch.cuda.current_stream(dev).cuda_stream


def current_raw_stream(dev):
    """The current stream of device dev, as its handle."""
    return _raw_stream(dev)


def _refuse(t, name, dev, dtype, shape):
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, is %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, has %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("tensors are on several devices: %s is not on device %d" % (name, dev))


def _arg(t, name, dev, dtype, shape):
    """The address of an optional tensor argument, after its checks: dtype,
    shape, device and C-contiguity."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, dev, dtype, shape)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _fits(name, a, b):
    """Refuses counts beyond the operators' (a C int would take their low bits)."""
    if a > MAX_COUNT or b > MAX_COUNT:
        raise AceError(ACE_ERR_UNSUPPORTED, "%s of %d x %d" % (name, a, b))


def check_arg(t, name, dev, dtype, shape):
    """The checks of an optional tensor argument, for objects that keep tensors
    for later calls."""
    _arg(t, name, dev, dtype, shape)


def _rows(t, name, dev, dtype, shape):
    """(address, row stride) of an optional [rows][n] tensor whose rows may lie
    apart; elements of a row are neighbours."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, dev, dtype, shape)
    rows, n = shape
    _fits(name, rows, n)
    ld, step = t.stride()
    if (n > 1 and step != 1) or (rows > 1 and ld < n):
        raise ValueError("%s must have rows of neighbouring elements" % name)
    return t.data_ptr(), (ld if rows > 1 else n)


def _run(fn, name, dev, stream, *args):
    """fn(*args, stream) with the tensors' device as the current one (the
    library launches on the current device, and the default stream is that
    device's)."""
    if dev < 0:
        raise ValueError("%s: tensors must be on a CUDA device" % name)
    if dev == torch.cuda.current_device():
        code = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if code != ACE_OK:
        raise AceError(code, name)


def ace_add_rmsnorm(x, gamma, residual=None, sum=None, y=None, q=None, q_scale=None, eps=1e-6,
                    stream=None):
    """sum = x + residual, y = RMSNorm(sum) gamma, and its int8 rows q with
    scales q_scale, whichever outputs are given (see include/ace.h).  x,
    residual, sum, y [T][d]; q [T][d] int8; q_scale [T] fp32; rows may be
    strided."""
    if x.dim() != 2:
        raise ValueError("x must be [T][d]")
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    T, d = shape
    code = _dtype_code(x)
    px, ldx = _rows(x, "x", dev, dt, shape)
    pr, ldr = _rows(residual, "residual", dev, dt, shape)
    ps, lds = _rows(sum, "sum", dev, dt, shape)
    py, ldy = _rows(y, "y", dev, dt, shape)
    pq, ldq = _rows(q, "q", dev, torch.int8, shape)
    _run(_lib.ace_add_rmsnorm, "ace_add_rmsnorm", dev, stream, px, ldx, pr, ldr, T, d, code,
         _arg(gamma, "gamma", dev, torch.float32, (d,)), eps, ps, lds, py, ldy, pq, ldq,
         _arg(q_scale, "q_scale", dev, torch.float32, (T,)))


def make_router_layer(gamma, w_router, router_bias=None):
    """An ``ace_layer`` holding only gamma and the router (for
    ace_moe_logits): E, d from w_router [E][d]; gamma [d] and router_bias [E]
    fp32 on the same device.  The caller keeps the tensors alive while the
    struct is in use."""
    if w_router.dim() != 2:
        raise ValueError("w_router must be [E][d]")
    E, d = w_router.shape
    dev = w_router.get_device()
    return ace_layer(d=d, E=E, m=64, k=1, dtype=_dtype_code(w_router),
                     gamma=_arg(gamma, "gamma", dev, torch.float32, (d,)),
                     w_router=_arg(w_router, "w_router", dev, w_router.dtype, (E, d)),
                     router_bias=_arg(router_bias, "router_bias", dev, torch.float32, (E,)))


def ace_logits_workspace_size(layer, max_tokens):
    return int(_lib.ace_logits_workspace_size(layer, int(max_tokens)))


def ace_moe_logits(layer, u, logits, ws, eps_rms=1e-6, stream=None):
    """logits [T][E] fp32 = RMSNorm(u) gamma . w_router (+ bias) (see
    include/ace.h); u [T][d] in the layer's dtype."""
    dev = u.get_device()
    if u.dim() != 2 or u.shape[1] != layer.d or _dtype_code(u) != layer.dtype:
        raise ValueError("u must be [T][%d] in the layer's dtype" % layer.d)
    T = u.shape[0]
    _fits("u", T, 1)
    if ws.get_device() != dev:
        raise ValueError("tensors are on several devices: ws is not on device %d" % dev)
    _run(_lib.ace_moe_logits, "ace_moe_logits", dev, stream, layer,
         _arg(u, "u", dev, u.dtype, u.shape), T, eps_rms,
         _arg(logits, "logits", dev, torch.float32, (T, layer.E)), ws.data_ptr(),
         ws.numel() * ws.element_size())
    return logits


@functools.lru_cache(maxsize=64)
def _gate_opts(score, n_groups, topk_groups, group_score, renorm, scale, tau):
    return ace_gate_opts(SCORES[score], n_groups, topk_groups, GROUP_SCORES[group_score],
                         1 if renorm else 0, scale, tau)


def check_gate(E, k, score="softmax", n_groups=1, topk_groups=1, group_score="max", renorm=True,
               scale=1.0):
    """Refuses options that ace_gate_topk would refuse for k of E experts."""
    opts = _gate_opts(score, int(n_groups), int(topk_groups), group_score, bool(renorm), float(scale), 0.0)
    _check(_lib.ace_gate_topk(None, E, ACE_F32, 0, E, k, None, opts, None, None, None, None, None),
           "ace_gate_topk")


def ace_gate_topk(logits, idx, weight, bias=None, score="softmax", n_groups=1, topk_groups=1,
                  group_score="max", renorm=True, scale=1.0, factor=None, tau=0.0, keep=None,
                  stream=None):
    """Experts idx [T][k] int32 and weights [T][k] fp32 of logits [T][E] (fp32
    or bf16), and the skip mask keep [T][k] uint8 if given (see
    include/ace.h)."""
    if logits.dim() != 2 or idx.dim() != 2:
        raise ValueError("logits must be [T][E] and idx [T][k]")
    T, E = logits.shape
    k, dev = idx.shape[1], logits.get_device()
    _fits("idx", T, k)
    pl, ld = _rows(logits, "logits", dev, logits.dtype, (T, E))
    opts = _gate_opts(score, int(n_groups), int(topk_groups), group_score, bool(renorm), float(scale),
                      float(tau))
    _run(_lib.ace_gate_topk, "ace_gate_topk", dev, stream, pl, ld, _dtype_code(logits), T, E, k,
         _arg(bias, "bias", dev, torch.float32, (E,)), opts,
         _arg(idx, "idx", dev, torch.int32, (T, k)),
         _arg(weight, "weight", dev, torch.float32, (T, k)),
         _arg(factor, "factor", dev, torch.float32, (E,)), _arg(keep, "keep", dev, torch.uint8, (T, k)))
    return idx, weight


def ace_moe_group(idx, E, offsets, slot_of, keep=None, gate=None, slot_token=None, slot_gate=None,
                  stream=None):
    """The kept slots of idx [T][k] in expert order: offsets [E + 1] and
    slot_of [T][k], and slot_token / slot_gate [T * k] if given (see
    include/ace.h)."""
    if idx.dim() != 2:
        raise ValueError("idx must be [T][k]")
    shape, dev = idx.shape, idx.get_device()
    T, k = shape
    _fits("idx", T, k)
    _fits("offsets", E, 1)
    _run(_lib.ace_moe_group, "ace_moe_group", dev, stream, _arg(idx, "idx", dev, torch.int32, shape),
         _arg(keep, "keep", dev, torch.uint8, shape), _arg(gate, "gate", dev, torch.float32, shape), T, k,
         E, _arg(offsets, "offsets", dev, torch.int32, (E + 1,)),
         _arg(slot_of, "slot_of", dev, torch.int32, shape),
         _arg(slot_token, "slot_token", dev, torch.int32, (T * k,)),
         _arg(slot_gate, "slot_gate", dev, torch.float32, (T * k,)))
    return offsets, slot_of


# ace_i8_product's fields in native layout: packing them takes half the time of the
# ctypes structure
_I8_PRODUCT = struct.Struct("@PqiPPPiiiPPP")
assert _I8_PRODUCT.size == ctypes.sizeof(ace_i8_product)


def ace_matmul_i8(xq, x_scale, wq, w_scale, out, ws, offsets=None, row_of=None, slot_scale=None,
                  stream=None):
    """out [S][N] (bf16 or fp32) = scaled int8 product of xq [n][K] with
    wq [N][K], or with wq [E][N][K] by the slots' experts (offsets [E + 1]);
    row_of [S] reads the slots' rows of xq (see include/ace.h)."""
    if xq.dim() != 2 or out.dim() != 2 or wq.dim() not in (2, 3):
        raise ValueError("xq must be [n][K], wq [N][K] or [E][N][K], out [S][N]")
    wshape, dev = wq.shape, xq.get_device()
    E = wshape[0] if len(wshape) == 3 else 1
    if E != 1 and offsets is None:
        raise ValueError("wq of several experts needs offsets")
    N, K = wshape[-2:]
    _fits("wq", E, N)
    n, S = xq.shape[0], out.shape[0]
    px, ldx = _rows(xq, "xq", dev, torch.int8, (n, K))
    po, ldo = _rows(out, "out", dev, out.dtype, (S, N))
    if ws.get_device() != dev:
        raise ValueError("tensors are on several devices: ws is not on device %d" % dev)
    p = _I8_PRODUCT.pack(px, ldx, n, _arg(x_scale, "x_scale", dev, torch.float32, (n,)),
                         _arg(wq, "wq", dev, torch.int8, wshape),
                         _arg(w_scale, "w_scale", dev, torch.float32, wshape[:-1]), E, N, K,
                         _arg(offsets, "offsets", dev, torch.int32, (E + 1,)) or 0,
                         _arg(row_of, "row_of", dev, torch.int32, (S,)) or 0,
                         _arg(slot_scale, "slot_scale", dev, torch.float32, (S,)) or 0)
    _run(_lib.ace_matmul_i8, "ace_matmul_i8", dev, stream, p, S, po, ldo, _dtype_code(out),
         ws.data_ptr(), ws.numel() * ws.element_size())
    return out


def ace_swiglu(gu, y=None, q=None, q_scale=None, n_valid=None, stream=None):
    """h = SiLU(g) u of rows gu [S][2 m] = [g | u]: y [S][m] and / or its int8
    rows q [S][m] with scales q_scale [S]; rows from n_valid[0] on (int32,
    device) are left alone (see include/ace.h)."""
    if gu.dim() != 2 or gu.shape[1] % 2:
        raise ValueError("gu must be [S][2 m]")
    shape, dt, dev = gu.shape, gu.dtype, gu.get_device()
    S, m = shape[0], shape[1] // 2
    pgu, ldgu = _rows(gu, "gu", dev, dt, shape)
    py, ldy = _rows(y, "y", dev, dt, (S, m))
    pq, ldq = _rows(q, "q", dev, torch.int8, (S, m))
    _run(_lib.ace_swiglu, "ace_swiglu", dev, stream, pgu, ldgu, S, m, _dtype_code(gu),
         _arg(n_valid, "n_valid", dev, torch.int32, (1,)), py, ldy, pq, ldq,
         _arg(q_scale, "q_scale", dev, torch.float32, (S,)))


def _host_f32(t):
    return t.detach().to("cpu", torch.float32).contiguous()


def ace_tables_save(path, a_gsp, a_rcr, amax, sigma=None):
    """Write ace_build_tables's outputs ([L][E] each, sigma [L][E][3] or None;
    any device) to a tables file (see include/ace.h)."""
    g, r, mx = (_host_f32(t).reshape(-1, a_gsp.shape[-1]) for t in (a_gsp, a_rcr, amax))
    L, E = g.shape
    sg = None if sigma is None else _host_f32(sigma)
    code = _lib.ace_tables_save(os.fsencode(path), L, E, _ptr(g), _ptr(r), _ptr(mx), _ptr(sg))
    _check(code, "ace_tables_save")


def ace_tables_info(path):
    """(n_layers, E, has_sigma) of a tables file."""
    L, E, hs = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    code = _lib.ace_tables_info(os.fsencode(path), ctypes.byref(L), ctypes.byref(E),
                                ctypes.byref(hs))
    _check(code, "ace_tables_info")
    return L.value, E.value, bool(hs.value)


def ace_tables_load(path, device="cpu", with_sigma=False):
    """(a_gsp, a_rcr, amax[, sigma]) from a tables file, fp32 on `device`."""
    L, E, hs = ace_tables_info(path)
    g, r, mx = (torch.empty(L, E, dtype=torch.float32) for _ in range(3))
    sg = torch.empty(L, E, 3, dtype=torch.float32) if with_sigma else None
    code = _lib.ace_tables_load(os.fsencode(path), L, E, _ptr(g), _ptr(r), _ptr(mx), _ptr(sg))
    _check(code, "ace_tables_load")
    out = tuple(t.to(device) for t in (g, r, mx))
    return out + ((sg.to(device),) if with_sigma else ())


def ace_moe_decode_noalloc(layer, u, tau, y, renorm=True, eps_rms=1e-6, stream=None,
                           fusion="max"):
    """Decode forward (1-8 tokens) with the library's fixed scratch array
    instead of a caller workspace; see include/ace.h."""
    opts = ace_fwd_opts(tau=float(tau), renorm_topk=int(bool(renorm)), fusion=_fusion(fusion),
                        eps_rms=float(eps_rms))
    code = _lib.ace_moe_decode_noalloc(ctypes.byref(layer), _ptr(u), int(u.shape[0]),
                                       ctypes.byref(opts), _ptr(y), _stream(stream))
    _check(code, "ace_moe_decode_noalloc")
    return y


def ace_stack_workspace_size(layers, max_tokens):
    arr = (ace_layer * len(layers))(*layers)
    return int(_lib.ace_stack_workspace_size(arr, len(layers), int(max_tokens)))


def ace_moe_stack_forward(layers, u, taus, y, ws, renorm=True, eps_rms=1e-6, stream=None,
                          fusion="max"):
    """len(layers) layers in sequence, each output the next input; taus[l]
    is layer l's threshold.  See include/ace.h."""
    n = len(layers)
    arr = (ace_layer * n)(*layers)
    opts = (ace_fwd_opts * n)(*[ace_fwd_opts(tau=float(t), renorm_topk=int(bool(renorm)),
                                             fusion=_fusion(fusion), eps_rms=float(eps_rms))
                                for t in taus])
    code = _lib.ace_moe_stack_forward(arr, n, _ptr(u), int(u.shape[0]), opts, _ptr(y), _ptr(ws),
                                      ws.numel(), _stream(stream))
    _check(code, "ace_moe_stack_forward")
    return y


def ace_tables_workspace_size(layer):
    return int(_lib.ace_tables_workspace_size(ctypes.byref(layer)))


def ace_build_tables(layers, a_gsp, a_rcr, amax, ws, sigma=None, gsp_norm=ACE_GSP_FRO, eps=1e-6,
                     rho=1.0, power_iters=200, stream=None):
    arr = (ace_layer * len(layers))(*layers)
    opts = ace_table_opts(gsp_norm=gsp_norm, eps=float(eps), rho=float(rho),
                          power_iters=int(power_iters))
    code = _lib.ace_build_tables(arr, len(layers), ctypes.byref(opts), _ptr(a_gsp), _ptr(a_rcr),
                                 _ptr(amax), _ptr(sigma), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "ace_build_tables")


def ace_tau_workspace_size():
    return int(_lib.ace_tau_workspace_size())


def ace_tau_quantile(score, n_skip, tau, ws, stream=None):
    """tau[0] = the (n_skip + 1)-th smallest non-top-1 score of the pool
    score [n_tok][k] (device fp32); see include/ace.h."""
    n_tok, k = score.shape
    code = _lib.ace_tau_quantile(_ptr(score), int(n_tok), int(k), int(n_skip), _ptr(tau),
                                 _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "ace_tau_quantile")
    return tau


def ace_read_status(ws, stream=None):
    """Synchronise the stream; return (status code, flag bits)."""
    flags = ctypes.c_uint32(0)
    code = _lib.ace_read_status(_ptr(ws), ws.numel(), ctypes.byref(flags), _stream(stream))
    return code, int(flags.value)


def ace_noalloc_read_status(stream=None):
    """Synchronise the stream; (status code, flag bits) of the last
    ace_moe_decode_noalloc call on the current device."""
    flags = ctypes.c_uint32(0)
    code = _lib.ace_noalloc_read_status(ctypes.byref(flags), _stream(stream))
    return code, int(flags.value)


def ace_set_peer_wait_limit_ns(ns):
    """Set the limit of cross-CTA waits (0: the 2 s default); returns the
    previous limit."""
    return int(_lib.ace_set_peer_wait_limit_ns(int(ns)))


class DebugOut:
    """Device buffers for the forward's intermediates, and the C struct that
    points at them."""

    def __init__(self, T, k, E, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.topk_idx = torch.empty(T, k, **i32)
        self.gate = torch.empty(T, k, **f32)
        self.score = torch.empty(T, k, **f32)
        self.keep = torch.empty(T, k, dtype=torch.uint8, device=device)
        self.expert_offsets = torch.empty(E + 1, **i32)
        self.slot_token = torch.empty(max(T * k, 1), **i32)
        self.slot_rank = torch.empty(max(T * k, 1), **i32)
        self.n_kept = torch.empty(1, **i32)
        self.logits = torch.empty(T, E, **f32)
        self.c = ace_debug_out(**{f: _ptr(getattr(self, f)) for f, _ in ace_debug_out._fields_
                                  if not f.startswith("ev_") and f != "trace"})


def event_handle(ev):
    """The cudaEvent_t behind a torch.cuda.Event, as a void* for the C ABI
    (torch creates the CUDA event at its first record, so record it once)."""
    if not ev.cuda_event:
        ev.record()
    return ctypes.c_void_p(ev.cuda_event)


def timing_debug(ev_begin, ev_mid, ev_end):
    """An ace_debug_out that only records the expert-GEMM timing events."""
    return ace_debug_out(ev_experts_begin=event_handle(ev_begin),
                         ev_experts_mid=event_handle(ev_mid),
                         ev_experts_end=event_handle(ev_end))
