"""Python binding of libssmscan (ctypes).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, and their device pointers are passed to the C ABI together with
the current HIP stream.  Every step of the computation runs in the library's
HIP kernels; there is no fallback.  If ``libssmscan.so`` has not been built
the import fails with an explanation.

Functions mirror the C entry points:

    scan_fwd(x, delta, A, B, C, D, h_init=None, y=None, h_final=None)
        -> (y, h_final)
    step(x, delta, A, B, C, D, h, y=None) -> y       (h is updated in place)
    scan_gated_fwd, scan_gated_bwd, step_gated       the gated linear recurrence
    layer_norm_fwd, layer_norm_bwd                   layer norm, by rows or heads
    linear_attn_fwd, linear_attn_bwd, step_linear_attn
                                                     linear attention with a decay per head
    qk_norm_rope_fwd, qk_norm_rope_bwd               norm and rotation of queries and keys
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# SSMSCAN_LIB selects another build of the same library (the sanitizer build
# of the host code, for example); by default the in-tree one.
LIB_PATH = os.environ.get("SSMSCAN_LIB") or os.path.join(_HERE, "libssmscan.so")

SSM_F32, SSM_BF16 = 0, 1
SSM_OPT_SEGMENT_LEN, SSM_OPT_FORCE_GENERAL, SSM_OPT_PROFILE, SSM_OPT_STEP_CHANNELS = 1, 2, 3, 4
SSM_DELTA_SOFTPLUS, SSM_EULER_B = 1, 2  # ssm_flags
SSM_ROPE_INTERLEAVED = 1  # ssm_rope_flags
KERNEL_KINDS = ("bc_prep", "scan_aggregate", "scan_carry", "scan_output", "step", "state_init",
                "bwd_aggregate", "bwd_carry", "bwd_main", "bwd_reduce", "ssd_aggregate", "ssd_carry",
                "ssd_output", "gated_fwd", "gated_bwd", "gated_reduce", "norm_fwd", "norm_bwd", "norm_reduce",
                "lin_aggregate", "lin_carry", "lin_output", "lin_reduce", "rope_fwd", "rope_bwd", "rope_reduce")
STATUS = {0: "SSM_OK", 1: "SSM_ERR_NULLPTR", 2: "SSM_ERR_BAD_DIM", 3: "SSM_ERR_BAD_DTYPE",
          4: "SSM_ERR_UNSUPPORTED_N", 5: "SSM_ERR_ALIGN", 6: "SSM_ERR_ALIAS", 7: "SSM_ERR_NOMEM",
          8: "SSM_ERR_HIP", 9: "SSM_ERR_BAD_OPTION", 10: "SSM_ERR_CAPTURE"}

# Every symbol include/ssmscan.h declares.
EXPORTS = ("ssm_scan_fwd", "ssm_scan_fwd_ex", "ssm_step", "ssm_step_ex", "ssm_strerror",
           "ssm_last_error", "ssm_version", "ssm_set_option", "ssm_get_option",
           "ssm_scan_plan", "ssm_release_workspaces", "ssm_profile_read", "ssm_scan_varlen_fwd",
           "ssm_scan_fused_fwd", "ssm_step_fused", "ssm_scan_bwd", "ssm_scan_complex_fwd",
           "ssm_step_complex", "ssm_scan_ssd_fwd", "ssm_scan_bwd_plan", "ssm_probe_issue",
           "ssm_scan_fwd_noalloc", "ssm_probe_hbm", "ssm_scan_varlen_bwd",
           "ssm_scan_complex_bwd", "ssm_scan_gated_fwd", "ssm_scan_gated_bwd", "ssm_step_gated",
           "ssm_gated_carry_steps", "ssm_layer_norm_fwd", "ssm_layer_norm_bwd",
           "ssm_linear_attn_fwd", "ssm_linear_attn_bwd", "ssm_step_linear_attn", "ssm_qk_norm_rope_fwd",
           "ssm_qk_norm_rope_bwd")


class SSMError(RuntimeError):
    def __init__(self, code, where, detail):
        self.code = code
        super().__init__(f"{where} failed: {STATUS.get(code, code)}: {detail}")


_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_lib = None


def lib():
    """The loaded libssmscan (raises ImportError if it was never built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m selective_state_space_18_amd.build` (needs ROCm hipcc)")
    L = ctypes.CDLL(LIB_PATH)
    L.ssm_scan_fwd.argtypes = [_vp] * 8 + [_i64] * 4 + [ctypes.c_int, _vp]
    L.ssm_scan_fwd_ex.argtypes = [_vp] * 9 + [_i64] * 4 + [ctypes.c_int, _vp]
    L.ssm_scan_fwd_noalloc.argtypes = [_vp] * 9 + [_i64] * 4 + [ctypes.c_int, _vp]
    L.ssm_scan_varlen_fwd.argtypes = [_vp] * 7 + [_i64] + [_vp] * 3 + [_i64] * 3 + [ctypes.c_int, _vp]
    L.ssm_scan_varlen_fwd.restype = ctypes.c_int
    L.ssm_scan_fused_fwd.argtypes = [_vp] * 8 + [_i64] + [_vp] * 3 + [_i64] * 4 + [ctypes.c_int, ctypes.c_uint, _vp]
    L.ssm_scan_fused_fwd.restype = ctypes.c_int
    L.ssm_scan_complex_fwd.argtypes = [_vp] * 10 + [_i64] * 4 + [ctypes.c_int, ctypes.c_uint, _vp]
    L.ssm_scan_complex_fwd.restype = ctypes.c_int
    L.ssm_scan_ssd_fwd.argtypes = [_vp] * 10 + [_i64] * 5 + [ctypes.c_int, ctypes.c_uint, _vp]
    L.ssm_scan_ssd_fwd.restype = ctypes.c_int
    L.ssm_step_complex.argtypes = [_vp] * 9 + [_i64] * 3 + [ctypes.c_int, ctypes.c_uint, _vp]
    L.ssm_step_complex.restype = ctypes.c_int
    L.ssm_scan_bwd.argtypes = [_vp] * 18 + [_i64] * 4 + [ctypes.c_int, ctypes.c_uint, _vp]
    L.ssm_scan_bwd.restype = ctypes.c_int
    L.ssm_scan_varlen_bwd.argtypes = [_vp] * 8 + [_i64] + [_vp] * 11 + [_i64] * 3 + [ctypes.c_int, ctypes.c_uint,
                                                                                    _vp]
    L.ssm_scan_varlen_bwd.restype = ctypes.c_int
    L.ssm_scan_complex_bwd.argtypes = [_vp] * 18 + [_i64] * 4 + [ctypes.c_int, ctypes.c_uint, _vp]
    L.ssm_scan_complex_bwd.restype = ctypes.c_int
    L.ssm_step_fused.argtypes = [_vp] * 9 + [_i64] * 3 + [ctypes.c_int, ctypes.c_uint, _vp]
    L.ssm_step_fused.restype = ctypes.c_int
    L.ssm_step.argtypes = [_vp] * 8 + [_i64] * 3 + [_vp]
    L.ssm_step_ex.argtypes = [_vp] * 8 + [_i64] * 3 + [ctypes.c_int, _vp]
    for f in ("ssm_scan_fwd", "ssm_scan_fwd_ex", "ssm_scan_fwd_noalloc", "ssm_step", "ssm_step_ex"):
        getattr(L, f).restype = ctypes.c_int
    L.ssm_scan_gated_fwd.argtypes = [_vp] * 5 + [_i64] + [_vp] * 4 + [_i64] * 3 + [ctypes.c_int, _vp]
    L.ssm_scan_gated_bwd.argtypes = [_vp] * 5 + [_i64] + [_vp] * 9 + [_i64] * 3 + [ctypes.c_int, _vp]
    L.ssm_step_gated.argtypes = [_vp] * 7 + [_i64] * 2 + [ctypes.c_int, _vp]
    L.ssm_gated_carry_steps.argtypes = []
    L.ssm_gated_carry_steps.restype = _i64
    L.ssm_layer_norm_fwd.argtypes = [_vp] * 8 + [_i64] * 3 + [ctypes.c_float, ctypes.c_int, _vp]
    L.ssm_layer_norm_bwd.argtypes = [_vp] * 9 + [_i64] * 3 + [ctypes.c_int, _vp]
    L.ssm_linear_attn_fwd.argtypes = [_vp] * 5 + [_i64] + [_vp] * 3 + [_i64] * 6 + [ctypes.c_float, ctypes.c_int, _vp]
    L.ssm_linear_attn_bwd.argtypes = [_vp] * 5 + [_i64] + [_vp] * 7 + [_i64] * 6 + [ctypes.c_float, ctypes.c_int, _vp]
    L.ssm_step_linear_attn.argtypes = [_vp] * 7 + [_i64] * 5 + [ctypes.c_float, ctypes.c_int, _vp]
    L.ssm_qk_norm_rope_fwd.argtypes = [_vp] * 8 + [_i64] * 5 + [ctypes.c_float, ctypes.c_uint, ctypes.c_int, _vp]
    L.ssm_qk_norm_rope_bwd.argtypes = [_vp] * 12 + [_i64] * 5 + [ctypes.c_float, ctypes.c_uint, ctypes.c_int, _vp]
    for f in ("ssm_scan_gated_fwd", "ssm_scan_gated_bwd", "ssm_step_gated", "ssm_layer_norm_fwd",
              "ssm_layer_norm_bwd", "ssm_linear_attn_fwd", "ssm_linear_attn_bwd", "ssm_step_linear_attn",
              "ssm_qk_norm_rope_fwd", "ssm_qk_norm_rope_bwd"):
        getattr(L, f).restype = ctypes.c_int
    L.ssm_strerror.argtypes = [ctypes.c_int]
    L.ssm_strerror.restype = ctypes.c_char_p
    L.ssm_last_error.argtypes = []
    L.ssm_last_error.restype = ctypes.c_char_p
    L.ssm_version.argtypes = []
    L.ssm_version.restype = ctypes.c_int
    L.ssm_set_option.argtypes = [ctypes.c_int, _i64]
    L.ssm_set_option.restype = ctypes.c_int
    L.ssm_get_option.argtypes = [ctypes.c_int]
    L.ssm_get_option.restype = _i64
    L.ssm_scan_plan.argtypes = [_i64] * 4 + [ctypes.c_int, ctypes.c_int,
                                             ctypes.POINTER(_i64), ctypes.POINTER(_i64)]
    L.ssm_scan_plan.restype = ctypes.c_int
    L.ssm_scan_bwd_plan.argtypes = [_i64] * 4 + [ctypes.c_int, ctypes.c_int] + [ctypes.POINTER(_i64)] * 4
    L.ssm_scan_bwd_plan.restype = ctypes.c_int
    L.ssm_probe_issue.argtypes = [ctypes.c_int, _i64, _i64, _vp, _vp, ctypes.POINTER(_i64), ctypes.POINTER(_i64)]
    L.ssm_probe_issue.restype = ctypes.c_int
    L.ssm_probe_hbm.argtypes = [ctypes.c_int, _vp, _i64, _vp]
    L.ssm_probe_hbm.restype = ctypes.c_int
    L.ssm_release_workspaces.argtypes = []
    L.ssm_release_workspaces.restype = ctypes.c_int
    L.ssm_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i64), ctypes.c_int]
    L.ssm_profile_read.restype = ctypes.c_int
    _lib = L
    return L


def _check(rc, where):
    if rc != 0:
        detail = lib().ssm_last_error().decode(errors="replace")
        raise SSMError(rc, where, detail)


def last_error() -> str:
    return lib().ssm_last_error().decode(errors="replace")


def version() -> int:
    return lib().ssm_version()


def set_option(option: int, value: int) -> None:
    _check(lib().ssm_set_option(int(option), int(value)), "ssm_set_option")


def get_option(option: int) -> int:
    return int(lib().ssm_get_option(int(option)))


def plan(Bsz, L, Dm, N, dtype=SSM_BF16, compute_units=0):
    """(segments, segment_len) the scan would use."""
    s, sl = _i64(), _i64()
    _check(lib().ssm_scan_plan(Bsz, L, Dm, N, dtype, compute_units, ctypes.byref(s), ctypes.byref(sl)),
           "ssm_scan_plan")
    return s.value, sl.value


def bwd_plan(Bsz, L, Dm, N, dtype=SSM_BF16, compute_units=0):
    """(segments, segment_len, seg_per_group, groups) the backward would use."""
    out = [_i64() for _ in range(4)]
    _check(lib().ssm_scan_bwd_plan(Bsz, L, Dm, N, dtype, compute_units, *(ctypes.byref(v) for v in out)),
           "ssm_scan_bwd_plan")
    return tuple(v.value for v in out)


PROBE_KINDS = ("fma_f32", "exp_f32", "fma_exp_f32", "fma_f64", "empty", "fmac_f32", "mul_f32", "add_f32",
               "fma_f32_vgpr", "scan_step_mix")
HBM_PROBES = {"read": 16, "rmw": 17, "write": 18}


def probe_issue(kind: str, blocks: int, iters: int, sink: torch.Tensor):
    """Launch an issue-rate probe on the current stream (the caller times it).
    Returns (VALU instructions per iteration, transcendental ones) per lane."""
    if sink.device.type != "cuda" or sink.dtype != torch.float32 or sink.numel() < blocks * 256:
        raise ValueError("sink must be a CUDA float32 tensor of at least blocks * 256 elements")
    v, t = _i64(), _i64()
    _check(lib().ssm_probe_issue(PROBE_KINDS.index(kind), blocks, iters, _ptr(sink), _stream(sink.device),
                                 ctypes.byref(v), ctypes.byref(t)), "ssm_probe_issue")
    return v.value, t.value


def probe_hbm(kind: str, buf: torch.Tensor) -> int:
    """Launch a streaming memory probe over buf on the current stream (the
    caller times it); returns the bytes it moves."""
    if buf.device.type != "cuda" or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous CUDA tensor")
    nbytes = buf.numel() * buf.element_size()
    _check(lib().ssm_probe_hbm(HBM_PROBES[kind], _ptr(buf), nbytes, _stream(buf.device)), "ssm_probe_hbm")
    return 2 * nbytes if kind == "rmw" else nbytes


def profile_read():
    """{kernel kind: (total ms, launches)} since the last read (SSM_OPT_PROFILE)."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (_i64 * n)()
    _check(lib().ssm_profile_read(ms, cnt, n), "ssm_profile_read")
    return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_KINDS)}


def release_workspaces() -> None:
    _check(lib().ssm_release_workspaces(), "ssm_release_workspaces")


_DT = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
    return _DT[t.dtype]


def _need(t, name, shape, dtype, device):
    # one expression for the usual case: a decode step makes seven of these
    # checks, and each attribute of a tensor costs about 0.1 us
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype and t.device == device
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    # the handle alone: building a torch.cuda.Stream around it takes 1.8 us
    return torch._C._cuda_getCurrentRawStream(device.index)


def _launch(entry, device, *args):
    """Call a C entry point on `device`'s current stream (its last argument)."""
    f = getattr(lib(), entry)
    if torch.cuda.current_device() == device.index:  # entering a device costs more than asking for it
        rc = f(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            rc = f(*args, _stream(device))
    _check(rc, entry)


def _flags(delta_softplus, euler_b):
    return (SSM_DELTA_SOFTPLUS if delta_softplus else 0) | (SSM_EULER_B if euler_b else 0)


def _bias(delta_bias, Dm, dev):
    if delta_bias is not None:
        _need(delta_bias, "delta_bias", (Dm,), torch.float32, dev)
    return delta_bias


def scan_fwd(x, delta, A, B, C, D, h_init=None, y=None, h_final=None, want_state=True,
             delta_bias=None, delta_softplus=False, euler_b=False):
    """Selective scan over [Bsz, L, Dm] with state size N = A.shape[1].

    x, delta: [Bsz, L, Dm]; B, C: [Bsz, L, N] (all the same dtype, fp32 or bf16);
    A: [Dm, N] fp32; D: [Dm] fp32; h_init: optional [Bsz, Dm, N] fp32.
    Options: delta_bias [Dm] fp32 is added to delta, delta_softplus applies
    softplus to the sum, euler_b uses the input term delta*B.
    Returns (y [Bsz, L, Dm] in x's dtype, h_final [Bsz, Dm, N] fp32 or None).
    """
    if delta_bias is not None or delta_softplus or euler_b:
        return scan_fused_fwd(x, delta, A, B, C, D, h_init=h_init, y=y, h_final=h_final,
                              want_state=want_state, delta_bias=delta_bias,
                              delta_softplus=delta_softplus, euler_b=euler_b)
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    Bsz, L, Dm = x.shape
    N = A.shape[1]
    dt = x.dtype
    code = _dtype_code(x)
    _need(x, "x", (Bsz, L, Dm), dt, dev)
    _need(delta, "delta", (Bsz, L, Dm), dt, dev)
    _need(A, "A", (Dm, N), torch.float32, dev)
    _need(B, "B", (Bsz, L, N), dt, dev)
    _need(C, "C", (Bsz, L, N), dt, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    if h_init is not None:
        _need(h_init, "h_init", (Bsz, Dm, N), torch.float32, dev)
    if y is None:
        y = torch.empty((Bsz, L, Dm), dtype=dt, device=dev)
    _need(y, "y", (Bsz, L, Dm), dt, dev)
    if h_final is None and want_state:
        h_final = torch.empty((Bsz, Dm, N), dtype=torch.float32, device=dev)
    if h_final is not None:
        _need(h_final, "h_final", (Bsz, Dm, N), torch.float32, dev)
    with torch.cuda.device(dev):
        if h_init is None:
            rc = lib().ssm_scan_fwd(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                    _ptr(y), _ptr(h_final), Bsz, L, Dm, N, code, _stream(dev))
        else:
            rc = lib().ssm_scan_fwd_ex(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                       _ptr(h_init), _ptr(y), _ptr(h_final), Bsz, L, Dm, N, code,
                                       _stream(dev))
    _check(rc, "ssm_scan_fwd")
    return y, h_final


def scan_fwd_noalloc(x, delta, A, B, C, D, h_init=None, y=None, h_final=None):
    """ssm_scan_fwd_noalloc: the scan of scan_fwd (no options) on the library's
    fixed 64 MiB device array instead of allocated scratch.  The C call
    allocates nothing; pass y and h_final to keep this wrapper from
    allocating them.  Returns (y, h_final)."""
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    Bsz, L, Dm = x.shape
    N = A.shape[1]
    dt = x.dtype
    code = _dtype_code(x)
    _need(x, "x", (Bsz, L, Dm), dt, dev)
    _need(delta, "delta", (Bsz, L, Dm), dt, dev)
    _need(A, "A", (Dm, N), torch.float32, dev)
    _need(B, "B", (Bsz, L, N), dt, dev)
    _need(C, "C", (Bsz, L, N), dt, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    if h_init is not None:
        _need(h_init, "h_init", (Bsz, Dm, N), torch.float32, dev)
    if y is None:
        y = torch.empty((Bsz, L, Dm), dtype=dt, device=dev)
    _need(y, "y", (Bsz, L, Dm), dt, dev)
    if h_final is None:
        h_final = torch.empty((Bsz, Dm, N), dtype=torch.float32, device=dev)
    _need(h_final, "h_final", (Bsz, Dm, N), torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_scan_fwd_noalloc(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(h_init),
                                        _ptr(y), _ptr(h_final), Bsz, L, Dm, N, code, _stream(dev))
    _check(rc, "ssm_scan_fwd_noalloc")
    return y, h_final


def scan_varlen_fwd(x, delta, A, B, C, D, cu_seqlens, h_init=None, y=None, h_final=None, want_state=True,
                    delta_bias=None, delta_softplus=False, euler_b=False):
    """Packed variable-length scan: sequences concatenated along time.

    x, delta: [L, Dm]; B, C: [L, N] (same dtype); A: [Dm, N] fp32; D: [Dm] fp32;
    cu_seqlens: [nseq+1] int64 device tensor of sequence start offsets
    (cu_seqlens[0] = 0, cu_seqlens[-1] = L); h_init: optional [nseq, Dm, N] fp32.
    Options as in scan_fwd.
    Returns (y [L, Dm], h_final [nseq, Dm, N] fp32 or None).
    """
    if delta_bias is not None or delta_softplus or euler_b:
        return scan_fused_fwd(x, delta, A, B, C, D, cu_seqlens=cu_seqlens, h_init=h_init, y=y,
                              h_final=h_final, want_state=want_state, delta_bias=delta_bias,
                              delta_softplus=delta_softplus, euler_b=euler_b)
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    L, Dm = x.shape
    N = A.shape[1]
    nseq = cu_seqlens.shape[0] - 1
    dt = x.dtype
    code = _dtype_code(x)
    _need(x, "x", (L, Dm), dt, dev)
    _need(delta, "delta", (L, Dm), dt, dev)
    _need(A, "A", (Dm, N), torch.float32, dev)
    _need(B, "B", (L, N), dt, dev)
    _need(C, "C", (L, N), dt, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", (nseq + 1,), torch.int64, dev)
    if h_init is not None:
        _need(h_init, "h_init", (nseq, Dm, N), torch.float32, dev)
    if y is None:
        y = torch.empty((L, Dm), dtype=dt, device=dev)
    _need(y, "y", (L, Dm), dt, dev)
    if h_final is None and want_state:
        h_final = torch.empty((nseq, Dm, N), dtype=torch.float32, device=dev)
    if h_final is not None:
        _need(h_final, "h_final", (nseq, Dm, N), torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_scan_varlen_fwd(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                       _ptr(cu_seqlens), nseq, _ptr(h_init), _ptr(y), _ptr(h_final),
                                       L, Dm, N, code, _stream(dev))
    _check(rc, "ssm_scan_varlen_fwd")
    return y, h_final


def scan_fused_fwd(x, delta, A, B, C, D, cu_seqlens=None, h_init=None, y=None, h_final=None,
                   want_state=True, delta_bias=None, delta_softplus=False, euler_b=False):
    """ssm_scan_fused_fwd: the scan with every option.

    cu_seqlens None: dense batch, shapes as in scan_fwd.  Otherwise packed
    sequences, shapes as in scan_varlen_fwd.  Returns (y, h_final).
    """
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    N = A.shape[1]
    dt = x.dtype
    code = _dtype_code(x)
    if cu_seqlens is None:
        Bsz, L, Dm = x.shape
        nseq, rows, sdim = 0, (Bsz, L), Bsz
    else:
        L, Dm = x.shape
        Bsz = 1
        nseq = cu_seqlens.shape[0] - 1
        rows, sdim = (L,), nseq
        _need(cu_seqlens, "cu_seqlens", (nseq + 1,), torch.int64, dev)
    _need(x, "x", (*rows, Dm), dt, dev)
    _need(delta, "delta", (*rows, Dm), dt, dev)
    _need(A, "A", (Dm, N), torch.float32, dev)
    _need(B, "B", (*rows, N), dt, dev)
    _need(C, "C", (*rows, N), dt, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    _bias(delta_bias, Dm, dev)
    if h_init is not None:
        _need(h_init, "h_init", (sdim, Dm, N), torch.float32, dev)
    if y is None:
        y = torch.empty((*rows, Dm), dtype=dt, device=dev)
    _need(y, "y", (*rows, Dm), dt, dev)
    if h_final is None and want_state:
        h_final = torch.empty((sdim, Dm, N), dtype=torch.float32, device=dev)
    if h_final is not None:
        _need(h_final, "h_final", (sdim, Dm, N), torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_scan_fused_fwd(_ptr(x), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C),
                                      _ptr(D), _ptr(cu_seqlens), nseq, _ptr(h_init), _ptr(y), _ptr(h_final),
                                      Bsz, L, Dm, N, code, _flags(delta_softplus, euler_b), _stream(dev))
    _check(rc, "ssm_scan_fused_fwd")
    return y, h_final


def scan_bwd(x, delta, A, B, C, D, dy, h_init=None, dh_final=None, delta_bias=None, delta_softplus=False,
             euler_b=False, want_dh_init=True, out=None):
    """ssm_scan_bwd: gradients of the scan (dense batch).

    Forward inputs as in scan_fwd (with the same options), dy [Bsz, L, Dm] in
    x's dtype and optional dh_final [Bsz, Dm, N] fp32.  Returns a dict with dx,
    ddelta (x's dtype), dA [Dm, N], dB, dC [Bsz, L, N], dD [Dm] (fp32),
    dh_init [Bsz, Dm, N] (if want_dh_init) and ddelta_bias [Dm] (if
    delta_bias is given).  `out` may supply any of these tensors.
    """
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    Bsz, L, Dm = x.shape
    N = A.shape[1]
    dt = x.dtype
    code = _dtype_code(x)
    for t, name, shape, tdt in ((x, "x", (Bsz, L, Dm), dt), (delta, "delta", (Bsz, L, Dm), dt),
                                (A, "A", (Dm, N), torch.float32), (B, "B", (Bsz, L, N), dt),
                                (C, "C", (Bsz, L, N), dt), (D, "D", (Dm,), torch.float32),
                                (dy, "dy", (Bsz, L, Dm), dt)):
        _need(t, name, shape, tdt, dev)
    _bias(delta_bias, Dm, dev)
    if h_init is not None:
        _need(h_init, "h_init", (Bsz, Dm, N), torch.float32, dev)
    if dh_final is not None:
        _need(dh_final, "dh_final", (Bsz, Dm, N), torch.float32, dev)
    o = dict(out or {})
    shapes = {"dx": ((Bsz, L, Dm), dt), "ddelta": ((Bsz, L, Dm), dt), "dA": ((Dm, N), torch.float32),
              "dB": ((Bsz, L, N), torch.float32), "dC": ((Bsz, L, N), torch.float32), "dD": ((Dm,), torch.float32)}
    if want_dh_init:
        shapes["dh_init"] = ((Bsz, Dm, N), torch.float32)
    if delta_bias is not None:
        shapes["ddelta_bias"] = ((Dm,), torch.float32)
    for k, (shape, tdt) in shapes.items():
        if o.get(k) is None:
            o[k] = torch.empty(shape, dtype=tdt, device=dev)
        _need(o[k], k, shape, tdt, dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_scan_bwd(_ptr(x), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                _ptr(h_init), _ptr(dy), _ptr(dh_final), _ptr(o["dx"]), _ptr(o["ddelta"]),
                                _ptr(o.get("ddelta_bias")), _ptr(o["dA"]), _ptr(o["dB"]), _ptr(o["dC"]),
                                _ptr(o["dD"]), _ptr(o.get("dh_init")), Bsz, L, Dm, N, code,
                                _flags(delta_softplus, euler_b), _stream(dev))
    _check(rc, "ssm_scan_bwd")
    return o


def scan_varlen_bwd(x, delta, A, B, C, D, cu_seqlens, dy, h_init=None, dh_final=None, delta_bias=None,
                    delta_softplus=False, euler_b=False, want_dh_init=True, out=None):
    """ssm_scan_varlen_bwd: gradients of the packed variable-length scan.

    Forward inputs as in scan_varlen_fwd (x, delta [L, Dm]; B, C [L, N];
    cu_seqlens [nseq+1] int64; h_init [nseq, Dm, N] or None; same options),
    dy [L, Dm] in x's dtype and optional dh_final [nseq, Dm, N] fp32.  Returns
    a dict with dx, ddelta [L, Dm] (x's dtype), dA [Dm, N], dB, dC [L, N], dD
    [Dm] (fp32), dh_init [nseq, Dm, N] (if want_dh_init) and ddelta_bias [Dm]
    (if delta_bias is given).  `out` may supply any of these tensors.
    """
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    L, Dm = x.shape
    N = A.shape[1]
    nseq = cu_seqlens.shape[0] - 1
    dt = x.dtype
    code = _dtype_code(x)
    for t, name, shape, tdt in ((x, "x", (L, Dm), dt), (delta, "delta", (L, Dm), dt),
                                (A, "A", (Dm, N), torch.float32), (B, "B", (L, N), dt), (C, "C", (L, N), dt),
                                (D, "D", (Dm,), torch.float32), (cu_seqlens, "cu_seqlens", (nseq + 1,), torch.int64),
                                (dy, "dy", (L, Dm), dt)):
        _need(t, name, shape, tdt, dev)
    _bias(delta_bias, Dm, dev)
    if h_init is not None:
        _need(h_init, "h_init", (nseq, Dm, N), torch.float32, dev)
    if dh_final is not None:
        _need(dh_final, "dh_final", (nseq, Dm, N), torch.float32, dev)
    o = dict(out or {})
    shapes = {"dx": ((L, Dm), dt), "ddelta": ((L, Dm), dt), "dA": ((Dm, N), torch.float32),
              "dB": ((L, N), torch.float32), "dC": ((L, N), torch.float32), "dD": ((Dm,), torch.float32)}
    if want_dh_init:
        shapes["dh_init"] = ((nseq, Dm, N), torch.float32)
    if delta_bias is not None:
        shapes["ddelta_bias"] = ((Dm,), torch.float32)
    for k, (shape, tdt) in shapes.items():
        if o.get(k) is None:
            o[k] = torch.empty(shape, dtype=tdt, device=dev)
        _need(o[k], k, shape, tdt, dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_scan_varlen_bwd(_ptr(x), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                       _ptr(cu_seqlens), nseq, _ptr(h_init), _ptr(dy), _ptr(dh_final),
                                       _ptr(o["dx"]), _ptr(o["ddelta"]), _ptr(o.get("ddelta_bias")), _ptr(o["dA"]),
                                       _ptr(o["dB"]), _ptr(o["dC"]), _ptr(o["dD"]), _ptr(o.get("dh_init")), L, Dm,
                                       N, code, _flags(delta_softplus, euler_b), _stream(dev))
    _check(rc, "ssm_scan_varlen_bwd")
    return o


def _pairs(t, name, shape, dev):
    """A complex64 tensor, or a float32 tensor with a trailing (re, im) axis,
    as the float32 (re, im) view the library takes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype == torch.complex64:
        t = torch.view_as_real(t)
    _need(t, name, (*shape, 2), torch.float32, dev)
    return t


def scan_complex_fwd(x, delta, A, B, C, D, h_init=None, y=None, h_final=None, want_state=True,
                     delta_bias=None, delta_softplus=False, euler_b=False):
    """ssm_scan_complex_fwd: scan with complex diagonal A.

    A: complex64 [Dm, N] (or float32 [Dm, N, 2]); h_init: complex64 [Bsz, Dm, N]
    or None; everything else as scan_fwd.  Returns (y [Bsz, L, Dm] real,
    h_final complex64 [Bsz, Dm, N] or None)."""
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    Bsz, L, Dm = x.shape
    N = A.shape[1]
    dt = x.dtype
    code = _dtype_code(x)
    _need(x, "x", (Bsz, L, Dm), dt, dev)
    _need(delta, "delta", (Bsz, L, Dm), dt, dev)
    A2 = _pairs(A, "A", (Dm, N), dev)
    _need(B, "B", (Bsz, L, N), dt, dev)
    _need(C, "C", (Bsz, L, N), dt, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    _bias(delta_bias, Dm, dev)
    hi2 = None if h_init is None else _pairs(h_init, "h_init", (Bsz, Dm, N), dev)
    if y is None:
        y = torch.empty((Bsz, L, Dm), dtype=dt, device=dev)
    _need(y, "y", (Bsz, L, Dm), dt, dev)
    if h_final is None and want_state:
        h_final = torch.empty((Bsz, Dm, N), dtype=torch.complex64, device=dev)
    hf2 = None if h_final is None else _pairs(h_final, "h_final", (Bsz, Dm, N), dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_scan_complex_fwd(_ptr(x), _ptr(delta), _ptr(delta_bias), _ptr(A2), _ptr(B), _ptr(C),
                                        _ptr(D), _ptr(hi2), _ptr(y), _ptr(hf2), Bsz, L, Dm, N, code,
                                        _flags(delta_softplus, euler_b), _stream(dev))
    _check(rc, "ssm_scan_complex_fwd")
    return y, h_final


def scan_complex_bwd(x, delta, A, B, C, D, dy, h_init=None, dh_final=None, delta_bias=None, delta_softplus=False,
                     euler_b=False, want_dh_init=True, out=None):
    """ssm_scan_complex_bwd: gradients of the complex-A scan.

    Forward inputs as in scan_complex_fwd (A complex64 [Dm, N] or float32
    [Dm, N, 2]; h_init complex64 [Bsz, Dm, N] or None), dy [Bsz, L, Dm] in x's
    dtype and optional dh_final complex64 [Bsz, Dm, N].  Returns a dict with
    dx, ddelta (x's dtype), dA complex64 [Dm, N] (dL/dRe A + i dL/dIm A), dB,
    dC [Bsz, L, N], dD [Dm] (fp32), dh_init complex64 [Bsz, Dm, N] (if
    want_dh_init) and ddelta_bias [Dm] (if delta_bias is given).  `out` may
    supply any of these tensors (the complex ones as complex64 or as float32
    with a trailing (re, im) axis).
    """
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    Bsz, L, Dm = x.shape
    N = A.shape[1]
    dt = x.dtype
    code = _dtype_code(x)
    for t, name, shape, tdt in ((x, "x", (Bsz, L, Dm), dt), (delta, "delta", (Bsz, L, Dm), dt),
                                (B, "B", (Bsz, L, N), dt), (C, "C", (Bsz, L, N), dt),
                                (D, "D", (Dm,), torch.float32), (dy, "dy", (Bsz, L, Dm), dt)):
        _need(t, name, shape, tdt, dev)
    A2 = _pairs(A, "A", (Dm, N), dev)
    _bias(delta_bias, Dm, dev)
    hi2 = None if h_init is None else _pairs(h_init, "h_init", (Bsz, Dm, N), dev)
    dhf2 = None if dh_final is None else _pairs(dh_final, "dh_final", (Bsz, Dm, N), dev)
    o = dict(out or {})
    shapes = {"dx": ((Bsz, L, Dm), dt), "ddelta": ((Bsz, L, Dm), dt), "dB": ((Bsz, L, N), torch.float32),
              "dC": ((Bsz, L, N), torch.float32), "dD": ((Dm,), torch.float32)}
    if delta_bias is not None:
        shapes["ddelta_bias"] = ((Dm,), torch.float32)
    for k, (shape, tdt) in shapes.items():
        if o.get(k) is None:
            o[k] = torch.empty(shape, dtype=tdt, device=dev)
        _need(o[k], k, shape, tdt, dev)
    cplx = {"dA": (Dm, N)}
    if want_dh_init:
        cplx["dh_init"] = (Bsz, Dm, N)
    pairs = {}
    for k, shape in cplx.items():
        if o.get(k) is None:
            o[k] = torch.empty(shape, dtype=torch.complex64, device=dev)
        pairs[k] = _pairs(o[k], k, shape, dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_scan_complex_bwd(_ptr(x), _ptr(delta), _ptr(delta_bias), _ptr(A2), _ptr(B), _ptr(C),
                                        _ptr(D), _ptr(hi2), _ptr(dy), _ptr(dhf2), _ptr(o["dx"]), _ptr(o["ddelta"]),
                                        _ptr(o.get("ddelta_bias")), _ptr(pairs["dA"]), _ptr(o["dB"]),
                                        _ptr(o["dC"]), _ptr(o["dD"]), _ptr(pairs.get("dh_init")), Bsz, L, Dm, N,
                                        code, _flags(delta_softplus, euler_b), _stream(dev))
    _check(rc, "ssm_scan_complex_bwd")
    return o


def scan_ssd_fwd(x, delta, A, B, C, D, head_dim=64, h_init=None, y=None, h_final=None, want_state=True,
                 delta_bias=None, delta_softplus=False, euler_b=False):
    """ssm_scan_ssd_fwd: scan with one scalar decay per head of head_dim channels.

    x: [Bsz, L, Dm]; delta: [Bsz, L, H] (H = Dm / head_dim); B, C: [Bsz, L, N]
    (all the same dtype); A: [H] fp32; D: [Dm] fp32; delta_bias: [H] fp32 or
    None; h_init: optional [Bsz, Dm, N] fp32.  Returns (y [Bsz, L, Dm],
    h_final [Bsz, Dm, N] fp32 or None)."""
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    Bsz, L, Dm = x.shape
    N = B.shape[2]
    P = int(head_dim)
    if P <= 0 or Dm % P:
        raise ValueError(f"Dm = {Dm} is not a multiple of head_dim = {P}")
    H = Dm // P
    dt = x.dtype
    code = _dtype_code(x)
    _need(x, "x", (Bsz, L, Dm), dt, dev)
    _need(delta, "delta", (Bsz, L, H), dt, dev)
    _need(A, "A", (H,), torch.float32, dev)
    _need(B, "B", (Bsz, L, N), dt, dev)
    _need(C, "C", (Bsz, L, N), dt, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    if delta_bias is not None:
        _need(delta_bias, "delta_bias", (H,), torch.float32, dev)
    if h_init is not None:
        _need(h_init, "h_init", (Bsz, Dm, N), torch.float32, dev)
    if y is None:
        y = torch.empty((Bsz, L, Dm), dtype=dt, device=dev)
    _need(y, "y", (Bsz, L, Dm), dt, dev)
    if h_final is None and want_state:
        h_final = torch.empty((Bsz, Dm, N), dtype=torch.float32, device=dev)
    if h_final is not None:
        _need(h_final, "h_final", (Bsz, Dm, N), torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_scan_ssd_fwd(_ptr(x), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                    _ptr(h_init), _ptr(y), _ptr(h_final), Bsz, L, Dm, N, P, code,
                                    _flags(delta_softplus, euler_b), _stream(dev))
    _check(rc, "ssm_scan_ssd_fwd")
    return y, h_final


def step_complex(x, delta, A, B, C, D, h, y=None, delta_bias=None, delta_softplus=False, euler_b=False):
    """ssm_step_complex: one decode step with complex A; h complex64
    [Bsz, Dm, N] (or float32 [..., 2]) is updated in place.  Returns y."""
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    Bsz, Dm = x.shape
    N = A.shape[1]
    dt = x.dtype
    code = _dtype_code(x)
    _need(x, "x", (Bsz, Dm), dt, dev)
    _need(delta, "delta", (Bsz, Dm), dt, dev)
    A2 = _pairs(A, "A", (Dm, N), dev)
    _need(B, "B", (Bsz, N), dt, dev)
    _need(C, "C", (Bsz, N), dt, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    _bias(delta_bias, Dm, dev)
    h2 = _pairs(h, "h", (Bsz, Dm, N), dev)
    if y is None:
        y = torch.empty((Bsz, Dm), dtype=dt, device=dev)
    _need(y, "y", (Bsz, Dm), dt, dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_step_complex(_ptr(x), _ptr(delta), _ptr(delta_bias), _ptr(A2), _ptr(B), _ptr(C), _ptr(D),
                                    _ptr(h2), _ptr(y), Bsz, Dm, N, code, _flags(delta_softplus, euler_b),
                                    _stream(dev))
    _check(rc, "ssm_step_complex")
    return y


def step_fused(x, delta, A, B, C, D, h, y=None, delta_bias=None, delta_softplus=False, euler_b=False):
    """ssm_step_fused: one decode step with the scan's options; h is updated in place."""
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    Bsz, Dm = x.shape
    N = A.shape[1]
    dt = x.dtype
    code = _dtype_code(x)
    _need(x, "x", (Bsz, Dm), dt, dev)
    _need(delta, "delta", (Bsz, Dm), dt, dev)
    _need(A, "A", (Dm, N), torch.float32, dev)
    _need(B, "B", (Bsz, N), dt, dev)
    _need(C, "C", (Bsz, N), dt, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    _need(h, "h", (Bsz, Dm, N), torch.float32, dev)
    _bias(delta_bias, Dm, dev)
    if y is None:
        y = torch.empty((Bsz, Dm), dtype=dt, device=dev)
    _need(y, "y", (Bsz, Dm), dt, dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_step_fused(_ptr(x), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                  _ptr(h), _ptr(y), Bsz, Dm, N, code, _flags(delta_softplus, euler_b),
                                  _stream(dev))
    _check(rc, "ssm_step_fused")
    return y


def step(x, delta, A, B, C, D, h, y=None, delta_bias=None, delta_softplus=False, euler_b=False):
    """One decode step: h [Bsz, Dm, N] fp32 is updated in place; returns y [Bsz, Dm].

    x, delta: [Bsz, Dm]; B, C: [Bsz, N] (same dtype: bf16, or fp32);
    A: [Dm, N] fp32; D: [Dm] fp32.  Options as in scan_fwd.
    """
    if delta_bias is not None or delta_softplus or euler_b:
        return step_fused(x, delta, A, B, C, D, h, y=y, delta_bias=delta_bias,
                          delta_softplus=delta_softplus, euler_b=euler_b)
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    Bsz, Dm = x.shape
    N = A.shape[1]
    dt = x.dtype
    code = _dtype_code(x)
    _need(x, "x", (Bsz, Dm), dt, dev)
    _need(delta, "delta", (Bsz, Dm), dt, dev)
    _need(A, "A", (Dm, N), torch.float32, dev)
    _need(B, "B", (Bsz, N), dt, dev)
    _need(C, "C", (Bsz, N), dt, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    _need(h, "h", (Bsz, Dm, N), torch.float32, dev)
    if y is None:
        y = torch.empty((Bsz, Dm), dtype=dt, device=dev)
    _need(y, "y", (Bsz, Dm), dt, dev)
    with torch.cuda.device(dev):
        if code == SSM_BF16:
            rc = lib().ssm_step(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(h),
                                _ptr(y), Bsz, Dm, N, _stream(dev))
        else:
            rc = lib().ssm_step_ex(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(h),
                                   _ptr(y), Bsz, Dm, N, code, _stream(dev))
    _check(rc, "ssm_step")
    return y


def gated_carry_steps() -> int:
    """Steps per row of the carry scan_gated_fwd returns."""
    return int(lib().ssm_gated_carry_steps())


def _gated_shape(x, cu_seqlens):
    """(leading shape of x, Bsz, L, Dm, sequences, state rows) of a gated call."""
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    if cu_seqlens is None:
        Bsz, L, Dm = x.shape
        return (Bsz, L), Bsz, L, Dm, 0, Bsz
    L, Dm = x.shape
    nseq = cu_seqlens.shape[0] - 1
    _need(cu_seqlens, "cu_seqlens", (nseq + 1,), torch.int64, dev)
    return (L,), 1, L, Dm, nseq, nseq


def scan_gated_fwd(x, r, i, A, cu_seqlens=None, h_init=None, want_state=True, want_carry=False, out=None):
    """ssm_scan_gated_fwd: gated linear recurrence.

    x, r, i: [Bsz, L, Dm] (same dtype, fp32 or bf16); A: [Dm] fp32, not
    positive; h_init: optional [Bsz, Dm] fp32.  With cu_seqlens (int64
    [nseq+1], on the device) the sequences are packed: x, r, i [L, Dm], h_init
    [nseq, Dm].  Returns a dict with y (x's shape and dtype), h_final
    [Bsz or nseq, Dm] fp32 (if want_state) and carry [Bsz, ceil(L /
    gated_carry_steps()), Dm] fp32 (if want_carry; for scan_gated_bwd).  `out`
    may supply any of these tensors.
    """
    lead, Bsz, L, Dm, nseq, rows = _gated_shape(x, cu_seqlens)
    dev, dt = x.device, x.dtype
    code = _dtype_code(x)
    for t, name, shape, tdt in ((x, "x", (*lead, Dm), dt), (r, "r", (*lead, Dm), dt), (i, "i", (*lead, Dm), dt),
                                (A, "A", (Dm,), torch.float32)):
        _need(t, name, shape, tdt, dev)
    if h_init is not None:
        _need(h_init, "h_init", (rows, Dm), torch.float32, dev)
    shapes = {"y": None}
    if want_state:
        shapes["h_final"] = (rows, Dm)
    if want_carry:
        c = gated_carry_steps()
        shapes["carry"] = (Bsz, (L + c - 1) // c, Dm)
    o = _outputs(out, x, shapes)
    _launch("ssm_scan_gated_fwd", dev, _ptr(x), _ptr(r), _ptr(i), _ptr(A), _ptr(cu_seqlens), nseq, _ptr(h_init),
            _ptr(o["y"]), _ptr(o.get("h_final")), _ptr(o.get("carry")), Bsz, L, Dm, code)
    return o


def _outputs(out, like, shapes):
    """The call's outputs: those the caller supplied, checked, and new ones.
    shapes: name -> shape of an fp32 tensor, or None for one like `like`."""
    o = {} if out is None else dict(out)
    for k in o:
        if k not in shapes:
            raise ValueError(f"out has {k!r}, which this call does not return ({', '.join(shapes)})")
    for k, shape in shapes.items():
        t = o.get(k)
        if t is not None:
            _need(t, k, like.shape if shape is None else shape, like.dtype if shape is None else torch.float32,
                  like.device)
        elif shape is None:
            o[k] = torch.empty_like(like)
        else:
            o[k] = torch.empty(shape, dtype=torch.float32, device=like.device)
    return o


def scan_gated_bwd(x, r, i, A, dy, cu_seqlens=None, h_init=None, dh_final=None, carry=None, want_dh_init=True,
                   out=None):
    """ssm_scan_gated_bwd: gradients of the gated linear recurrence.

    Forward inputs as in scan_gated_fwd, dy in x's shape and dtype, optional
    dh_final [Bsz or nseq, Dm] fp32.  carry: the forward's carry
    (want_carry=True); without it the states are computed again.  Returns a
    dict with dx, dr, di (x's shape and dtype), dA [Dm] fp32 and dh_init
    [Bsz or nseq, Dm] fp32 (if want_dh_init).  `out` may supply any of these
    tensors.
    """
    lead, Bsz, L, Dm, nseq, rows = _gated_shape(x, cu_seqlens)
    dev, dt = x.device, x.dtype
    code = _dtype_code(x)
    for t, name, shape, tdt in ((x, "x", (*lead, Dm), dt), (r, "r", (*lead, Dm), dt), (i, "i", (*lead, Dm), dt),
                                (A, "A", (Dm,), torch.float32), (dy, "dy", (*lead, Dm), dt)):
        _need(t, name, shape, tdt, dev)
    for t, name in ((h_init, "h_init"), (dh_final, "dh_final")):
        if t is not None:
            _need(t, name, (rows, Dm), torch.float32, dev)
    if carry is not None:
        c = gated_carry_steps()
        _need(carry, "carry", (Bsz, (L + c - 1) // c, Dm), torch.float32, dev)
    shapes = {"dx": None, "dr": None, "di": None, "dA": (Dm,)}
    if want_dh_init:
        shapes["dh_init"] = (rows, Dm)
    o = _outputs(out, x, shapes)
    _launch("ssm_scan_gated_bwd", dev, _ptr(x), _ptr(r), _ptr(i), _ptr(A), _ptr(cu_seqlens), nseq, _ptr(h_init),
            _ptr(carry), _ptr(dy), _ptr(dh_final), _ptr(o["dx"]), _ptr(o["dr"]), _ptr(o["di"]), _ptr(o["dA"]),
            _ptr(o.get("dh_init")), Bsz, L, Dm, code)
    return o


def step_gated(x, r, i, A, h, h_out=None, y=None):
    """ssm_step_gated: one decode step of the gated linear recurrence.

    x, r, i: [Bsz, Dm] (same dtype); A: [Dm] fp32; h: [Bsz, Dm] fp32, updated
    in place unless h_out [Bsz, Dm] fp32 is given.  Returns y [Bsz, Dm].
    """
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    Bsz, Dm = x.shape
    dt = x.dtype
    code = _dtype_code(x)
    if h_out is None:
        h_out = h
    if y is None:
        y = torch.empty_like(x)
    shape = (Bsz, Dm)
    _need(x, "x", shape, dt, dev)
    _need(r, "r", shape, dt, dev)
    _need(i, "i", shape, dt, dev)
    _need(A, "A", (Dm,), torch.float32, dev)
    _need(h, "h", shape, torch.float32, dev)
    if h_out is not h:
        _need(h_out, "h_out", shape, torch.float32, dev)
    _need(y, "y", shape, dt, dev)
    _launch("ssm_step_gated", dev, x.data_ptr(), r.data_ptr(), i.data_ptr(), A.data_ptr(), h.data_ptr(),
            h_out.data_ptr(), y.data_ptr(), Bsz, Dm, code)
    return y


def _norm_shape(x, group):
    """(rows, channels, channels of a group, shape of the statistics)."""
    if x.device.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: x must be a device tensor")
    shape = x.shape
    if not shape:
        raise ValueError("x needs at least one axis")
    Dm = shape[-1]
    P = Dm if group is None else int(group)
    if P <= 0 or Dm % P:
        raise ValueError(f"the last axis ({Dm}) is not a multiple of group = {P}")
    return x.numel() // Dm, Dm, P, (*shape[:-1], Dm // P)


def layer_norm_fwd(x, weight=None, bias=None, residual=None, group=None, eps=1e-5, want_stats=False, out=None):
    """ssm_layer_norm_fwd: layer norm over groups of channels of the last axis.

    x, residual: [..., Dm] (same dtype, fp32 or bf16); weight, bias: [Dm] fp32
    or None; group: channels normalised together (None: all Dm).  Returns a
    dict with y (x's shape and dtype), sum = x + residual (if residual is
    given) and mean, rstd [..., Dm / group] fp32 (if want_stats; for
    layer_norm_bwd).  `out` may supply any of these tensors; out["sum"] may be
    residual itself.
    """
    rows, Dm, P, stats = _norm_shape(x, group)
    dev, dt = x.device, x.dtype
    code = _dtype_code(x)
    shape = x.shape
    _need(x, "x", shape, dt, dev)
    if residual is not None:
        _need(residual, "residual", shape, dt, dev)
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _need(t, name, (Dm,), torch.float32, dev)
    shapes = {"y": None}
    if residual is not None:
        shapes["sum"] = None
    if want_stats:
        shapes["mean"] = shapes["rstd"] = stats
    o = _outputs(out, x, shapes)
    _launch("ssm_layer_norm_fwd", dev, _ptr(x), _ptr(residual), _ptr(weight), _ptr(bias), _ptr(o.get("sum")),
            _ptr(o["y"]), _ptr(o.get("mean")), _ptr(o.get("rstd")), rows, Dm, P, eps, code)
    return o


def layer_norm_bwd(s, weight, mean, rstd, dy, dsum=None, group=None, want_params=True, out=None):
    """ssm_layer_norm_bwd: gradients of the layer norm.

    s: the normalised values (the forward's sum, or x when there was no
    residual), mean, rstd: the forward's statistics, dy: s's shape and dtype;
    weight: [Dm] fp32 or None; dsum: optional gradient that reaches s directly
    (the residual path).  Returns a dict with dx (s's shape and dtype) and, if
    want_params, dweight and dbias [Dm] fp32.  `out` may supply any of these
    tensors.
    """
    rows, Dm, P, stats = _norm_shape(s, group)
    dev, dt = s.device, s.dtype
    code = _dtype_code(s)
    shape = s.shape
    _need(s, "s", shape, dt, dev)
    _need(dy, "dy", shape, dt, dev)
    if dsum is not None:
        _need(dsum, "dsum", shape, dt, dev)
    if weight is not None:
        _need(weight, "weight", (Dm,), torch.float32, dev)
    _need(mean, "mean", stats, torch.float32, dev)
    _need(rstd, "rstd", stats, torch.float32, dev)
    shapes = {"dx": None}
    if want_params:
        shapes["dweight"] = shapes["dbias"] = (Dm,)
    o = _outputs(out, s, shapes)
    _launch("ssm_layer_norm_bwd", dev, _ptr(s), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dy), _ptr(dsum),
            _ptr(o["dx"]), _ptr(o.get("dweight")), _ptr(o.get("dbias")), rows, Dm, P, code)
    return o


def _attn_shape(q, k, v, log_decay, cu_seqlens):
    """(leading shape, Bsz, L, H, Hkv, Dk, Dv, sequences, state rows) of a
    linear attention call, its tensors checked."""
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: q must be a device tensor")
    *lead, H, Dk = q.shape
    Hkv, Dv = v.shape[-2:]
    lead = tuple(lead)
    if cu_seqlens is None:
        Bsz, L = lead
        nseq, rows = 0, Bsz
    else:
        Bsz, (L,) = 1, lead
        nseq = rows = cu_seqlens.shape[0] - 1
        _need(cu_seqlens, "cu_seqlens", (nseq + 1,), torch.int64, dev)
    for t, name, shape, tdt in ((q, "q", (*lead, H, Dk), dt), (k, "k", (*lead, Hkv, Dk), dt),
                                (v, "v", (*lead, Hkv, Dv), dt), (log_decay, "log_decay", (H,), torch.float32)):
        _need(t, name, shape, tdt, dev)
    return lead, Bsz, L, H, Hkv, Dk, Dv, nseq, rows


def _outputs_of(out, dev, shapes):
    """The call's outputs: those the caller supplied, checked, and new ones.
    shapes: name -> (shape, dtype)."""
    o = {} if out is None else dict(out)
    for k in o:
        if k not in shapes:
            raise ValueError(f"out has {k!r}, which this call does not return ({', '.join(shapes)})")
    for k, (shape, dt) in shapes.items():
        if o.get(k) is not None:
            _need(o[k], k, shape, dt, dev)
        else:
            o[k] = torch.empty(shape, dtype=dt, device=dev)
    return o


def linear_attn_fwd(q, k, v, log_decay, cu_seqlens=None, h_init=None, scale=None, want_state=True, out=None):
    """ssm_linear_attn_fwd: linear attention with one decay per head.

    q: [Bsz, L, H, Dk]; k: [Bsz, L, Hkv, Dk]; v: [Bsz, L, Hkv, Dv] (same dtype,
    fp32 or bf16; H a multiple of Hkv); log_decay: [H] fp32, not positive;
    h_init: optional [Bsz, H, Dv, Dk] fp32; scale: of y, 1 / sqrt(Dk) if None.
    With cu_seqlens (int64 [nseq+1], on the device) the sequences are packed:
    q, k, v without a batch axis, h_init [nseq, H, Dv, Dk].  Returns a dict
    with y ([Bsz, L, H, Dv], q's dtype) and h_final (like h_init, if
    want_state).  `out` may supply any of these tensors.
    """
    lead, Bsz, L, H, Hkv, Dk, Dv, nseq, rows = _attn_shape(q, k, v, log_decay, cu_seqlens)
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    state = (rows, H, Dv, Dk)
    if h_init is not None:
        _need(h_init, "h_init", state, torch.float32, dev)
    shapes = {"y": ((*lead, H, Dv), dt)}
    if want_state:
        shapes["h_final"] = (state, torch.float32)
    o = _outputs_of(out, dev, shapes)
    _launch("ssm_linear_attn_fwd", dev, _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(cu_seqlens), nseq,
            _ptr(h_init), _ptr(o["y"]), _ptr(o.get("h_final")), Bsz, L, H, Hkv, Dk, Dv,
            Dk ** -0.5 if scale is None else scale, code)
    return o


def linear_attn_bwd(q, k, v, log_decay, dy, cu_seqlens=None, h_init=None, dh_final=None, scale=None,
                    want_dh_init=True, out=None):
    """ssm_linear_attn_bwd: gradients of linear attention.

    Forward inputs as in linear_attn_fwd, dy: [Bsz, L, H, Dv] (q's dtype),
    dh_final: optional, like h_init.  Returns a dict with dq, dk, dv (like q,
    k, v) and dh_init (like h_init, if want_dh_init).  `out` may supply any of
    these tensors.
    """
    lead, Bsz, L, H, Hkv, Dk, Dv, nseq, rows = _attn_shape(q, k, v, log_decay, cu_seqlens)
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    state = (rows, H, Dv, Dk)
    _need(dy, "dy", (*lead, H, Dv), dt, dev)
    for t, name in ((h_init, "h_init"), (dh_final, "dh_final")):
        if t is not None:
            _need(t, name, state, torch.float32, dev)
    shapes = {"dq": (q.shape, dt), "dk": (k.shape, dt), "dv": (v.shape, dt)}
    if want_dh_init:
        shapes["dh_init"] = (state, torch.float32)
    o = _outputs_of(out, dev, shapes)
    _launch("ssm_linear_attn_bwd", dev, _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(cu_seqlens), nseq,
            _ptr(h_init), _ptr(dy), _ptr(dh_final), _ptr(o["dq"]), _ptr(o["dk"]), _ptr(o["dv"]),
            _ptr(o.get("dh_init")), Bsz, L, H, Hkv, Dk, Dv, Dk ** -0.5 if scale is None else scale, code)
    return o


def step_linear_attn(q, k, v, log_decay, h, h_out=None, y=None, scale=None):
    """ssm_step_linear_attn: one decode step of linear attention.

    q: [Bsz, H, Dk]; k: [Bsz, Hkv, Dk]; v: [Bsz, Hkv, Dv] (same dtype);
    log_decay: [H] fp32; h: [Bsz, H, Dv, Dk] fp32, updated in place unless
    h_out (like h) is given; scale as in linear_attn_fwd.  Returns
    y [Bsz, H, Dv].
    """
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: q must be a device tensor")
    Bsz, H, Dk = q.shape
    Hkv, Dv = v.shape[-2:]
    code = _dtype_code(q)
    if h_out is None:
        h_out = h
    if y is None:
        y = torch.empty((Bsz, H, Dv), dtype=dt, device=dev)
    _need(q, "q", (Bsz, H, Dk), dt, dev)
    _need(k, "k", (Bsz, Hkv, Dk), dt, dev)
    _need(v, "v", (Bsz, Hkv, Dv), dt, dev)
    _need(log_decay, "log_decay", (H,), torch.float32, dev)
    _need(h, "h", (Bsz, H, Dv, Dk), torch.float32, dev)
    if h_out is not h:
        _need(h_out, "h_out", (Bsz, H, Dv, Dk), torch.float32, dev)
    _need(y, "y", (Bsz, H, Dv), dt, dev)
    _launch("ssm_step_linear_attn", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), h.data_ptr(),
            h_out.data_ptr(), y.data_ptr(), Bsz, H, Hkv, Dk, Dv, Dk ** -0.5 if scale is None else scale, code)
    return y


def _rope_shape(q, k, positions, freqs, q_weight, k_weight):
    """(rows, Hq, Hk, D, R) of a norm and rotation, its tensors checked."""
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("libssmscan runs on the GPU: q must be a device tensor")
    *lead, Hq, D = q.shape
    lead, Hk = tuple(lead), k.shape[-2]
    R = 0 if freqs is None else 2 * freqs.shape[0]
    _need(q, "q", (*lead, Hq, D), dt, dev)
    _need(k, "k", (*lead, Hk, D), dt, dev)
    if R:
        _need(positions, "positions", lead, torch.int64, dev)
        _need(freqs, "freqs", (R // 2,), torch.float32, dev)
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _need(t, name, (D,), torch.float32, dev)
    rows = 1
    for n in lead:
        rows *= n
    return rows, Hq, Hk, D, R


def qk_norm_rope_fwd(q, k, positions=None, freqs=None, q_weight=None, k_weight=None, interleaved=False, eps=1e-6,
                     out=None):
    """ssm_qk_norm_rope_fwd: norm over each head of q and k, and the rotation
    of their positions.

    q: [..., Hq, D]; k: [..., Hk, D] (same dtype, fp32 or bf16); positions:
    [...] int64; freqs: [R / 2] fp32, radians per position (None: the norm
    alone); q_weight, k_weight: [D] fp32 or None; interleaved: pairs (2i,
    2i+1) instead of (i, i + R/2).  Returns a dict with q and k.  `out` may
    supply either tensor, which may be the input itself.
    """
    rows, Hq, Hk, D, R = _rope_shape(q, k, positions, freqs, q_weight, k_weight)
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    o = _outputs_of(out, dev, {"q": (q.shape, dt), "k": (k.shape, dt)})
    _launch("ssm_qk_norm_rope_fwd", dev, _ptr(q), _ptr(k), _ptr(positions), _ptr(freqs), _ptr(q_weight),
            _ptr(k_weight), _ptr(o["q"]), _ptr(o["k"]), rows, Hq, Hk, D, R, eps,
            SSM_ROPE_INTERLEAVED if interleaved else 0, code)
    return o


def qk_norm_rope_bwd(q, k, dq, dk, positions=None, freqs=None, q_weight=None, k_weight=None, interleaved=False,
                     eps=1e-6, want_params=True, out=None):
    """ssm_qk_norm_rope_bwd: gradients of the norm and rotation.

    q, k: the forward's inputs; dq, dk: gradients of its outputs (same shapes
    and dtype); the rest as in qk_norm_rope_fwd.  Returns a dict with dq, dk
    and, if want_params, dq_weight and dk_weight [D] fp32.  `out` may supply
    any of these tensors.
    """
    rows, Hq, Hk, D, R = _rope_shape(q, k, positions, freqs, q_weight, k_weight)
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    _need(dq, "dq", q.shape, dt, dev)
    _need(dk, "dk", k.shape, dt, dev)
    shapes = {"dq": (q.shape, dt), "dk": (k.shape, dt)}
    if want_params:
        shapes["dq_weight"] = shapes["dk_weight"] = ((D,), torch.float32)
    o = _outputs_of(out, dev, shapes)
    _launch("ssm_qk_norm_rope_bwd", dev, _ptr(q), _ptr(k), _ptr(dq), _ptr(dk), _ptr(positions), _ptr(freqs),
            _ptr(q_weight), _ptr(k_weight), _ptr(o["dq"]), _ptr(o["dk"]), _ptr(o.get("dq_weight")),
            _ptr(o.get("dk_weight")), rows, Hq, Hk, D, R, eps, SSM_ROPE_INTERLEAVED if interleaved else 0, code)
    return o
