"""Quantized latent-MoE expert stage on MI355X (gfx950): Python binding.

Thin ctypes marshalling over ``liblatmoe.so`` (the C ABI in
``include/lat_moe.h``).  Every step of the stage runs in the library's HIP
kernels; torch tensors only provide device memory and the current stream.
There is no fallback: if the library is not built, calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblatmoe.so")

LAT_MOE_MAX_E = 1024
# down-weight formats of lat_moe_expert_forward_fmt (both 18-byte blocks of 32)
DOWN_IQ4_NL = 0
DOWN_Q4_0 = 1
# gate/up-weight formats of lat_moe_expert_forward_fmt
GATEUP_Q3_K = 0
GATEUP_Q4_0 = 1

# Symbols the C header declares (checked by the CPU test suite).
EXPORTED = (
    "lat_moe_workspace_size",
    "lat_moe_expert_forward",
    "lat_moe_expert_forward_ex",
    "lat_moe_expert_forward_fmt",
    "lat_moe_expert_forward_noalloc",
    "lat_moe_quantize_q8_1",
    "lat_moe_dense_q8_0",
    "lat_moe_dense_q8_0_debug",
    "lat_moe_dense_q4_0",
    "lat_moe_dense_q4_0_debug",
    "lat_moe_router_topk",
    "lat_moe_router_topk_ex",
    "lat_moe_quantize_fp8",
    "lat_moe_rmsnorm",
    "lat_moe_dense_fp8",
    "lat_moe_dense_fp8_ex",
    "lat_moe_ffn_fp8_workspace_size",
    "lat_moe_ffn_fp8",
    "lat_moe_ffn_fp8_ex",
    "lat_moe_dense_16",
    "lat_moe_gated_16",
    "lat_moe_strerror",
    "lat_moe_version",
)


class Shapes(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("L", ctypes.c_int32), ("F", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32)]


class Debug(ctypes.Structure):
    _fields_ = [
        ("h_q8_1", ctypes.c_void_p),
        ("perm", ctypes.c_void_p),
        ("offsets", ctypes.c_void_p),
        ("dropped", ctypes.c_void_p),
        ("gateup_i32", ctypes.c_void_p),
        ("gu_row0", ctypes.c_int32),
        ("gu_rows", ctypes.c_int32),
        ("down_i32", ctypes.c_void_p),
        ("dn_row0", ctypes.c_int32),
        ("dn_rows", ctypes.c_int32),
        ("stage_events", ctypes.POINTER(ctypes.c_void_p)),
        ("deterministic", ctypes.c_int32),
    ]


class Routing(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float)]


class LatMoeError(RuntimeError):
    pass


_lib = None


def lib() -> ctypes.CDLL:
    """Load liblatmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise LatMoeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "(or python quantized_latent_moe_amd/build.py)")
        c = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        c.lat_moe_workspace_size.argtypes = [ctypes.POINTER(Shapes)]
        c.lat_moe_workspace_size.restype = ctypes.c_size_t
        c.lat_moe_expert_forward.argtypes = [P, P, P, P, P, ctypes.POINTER(Shapes), P, P, ctypes.c_size_t, P]
        c.lat_moe_expert_forward.restype = ctypes.c_int
        c.lat_moe_expert_forward_ex.argtypes = [P, P, P, P, P, ctypes.POINTER(Shapes), P, P, ctypes.c_size_t, P,
                                                ctypes.POINTER(Debug)]
        c.lat_moe_expert_forward_ex.restype = ctypes.c_int
        c.lat_moe_expert_forward_fmt.argtypes = [P, P, P, P, ctypes.c_int32, P, ctypes.c_int32,
                                                 ctypes.POINTER(Shapes), P, P, ctypes.c_size_t, P,
                                                 ctypes.POINTER(Debug)]
        c.lat_moe_expert_forward_fmt.restype = ctypes.c_int
        c.lat_moe_expert_forward_noalloc.argtypes = [P, P, P, P, P, ctypes.POINTER(Shapes), P, P]
        c.lat_moe_expert_forward_noalloc.restype = ctypes.c_int
        c.lat_moe_quantize_q8_1.argtypes = [P, ctypes.c_int64, ctypes.c_int32, P, P]
        c.lat_moe_quantize_q8_1.restype = ctypes.c_int
        i32, i64 = ctypes.c_int32, ctypes.c_int64
        c.lat_moe_dense_q8_0.argtypes = [P, P, i64, i32, i32, P, P, P]
        c.lat_moe_dense_q8_0.restype = ctypes.c_int
        c.lat_moe_dense_q8_0_debug.argtypes = [P, P, i64, i32, i32, P, P, P, P, i32, i32]
        c.lat_moe_dense_q8_0_debug.restype = ctypes.c_int
        c.lat_moe_dense_q4_0.argtypes = [P, P, i64, i32, i32, P, P, P]
        c.lat_moe_dense_q4_0.restype = ctypes.c_int
        c.lat_moe_dense_q4_0_debug.argtypes = [P, P, i64, i32, i32, P, P, P, P, i32, i32]
        c.lat_moe_dense_q4_0_debug.restype = ctypes.c_int
        c.lat_moe_router_topk.argtypes = [P, i64, i32, i32, P, P, P]
        c.lat_moe_router_topk.restype = ctypes.c_int
        f32, size = ctypes.c_float, ctypes.c_size_t
        c.lat_moe_quantize_fp8.argtypes = [P, i32, i64, i32, P, P, P]
        c.lat_moe_quantize_fp8.restype = ctypes.c_int
        c.lat_moe_rmsnorm.argtypes = [P, i32, P, i32, P, f32, i64, i32, P, P, i32, P, P, P, P]
        c.lat_moe_rmsnorm.restype = ctypes.c_int
        c.lat_moe_dense_fp8.argtypes = [P, P, P, P, i64, i32, i32, P, P, P, P]
        c.lat_moe_dense_fp8.restype = ctypes.c_int
        c.lat_moe_dense_fp8_ex.argtypes = [P, P, P, P, i64, i32, i32, P, P, P, i32, P]
        c.lat_moe_dense_fp8_ex.restype = ctypes.c_int
        c.lat_moe_ffn_fp8_workspace_size.argtypes = [i64, i32, i32]
        c.lat_moe_ffn_fp8_workspace_size.restype = size
        c.lat_moe_ffn_fp8.argtypes = [P, P, P, P, P, P, i64, i32, i32, P, P, P, P, P, size, P]
        c.lat_moe_ffn_fp8.restype = ctypes.c_int
        c.lat_moe_ffn_fp8_ex.argtypes = [P, P, P, P, P, P, i64, i32, i32, P, P, P, P, i32, P, size, P]
        c.lat_moe_ffn_fp8_ex.restype = ctypes.c_int
        c.lat_moe_router_topk_ex.argtypes = [P, P, i64, i32, i32, ctypes.POINTER(Routing), P, P, P]
        c.lat_moe_router_topk_ex.restype = ctypes.c_int
        c.lat_moe_dense_16.argtypes = [P, i64, P, i32, i64, i32, i32, P, i32, P, i32, i64, P, i32, i64, P, P]
        c.lat_moe_dense_16.restype = ctypes.c_int
        c.lat_moe_gated_16.argtypes = [P, i64, P, i32, i64, i32, i32, P, i32, P, i32, i64, P]
        c.lat_moe_gated_16.restype = ctypes.c_int
        c.lat_moe_strerror.argtypes = [ctypes.c_int]
        c.lat_moe_strerror.restype = ctypes.c_char_p
        c.lat_moe_version.restype = ctypes.c_int
        _lib = c
    return _lib


def strerror(code: int) -> str:
    return lib().lat_moe_strerror(int(code)).decode()


def _check(rc: int) -> None:
    if rc != 0:
        raise LatMoeError(f"lat_moe error {rc}: {strerror(rc)}")


def shapes(T: int, L: int, F: int, E: int, k: int) -> Shapes:
    return Shapes(int(T), int(L), int(F), int(E), int(k))


def workspace_size(s: Shapes) -> int:
    return int(lib().lat_moe_workspace_size(ctypes.byref(s)))


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return int(stream)
    import torch
    return torch.cuda.current_stream().cuda_stream


def expert_forward(x_q8_1, router_idx, router_w, gateup_q3k, down_iq4nl, s: Shapes, y, workspace,
                   stream=None) -> None:
    """Enqueue the expert stage; all tensors on the current GPU (uint8 blocks,
    int32 ids, fp32 weights, fp32 y [T, L], uint8 workspace)."""
    rc = lib().lat_moe_expert_forward(_ptr(x_q8_1), _ptr(router_idx), _ptr(router_w), _ptr(gateup_q3k),
                                      _ptr(down_iq4nl), ctypes.byref(s), _ptr(y), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc)


NOALLOC_SCRATCH_BYTES = 64 << 20
ESCRATCH = 5


def expert_forward_noalloc(x_q8_1, router_idx, router_w, gateup_q3k, down_iq4nl, s: Shapes, y, stream=None) -> None:
    """As expert_forward without a workspace: the library's fixed per-GPU
    scratch (NOALLOC_SCRATCH_BYTES) is used, and nothing is allocated."""
    rc = lib().lat_moe_expert_forward_noalloc(_ptr(x_q8_1), _ptr(router_idx), _ptr(router_w), _ptr(gateup_q3k),
                                              _ptr(down_iq4nl), ctypes.byref(s), _ptr(y), _stream(stream))
    _check(rc)


def _debug(h_q8_1, perm, offsets, dropped, gateup_i32, gu_row0, down_i32, dn_row0, stage_events, deterministic):
    ev = None
    if stage_events is not None:
        if len(stage_events) != 5:
            raise ValueError("stage_events needs 5 events")
        ev = (ctypes.c_void_p * 5)(*[int(e.cuda_event) for e in stage_events])
    d = Debug(_ptr(h_q8_1), _ptr(perm), _ptr(offsets), _ptr(dropped), _ptr(gateup_i32), int(gu_row0),
              0 if gateup_i32 is None else int(gateup_i32.shape[1]), _ptr(down_i32), int(dn_row0),
              0 if down_i32 is None else int(down_i32.shape[1]),
              ctypes.cast(ev, ctypes.POINTER(ctypes.c_void_p)) if ev is not None else None,
              1 if deterministic else 0)
    return d, ev


def expert_forward_ex(x_q8_1, router_idx, router_w, gateup_q3k, down_iq4nl, s: Shapes, y, workspace, *,
                      deterministic: bool = True, h_q8_1=None, perm=None, offsets=None, dropped=None, gateup_i32=None,
                      gu_row0=0, down_i32=None, dn_row0=0, stage_events=None, stream=None) -> None:
    """As expert_forward, with the options and optional debug outputs of
    lat_moe_debug: deterministic=False sums each token's experts into y by
    fp32 atomic adds (no slot buffer, no combine kernel); gateup_i32 is
    [T*k, rows, L/32] int32 and down_i32 [T*k, rows, F/32]; stage_events is a
    list of five recorded torch.cuda.Event(enable_timing=True)."""
    d, ev = _debug(h_q8_1, perm, offsets, dropped, gateup_i32, gu_row0, down_i32, dn_row0, stage_events,
                   deterministic)
    rc = lib().lat_moe_expert_forward_ex(_ptr(x_q8_1), _ptr(router_idx), _ptr(router_w), _ptr(gateup_q3k),
                                         _ptr(down_iq4nl), ctypes.byref(s), _ptr(y), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream),
                                         ctypes.byref(d))
    _check(rc)


def expert_forward_fmt(x_q8_1, router_idx, router_w, gateup, down, down_format: int, s: Shapes, y, workspace, *,
                       gateup_format: int = GATEUP_Q3_K, debug: bool = False, deterministic: bool = True,
                       h_q8_1=None, perm=None, offsets=None, dropped=None, gateup_i32=None, gu_row0=0, down_i32=None,
                       dn_row0=0, stage_events=None, stream=None) -> None:
    """The expert stage with gate/up weights in gateup_format (GATEUP_Q3_K:
    [E, 2F, L/256, 110]; GATEUP_Q4_0: [E, 2F, L/32, 18]) and down weights in
    down_format (DOWN_IQ4_NL or DOWN_Q4_0, both [E, L, F/32, 18] uint8); with
    debug=True (or deterministic=False) the options and optional outputs of
    expert_forward_ex are passed, otherwise no debug struct is."""
    d = None
    if debug or not deterministic:
        d, ev = _debug(h_q8_1, perm, offsets, dropped, gateup_i32, gu_row0, down_i32, dn_row0, stage_events,
                       deterministic)
    rc = lib().lat_moe_expert_forward_fmt(_ptr(x_q8_1), _ptr(router_idx), _ptr(router_w), _ptr(gateup),
                                          int(gateup_format), _ptr(down), int(down_format), ctypes.byref(s), _ptr(y),
                                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _stream(stream), ctypes.byref(d) if d is not None else None)
    _check(rc)


def quantize_q8_1(x, out, stream=None) -> None:
    """fp32 [rows, cols] -> q8_1 blocks (uint8 [rows, cols/32, 36])."""
    rows, cols = x.shape
    _check(lib().lat_moe_quantize_q8_1(_ptr(x), int(rows), int(cols), _ptr(out), _stream(stream)))


def dense_q8_0(x_q8_1, w_q8_0, T: int, N: int, K: int, y_f32=None, y_q8_1=None, *, dots_i32=None, row0: int = 0,
               stream=None) -> None:
    """Latent D / U projection: q8_1 rows x_q8_1 (uint8 [T, K/32, 36]) against
    Q8_0 weights (uint8 [N, K/32, 34]) -> y_f32 (fp32 [T, N]) and/or y_q8_1
    (uint8 [T, N/32, 36]); dots_i32 (int32 [T, rows, K/32]) takes the block
    dots of weight rows row0 .. row0+rows-1."""
    rows = 0 if dots_i32 is None else int(dots_i32.shape[1])
    _check(lib().lat_moe_dense_q8_0_debug(_ptr(x_q8_1), _ptr(w_q8_0), int(T), int(N), int(K), _ptr(y_f32),
                                          _ptr(y_q8_1), _stream(stream), _ptr(dots_i32), int(row0), rows))


def dense_q4_0(x_q8_1, w_q4_0, T: int, N: int, K: int, y_f32=None, y_q8_1=None, *, dots_i32=None, row0: int = 0,
               stream=None) -> None:
    """As dense_q8_0 with Q4_0 weights (uint8 [N, K/32, 18])."""
    rows = 0 if dots_i32 is None else int(dots_i32.shape[1])
    _check(lib().lat_moe_dense_q4_0_debug(_ptr(x_q8_1), _ptr(w_q4_0), int(T), int(N), int(K), _ptr(y_f32),
                                          _ptr(y_q8_1), _stream(stream), _ptr(dots_i32), int(row0), rows))


def router_topk(logits, k: int, router_idx, router_w, stream=None) -> None:
    """fp32 logits [T, E] -> top-k expert ids (int32 [T, k]) and renormalised
    softmax weights (fp32 [T, k]), the expert stage's routing inputs."""
    T, E = logits.shape
    _check(lib().lat_moe_router_topk(_ptr(logits), int(T), int(E), int(k), _ptr(router_idx), _ptr(router_w),
                                     _stream(stream)))


# ---- e4m3 rows and weights: a scale for each 128 values of a row, or for each 128 x 128 block of a matrix ----

FP8_BLOCK = 128


_TORCH = None
_INT32 = None


def _torch():
    """What the calls below use of torch (imported on first use, as everywhere
    in this module): element types, the type codes of rows, and the current
    device's index and its current stream's handle."""
    global _TORCH, _INT32
    if _TORCH is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # about 0.1 us, a Stream object about 3
        # the GPU is in use where a tensor on it is at hand: no need to look whether it is, as torch.cuda does
        cur = getattr(torch._C, "_cuda_getDevice", None)
        _INT32 = torch.int32
        _TORCH = (torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.uint8,
                  {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}, cur or torch.cuda.current_device,
                  raw or (lambda device: torch.cuda.current_stream(device).cuda_stream))
    return _TORCH


def _tensor(name: str, t, dtype, shape, device: int) -> int:
    """Data pointer of a contiguous tensor of this type and shape on the
    current GPU; raises ValueError for anything else."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}: expected the current GPU (cuda:{device})")
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)}, got "
                     f"{'' if t.is_contiguous() else 'non-contiguous '}{t.dtype} {tuple(t.shape)}")


def _device(name: str, t, current_device) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}: expected the current GPU")
    return current_device()


def _rows(name: str, t, kinds) -> int:
    """The type code of a two-dimensional tensor of rows."""
    if t.dim() != 2 or t.dtype not in kinds or t.shape[1] >> 31:
        raise ValueError(f"{name}: expected a 2-dimensional float32, bfloat16 or float16 tensor, got {t.dtype} "
                         f"{tuple(t.shape)}")
    return kinds[t.dtype]


def quantize_fp8(x, codes, scales, stream=None) -> None:
    """Rows x [rows, cols] (float32, bfloat16 or float16) -> e4m3 codes
    (float8_e4m3fn [rows, cols]) and scales (float32 [rows, ceil(cols/128)])."""
    e4m3, f32, _, _, kinds, cur, raw = _torch()
    kind = _rows("x", x, kinds)
    rows, cols = shape = x.shape
    dev = _device("x", x, cur)
    rc = lib().lat_moe_quantize_fp8(_tensor("x", x, x.dtype, shape, dev), kind, rows, cols,
                                    _tensor("codes", codes, e4m3, shape, dev),
                                    _tensor("scales", scales, f32, (rows, -(-cols // 128)), dev),
                                    raw(dev) if stream is None else int(stream))
    if rc:
        _check(rc)


def rmsnorm(x, weight, eps: float, *, residual=None, residual_out=None, y=None, y_q8_1=None, y_fp8=None,
            y_scales=None, stream=None) -> None:
    """Root-mean-square norm of x + residual (or of x) with weight (float32
    [C]), and its roundings: x, residual, residual_out and y are [T, C] in
    float32, bfloat16 or float16 (residual and residual_out in one type);
    y_q8_1 is uint8 [T, C/32, 36]; y_fp8 float8_e4m3fn [T, C] with y_scales
    float32 [T, ceil(C/128)].  Outputs that are None are not made;
    residual_out may be residual, and y may be x."""
    e4m3, f32, _, u8, kinds, cur, raw = _torch()
    kind = _rows("x", x, kinds)
    T, C = shape = x.shape
    dev = _device("x", x, cur)
    r_kind = y_kind = 0
    rp = op = yp = qp = cp = sp = None
    if residual is not None:
        r_kind = _rows("residual", residual, kinds)
        rp = _tensor("residual", residual, residual.dtype, shape, dev)
    if residual_out is not None:
        r_kind = _rows("residual_out", residual_out, kinds)
        op = _tensor("residual_out", residual_out, residual_out.dtype if residual is None else residual.dtype, shape,
                     dev)
    if y is not None:
        y_kind = _rows("y", y, kinds)
        yp = _tensor("y", y, y.dtype, shape, dev)
    if y_q8_1 is not None:
        qp = _tensor("y_q8_1", y_q8_1, u8, (T, C // 32, 36), dev)
    if y_fp8 is not None:
        cp = _tensor("y_fp8", y_fp8, e4m3, shape, dev)
    if y_scales is not None:
        sp = _tensor("y_scales", y_scales, f32, (T, -(-C // 128)), dev)
    rc = lib().lat_moe_rmsnorm(_tensor("x", x, x.dtype, shape, dev), kind, rp, r_kind,
                               _tensor("weight", weight, f32, (C,), dev), eps, T, C, op, yp, y_kind, qp, cp, sp,
                               raw(dev) if stream is None else int(stream))
    if rc:
        _check(rc)


def _matrix(name: str, codes, scales, lead, N: int, K: int, e4m3, f32, dev):
    """Pointers of an e4m3 matrix: codes [lead * N, K], scales
    [(lead,) ceil(N/128), ceil(K/128)]."""
    if N >> 31 or K >> 31:
        raise ValueError(f"{name}: {N} x {K} is beyond 32-bit sizes")
    blocks = (-(-N // 128), -(-K // 128))
    return (_tensor(name, codes, e4m3, ((lead or 1) * N, K), dev),
            _tensor(name + "'s scales", scales, f32, (lead, *blocks) if lead else blocks, dev))


def _products(exact) -> int:
    """How products with more than 16 rows are computed.  None: exactly where
    an fp32 y is asked for (the gated block's gate and up products never);
    True: exactly; False: by the e4m3 matrix unit."""
    if exact is None:
        return 0
    if exact is not True and exact is not False:
        raise ValueError(f"exact has to be True, False or None, got {exact!r}")
    return 1 if exact else 2


def dense_fp8(x_fp8, x_scales, w_fp8, w_scales, *, y_f32=None, y_bf16=None, y_q8_1=None, exact=None,
              stream=None) -> None:
    """Projection of e4m3 rows x_fp8 (float8_e4m3fn [T, K]) with x_scales
    (float32 [T, ceil(K/128)]) by e4m3 weights w_fp8 (float8_e4m3fn [N, K])
    with w_scales (float32 [ceil(N/128), ceil(K/128)]) -> y_f32 (float32
    [T, N]), y_bf16 (bfloat16 [T, N]) and/or y_q8_1 (uint8 [T, N/32, 36]).
    With more than 16 rows the products are exact if y_f32 is given, and pass
    through the e4m3 matrix unit, which cuts small ones beside large ones,
    otherwise (about twice as fast); exact=True or False chooses."""
    e4m3, f32, bf16, u8, _, cur, raw = _torch()
    if x_fp8.dim() != 2 or w_fp8.dim() != 2:
        raise ValueError("x_fp8 and w_fp8 have to be 2-dimensional")
    T, K = shape = x_fp8.shape
    N = w_fp8.shape[0]
    dev = _device("x_fp8", x_fp8, cur)
    w, ws = _matrix("w_fp8", w_fp8, w_scales, 0, N, K, e4m3, f32, dev)
    rc = lib().lat_moe_dense_fp8_ex(_tensor("x_fp8", x_fp8, e4m3, shape, dev),
                                    _tensor("x_scales", x_scales, f32, (T, -(-K // 128)), dev), w, ws, T, N, K,
                                    None if y_f32 is None else _tensor("y_f32", y_f32, f32, (T, N), dev),
                                    None if y_bf16 is None else _tensor("y_bf16", y_bf16, bf16, (T, N), dev),
                                    None if y_q8_1 is None else _tensor("y_q8_1", y_q8_1, u8, (T, N // 32, 36), dev),
                                    _products(exact), raw(dev) if stream is None else int(stream))
    if rc:
        _check(rc)


def ffn_fp8_workspace_size(T: int, C: int, F: int) -> int:
    """Bytes of workspace ffn_fp8 needs (0 if the shapes are unsupported)."""
    if max(C, F) >> 31:
        return 0
    return int(lib().lat_moe_ffn_fp8_workspace_size(int(T), int(C), int(F)))


def ffn_fp8(x_fp8, x_scales, gateup_fp8, gateup_scales, down_fp8, down_scales, workspace, *, y_f32=None, y_bf16=None,
            h_fp8=None, h_scales=None, exact=None, stream=None) -> None:
    """Gated feed-forward block on e4m3 rows x_fp8 [T, C] (x_scales [T,
    ceil(C/128)]): silu(x gate^T) * (x up^T), rounded to e4m3 rows, times
    down^T.  gateup_fp8 is [2F, C], the gate rows first, with gateup_scales
    [2, ceil(F/128), ceil(C/128)]; down_fp8 [C, F] with down_scales
    [ceil(C/128), ceil(F/128)]; y_f32 and/or y_bf16 are [T, C]; h_fp8 [T, F]
    and h_scales [T, ceil(F/128)] take H if they are given; workspace is a
    uint8 tensor of at least ffn_fp8_workspace_size(T, C, F) bytes.  With more
    than 16 rows the gate and up products pass through the e4m3 matrix unit, so
    that 0.24% of H's codes differ from those of exact products, and the down
    products are exact if y_f32 is given; exact=True makes all exact, False
    none."""
    e4m3, f32, bf16, u8, _, cur, raw = _torch()
    if x_fp8.dim() != 2 or down_fp8.dim() != 2:
        raise ValueError("x_fp8 and down_fp8 have to be 2-dimensional")
    T, C = shape = x_fp8.shape
    F = down_fp8.shape[1]
    dev = _device("x_fp8", x_fp8, cur)
    gu, gus = _matrix("gateup_fp8", gateup_fp8, gateup_scales, 2, F, C, e4m3, f32, dev)
    dn, dns = _matrix("down_fp8", down_fp8, down_scales, 0, C, F, e4m3, f32, dev)
    nbytes = workspace.numel()
    rc = lib().lat_moe_ffn_fp8_ex(_tensor("x_fp8", x_fp8, e4m3, shape, dev),
                                  _tensor("x_scales", x_scales, f32, (T, -(-C // 128)), dev), gu, gus, dn, dns, T, C, F,
                                  None if y_f32 is None else _tensor("y_f32", y_f32, f32, shape, dev),
                                  None if y_bf16 is None else _tensor("y_bf16", y_bf16, bf16, shape, dev),
                                  None if h_fp8 is None else _tensor("h_fp8", h_fp8, e4m3, (T, F), dev),
                                  None if h_scales is None else _tensor("h_scales", h_scales, f32, (T, -(-F // 128)),
                                                                        dev),
                                  _products(exact), _tensor("workspace", workspace, u8, (nbytes,), dev), nbytes,
                                  raw(dev) if stream is None else int(stream))
    if rc:
        _check(rc)


# ---- routing by other rules ----

SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}


def _choice(name: str, value, choices) -> int:
    code = choices.get(value)
    if code is None:
        raise ValueError(f"{name} has to be one of {', '.join(choices)}, got {value!r}")
    return code


def router_topk_ex(logits, k: int, router_idx, router_w, *, bias=None, score: str = "softmax", groups: int = 1,
                   top_groups: Optional[int] = None, group_score: str = "top2", renormalise: bool = True,
                   scale: float = 1.0, stream=None) -> None:
    """float32 logits [T, E] -> top-k expert ids (int32 [T, k]) and weights
    (float32 [T, k]) by scores with a choice of rules: softmax or sigmoid of
    the logits; experts ranked by score + bias (float32 [E]; it does not enter
    the weights); picks from the top_groups best of `groups` groups of
    neighbouring experts, a group ranked by its largest candidate ("max") or
    the sum of its two largest ("top2"); weights divided by their sum if
    renormalise, and multiplied by scale.  Logits or biases of -inf close an
    expert."""
    _, f32, _, _, _, cur, raw = _TORCH or _torch()
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError("logits have to be 2-dimensional")
    T, E = shape
    kept = groups if top_groups is None else top_groups
    if (E | k | groups | kept) >> 31 not in (0, -1):  # the call would take them modulo 2^32
        raise ValueError("sizes beyond 32 bits")
    dev = logits.get_device()
    if dev < 0 or dev != cur():
        raise ValueError(f"logits are on {logits.device}: expected the current GPU")
    rules = Routing(_choice("score", score, SCORES), groups, kept,
                    _choice("group_score", group_score, GROUP_SCORES), renormalise, scale)
    rc = (_lib or lib()).lat_moe_router_topk_ex(_tensor("logits", logits, f32, shape, dev),
                                      None if bias is None else _tensor("bias", bias, f32, (E,), dev), T, E, k,
                                      rules, _tensor("router_idx", router_idx, _INT32, (T, k), dev),
                                      _tensor("router_w", router_w, f32, (T, k), dev),
                                      raw(dev) if stream is None else int(stream))
    if rc:
        _check(rc)


# ---- rows and weights in 16 bits ----

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _strided(name: str, t, kinds, shape, device: int) -> tuple:
    """Pointer, type code and row stride of a tensor of rows on the current
    GPU, whose rows may lie apart."""
    kind = kinds.get(t.dtype)
    if kind is not None and t.shape == shape and t.get_device() == device:
        if t.is_contiguous():
            return t.data_ptr(), kind, shape[1]
        if t.stride(1) == 1 or shape[1] == 1:
            return t.data_ptr(), kind, t.stride(0) if shape[0] > 1 else shape[1]
        raise ValueError(f"{name}: the values of a row have to be neighbours, got strides {t.stride()}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}: expected the current GPU (cuda:{device})")
    raise ValueError(f"{name}: expected a float32, bfloat16 or float16 tensor of shape {tuple(shape)}, got {t.dtype} "
                     f"{tuple(t.shape)}")


def _operands(x, w) -> tuple:
    """What a 16-bit product needs to know of its operands: the current GPU,
    x's pointer, row stride and type code, w's pointer, T, N and K."""
    kinds, cur = (_TORCH or _torch())[4:6]
    kind, shape, shape_w = kinds.get(x.dtype), x.shape, w.shape
    if not kind or len(shape) != 2 or len(shape_w) != 2:
        raise ValueError(f"x and w have to be 2-dimensional and bfloat16 or float16, got {x.dtype} {tuple(shape)} and "
                         f"{tuple(shape_w)}")
    T, K = shape
    N = shape_w[0]
    if (K | N) >> 31:
        raise ValueError("x or w is beyond 32-bit sizes")
    dev = x.get_device()
    if dev < 0 or dev != cur():
        raise ValueError(f"x is on {x.device}: expected the current GPU")
    if x.is_contiguous():
        stride = K
    elif x.stride(1) == 1 or K == 1:
        stride = x.stride(0) if T > 1 else K
    else:
        raise ValueError(f"x: the values of a row have to be neighbours, got strides {x.stride()}")
    return dev, x.data_ptr(), stride, kind, _tensor("w", w, x.dtype, (N, K), dev), T, N, K


def dense_16(x, w, *, bias=None, activation: str = "none", residual=None, y=None, y_q8_1=None, stream=None) -> None:
    """Projection act(x w^T + bias) + residual of bfloat16 or float16 rows
    x [T, K] by weights w [N, K] of the same type -> y [T, N] (float32,
    bfloat16 or float16) and/or y_q8_1 (uint8 [T, N/32, 36]).  bias is float32
    [N], residual [T, N] in float32, bfloat16 or float16 (it may be y);
    activation is one of ACTIVATIONS.  The rows of x, residual and y may lie
    apart (those of x by a multiple of 8 values)."""
    dev, xp, xs, kind, wp, T, N, K = _operands(x, w)
    _, f32, _, u8, kinds, _, raw = _TORCH
    rp = yp = qp = bp = None
    rk = rs = yk = ys = 0
    if residual is not None:
        rp, rk, rs = _strided("residual", residual, kinds, (T, N), dev)
    if y is not None:
        yp, yk, ys = _strided("y", y, kinds, (T, N), dev)
    if y_q8_1 is not None:
        qp = _tensor("y_q8_1", y_q8_1, u8, (T, N // 32, 36), dev)
    if bias is not None:
        bp = _tensor("bias", bias, f32, (N,), dev)
    rc = (_lib or lib()).lat_moe_dense_16(xp, xs, wp, kind, T, N, K, bp, _choice("activation", activation, ACTIVATIONS),
                                          rp, rk, rs, yp, yk, ys, qp, raw(dev) if stream is None else int(stream))
    if rc:
        _check(rc)


def gated_16(x, w, h, *, bias=None, activation: str = "silu", stream=None) -> None:
    """Gate and up projections of a gated block on bfloat16 or float16 rows
    x [T, K]: h = act(x gate^T + gate bias) * (x up^T + up bias).  w is [2F, K]
    of x's type, the gate rows first; bias float32 [2F]; h [T, F] in float32,
    bfloat16 or float16.  The rows of x and h may lie apart (those of x by a
    multiple of 8 values).  dense_16 with a residual is the block's other
    half."""
    dev, xp, xs, kind, wp, T, rows, K = _operands(x, w)
    _, f32, _, _, kinds, _, raw = _TORCH
    if rows % 2:
        raise ValueError(f"w: expected gate rows and as many up rows, got {rows} rows")
    F = rows // 2
    hp, hk, hs = _strided("h", h, kinds, (T, F), dev)
    bp = None if bias is None else _tensor("bias", bias, f32, (rows,), dev)
    rc = (_lib or lib()).lat_moe_gated_16(xp, xs, wp, kind, T, F, K, bp, _choice("activation", activation, ACTIVATIONS),
                                          hp, hk, hs, raw(dev) if stream is None else int(stream))
    if rc:
        _check(rc)


def version() -> int:
    return int(lib().lat_moe_version())
