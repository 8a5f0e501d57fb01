"""Quantize-then-GEMM for one linear-layer GEMM, on top of the C ABI.

Buffer management and call sequencing only (torch allocates device memory,
every computation is a libpbs kernel).  Which copy each GEMM consumes
("How to optimize Transformer-based models for low-precision training",
"Using autocast mode vs pre-quantized mode": Fprop, Dgrad and Wgrad are
separate GEMMs), with X [M, K], W stored [N, K], dY [M, N]:

  fprop: A = X row copy,  B = W row copy
  dgrad: A = dY row copy, B = W col copy
  wgrad: A = X col copy,  B = dY col copy

Format roles: per-tensor FP8 uses E4M3 for X and W, E5M2 for dY;
sub-channel FP8 (fp32 or power-of-two block scales), channel-wise FP8 (one
fp32 scale per row of each copy) and MXFP8 use E4M3; NVFP4 and MXFP4 use E2M1.  Weights
take 2D blocks (128x128 sub-channel, 16x16 NVFP4; MXFP4 keeps 1x32 blocks
along the contraction axis for every operand); the sub-channel pairings
take 1x128 blocks on every tensor (1D1D) or 128x128 on every tensor (2D2D).  NVFP4 and MXFP4 apply the
random Hadamard transform to both Wgrad operands and stochastic rounding
to dY.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass

import torch

from . import (PBS_COL, PBS_DGRAD, PBS_FLAG_RHT16, PBS_FLAG_SR, PBS_FMT_BF16, PBS_FMT_E2M1,
               PBS_FMT_E4M3, PBS_FMT_E5M2, PBS_FMT_F32, PBS_FPROP, PBS_RECIPE_BF16,
               PBS_RECIPE_FP8_BLOCK128, PBS_RECIPE_FP8_BLOCK128_1D1D, PBS_RECIPE_FP8_BLOCK128_2D2D,
               PBS_RECIPE_FP8_BLOCK128_POW2,
               PBS_RECIPE_FP8_CHANNEL, PBS_RECIPE_FP8_CURRENT,
               PBS_RECIPE_FP8_DELAYED,
               PBS_RECIPE_MXFP4, PBS_RECIPE_MXFP8, PBS_RECIPE_NVFP4, PBS_ROW, PBS_WGRAD, pbs_amax,
               pbs_cast,
               pbs_delayed_init, pbs_delayed_scale, pbs_delayed_scale_inv, pbs_delayed_state_bytes,
               pbs_delayed_update, pbs_gemm, pbs_gemm_amax, pbs_layernorm, pbs_layernorm_grad,
               pbs_layernorm_grad_bytes, pbs_linear_distill, pbs_linear_distill_grad, pbs_linear_loss_bytes,
               pbs_linear_xent, pbs_linear_xent_grad, pbs_muon, pbs_orthogonalize,
               pbs_orthogonalize_bytes, pbs_qk_norm_rope, pbs_qk_norm_rope_grad,
               pbs_qk_norm_rope_grad_bytes, pbs_scale_from_amax)

RECIPES = {
    "bf16": PBS_RECIPE_BF16,
    "fp8_current": PBS_RECIPE_FP8_CURRENT,
    "fp8_delayed": PBS_RECIPE_FP8_DELAYED,
    "fp8_block128": PBS_RECIPE_FP8_BLOCK128,
    "mxfp8": PBS_RECIPE_MXFP8,
    "nvfp4": PBS_RECIPE_NVFP4,
    "mxfp4": PBS_RECIPE_MXFP4,
    "fp8_channel": PBS_RECIPE_FP8_CHANNEL,
    "fp8_block128_1d1d": PBS_RECIPE_FP8_BLOCK128_1D1D,
    "fp8_block128_2d2d": PBS_RECIPE_FP8_BLOCK128_2D2D,
    "fp8_block128_pow2": PBS_RECIPE_FP8_BLOCK128_POW2,
}
# sources that take 2D blocks, per recipe
TWO_D = {"fp8_block128": ("w",), "nvfp4": ("w",), "fp8_block128_2d2d": ("x", "w", "dy"),
         "fp8_block128_pow2": ("w",)}
SUBCHANNEL = ("fp8_block128", "fp8_block128_1d1d", "fp8_block128_2d2d")
LAYOUTS = {"fprop": PBS_FPROP, "dgrad": PBS_DGRAD, "wgrad": PBS_WGRAD}
ROLES = {"fprop": (("x", "row"), ("w", "row")),
         "dgrad": (("dy", "row"), ("w", "col")),
         "wgrad": (("x", "col"), ("dy", "col"))}
FMAX = {PBS_FMT_E4M3: 448.0, PBS_FMT_E5M2: 57344.0}
NVFP4_FMAX = 2688.0
RHT_SEED = 42
SR_SEED = 42
HIST_LEN = 16


@dataclass
class QTensor:
    """One quantized copy, contraction axis last: codes [rows, cols(/2)]."""
    recipe: str
    fmt: int
    rows: int
    cols: int
    codes: torch.Tensor
    scales: torch.Tensor | None = None
    tensor_scale_inv: torch.Tensor | None = None
    weight_2d: bool = False


def fmt_for(recipe, src):
    if recipe in ("fp8_current", "fp8_delayed"):
        return PBS_FMT_E5M2 if src == "dy" else PBS_FMT_E4M3
    if recipe in ("nvfp4", "mxfp4"):
        return PBS_FMT_E2M1
    if recipe == "bf16":
        return PBS_FMT_BF16
    return PBS_FMT_E4M3


def _empty_copy(recipe, rows, cols, w2d, device):
    """Allocate codes / scales for one copy of stored shape [rows, cols]."""
    if recipe == "nvfp4":
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        sc = (torch.empty((rows // 16, cols // 16), dtype=torch.uint8, device=device) if w2d
              else torch.empty((rows, cols // 16), dtype=torch.uint8, device=device))
        return codes, sc
    if recipe == "mxfp4":
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        return codes, torch.empty((rows, cols // 32), dtype=torch.uint8, device=device)
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=device)
    if recipe == "fp8_block128_pow2":      # one 32-bit word per block: its E8M0 code in every byte
        sc = (torch.empty((rows // 128, cols // 128), dtype=torch.int32, device=device) if w2d
              else torch.empty((rows, cols // 128), dtype=torch.int32, device=device))
    elif recipe in SUBCHANNEL:
        sc = (torch.empty((rows // 128, cols // 128), dtype=torch.float32, device=device) if w2d
              else torch.empty((rows, cols // 128), dtype=torch.float32, device=device))
    elif recipe == "mxfp8":
        sc = torch.empty((rows, cols // 32), dtype=torch.uint8, device=device)
    elif recipe == "fp8_channel":
        sc = torch.empty((rows,), dtype=torch.float32, device=device)
    else:
        sc = None
    return codes, sc


class DelayedState:
    """Device-resident amax history for one tensor (delayed scaling)."""

    def __init__(self, fmt, device, hist_len=HIST_LEN, stream=None):
        self.fmt = fmt
        self.fmax = FMAX[fmt]
        n = pbs_delayed_state_bytes(hist_len)
        self.buf = torch.empty(((n + 15) // 16) * 16, dtype=torch.uint8, device=device)
        self.amax = torch.zeros(1, dtype=torch.float32, device=device)
        pbs_delayed_init(self.buf, hist_len, stream)

    @property
    def scale_inv(self):
        """The state's scale_inv word as a one-element device tensor (a view)."""
        return self.buf[4:8].view(torch.float32)

    @property
    def scale_ptr(self):
        return pbs_delayed_scale(self.buf)

    @property
    def scale_inv_ptr(self):
        return pbs_delayed_scale_inv(self.buf)

    def update(self, stream=None):
        pbs_delayed_update(self.buf, self.amax, self.fmax, stream)


class Workspace:
    """Reusable per-tensor scalars so repeated quantization allocates nothing."""

    def __init__(self, device):
        self.device = device
        self._cache = {}

    def scalars(self, key, n=3):
        t = self._cache.get(key)
        if t is None:
            t = torch.zeros(n, dtype=torch.float32, device=self.device)
            self._cache[key] = t
        return t


def _copy_scalar(dst, src, stream=None):
    """Stream-ordered device-to-device copy of one fp32 (no arithmetic)."""
    if stream is None:
        dst.copy_(src)
        return
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    with torch.cuda.stream(stream):
        dst.copy_(src)


def _new_scalars(dev):
    return torch.zeros(3, dtype=torch.float32, device=dev)   # amax, scale, scale_inv


def _cast_into(recipe, x, src, pass_, rmask, bufs, scal, w2d, state, stream, known_amax):
    """The amax / scale / cast calls of one recipe into the copies `bufs`
    (row codes, row scales, col codes, col scales; unused ones None).
    Returns the device tensor scale_inv the copies carry (or None)."""
    R, C = x.shape
    fmt = fmt_for(recipe, src)
    rec = RECIPES[recipe]
    row_c, row_s, col_c, col_s = bufs
    if recipe == "fp8_current":
        am = known_amax if known_amax is not None else scal[0:1]
        if known_amax is None:
            pbs_amax(x, R, C, 0, 0, am, stream)
        pbs_scale_from_amax(am, FMAX[fmt], scal[1:2], scal[2:3], stream)
        pbs_cast(rec, x, R, C, fmt, rmask, 0, 0, 0, scal[1:2], None, row_c, row_s, col_c, col_s, stream)
        return scal[2:3]
    if recipe == "fp8_delayed":
        if state is None:
            raise ValueError("delayed scaling needs a DelayedState")
        pbs_cast(rec, x, R, C, fmt, rmask, 0, 0, 0, state.scale_ptr, state.amax, row_c, row_s,
                 col_c, col_s, stream)
        # the copy keeps the scale it was cast with: a stream-ordered 4-byte
        # device copy of the state's scale_inv, which later updates replace
        _copy_scalar(scal[2:3], state.scale_inv, stream)
        return scal[2:3]
    if recipe in SUBCHANNEL + ("mxfp8", "fp8_channel", "fp8_block128_pow2"):
        pbs_cast(rec, x, R, C, fmt, rmask, int(w2d), 0, 0, None, None, row_c, row_s, col_c, col_s, stream)
        return None
    if recipe == "nvfp4":
        rht = pass_ == "wgrad"
        flags = (PBS_FLAG_RHT16 if rht else 0) | (PBS_FLAG_SR if src == "dy" else 0)
        if known_amax is not None and rht:
            raise ValueError("the Hadamard-transformed tensor's amax is not the producer's")
        am = known_amax if known_amax is not None else scal[0:1]
        if known_amax is None:
            pbs_amax(x, R, C, PBS_FLAG_RHT16 if rht else 0, RHT_SEED, am, stream)
        pbs_scale_from_amax(am, NVFP4_FMAX, scal[1:2], scal[2:3], stream)
        seed = SR_SEED if src == "dy" else RHT_SEED
        if rht and src == "dy" and RHT_SEED != SR_SEED:
            raise ValueError("one seed drives both the RHT signs and SR")
        pbs_cast(rec, x, R, C, fmt, rmask, int(w2d), flags, seed, scal[1:2], None, row_c, row_s,
                 col_c, col_s, stream)
        return scal[2:3]
    if recipe == "mxfp4":
        flags = (PBS_FLAG_RHT16 if pass_ == "wgrad" else 0) | (PBS_FLAG_SR if src == "dy" else 0)
        if flags == (PBS_FLAG_RHT16 | PBS_FLAG_SR) and RHT_SEED != SR_SEED:
            raise ValueError("one seed drives both the RHT signs and SR")
        pbs_cast(rec, x, R, C, fmt, rmask, 0, flags, SR_SEED if src == "dy" else RHT_SEED, None, None,
                 row_c, row_s, col_c, col_s, stream)
        return None
    raise ValueError(recipe)


def quantize(recipe, x, src, orient, pass_, state=None, out=None, ws=None, stream=None, known_amax=None):
    """Quantize bf16 tensor ``x`` [R, C] for use as the ``src`` operand of ``pass_``.

    Returns a QTensor whose stored shape is [R, C] (row) or [C, R] (col).
    ``out`` may be a QTensor from an earlier call with the same shape, reused
    in place.  ``state`` is a DelayedState for the delayed recipe.
    ``known_amax`` (a device fp32 of one element holding max |x|, e.g. from
    the epilogue of the GEMM that produced x) replaces the amax pass of the
    per-tensor current-scaling and NVFP4 recipes; not with the Hadamard
    transform, whose maximum is taken over the transformed values.
    """
    R, C = x.shape
    rows, cols = (R, C) if orient == "row" else (C, R)
    if recipe == "bf16":
        if orient != "row":
            raise ValueError("bf16 operands are consumed in natural storage")
        return QTensor("bf16", PBS_FMT_BF16, R, C, x)
    w2d = src in TWO_D.get(recipe, ())
    if out is None:
        codes, sc = _empty_copy(recipe, rows, cols, w2d, x.device)
        scal = _new_scalars(x.device)
        out = QTensor(recipe, fmt_for(recipe, src), rows, cols, codes, sc, scal[2:3], w2d)
        out._scal = scal
    bufs = ((out.codes, out.scales, None, None) if orient == "row" else (None, None, out.codes, out.scales))
    rmask = PBS_ROW if orient == "row" else PBS_COL
    out.tensor_scale_inv = _cast_into(recipe, x, src, pass_, rmask, bufs, out._scal, w2d, state, stream,
                                      known_amax)
    return out


def quantize_both(recipe, x, src, state=None, outs=None, stream=None, known_amax=None):
    """Row and col copies of bf16 ``x`` [R, C] from one read of x (pbs_cast
    with both orientations), for a tensor whose two copies get the same
    treatment: every recipe's weights, and the activations and gradients of
    every recipe but the 4-bit ones (whose col copies take the Hadamard
    transform, and whose gradients round stochastically).  Returns
    (row QTensor [R, C], col QTensor [C, R]); ``outs`` may be such a pair,
    reused in place."""
    if recipe == "bf16":
        raise ValueError("bf16 operands are consumed in natural storage")
    if recipe in ("nvfp4", "mxfp4") and src != "w":
        raise ValueError("the 4-bit recipes' activation and gradient copies differ (Hadamard, SR)")
    R, C = x.shape
    w2d = src in TWO_D.get(recipe, ())
    if outs is None:
        rc, rs = _empty_copy(recipe, R, C, w2d, x.device)
        cc, cs = _empty_copy(recipe, C, R, w2d, x.device)
        scal = _new_scalars(x.device)
        fmt = fmt_for(recipe, src)
        outs = (QTensor(recipe, fmt, R, C, rc, rs, scal[2:3], w2d), QTensor(recipe, fmt, C, R, cc, cs, scal[2:3], w2d))
        outs[0]._scal = outs[1]._scal = scal
    row, col = outs
    tsi = _cast_into(recipe, x, src, "fprop", PBS_ROW | PBS_COL, (row.codes, row.scales, col.codes, col.scales),
                     row._scal, w2d, state, stream, known_amax)
    row.tensor_scale_inv = col.tensor_scale_inv = tsi
    return row, col


def gemm(recipe, pass_, A, B, M, N, K, out_dtype=torch.bfloat16, C=None, stream=None, c_amax=None):
    """C[M, N] for one pass from the two operands (QTensor for quantized recipes).

    For the bf16 recipe A and B are the natural-storage bf16 tensors of the
    pass (fprop: X, W; dgrad: dY, W; wgrad: X, dY).  With ``c_amax`` (a
    device fp32 tensor of one element) the epilogue also writes max |C| there
    (pbs_gemm_amax).
    """
    dev = (A.codes if isinstance(A, QTensor) else A).device
    if C is None:
        C = torch.empty((M, N), dtype=out_dtype, device=dev)
    c_fmt = PBS_FMT_BF16 if C.dtype == torch.bfloat16 else PBS_FMT_F32
    rec = RECIPES[recipe]
    lay = LAYOUTS[pass_]
    if recipe == "bf16":
        a = A.codes if isinstance(A, QTensor) else A
        b = B.codes if isinstance(B, QTensor) else B
        args = (rec, lay, M, N, K, a, PBS_FMT_BF16, None, None, b, PBS_FMT_BF16, None, None, C, c_fmt)
    else:
        args = (rec, lay, M, N, K, A.codes, A.fmt, A.scales, A.tensor_scale_inv, B.codes, B.fmt,
                B.scales, B.tensor_scale_inv, C, c_fmt)
    if c_amax is None:
        pbs_gemm(*args, stream)
    else:
        pbs_gemm_amax(*args, c_amax, stream)
    return C


def pass_dims(pass_, M_tok, K_in, N_out):
    """(M, N, K) of the GEMM for a linear layer with X [M_tok, K_in], W [N_out, K_in]."""
    return {"fprop": (M_tok, N_out, K_in),
            "dgrad": (M_tok, K_in, N_out),
            "wgrad": (K_in, N_out, M_tok)}[pass_]


def sources(pass_, x, w, dy):
    return {"x": x, "w": w, "dy": dy}


def quantize_pass(recipe, pass_, x, w, dy, states=None, outs=None, stream=None):
    """Quantize both operands of one pass.  Returns (A, B)."""
    src = {"x": x, "w": w, "dy": dy}
    (sa, oa), (sb, ob) = ROLES[pass_]
    if recipe == "bf16":
        return src[sa], src[sb]
    states = states or {}
    outs = outs or {}
    A = quantize(recipe, src[sa], sa, oa, pass_, states.get(sa), outs.get("A"), stream=stream)
    B = quantize(recipe, src[sb], sb, ob, pass_, states.get(sb), outs.get("B"), stream=stream)
    return A, B


# ---------------------------------------------------------------------------
# the ends of a step: the norm ahead of a linear layer, the losses of the head
#
# Outputs and workspaces are allocated on the call's device and stream.  A call
# on another stream than the current one (``stream``) is ordered against the
# other streams' work, and its tensors are kept until it is done, by the
# caller, as for torch's own operators under ``torch.cuda.stream``.
# ---------------------------------------------------------------------------
FMT_OF = {torch.bfloat16: PBS_FMT_BF16, torch.float32: PBS_FMT_F32}
BF16_F32 = (torch.bfloat16, torch.float32)
F32 = (torch.float32,)
I64 = (torch.int64,)


def _matrix(name, t, device, shape=None):
    """Checks a [rows, cols] operand of bf16 or fp32 whose rows are contiguous; returns (format, row stride)."""
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: want shape {tuple(shape) if shape else '[rows, cols]'}, got {tuple(t.shape)}")
    fmt = FMT_OF.get(t.dtype)
    if fmt is None:
        raise ValueError(f"{name}: want bf16 or fp32, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, want {device}")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    if rows <= 1:
        ld = max(cols, 1)
    elif ld < cols:
        raise ValueError(f"{name}: rows overlap (row stride {ld}, {cols} columns)")
    return fmt, ld


def _vector(name, t, n, dtypes, device):
    """Checks a contiguous vector of n values; returns its address (None: none)."""
    if t is None:
        return None
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name}: want {n} contiguous values, got shape {tuple(t.shape)}, strides {t.stride()}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: got {t.dtype}, want {' or '.join(str(d) for d in dtypes)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, want {device}")
    return t.data_ptr()


def _given(**tensors):
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} is missing")


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """The context that runs a call on `device` and on `stream` (None: the
    device's current stream), so that what the call allocates belongs there."""
    if device.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    if stream is None:
        return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors on {device}")
    return torch.cuda.stream(stream)


def _current(device):
    """The address of the device's current stream, without building a Stream."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def layernorm(x, gamma=None, beta=None, eps=1e-5, out_dtype=None, y=None, amax=None, stream=None):
    """Layer norm of the rows of ``x`` [R, C] (bf16 or fp32).  Returns (y,
    mean [R], rstd [R]), the statistics in fp32 for ``layernorm_grad``.

    ``gamma`` / ``beta`` [C]: both bf16 or both fp32 (None: 1 / 0).  ``y`` may
    be given ([R, C], bf16 or fp32; ``x`` itself for in place, else apart from
    it), else it is allocated in ``out_dtype`` (None: x's).  ``amax`` (a device fp32 of one
    element) receives max |y| as stored: ``quantize(..., known_amax=amax)``
    then needs no pass of its own.
    """
    dev = x.device
    x_fmt, ldx = _matrix("x", x, dev)
    R, C = x.shape
    if C < 1:
        raise ValueError("x: no columns")
    g, b = _vector("gamma", gamma, C, BF16_F32, dev), _vector("beta", beta, C, BF16_F32, dev)
    if g is not None and b is not None and gamma.dtype != beta.dtype:
        raise ValueError("gamma and beta must have the same type")
    w = gamma if g is not None else beta
    a = _vector("amax", amax, 1, F32, dev)
    if y is None:
        if out_dtype is not None and out_dtype not in FMT_OF:
            raise ValueError(f"out_dtype: want bf16 or fp32, got {out_dtype}")
    else:
        if out_dtype not in (None, y.dtype):
            raise ValueError("out_dtype is not y's")
        y_fmt, ldy = _matrix("y", y, dev, x.shape)
    with _on(dev, stream):
        if y is None:
            y = torch.empty((R, C), dtype=out_dtype or x.dtype, device=dev)
            y_fmt, ldy = FMT_OF[y.dtype], C
        mean = torch.empty(R, dtype=torch.float32, device=dev)
        rstd = torch.empty(R, dtype=torch.float32, device=dev)
        pbs_layernorm(x.data_ptr(), x_fmt, R, C, ldx, g, b, PBS_FMT_F32 if w is None else FMT_OF[w.dtype], eps,
                      y.data_ptr(), y_fmt, ldy, mean.data_ptr(), rstd.data_ptr(), a, _current(dev))
    return y, mean, rstd


def layernorm_grad(dy, x, gamma, mean, rstd, dx=None, stream=None):
    """Gradients of ``layernorm``: returns (dx [R, C] in x's type, dgamma [C],
    dbeta [C] in fp32) from dy [R, C] (bf16 or fp32), the forward's x, gamma
    (None: 1) and the statistics it returned.  ``dx`` may be given: x or dy
    itself, or apart from them."""
    dev = x.device
    x_fmt, ldx = _matrix("x", x, dev)
    R, C = x.shape
    if C < 1:
        raise ValueError("x: no columns")
    y_fmt, lddy = _matrix("dy", dy, dev, x.shape)
    g = _vector("gamma", gamma, C, BF16_F32, dev)
    _given(mean=mean, rstd=rstd)
    m, r = _vector("mean", mean, R, F32, dev), _vector("rstd", rstd, R, F32, dev)
    lddx = C
    if dx is not None:
        d_fmt, lddx = _matrix("dx", dx, dev, x.shape)
        if d_fmt != x_fmt:
            raise ValueError(f"dx: want x's type, got {dx.dtype}")
    with _on(dev, stream):
        if dx is None:
            dx = torch.empty((R, C), dtype=x.dtype, device=dev)
        dgamma = torch.empty(C, dtype=torch.float32, device=dev)
        dbeta = torch.empty(C, dtype=torch.float32, device=dev)
        n = pbs_layernorm_grad_bytes(R, C)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        pbs_layernorm_grad(dy.data_ptr(), y_fmt, lddy, x.data_ptr(), x_fmt, ldx, R, C, g,
                           PBS_FMT_F32 if g is None else FMT_OF[gamma.dtype], m, r, dx.data_ptr(), lddx,
                           dgamma.data_ptr(), dbeta.data_ptr(), ws.data_ptr(), n, _current(dev))
    return dx, dgamma, dbeta


def _head(x, w):
    """Checks the head's operands; returns (tokens, vocab, hidden)."""
    for name, t in (("x", x), ("w", w)):
        if t.dim() != 2 or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name}: want a contiguous bf16 matrix, got {t.dtype} {tuple(t.shape)}, strides "
                             f"{t.stride()}")
    T, H = x.shape
    V = w.shape[0]
    if w.shape[1] != H or V < 1:
        raise ValueError(f"w {tuple(w.shape)} does not fit x {tuple(x.shape)}")
    if w.device != x.device:
        raise ValueError(f"w: on {w.device}, want {x.device}")
    return T, V, H


def _teacher(top_ids, top_logits, T, device):
    if (top_ids.dim() != 2 or top_ids.shape[0] != T or top_ids.shape[1] < 1 or not top_ids.is_contiguous() or
            top_ids.dtype != torch.int64):
        raise ValueError(f"top_ids: want contiguous int64 [{T}, top], got {top_ids.dtype} {tuple(top_ids.shape)}")
    if top_logits.shape != top_ids.shape or not top_logits.is_contiguous() or top_logits.dtype not in FMT_OF:
        raise ValueError(f"top_logits: want contiguous bf16 or fp32 {tuple(top_ids.shape)}, got {top_logits.dtype} "
                         f"{tuple(top_logits.shape)}")
    if top_ids.device != device or top_logits.device != device:
        raise ValueError(f"the teacher's tensors must be on {device}")
    return top_ids.shape[1]


def _loss(dev, stream, T, V, H, top, call):
    """Allocates a loss's outputs and workspace and makes the call."""
    with _on(dev, stream):
        n = pbs_linear_loss_bytes(T, V, H, top)[0]
        loss = torch.empty(T, dtype=torch.float32, device=dev)
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        call(loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), n, _current(dev))
    return loss, lse


def _loss_grad(dev, stream, T, V, H, top, piece, need_dx, need_dw, dw_dtype, call):
    """The same for a gradient."""
    if not (need_dx or need_dw):
        raise ValueError("neither dx nor dw is wanted")
    if dw_dtype not in FMT_OF:
        raise ValueError(f"dw_dtype: want bf16 or fp32, got {dw_dtype}")
    with _on(dev, stream):
        n = pbs_linear_loss_bytes(T, V, H, top, piece)[1]
        dx = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if need_dx else None
        dw = torch.empty((V, H), dtype=dw_dtype, device=dev) if need_dw else None
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        call(piece, dx, dw, FMT_OF[dw_dtype], ws.data_ptr(), n, _current(dev))
    return dx, dw


def linear_xent(x, w, targets, stream=None):
    """Softmax cross entropy of the logits x w^T, which are never kept: x
    [T, H] and w [V, H] bf16, ``targets`` [T] int64 (negative: the token is
    left out, its loss and lse are 0).  Returns (loss [T], lse [T]) in fp32;
    lse = log sum exp of a token's logits is what ``linear_xent_grad`` takes.
    """
    T, V, H = _head(x, w)
    _given(targets=targets)
    t = _vector("targets", targets, T, I64, x.device)
    return _loss(x.device, stream, T, V, H, 0,
                 lambda *a: pbs_linear_xent(x.data_ptr(), w.data_ptr(), T, V, H, t, *a))


def linear_xent_grad(dloss, x, w, targets, lse, piece=0, need_dx=True, need_dw=True, dw_dtype=torch.bfloat16,
                     stream=None):
    """Gradients of sum(dloss * loss) of ``linear_xent``: (dx [T, H] bf16, dw
    [V, H] in ``dw_dtype``), None for one that is not needed.  The workspace
    holds the logits' gradient for ``piece`` ids at a time (0: up to 1 GiB of
    it, or 2048 ids where those take more)."""
    T, V, H = _head(x, w)
    _given(dloss=dloss, targets=targets, lse=lse)
    t = _vector("targets", targets, T, I64, x.device)
    d, s = _vector("dloss", dloss, T, F32, x.device), _vector("lse", lse, T, F32, x.device)
    return _loss_grad(x.device, stream, T, V, H, 0, piece, need_dx, need_dw, dw_dtype,
                      lambda *a: pbs_linear_xent_grad(d, x.data_ptr(), w.data_ptr(), T, V, H, t, s, *a))


def linear_distill(x, w, top_ids, top_logits, temperature=1.0, stream=None):
    """Kullback-Leibler divergence from softmax(top_logits / temperature) over
    a teacher's stored logits to softmax(x w^T / temperature) over the whole
    vocabulary.  ``top_ids`` [T, k] int64 (negative: unused slot), ``top_logits``
    [T, k] bf16 or fp32.  Returns (loss [T], lse [T]) in fp32, both 0 for a
    token without used slots; no factor temperature^2 is applied."""
    T, V, H = _head(x, w)
    top = _teacher(top_ids, top_logits, T, x.device)
    return _loss(x.device, stream, T, V, H, top,
                 lambda *a: pbs_linear_distill(x.data_ptr(), w.data_ptr(), T, V, H, top_ids.data_ptr(),
                                               top_logits.data_ptr(), FMT_OF[top_logits.dtype], top, temperature, *a))


def linear_distill_grad(dloss, x, w, top_ids, top_logits, temperature, lse, piece=0, need_dx=True, need_dw=True,
                        dw_dtype=torch.bfloat16, stream=None):
    """Gradients of sum(dloss * loss) of ``linear_distill``, as
    ``linear_xent_grad`` returns them."""
    T, V, H = _head(x, w)
    top = _teacher(top_ids, top_logits, T, x.device)
    _given(dloss=dloss, lse=lse)
    d, s = _vector("dloss", dloss, T, F32, x.device), _vector("lse", lse, T, F32, x.device)
    return _loss_grad(x.device, stream, T, V, H, top, piece, need_dx, need_dw, dw_dtype,
                      lambda *a: pbs_linear_distill_grad(d, x.data_ptr(), w.data_ptr(), T, V, H, top_ids.data_ptr(),
                                                         top_logits.data_ptr(), FMT_OF[top_logits.dtype], top,
                                                         temperature, s, *a))


# ---------------------------------------------------------------------------
# the QKV projection's output: norm and rotation of the queries and keys
# ---------------------------------------------------------------------------
F64 = (torch.float64,)


def rope_frequencies(rot_dim, base=10000.0, device="cuda"):
    """base^(-2 i / rot_dim) for the pairs i of a rotation, fp64 [rot_dim / 2]:
    the angle a pair turns by from one position to the next."""
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError(f"rot_dim: want an even number, got {rot_dim}")
    return torch.tensor([float(base) ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], dtype=torch.float64,
                        device=device)


def _heads4(name, t, device, shape=None, dtype=None):
    """Checks a [batch, seq, heads, head_dim] tensor whose last axis is contiguous; returns its strides."""
    if t.dim() != 4 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: want shape {tuple(shape) if shape else '[batch, seq, heads, head_dim]'}, got "
                         f"{tuple(t.shape)}")
    if t.dtype not in FMT_OF or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name}: want {dtype or 'bf16 or fp32'}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, want {device}")
    sb, ss, sh, sd = t.stride()
    if sd != 1 and t.shape[3] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return sb, ss, sh


def _qk_common(q, k, q_weight, k_weight, positions, freqs, norm, eps):
    """Checks what the pass and its gradient share; returns (device, x format,
    (batch, seq, head_dim), the strides of q and k, heads, kv_heads, the call's
    arguments from the weights to interleaved, less that)."""
    if q is None:
        raise ValueError("q is missing")
    dev = q.device
    sq = _heads4("q", q, dev)
    B, S, H, D = q.shape
    sk, kv = None, 0
    if k is not None:
        kv = k.shape[2] if k.dim() == 4 else 0
        sk = _heads4("k", k, dev, torch.Size((B, S, kv, D)), q.dtype)
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    w = q_weight if q_weight is not None else k_weight
    qw, kw = _vector("q_weight", q_weight, D, BF16_F32, dev), _vector("k_weight", k_weight, D, BF16_F32, dev)
    if qw is not None and kw is not None and q_weight.dtype != k_weight.dtype:
        raise ValueError("q_weight and k_weight must have the same type")
    p, psb = None, 0
    if positions is not None:
        if positions.dtype != torch.int64 or positions.shape not in ((S,), (B, S)):
            raise ValueError(f"positions: want int64 [{S}] or [{B}, {S}], got {positions.dtype} {tuple(positions.shape)}")
        if positions.device != dev:
            raise ValueError(f"positions: on {positions.device}, want {dev}")
        if S > 1 and positions.stride(-1) != 1:
            raise ValueError("positions: the last axis must be contiguous")
        if positions.dim() == 2 and B > 1:
            psb = positions.stride(0)
            if psb != 0 and psb < S:
                raise ValueError("positions: rows overlap")
        p = positions.data_ptr()
    rot, f = 0, None
    if freqs is not None:
        rot = 2 * freqs.shape[0] if freqs.dim() == 1 else -1
        if rot < 0 or rot > D:
            raise ValueError(f"freqs: want at most {D // 2} values, got shape {tuple(freqs.shape)}")
        f = _vector("freqs", freqs, rot // 2, F64, dev)
    args = (qw, kw, PBS_FMT_F32 if w is None else FMT_OF[w.dtype], int(norm), float(eps), p, psb, f, rot)
    return dev, FMT_OF[q.dtype], (B, S, D), sq, sk, H, kv, args


def qk_norm_rope(q, k=None, q_weight=None, k_weight=None, positions=None, freqs=None, interleaved=False, eps=1e-6,
                 norm=True, q_out=None, k_out=None, out_dtype=None, stream=None):
    """RMS norm of each head of ``q`` [B, S, H, D] and ``k`` [B, S, Hk, D] (bf16
    or fp32; None: queries alone) and their rotation by position, in one pass.
    Returns (q_out, k_out).

    Any strides with a contiguous last axis: views of a packed projection, or
    ``t.transpose(1, 2)`` of [B, H, S, D], for the outputs too (``q_out``,
    ``k_out``: also q and k themselves), which are else allocated contiguous in
    ``out_dtype`` (None: q's).  ``q_weight`` / ``k_weight`` [D]: both bf16 or both
    fp32 (None: 1).  ``positions``: int64 [S] or [B, S] (None: 0 to S - 1).
    ``freqs``: fp64 [rot / 2] (``rope_frequencies``), the pairs' angle a position
    (None: no rotation); the first ``rot`` values of a head are turned, in pairs
    (i, i + rot / 2), or (2 i, 2 i + 1) if ``interleaved``.  ``norm=False``:
    rotation alone.
    """
    dev, x_fmt, (B, S, D), sq, sk, H, kv, args = _qk_common(q, k, q_weight, k_weight, positions, freqs, norm, eps)
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    given = q_out if q_out is not None else k_out
    if out_dtype is None:
        out_dtype = given.dtype if given is not None else q.dtype
    if out_dtype not in FMT_OF:
        raise ValueError(f"out_dtype: want bf16 or fp32, got {out_dtype}")
    oq = None if q_out is None else _heads4("q_out", q_out, dev, q.shape, out_dtype)
    ok = None if k_out is None else _heads4("k_out", k_out, dev, k.shape, out_dtype)
    with _on(dev, stream):
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=out_dtype, device=dev)
            oq = (S * H * D, H * D, D)
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=out_dtype, device=dev)
            ok = (S * kv * D, kv * D, D)
        kp, ko = (None, None) if k is None else (k.data_ptr(), k_out.data_ptr())
        pbs_qk_norm_rope(q.data_ptr(), sq, H, kp, sk, kv, x_fmt, B, S, D, *args, interleaved, q_out.data_ptr(), oq, ko, ok,
                         FMT_OF[out_dtype], _current(dev))
    return q_out, k_out


def qk_norm_rope_grad(dq, dk, q, k=None, q_weight=None, k_weight=None, positions=None, freqs=None, interleaved=False,
                      eps=1e-6, norm=True, dv=None, dq_out=None, dk_out=None, dv_out=None, amax=None, stream=None):
    """Gradients of ``qk_norm_rope``: returns (dq_out, dk_out in q's type,
    dq_weight [D], dk_weight [D] in fp32; None for k's without k) from ``dq``, ``dk``
    (the outputs' gradients, both bf16 or both fp32) and the forward's arguments.

    ``dq_out``, ``dk_out`` may be given (any strides; q / dq, k / dk themselves
    with the same type).  ``dv`` [B, S, Hk, D] (dq's type) is copied to ``dv_out``
    (q's type): with the three outputs as the parts of one packed tensor, that is
    the gradient of the projection's output, and ``amax`` (a device fp32 of one
    element) receives its max |value| as stored, for ``quantize(...,
    known_amax=amax)``.
    """
    dev, x_fmt, (B, S, D), sq, sk, H, kv, args = _qk_common(q, k, q_weight, k_weight, positions, freqs, norm, eps)
    if dq is None or (dk is None) != (k is None):
        raise ValueError("dq or dk is missing, or dk given without k")
    if k is None and dk_out is not None:
        raise ValueError("dk_out without k")
    if (dv is None) != (dv_out is None):
        raise ValueError("dv and dv_out go together")
    sdq = _heads4("dq", dq, dev, q.shape)
    sdk = None if k is None else _heads4("dk", dk, dev, k.shape, dq.dtype)
    sdv = odv = None
    if dv is not None:
        if k is None:
            raise ValueError("dv without k")
        sdv, odv = _heads4("dv", dv, dev, k.shape, dq.dtype), _heads4("dv_out", dv_out, dev, k.shape, q.dtype)
    oq = None if dq_out is None else _heads4("dq_out", dq_out, dev, q.shape, q.dtype)
    ok = None if dk_out is None else _heads4("dk_out", dk_out, dev, k.shape, q.dtype)
    a = _vector("amax", amax, 1, F32, dev)
    with _on(dev, stream):
        if dq_out is None:
            dq_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            oq = dq_out.stride()[:3]
        if k is not None and dk_out is None:
            dk_out = torch.empty(k.shape, dtype=q.dtype, device=dev)
            ok = dk_out.stride()[:3]
        dqw = torch.empty(D, dtype=torch.float32, device=dev)
        dkw = None if k is None else torch.empty(D, dtype=torch.float32, device=dev)
        n = pbs_qk_norm_rope_grad_bytes(B, S, D)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        pbs_qk_norm_rope_grad(dq, sdq, dk, sdk, dv, sdv, FMT_OF[dq.dtype], q, sq, H, k, sk, kv, x_fmt, B, S, D, *args,
                              interleaved, dq_out, oq, dk_out, ok, dv_out, odv, dqw, dkw, a, ws, n, _current(dev))
    return dq_out, dk_out, dqw, dkw


# ---------------------------------------------------------------------------
# the weights' update
# ---------------------------------------------------------------------------
# a, b, c of the Muon optimiser's five quintic steps
MUON_STEPS = ((3.4445, -4.7750, 2.0315),) * 5


def _matrices(name, t, device, shape=None, flip=False):
    """Checks a [rows, cols] or [batch, rows, cols] tensor of bf16 or fp32 with a contiguous last axis (with
    ``flip``: or the one before it); returns (format, row stride, batch stride, whether it lies transposed)."""
    if t.dim() not in (2, 3) or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: want shape {tuple(shape) if shape else '[rows, cols] or [batch, rows, cols]'}, got "
                         f"{tuple(t.shape)}")
    if t.dtype not in FMT_OF:
        raise ValueError(f"{name}: want bf16 or fp32, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, want {device}")
    rows, cols = t.shape[-2:]
    lr, lc = t.stride()[-2:]
    turned = flip and cols > 1 and lc != 1
    if turned:
        rows, cols, lr, lc = cols, rows, lc, lr
    if cols > 1 and lc != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    ld = max(cols, 1) if rows <= 1 else lr
    stride = t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else ld * max(rows, 1)
    return FMT_OF[t.dtype], ld, stride, turned


def orthogonalize(x, y=None, coefficients=MUON_STEPS, eps=1e-7, stream=None):
    """The nearest matrix with orthonormal rows or columns, approximately: X =
    x / (||x||_F + eps), then X <- a X + (b A + c A^2) X with A = X X^T (of the
    shorter side) for each (a, b, c) of ``coefficients``.  ``x`` [R, C] or [B, R,
    C] (each by itself), bf16 or fp32; returns bf16, ``y`` if given (any rows; x
    itself if that is bf16)."""
    dev = x.device
    x_fmt, ldx, sx, _ = _matrices("x", x, dev)
    B = x.shape[0] if x.dim() == 3 else 1
    R, C = x.shape[-2:]
    if y is not None:
        if y.dtype != torch.bfloat16:
            raise ValueError(f"y: want bf16, got {y.dtype}")
        _, ldy, sy, _ = _matrices("y", y, dev, x.shape)
        if y.data_ptr() == x.data_ptr() and x.numel() and (y.dtype != x.dtype or (ldy, sy) != (ldx, sx)):
            raise ValueError("y is on x's memory with another type or other strides")
    with _on(dev, stream):
        if y is None:
            y = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
            ldy, sy = max(C, 1), max(R, 1) * max(C, 1)
        n = pbs_orthogonalize_bytes(B, R, C)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        pbs_orthogonalize(x, x_fmt, ldx, sx, B, R, C, coefficients, eps, y, ldy, sy, ws, n, _current(dev))
    return y


def muon(w, momentum, grad, lr, beta=0.95, nesterov=True, weight_decay=0.0, scale=None, coefficients=MUON_STEPS, eps=1e-7,
         stream=None):
    """One step of Muon on ``w`` [R, C] or [B, R, C] (each matrix by itself),
    in place: momentum <- beta momentum + (1 - beta) grad; U = beta momentum +
    (1 - beta) grad (``nesterov``) or the momentum; w <- (1 - lr weight_decay) w -
    lr scale X with X = ``orthogonalize(U)``.  Returns w.

    ``w``, ``momentum`` and ``grad`` are bf16 or fp32 each, rows contiguous;
    ``grad`` may also lie transposed: what the Wgrad product writes, [in, out],
    is given as ``dw.t()``.  ``scale`` None: max(1, R / C)^0.5.  ``lr``: a number, or
    a device fp32 of one element (read when the work runs, so a captured graph
    follows a schedule)."""
    dev = w.device
    w_fmt, ldw, sw, _ = _matrices("w", w, dev)
    m_fmt, ldm, sm, _ = _matrices("momentum", momentum, dev, w.shape)
    g_fmt, ldg, sg, turned = _matrices("grad", grad, dev, w.shape, flip=True)
    B = w.shape[0] if w.dim() == 3 else 1
    R, C = w.shape[-2:]
    factor = None
    if isinstance(lr, torch.Tensor):
        factor, lr = _vector("lr", lr.reshape(-1), 1, F32, dev), 1.0
    if scale is None:
        scale = max(1.0, R / max(C, 1)) ** 0.5
    with _on(dev, stream):
        n = pbs_orthogonalize_bytes(B, R, C)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        pbs_muon(w, w_fmt, ldw, sw, momentum, m_fmt, ldm, sm, grad, g_fmt, turned, ldg, sg, B, R, C, beta, nesterov, lr, factor,
                 weight_decay, scale, coefficients, eps, ws, n, _current(dev))
    return w
