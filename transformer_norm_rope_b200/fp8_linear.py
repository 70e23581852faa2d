"""A linear layer, with a row normalization in front of it if wanted, on 8-bit operands.

y = act(norm(x) W^T + bias) with norm(x) and W in e4m3, one fp32 scale for each 128 values of a row of
norm(x) and for each 128 x 128 block of W: the 8-bit form of ``norm_linear`` (Janus-Pro inference page,
section 4.1; HY-Motion optimization page, section 3.1, whose quantisation section asks for FP8). Unlike
there the norm weight is not folded into W: the normalised rows are what is quantised, in the same pass
that normalises them.

Forward: ``gn_norm_quant_fp8`` (norm + codes), ``gn_linear_fp8`` (product, bias, activation).

Backward, with z = norm(x) W^T + bias and the codes taken for the values they stand for (the rounding to
codes has no gradient of its own):
  * dz = dy act'(z), quantised along its rows and along the tokens, and dbias: ``gn_quant_fp8``, one pass;
  * dxn = dz W: ``gn_linear_fp8`` on dz's rows and W's transpose (made once with W's codes);
  * dW = dz^T xn: ``gn_linear_fp8`` on dz transposed and the normalised rows, quantised along the tokens,
    fp32, a scale per row of either operand;
  * dx, dg, dbeta: the normalization's backward with dxn as the gradient of its output.
This module only orders the calls and allocates their outputs.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import transformer_norm_rope_b200 as gn


class Weight(NamedTuple):
    """A layer's weight W [N, K] in 8 bits: codes and scales, and those of its transpose (for dx; None if
    the weight was prepared for the forward only)."""

    q: object
    scale: object
    qt: Optional[object]
    scale_t: Optional[object]


def prepare(W, training: bool = True) -> Weight:
    """W [N, K] (bf16 or fp32) as its 8-bit form. Run it once per weight update."""
    if training:
        return Weight(*gn.quant_fp8(W, tile=True, transposed=True))
    return Weight(*gn.quant_fp8(W, tile=True), None, None)


def _act(z, act):
    """act(z) in z's layout: the product pads rows whose width is not whole 16 bytes, and the elementwise kernel
    takes the padding (whatever it holds) along."""
    if z.is_contiguous():
        return gn.act_fwd(z, epilogue=act)
    y = gn._empty(z.shape, z.stride(), z.dtype, z.device)
    flat = ((z.shape[0] - 1) * z.stride(0) + z.shape[1],)
    gn.act_fwd(z.as_strided(flat, (1,)), epilogue=act, out=y.as_strided(flat, (1,)))
    return y


def _whole_rows(t):
    """t [M, N] with its rows on 16-byte boundaries: t itself, or a copy (a gradient that autograd hands over is
    contiguous, or expanded, whatever its width)."""
    es = t.element_size()
    if t.dim() != 2 or (t.stride(1) == 1 and t.data_ptr() % 16 == 0
                        and (t.shape[0] <= 1 or (t.stride(0) >= t.shape[1] and t.stride(0) * es % 16 == 0))):
        return t
    return gn.empty_rows(t.shape, t.dtype, t.device).copy_(t)


def forward(x, weight: Weight, bias=None, norm: str = "none", g=None, beta=None, eps: float = 1e-5, gemma: bool = False,
            act: str = "none"):
    """y [M, N] bf16 = act(norm(x) W^T + bias) for x [M, K] (bf16 or, without a backward, fp32; bias fp32 [N])
    -> (y, mean or None, rstd or None). Rows of at most 32 KiB behind a norm, of any width without one."""
    if x.dim() != 2:
        raise ValueError(f"x {tuple(x.shape)} must be [M, K]: take its rows together")
    if norm == "none" and x.shape[1] * x.element_size() > 32768:  # no statistics, so any width: the same codes by tiles
        (q, s), mean, rstd = gn.quant_fp8(x), None, None
    else:
        q, s, mean, rstd = gn.norm_quant_fp8(x, g, beta, eps, norm=norm, gemma=gemma)
    return gn.linear_fp8(q, s, weight.q, weight.scale, bias, epilogue=act), mean, rstd


def forward_keeping_z(x, weight: Weight, bias=None, norm: str = "none", g=None, beta=None, eps: float = 1e-5,
                      gemma: bool = False, act: str = "none"):
    """The same layer keeping its pre-activation for the backward -> (y, mean, rstd, z) (y is z itself when
    act is "none")."""
    z, mean, rstd = forward(x, weight, bias, norm, g, beta, eps, gemma)
    return (z if act == "none" else _act(z, act)), mean, rstd, z


def backward(x, weight: Weight, z, dy, norm: str = "none", g=None, beta=None, mean=None, rstd=None, eps: float = 1e-5,
             gemma: bool = False, act: str = "none", want_dbias: bool = True):
    """Gradients of sum(dy * y) from the pre-activation and the statistics that ``forward_keeping_z`` kept ->
    (dx [M, K] bf16, dg, dbeta (fp32 [K], None where the norm has none), dW [N, K] fp32, dbias [N] fp32 or None)."""
    torch = gn._torch()
    if weight.qt is None:
        raise ValueError("the weight was prepared without its transpose: prepare(W, training=True)")
    if norm not in ("none", "ln", "rms"):
        raise ValueError(f"norm {norm!r}: 'none', 'ln' or 'rms'")
    if norm == "rms" and g is None:
        raise ValueError("the RMSNorm backward needs the norm weight g")
    q, s, qt, st, dbias = gn.act_grad_quant_fp8(z, _whole_rows(dy), epilogue=act, want_db=want_dbias)
    dxn = gn.linear_fp8(q, s, weight.qt, weight.scale_t)
    if norm == "ln":
        xn, _, _ = gn.layernorm_fwd(x, g, beta, eps, save_stats=False)
    elif norm == "rms":
        xn, _ = gn.rmsnorm_fwd(x, g, eps, gemma=gemma, save_stats=False)
    else:
        xn = x
    if x.shape[0] == 0:  # dW is a sum over no tokens
        dW = torch.zeros((z.shape[1], x.shape[1]), dtype=torch.float32, device=x.device)
    else:
        xt, xts = gn.quant_fp8(xn, by_rows=False, transposed=True)
        dW = gn.linear_fp8(qt, st, xt, xts, out_dtype=torch.float32)
    if norm == "ln":
        dx, dg, dbeta = gn.layernorm_bwd(x, g, beta, mean, rstd, dxn)
        return dx, dg, dbeta, dW, dbias
    if norm == "rms":
        dx, dg = gn.rmsnorm_bwd(x, g, rstd, dxn, gemma=gemma)
        return dx, dg, None, dW, dbias
    return dxn, None, None, dW, dbias


def _function_class():
    torch = gn._torch()

    class _Fp8Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, W, bias, g, beta, norm, eps, gemma, act):
            weight = prepare(W)
            d = None if bias is None else bias.float()
            y, mean, rstd, z = forward_keeping_z(x, weight, d, norm, g, beta, eps, gemma, act)
            ctx.save_for_backward(x, g, beta, mean, rstd, z, weight.qt, weight.scale_t)
            ctx.cfg = (norm, eps, gemma, act, W.dtype, None if bias is None else bias.dtype)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, g, beta, mean, rstd, z, qt, scale_t = ctx.saved_tensors
            norm, eps, gemma, act, w_dtype, b_dtype = ctx.cfg
            dx, dg, dbeta, dW, dbias = backward(x, Weight(None, None, qt, scale_t), z, dy, norm, g, beta, mean, rstd,
                                                eps, gemma, act, want_dbias=b_dtype is not None)

            def cast(t, like):
                return None if t is None or like is None else t.to(like.dtype)

            return (dx, dW.to(w_dtype), None if b_dtype is None else dbias.to(b_dtype), cast(dg, g), cast(dbeta, beta), None,
                    None, None, None)

    return _Fp8Linear


_FUNCTION = None


class Fp8LinearFunction:
    """torch.autograd.Function form for x [M, K] and W [N, K] in bf16: quantises W on every call and saves
    x, the statistics, the pre-activation and W's transposed codes."""

    @staticmethod
    def apply(x, W, bias=None, g=None, beta=None, norm: str = "none", eps: float = 1e-5, gemma: bool = False,
              act: str = "none"):
        global _FUNCTION
        if _FUNCTION is None:
            _FUNCTION = _function_class()
        return _FUNCTION.apply(x, W, bias, g, beta, norm, eps, gemma, act)


__all__ = ["Weight", "prepare", "forward", "forward_keeping_z", "backward", "Fp8LinearFunction"]
