"""The 8-bit linear layer (fp8_linear): its operators run together, as a layer and behind GroupNorm, against the
layer's formulas in 64 bits on the values that the codes stand for.

Tolerances. y: half a step of bf16 (2^-8) twice (z and y where an activation follows) plus the product's fp32 sums
(2^-17 of the sum of |a||b|). Gradients also go through codes: dz is held in codes, so dx and dW differ from the
formula by up to half an e4m3 step (2^-4, random in sign) of each of its terms; over n terms of one size the 2-norm
of the sum's error stays within 2^-4 of the 2-norm of the terms' own, sqrt(sum (a b)^2): checked at twice that on
every element's root mean square, that is on the tensor's 2-norm.
"""
import pytest
import torch

import transformer_norm_rope_b200 as gn
from transformer_norm_rope_b200 import fp8_linear as fl


def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def norm64(x, g, beta, norm, eps, gemma):
    if norm == "none":
        return x
    if norm == "rms":
        return x * (x.square().mean(-1, keepdim=True) + eps) ** -0.5 * (1 + g if gemma else g)
    mu = x.mean(-1, keepdim=True)
    return (x - mu) * ((x - mu).square().mean(-1, keepdim=True) + eps) ** -0.5 * g + beta


def values(q, s, tile=False):
    """what codes stand for, in double"""
    rows, cols = q.shape
    sx = s.double().repeat_interleave(128, 1)[:, :cols]
    if tile:
        sx = sx.repeat_interleave(128, 0)[:rows]
    return q.double() * sx


def layer(M, N, K, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = {"x": 1.5 * r(M, K) + 0.3, "W": r(N, K) / K ** 0.5, "g": 1 + 0.1 * r(K), "beta": 0.1 * r(K), "dy": r(M, N)}
    t = {k: v.to(torch.bfloat16).cuda() for k, v in t.items()}
    t["bias"] = (0.3 * r(N)).cuda()
    return t


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
@pytest.mark.parametrize("norm,gemma", [("none", False), ("ln", False), ("rms", False), ("rms", True)])
@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (37, 136, 264), (300, 520, 648), (1030, 2056, 1304)])
def test_layer(gpu, M, N, K, norm, gemma, act):
    t = layer(M, N, K)
    w = fl.prepare(t["W"])
    ng, nb = (None, None) if norm == "none" else (t["g"], t["beta"] if norm == "ln" else None)
    args = dict(norm=norm, g=ng, beta=nb, eps=1e-5, gemma=gemma, act=act)
    y, mean, rstd, z = fl.forward_keeping_z(t["x"], w, t["bias"], **args)
    y2, _, _ = fl.forward(t["x"], fl.prepare(t["W"], training=False), t["bias"], **args)
    q, s, _, _ = gn.norm_quant_fp8(t["x"], ng, nb, 1e-5, norm=norm, gemma=gemma)
    a, b = values(q, s), values(w.q, w.scale, tile=True)
    z64 = a @ b.t() + t["bias"].double()
    acc = 2.0 ** -17 * (a.abs() @ b.abs().t() + t["bias"].double().abs())
    assert ((z.double() - z64).abs() <= 2.0 ** -8 * z64.abs() + acc).all()
    v = act64(z64, act)
    for out in (y, y2):
        assert ((out.double() - v).abs() <= 2.0 ** -8 * v.abs() + (1.2 * (2.0 ** -8 * z64.abs() + acc) + 2.0 ** -11 * z64.abs() if act != "none" else acc)).all()

    dx, dg, dbeta, dW, dbias = fl.backward(t["x"], w, z, t["dy"], mean=mean, rstd=rstd, **args)
    # dz from the z that was kept; dW and dxn as the formula gives them on dz and the layer's operands
    zz = z.double().clone().requires_grad_(True)
    (dz,) = torch.autograd.grad((act64(zz, act) * t["dy"].double()).sum(), zz)
    assert ((dbias.double() - dz.sum(0)).abs() <= 2e-5 * dz.abs().sum(0) + 1e-6).all()
    xn = norm64(t["x"].double(), t["g"].double(), t["beta"].double(), norm, 1e-5, gemma)
    dW64 = dz.t() @ xn
    terms = (dz.square().t() @ xn.square()).sum().sqrt()  # 2-norm of all the terms
    # two operands in codes and xn through bf16: 2^-4 twice, random over the tokens
    assert (dW.double() - dW64).norm() <= 2 * 2.0 ** -4 * terms * 2 ** 0.5
    dxn64 = dz @ b
    xx, gg, bb = (v.double().clone().requires_grad_(True) for v in (t["x"], t["g"], t["beta"]))
    grads = torch.autograd.grad((norm64(xx, gg, bb, norm, 1e-5, gemma) * dxn64).sum(), (xx, gg, bb), allow_unused=True)
    dterms = (dz.square() @ b.square()).sum().sqrt()
    scale = 1.0 if norm == "none" else float((rstd.double().max() * (1 + t["g"].double().abs().max())))
    assert (dx.double() - grads[0]).norm() <= (2 * 2.0 ** -4 * dterms + 2 * 2.0 ** -8 * dxn64.norm()) * scale
    if norm != "none":
        assert (dg.double() - grads[1]).norm() <= (2 * 2.0 ** -4 * dterms + 2 * 2.0 ** -8 * dxn64.norm()) * float(xn.abs().max())
    if norm == "ln":
        assert (dbeta.double() - grads[2]).norm() <= (2 * 2.0 ** -4 * dterms + 2 * 2.0 ** -8 * dxn64.norm()) * M ** 0.5
    else:
        assert dbeta is None
    assert gpu.device_error() == 0


def odd_layer(M, N, K, seed=0):
    """layer() with x and W on rows of whole 16 bytes, at any width"""
    t = layer(M, N, K, seed)
    return {k: gn.empty_rows(v.shape, v.dtype, v.device).copy_(v) if k in ("x", "W") else v for k, v in t.items()}


def check_gradients(t, w, z, dy, mean, rstd, grads, norm, gemma, act):
    """The layer's gradients against the same formulas in 64 bits on the codes that the layer itself makes of dz and of
    the normalised rows (what those codes are of is checked apart), so that only roundings are left:
    * dW: fp32 sums, 2^-24 (M + M / 128 + 4) of the magnitudes;
    * dxn is bf16, half a step 2^-8 of each value, and the product's sums 2^-24 (N + N / 128 + 4) of the magnitudes: e;
    * dbeta = sum dxn, dg = sum dxn x^: e of each term, and 2e-5 of the magnitudes for the sums and for x^;
    * dx = rstd P(dxn g') with P a projection for each row: 2-norm of rstd max|g'| e, half a step of dx, and 2e-5 of
      rstd |dxn g'| for the evaluation. Without a norm dx is dxn.
    A gradient of zeros must not pass: each tolerance is below half of the gradient's own 2-norm."""
    dx, dg, dbeta, dW, dbias = grads
    M, N = z.shape
    q, s, qt, st, db = gn.act_grad_quant_fp8(z, dy, epilogue=act)
    if norm == "ln":
        xn = gn.layernorm_fwd(t["x"], t["g"], t["beta"], 1e-5)[0]
    elif norm == "rms":
        xn = gn.rmsnorm_fwd(t["x"], t["g"], 1e-5, gemma=gemma)[0]
    else:
        xn = t["x"]
    xt, xts = gn.quant_fp8(xn, by_rows=False, transposed=True)

    def holds(got, ref, tol, what, norms=False):
        assert got.shape == ref.shape and torch.isfinite(got).all(), what
        d = (got.double() - ref).abs()
        assert d.norm() <= tol.norm() if norms else (d <= tol).all(), f"{what}: {d.norm():.3g} off, {tol.norm():.3g} allowed"
        assert tol.norm() <= 0.5 * ref.norm(), f"{what}: the tolerance {tol.norm():.3g} says nothing about {ref.norm():.3g}"

    a, b = values(qt, st), values(xt, xts)
    holds(dW, a @ b.t(), 2.0 ** -24 * (M + M / 128 + 4) * (a.abs() @ b.abs().t()), "dW")
    if dbias is not None:
        assert torch.equal(dbias, db)
    a, b = values(q, s), values(w.qt, w.scale_t, tile=True)
    dxn = a @ b.t()
    e = 2.0 ** -8 * dxn.abs() + 2.0 ** -24 * (N + N / 128 + 4) * (a.abs() @ b.abs().t())
    if norm == "none":
        return holds(dx, dxn, e, "dx")
    x, g = t["x"].double(), t["g"].double() + (1 if gemma else 0)
    mu = x.mean(1, keepdim=True) if norm == "ln" else 0
    r = ((x - mu).square().mean(1, keepdim=True) + 1e-5) ** -0.5
    xh, gg = (x - mu) * r, dxn * g
    m2 = (gg * xh).mean(1, keepdim=True)
    dx64 = r * (gg - xh * m2 - (gg.mean(1, keepdim=True) if norm == "ln" else 0))
    holds(dx, dx64, r * g.abs().max() * e + 2.0 ** -8 * dx64.abs() + 2e-5 * r * gg.abs(), "dx", norms=True)
    holds(dg, (dxn * xh).sum(0), ((e + 2e-5 * dxn.abs()) * xh.abs()).sum(0), "dg")
    if norm == "ln":
        holds(dbeta, dxn.sum(0), (e + 2e-5 * dxn.abs()).sum(0), "dbeta")
    else:
        assert dbeta is None


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
@pytest.mark.parametrize("norm,gemma", [("none", False), ("ln", False), ("rms", True)])
@pytest.mark.parametrize("M,N,K", [(70, 300, 264), (33, 129, 200), (300, 333, 133), (1, 300, 264), (40, 1, 72), (2, 7, 136)])
def test_widths_that_are_not_whole_16_bytes(gpu, M, N, K, norm, gemma, act):
    """The product pads its rows at such widths: keeping z, the backward on a contiguous gradient, and autograd."""
    t = odd_layer(M, N, K)
    ng, nb = (None, None) if norm == "none" else (t["g"], t["beta"] if norm == "ln" else None)
    args = dict(norm=norm, g=ng, beta=nb, eps=1e-5, gemma=gemma, act=act)
    w = fl.prepare(t["W"])
    y, mean, rstd, z = fl.forward_keeping_z(t["x"], w, t["bias"], **args)
    assert y.shape == z.shape == (M, N)
    q, s, _, _ = gn.norm_quant_fp8(t["x"], ng, nb, 1e-5, norm=norm, gemma=gemma)
    a, b = values(q, s), values(w.q, w.scale, tile=True)
    z64 = a @ b.t() + t["bias"].double()
    tol = 2.0 ** -8 * z64.abs() + 2.0 ** -24 * (K + K / 128 + 5) * (a.abs() @ b.abs().t() + t["bias"].double().abs())
    assert ((z.double() - z64).abs() <= tol).all()
    v = act64(z.double(), act)  # y: the activation of the z that was kept, half a step and 2^-11 |z| for its hardware tanh
    assert ((y.double() - v).abs() <= 2.0 ** -8 * v.abs() + (2.0 ** -11 * z.double().abs() if act != "none" else 0)).all()

    assert t["dy"].is_contiguous()
    grads = fl.backward(t["x"], w, z, t["dy"], mean=mean, rstd=rstd, **args)
    dy = gn.empty_rows((M, N), torch.bfloat16, "cuda").copy_(t["dy"])
    if M > 1:  # one row's norms leave too few values for the 2-norms of check_gradients
        check_gradients(t, w, z, dy, mean, rstd, grads, norm, gemma, act)
    again = fl.backward(t["x"], w, z, dy, mean=mean, rstd=rstd, **args)
    assert all(p is None and q is None or torch.equal(p, q) for p, q in zip(grads, again))

    leaves = {k: t[k].detach().requires_grad_(True) for k in ("x", "W")}  # (clone() would pack their rows)
    bias = t["bias"].clone().requires_grad_(True)
    out = fl.Fp8LinearFunction.apply(leaves["x"], leaves["W"], bias, ng, nb, norm, 1e-5, gemma, act)
    assert torch.equal(out, y)
    out.backward(t["dy"])
    assert torch.equal(leaves["x"].grad, grads[0]) and torch.equal(leaves["W"].grad, grads[3].bfloat16()) and torch.equal(bias.grad, grads[4])
    leaves["x"].grad = leaves["W"].grad = None
    fl.Fp8LinearFunction.apply(leaves["x"], leaves["W"], None, ng, nb, norm, 1e-5, gemma, act).sum().backward()  # an expanded gradient
    assert torch.isfinite(leaves["x"].grad).all() and torch.isfinite(leaves["W"].grad).all()
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
@pytest.mark.parametrize("norm,gemma", [("none", False), ("ln", False), ("rms", False), ("rms", True)])
@pytest.mark.parametrize("M,N,K", [(37, 136, 264), (300, 520, 648), (1030, 2056, 1304)])
def test_gradients_on_the_layers_own_codes(gpu, M, N, K, norm, gemma, act):
    t = layer(M, N, K)
    ng, nb = (None, None) if norm == "none" else (t["g"], t["beta"] if norm == "ln" else None)
    args = dict(norm=norm, g=ng, beta=nb, eps=1e-5, gemma=gemma, act=act)
    w = fl.prepare(t["W"])
    _, mean, rstd, z = fl.forward_keeping_z(t["x"], w, t["bias"], **args)
    check_gradients(t, w, z, t["dy"], mean, rstd, fl.backward(t["x"], w, z, t["dy"], mean=mean, rstd=rstd, **args), norm, gemma, act)


@pytest.mark.gpu
@pytest.mark.parametrize("act,d1,d2,d3", [("silu", 1.1, 0.5, 0.309), ("gelu_tanh", 1.13, 0.798, 0.777)])
def test_bias_gradient_against_differences(gpu, act, d1, d2, d3):
    """Central differences of f(bias) = sum(y dy) through the layer itself, along v = sign(dbias), where the derivative
    sum |dbias| is at its largest. Off by at most (d1 to d3: the largest slope, curvature and third derivative):
    * the rounding of each y to bf16, 2^-8 |y| <= 2^-8 (|y0| + d1 h), over h: sum |dy| of it;
    * the third order, h^2 / 6 d3 sum |dy|;
    * dbias comes from z rounded to bf16: d2 2^-8 |z| sum |dy|; and 1 % of all that for fp32 sums.
    A bias gradient of zeros must not pass."""
    M, N, K, h = 16, 256, 512, 0.25
    t = layer(M, N, K, seed=3)
    w = fl.prepare(t["W"])
    dy = t["dy"].double()
    f = lambda d: (fl.forward(t["x"], w, d, act=act)[0].double() * dy).sum()  # noqa: E731
    y, _, _, z = fl.forward_keeping_z(t["x"], w, t["bias"], act=act)
    dbias = fl.backward(t["x"], w, z, t["dy"], act=act)[4].double()
    v = dbias.sign().float()
    num = (f(t["bias"] + h * v) - f(t["bias"] - h * v)) / (2 * h)
    ana = dbias.abs().sum()
    off = 2.0 ** -8 * (y.double().abs() + d1 * h) / h + h * h / 6 * d3 + d2 * 2.0 ** -8 * z.double().abs()
    tol = 1.01 * (off * dy.abs()).sum()
    assert tol <= 0.25 * num.abs(), f"the tolerance {tol:.3g} says nothing about {num:.3g}"
    assert (num - ana).abs() <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("act,d1,d2,d3", [("none", 1.0, 0.0, 0.0), ("silu", 1.1, 0.5, 0.309), ("gelu_tanh", 1.13, 0.798, 0.777)])
def test_weight_gradient_against_differences(gpu, act, d1, d2, d3):
    """Central differences through the layer itself as the scales of W's 128 x 128 blocks move by 1 +- h, each block in
    the direction that adds to f = sum(y dy): W's values move along V, its blocks times their directions, and z with
    them by exactly h zV, zV = x V^T (its codes are those of x). The derivative is sum(dW V). Off by
    * at most, as for the bias: (2^-8 (|y| + d1 h |zV|) / h + h^2 / 6 d3 |zV|^3) |dy| and d2 2^-8 |z zV dy|, summed;
    * the codes of dz and x in dW, half a step 2^-4 of each of dW's terms, two operands: independent roundings, so four
      times the 2-norm of the terms |dz x V|, 2^-4 sqrt(2 / 3) each (a rounding's spread is its half step over sqrt 3).
    A weight gradient of zeros must not pass."""
    M, N, K, h = 2, 512, 640, 0.125
    t = layer(M, N, K, seed=5)
    w = fl.prepare(t["W"])
    dy = t["dy"].double()
    y, _, _, z = fl.forward_keeping_z(t["x"], w, t["bias"], act=act)
    dW = fl.backward(t["x"], w, z, t["dy"], act=act)[3].double()
    W = values(w.q, w.scale, tile=True)
    per_block = (dW * W).reshape(N // 128, 128, K // 128, 128).sum((1, 3))
    c = per_block.sign()
    V = W * c.repeat_interleave(128, 0).repeat_interleave(128, 1)
    f = lambda k: (fl.forward(t["x"], w._replace(scale=w.scale * (1 + k * c).float()), t["bias"], act=act)[0].double() * dy).sum()  # noqa: E731
    num, ana = (f(h) - f(-h)) / (2 * h), per_block.abs().sum()
    q, s, _, _ = gn.norm_quant_fp8(t["x"], norm="none")
    x = values(q, s)
    zV = x @ V.t()
    off = (2.0 ** -8 * (y.double().abs() + d1 * h * zV.abs()) / h + h * h / 6 * d3 * zV.abs() ** 3 + d2 * 2.0 ** -8 * (z.double() * zV).abs())
    zz = z.double().clone().requires_grad_(True)
    (dz,) = torch.autograd.grad((act64(zz, act) * dy).sum(), zz)
    codes = 4 * 2.0 ** -4 * (2 / 3) ** 0.5 * (dz.square() * (x.square() @ V.square().t())).sum().sqrt()
    tol = 1.01 * (off * dy.abs()).sum() + codes
    assert tol <= 0.4 * num.abs(), f"the tolerance {tol:.3g} says nothing about {num:.3g}"
    assert (num - ana).abs() <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("dt,K", [("bf16", 16384), ("bf16", 16392), ("bf16", 20480), ("f32", 8192), ("f32", 8196), ("f32", 20480)])
@pytest.mark.parametrize("M", [3, 140])
def test_rows_wider_than_a_norm_takes(gpu, M, K, dt):
    """Without a norm in front any width is taken, forward and (bf16) backward; with one a row is at most 32 KiB."""
    N = 72
    t = odd_layer(M, N, K)  # (8196 bf16 values are not whole 16 bytes)
    x = t["x"] if dt == "bf16" else t["x"].float()
    w = fl.prepare(t["W"])
    y, mean, rstd = fl.forward(x, w, t["bias"])
    q, s = gn.quant_fp8(x)
    a, b = values(q, s), values(w.q, w.scale, tile=True)
    v = a @ b.t() + t["bias"].double()
    tol = 2.0 ** -8 * v.abs() + 2.0 ** -24 * (K + K / 128 + 5) * (a.abs() @ b.abs().t() + t["bias"].double().abs())
    assert mean is None and rstd is None and ((y.double() - v).abs() <= tol).all()
    if dt == "bf16":
        _, _, _, z = fl.forward_keeping_z(x, w, t["bias"])
        check_gradients(t, w, z, t["dy"], None, None, fl.backward(x, w, z, t["dy"]), "none", False, "none")
    if K * x.element_size() > 32768:
        with pytest.raises(gn.GnError) as e:
            fl.forward(x, w, norm="ln")
        assert e.value.status == gn.GN_ERR_UNSUPPORTED
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("norm", ["none", "ln", "rms"])
@pytest.mark.parametrize("N", [64, 300])
def test_no_tokens(gpu, N, norm, act):
    """A batch without tokens: empty y and dx, zeros for the parameters' gradients, by calls and by autograd."""
    K = 136
    t = odd_layer(0, N, K)
    ng, nb = (None, None) if norm == "none" else (t["g"], t["beta"] if norm == "ln" else None)
    args = dict(norm=norm, g=ng, beta=nb, eps=1e-5, act=act)
    w = fl.prepare(t["W"])
    junk = torch.full((N * K,), 5.0, device="cuda")  # what the allocator hands out next is not zero already
    del junk
    y, mean, rstd, z = fl.forward_keeping_z(t["x"], w, t["bias"], **args)
    assert y.shape == z.shape == (0, N) and fl.forward(t["x"], w, t["bias"], **args)[0].shape == (0, N)
    dx, dg, dbeta, dW, dbias = fl.backward(t["x"], w, z, t["dy"], mean=mean, rstd=rstd, **args)
    assert dx.shape == (0, K) and dW.shape == (N, K) and dbias.shape == (N,)
    assert all((v == 0).all() for v in (dW, dbias, dg, dbeta) if v is not None)
    assert (dg is None) == (norm == "none") and (dbeta is None) == (norm != "ln")
    x, W = (t[k].detach().requires_grad_(True) for k in ("x", "W"))
    fl.Fp8LinearFunction.apply(x, W, t["bias"], ng, nb, norm, 1e-5, False, act).sum().backward()
    assert x.grad.shape == (0, K) and (W.grad == 0).all()
    assert gpu.device_error() == 0


@pytest.mark.gpu
def test_autograd_function_and_its_graph(gpu):
    """The autograd form gives the module's gradients; a second layer's captured forward and backward replay to the
    same bits while the first one's eager graph lives on (of other leaves: a capture of the same leaves' backward
    would touch state that the eager graph holds)."""
    t = layer(260, 392, 520)
    leaves = {k: t[k].clone().requires_grad_(True) for k in ("x", "W", "g", "beta")}
    bias = t["bias"].bfloat16().requires_grad_(True)
    y = fl.Fp8LinearFunction.apply(leaves["x"], leaves["W"], bias, leaves["g"], leaves["beta"], "ln", 1e-5, False, "silu")
    y.backward(t["dy"])
    w = fl.prepare(t["W"])
    args = dict(norm="ln", g=t["g"], beta=t["beta"], act="silu")
    y2, mean, rstd, z = fl.forward_keeping_z(t["x"], w, bias.detach().float(), **args)
    dx, dg, dbeta, dW, dbias = fl.backward(t["x"], w, z, t["dy"], mean=mean, rstd=rstd, **args)
    assert torch.equal(y.detach(), y2) and torch.equal(leaves["x"].grad, dx) and torch.equal(leaves["W"].grad, dW.bfloat16())
    assert torch.equal(leaves["g"].grad, dg.bfloat16()) and torch.equal(leaves["beta"].grad, dbeta.bfloat16())
    assert torch.equal(bias.grad, dbias.bfloat16())

    def step():
        y, mean, rstd, z = fl.forward_keeping_z(t["x"], w, t["bias"], **args)
        return (y,) + tuple(fl.backward(t["x"], w, z, t["dy"], mean=mean, rstd=rstd, **args))

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_gradients_against_differences(gpu):
    """With the codes fixed the layer is linear in them: the directional derivative of sum(y dy) along the bias is
    exact up to bf16 (2^-8 of the magnitudes), and dW along a direction that keeps every code's block scale matches
    the difference of two forwards within the codes' rounding."""
    M, N, K = 64, 128, 256
    t = layer(M, N, K, seed=3)
    w = fl.prepare(t["W"])
    f = lambda d: (fl.forward(t["x"], w, d, act="silu")[0].double() * t["dy"].double()).sum()  # noqa: E731
    y, _, _, z = fl.forward_keeping_z(t["x"], w, t["bias"], act="silu")
    _, _, _, dW, dbias = fl.backward(t["x"], w, z, t["dy"], act="silu")
    v, h = torch.randn(N, device="cuda"), 0.25
    num = (f(t["bias"] + h * v) - f(t["bias"] - h * v)) / (2 * h)
    ana = (dbias.double() * v.double()).sum()
    mags = (t["dy"].double().abs() * (y.double().abs() * 2.0 ** -8 / h + h ** 2 * 0.2)).square().sum().sqrt() * v.double().abs().max() ** 3
    assert (num - ana).abs() <= 2 * mags + 0.02 * (dbias.double().norm() * v.double().norm()) / N ** 0.5
    # along W: the layer is linear in W's values, so the derivative of sum(z dy) along V is sum((a V^T) dy)
    q, s, _, _ = gn.norm_quant_fp8(t["x"], norm="none")
    V = torch.randn(N, K, device="cuda", dtype=torch.float64)
    zz = z.double().clone().requires_grad_(True)
    (dz,) = torch.autograd.grad((act64(zz, "silu") * t["dy"].double()).sum(), zz)
    num = ((values(q, s) @ V.t()) * dz).sum()
    ana = (dW.double() * V).sum()
    assert (num - ana).abs() <= 4 * 2.0 ** -4 * 2 ** 0.5 * (dz.square().t() @ t["x"].double().square()).sum().sqrt()


@pytest.mark.gpu
def test_groupnorm_in_front_of_the_layer(gpu):
    """An image block's projection: GroupNorm with SiLU over [N, H, W, C], then the 8-bit layer on its positions,
    and the way back to the image's gradient."""
    N, H, W, C, F, G = 2, 12, 11, 160, 264, 16
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    x, gw, gb, Wt, dy = r(N, H, W, C), 1 + 0.1 * r(C), 0.1 * r(C), r(F, C) / C ** 0.5, r(N * H * W, F)
    w = fl.prepare(Wt)
    n, mean, rstd = gn.groupnorm_fwd(x, G, gw, gb, epilogue="silu")
    y, _, _, z = fl.forward_keeping_z(n.view(-1, C), w)
    dn, _, _, dW, _ = fl.backward(n.view(-1, C), w, z, dy, want_dbias=False)
    dx, dgw, dgb = gn.groupnorm_bwd(x, G, gw, gb, mean, rstd, dn.view_as(n), epilogue="silu")

    xx, ww, bb, W64 = (v.double().clone().requires_grad_(True) for v in (x, gw, gb, Wt))
    xg = xx.reshape(N, H * W, G, C // G)
    mu = xg.mean((1, 3), keepdim=True)
    zz = ((xg - mu) * (((xg - mu) ** 2).mean((1, 3), keepdim=True) + 1e-5) ** -0.5).reshape(N * H * W, C) * ww + bb
    out = (zz * torch.sigmoid(zz)) @ W64.t()
    want = torch.autograd.grad((out * dy.double()).sum(), (xx, ww, bb, W64))
    # every operand of the three products has gone through codes: 2^-4 of each term at most, two operands, random
    for got, ref in ((y, out.detach()), (dx, want[0]), (dgw, want[1]), (dgb, want[2]), (dW, want[3])):
        assert rel(got, ref) <= 2 * 2.0 ** -4 * 2 ** 0.5
    assert gpu.device_error() == 0


def test_helper_refusals(monkeypatch):
    w = fl.Weight(torch.zeros(1), torch.zeros(1), None, None)
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="transpose"):
        fl.backward(x, w, x, x)
    w = fl.Weight(torch.zeros(1), torch.zeros(1), torch.zeros(1), torch.zeros(1))
    with pytest.raises(ValueError, match="norm"):
        fl.backward(x, w, x, x, norm="group")
    with pytest.raises(ValueError, match="norm weight"):
        fl.backward(x, w, x, x, norm="rms")
    w = fl.Weight(torch.zeros(1), torch.zeros(1), None, None)
    with pytest.raises(ValueError, match="M, K"):
        fl.forward(torch.zeros(2, 4, 8), w)


class OfDevice1(torch.Tensor):
    """A CPU tensor that says it lives on the second GPU."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))


class TwoGpus:
    """torch with two devices that only remember which of them is current; outputs are made on the CPU."""

    def __init__(self):
        self.current, outer = 0, self

        class device:
            def __init__(self, d):
                self.d = d.index

            def __enter__(self):
                self.before, outer.current = outer.current, self.d

            def __exit__(self, *exc):
                outer.current = self.before

        self.cuda = type("cuda", (), {"current_device": staticmethod(lambda: outer.current), "device": device})

    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, *shape, device=None, **kw):
        return torch.empty(*shape, **kw).as_subclass(OfDevice1)

    def empty_strided(self, *shape, device=None, **kw):
        return torch.empty_strided(*shape, **kw).as_subclass(OfDevice1)


@pytest.mark.parametrize("norm", ["none", "ln", "rms"])
def test_every_call_runs_on_the_tensors_device(monkeypatch, norm):
    """x on the second device while the first is current: every launch of the layer, forward and backward, goes to
    the second one's current stream (the streams' handles stand for their devices here)."""
    gpus, calls = TwoGpus(), []
    monkeypatch.setattr(gn, "_TORCH", gpus)
    monkeypatch.setattr(gn, "_WORKSPACE", {})
    monkeypatch.setattr(gn, "_stream", lambda stream=None: gpus.current)
    for f in gn.SIGNATURES:
        if gn.SIGNATURES[f][0] is gn._st:
            monkeypatch.setattr(gn, f, lambda *a, f=f: calls.append((f, a[-1], gpus.current)) or gn.GN_OK)
        elif f.endswith("_workspace"):
            monkeypatch.setattr(gn, f, lambda *a: 16)
    M, N, K = 32, 64, 128
    t = {k: torch.zeros(s, dtype=torch.bfloat16).as_subclass(OfDevice1) for k, s in dict(x=(M, K), W=(N, K), g=(K,), beta=(K,), dy=(M, N)).items()}
    args = dict(norm=norm, g=None if norm == "none" else t["g"], beta=t["beta"] if norm == "ln" else None, act="silu")
    w = fl.prepare(t["W"])
    y, mean, rstd, z = fl.forward_keeping_z(t["x"], w, **args)
    fl.backward(t["x"], w, z, t["dy"], mean=mean, rstd=rstd, **args)
    assert gpus.current == 0 and {"gn_act_fwd", "gn_linear_fp8", "gn_quant_fp8"} <= {c[0] for c in calls}
    assert all(stream == 1 and current == 1 for _, stream, current in calls), [c for c in calls if c[1:] != (1, 1)]
