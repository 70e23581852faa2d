"""GroupNorm of channels-last images against its definition in 64 bits.

Tolerances, per element (u = half a step of the stored type: 2^-8 of the value in bf16, 2^-24 in fp32):
* y: u |y| + 2e-6 (|z| + |b| + 1) for the fp32 evaluation, plus 2^-11 |z| where bf16 rows use the
  hardware tanh (relative error 2^-11) or the approximate exponential.
* mean, rstd: sums of at most a few thousand fp32 terms joined in a tree: 4e-6 of (|mu| + sigma) and of rstd.
* dx: u |dx| + 8e-6 of the sum of its terms' magnitudes (+ 2^-9 |dy w s| for the approximate derivative).
* dw, db: 4e-6 (+ 2^-9) of the sum of the magnitudes of their terms.
"""
import pytest
import torch

import transformer_norm_rope_b200 as gn

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def make(N, S, C, dt, seed=0, ld=None, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = r(N, S, C) * (0.5 + r(N, 1, C).abs()) + spread * r(N, 1, C)
    t = {"x": x, "dy": r(N, S, C), "w": 1 + 0.1 * r(C), "b": 0.1 * r(C)}
    t = {k: v.to(DT[dt]) for k, v in t.items()}
    dev = {}
    for k, v in t.items():
        if k in ("x", "dy"):
            base = torch.zeros(v.shape[:-1] + (ld or C,), dtype=v.dtype, device="cuda")
            base[..., :C] = v.cuda()
            dev[k] = base[..., :C]
        else:
            dev[k] = v.cuda()
    return dev


def reference(t, G, eps, act, w=True, b=True):
    """Everything in double from the definition; gradients by autograd of that definition."""
    x = t["x"].double().clone().requires_grad_(True)
    N, S, C = x.shape
    wd = (t["w"].double() if w else torch.ones(C, dtype=torch.float64, device=x.device)).requires_grad_(True)
    bd = (t["b"].double() if b else torch.zeros(C, dtype=torch.float64, device=x.device)).requires_grad_(True)
    xg = x.reshape(N, S, G, C // G)
    mu = xg.mean(dim=(1, 3), keepdim=True)
    var = ((xg - mu) ** 2).mean(dim=(1, 3), keepdim=True)
    s = (var + eps) ** -0.5
    xhat = ((xg - mu) * s).reshape(N, S, C)
    z = xhat * wd + bd
    y = act64(z, act)
    dy = t["dy"].double()
    (gz,) = torch.autograd.grad((y * dy).sum(), z, retain_graph=True)
    dx, dw, db = torch.autograd.grad((y * dy).sum(), (x, wd, bd))
    d = dict(y=y, z=z, mean=mu.reshape(N, G), rstd=s.reshape(N, G), dx=dx, dw=dw, db=db, g=gz, xhat=xhat)
    return {k: v.detach() for k, v in d.items()}, wd.detach(), bd.detach()


def within(got, ref, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    over = (got - ref).abs() - tol
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.numel()} over the tolerance, worst by {over.max():.3g}"


def check(t, G, dt, act, eps=1e-5, w=True, b=True, shape=None):
    N, S, C = t["x"].shape
    ref, wd, bd = reference(t, G, eps, act, w, b)
    args = (t["w"] if w else None, t["b"] if b else None)
    x, dy = (t["x"], t["dy"]) if shape is None else (t["x"].view(shape), t["dy"].view(shape))
    y, mean, rstd = gn.groupnorm_fwd(x, G, *args, eps, epilogue=act)
    dx, dw, db = gn.groupnorm_bwd(x, G, *args, mean, rstd, dy, epilogue=act)
    assert y.shape == x.shape and dx.shape == x.shape and y.dtype == dx.dtype == DT[dt]
    u = HALF_STEP[dt]
    fast = dt == "bf16" and act != "none"
    rep = lambda v: v.repeat_interleave(C // G, dim=-1)[:, None, :]  # noqa: E731
    y_tol = u * ref["y"].abs() + 2e-6 * (ref["z"].abs() + bd.abs() + 1) + (2.0 ** -11 * ref["z"].abs() if fast else 0)
    within(y.reshape(N, S, C), ref["y"], y_tol, "y")
    within(mean, ref["mean"], 4e-6 * (ref["mean"].abs() + 1 / ref["rstd"]), "mean")
    within(rstd, ref["rstd"], 4e-6 * ref["rstd"], "rstd")
    sw = rep(ref["rstd"]) * wd.abs()
    terms = sw * ref["g"].abs() + rep(ref["rstd"]) * (rep((ref["g"] * wd).reshape(N, S, G, -1).abs().mean(dim=(1, 3)))
                                                      + ref["xhat"].abs() * rep((ref["g"] * wd * ref["xhat"]).reshape(N, S, G, -1).abs().mean(dim=(1, 3))))
    within(dx.reshape(N, S, C), ref["dx"], u * ref["dx"].abs() + 8e-6 * terms
           + (2.0 ** -9 * (sw * t["dy"].double().abs() + terms) if fast else 0), "dx")
    c = 4e-6 + (2.0 ** -9 if fast else 0)
    dya = t["dy"].double().abs()
    within(dw, ref["dw"], c * ((ref["g"].abs() + (dya if fast else 0)) * ref["xhat"].abs()).sum((0, 1)) + 1e-6, "dw")
    within(db, ref["db"], c * (ref["g"].abs() + (dya if fast else 0)).sum((0, 1)) + 1e-6, "db")


# (N, S, C, G): one position; one value a group (variance 0); groups that cross 16-byte vectors; one
# group; as many groups as channels; widths that end inside a vector; many small images; long images
SHAPES = [(1, 1, 64, 8), (2, 1, 8, 8), (1, 63, 320, 32), (3, 17, 30, 3), (2, 50, 40, 1), (2, 33, 24, 24), (2, 65, 77, 7),
          (33, 5, 64, 4), (1, 4099, 128, 32), (2, 1031, 640, 32), (1, 300, 1536, 16), (1, 20000, 64, 32), (2, 4096, 640, 32), (1, 70000, 64, 4), (2, 30001, 48, 3), (1, 9000, 520, 1),
          (1, 17, 8192, 2), (1, 40, 4104, 27), (300, 7, 32, 2), (3, 2500, 1032, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,S,C,G", SHAPES)
def test_groupnorm(gpu, N, S, C, G, dt, act):
    es = 2 if dt == "bf16" else 4
    ld = (C * es + 15) // 16 * 16 // es
    check(make(N, S, C, dt, ld=ld), G, dt, act)
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [2.0, 30.0])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,S,C,G", [(15, 1017, 3, 3), (13, 179, 9, 9), (40, 1017, 5, 1), (20, 5000, 9, 9), (30, 6000, 3, 1), (8, 3156, 42, 6), (4, 9000, 264, 24)])
def test_statistics_of_narrow_images(gpu, N, S, C, G, dt, spread):
    """Few channels put many threads on each: their join must not round the mean once a thread. 2-norms over the groups,
    in u = 2^-24, independent roundings (uniform, 0.58 u each) adding up in squares:
    * mean: the threads' (averaged), the slab's, the products and the tree of the join (with halves of its sums: 0.82
      together), the division: 1.3 u of |mu|, and as much of sigma for the deviations: 2 u (|mu| + sigma) allowed;
    * rstd: half of the variance's few u, the root and the division: 3 u;
    * y (fp32): the mean's error times rstd and w, and the rounding of (x - mu), of its product, of w and of the sum."""
    t = make(N, S, C, dt, ld=(C + 7) // 8 * 8, spread=spread, seed=3)
    ref, wd, bd = reference(t, G, 1e-5, "none")
    y, mean, rstd = gn.groupnorm_fwd(t["x"], G, t["w"], t["b"])
    u = 2.0 ** -24
    off = lambda got, v: (got.double() - v).norm()  # noqa: E731
    em = 2 * u * (ref["mean"].abs() + 1 / ref["rstd"])
    assert off(mean, ref["mean"]) <= em.norm(), f"mean: {off(mean, ref['mean']) / ref['mean'].norm() / u:.3g} u"
    assert off(rstd, ref["rstd"]) <= 3 * u * ref["rstd"].norm(), f"rstd: {off(rstd, ref['rstd']) / ref['rstd'].norm() / u:.3g} u"
    if dt == "f32":
        rep = lambda v: v.repeat_interleave(C // G, dim=-1)[:, None, :]  # noqa: E731
        tol = ((rep(em * ref["rstd"]) + 3 * 0.58 * u * ref["xhat"].abs()) * wd.abs() + 0.58 * u * ref["y"].abs()
               + 3 * u * ref["xhat"].abs() * wd.abs())  # the last term: rstd's
        assert off(y, ref["y"]) <= tol.norm(), f"y: {off(y, ref['y']) / ref['y'].norm() / u:.3g} u"
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,S,C,G", [(15, 1017, 3, 3), (13, 179, 9, 9), (8, 50000, 3, 3), (2, 30000, 40, 8), (8, 3156, 42, 6), (4, 9000, 264, 24), (1, 60000, 24, 24)])
def test_parameter_gradients_of_narrow_images(gpu, N, S, C, G, dt):
    """dw and db are sums over all positions: no part of them may be a long chain. Against the same formula in 64 bits on
    the saved statistics, 2-norms over the channels, in u = 2^-24 of the 2-norm of a channel's terms. A chain of K
    roundings of growing partial sums of independent terms leaves 0.58 sqrt(K / 2), a tree of L levels 0.58 sqrt(L): a
    thread's positions (under 30 here: 2.2), a lane's threads (16: 1.6), lanes (5 levels: 1.3), slabs (a chain of 8 and 7
    levels: 1.9), images (a chain of 15: 1.6), x^ and its product (1): 4.1 in squares; 6 allowed."""
    t = make(N, S, C, dt, ld=(C + 7) // 8 * 8, seed=5)
    _, mean, rstd = gn.groupnorm_fwd(t["x"], G, t["w"], t["b"])
    _, dw, db = gn.groupnorm_bwd(t["x"], G, t["w"], t["b"], mean, rstd, t["dy"])
    rep = lambda v: v.double().repeat_interleave(C // G, dim=-1)[:, None, :]  # noqa: E731
    dy, xh = t["dy"].double(), (t["x"].double() - rep(mean)) * rep(rstd)
    for got, terms, what in ((db, dy, "db"), (dw, dy * xh, "dw")):
        off = (got.double() - terms.sum((0, 1))).norm() / terms.square().sum((0, 1)).sqrt().norm() * 2 ** 24
        assert off <= 6, f"{what}: {off:.3g} u"
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("N,S,C,G", [(1, 63, 320, 32), (2, 50, 40, 1), (2, 65, 77, 7), (1, 4099, 128, 32), (2, 1031, 640, 32), (3, 2500, 1032, 2), (2, 9000, 520, 1)])
def test_activations_of_bf16_images_are_evaluated_in_fp32(gpu, N, S, C, G, act):
    """Half a step of bf16 and fp32 evaluation, nothing coarser, on chip and in two passes. With t = z (SiLU) or
    2 k (z + c z^3) (GeLU), p = sigmoid(t) and q = 1 - p:
    * y = z p: 2^-22 (|t| + 4) of the value for the exponential's argument and the functions' ulps; z's own
      2e-6 (|z| + |b| + 1), as in check(), times the largest slope, 1.13;
    * act' = p (1 + z q t'): the same relative part of each of its two terms, and z's error times the largest
      curvature, 0.8: e, which reaches dx, dw and db times dy and what multiplies it there; their sums and the
      rest as in check().
    An activation that is off by 2^-11 of 1 must not pass."""
    t = make(N, S, C, "bf16", ld=(C + 7) // 8 * 8)
    ref, wd, bd = reference(t, G, 1e-5, act)
    y, mean, rstd = gn.groupnorm_fwd(t["x"], G, t["w"], t["b"], epilogue=act)
    dx, dw, db = gn.groupnorm_bwd(t["x"], G, t["w"], t["b"], mean, rstd, t["dy"], epilogue=act)
    z, dy, xh, s = ref["z"], t["dy"].double().abs(), ref["xhat"].abs(), ref["rstd"].repeat_interleave(C // G, dim=-1)[:, None, :]
    k = (2 / torch.pi) ** 0.5
    u, du = (z, torch.ones_like(z)) if act == "silu" else (2 * k * (z + 0.044715 * z ** 3), 2 * k * (1 + 3 * 0.044715 * z ** 2))
    p = torch.sigmoid(u)
    ez, rel = 2e-6 * (z.abs() + bd.abs() + 1), 2.0 ** -22 * (u.abs() + 4)
    y_tol = 2.0 ** -8 * ref["y"].abs() + rel * ref["y"].abs() + 1.13 * ez
    within(y, ref["y"], y_tol, "y")
    coarse = z * (p + 2.0 ** -12)  # (1 + tanh) / 2 with the hardware tanh's error
    assert ((coarse - ref["y"]).abs() > y_tol).any()

    e = (rel * (p + (z * p * (1 - p) * du).abs()) + 0.8 * ez) * dy  # of g = dy act'
    group = lambda v: v.reshape(N, S, G, -1).mean(dim=(1, 3)).repeat_interleave(C // G, dim=-1)[:, None, :]  # noqa: E731
    gw, ew = ref["g"].abs() * wd.abs(), e * wd.abs()
    through = lambda v: s * (v + group(v) + xh * group(v * xh))  # noqa: E731
    within(dx, ref["dx"], 2.0 ** -8 * ref["dx"].abs() + 8e-6 * through(gw) + through(ew), "dx")
    within(dw, ref["dw"], ((4e-6 * ref["g"].abs() + e) * xh).sum((0, 1)) + 1e-6, "dw")
    within(db, ref["db"], (4e-6 * ref["g"].abs() + e).sum((0, 1)) + 1e-6, "db")
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("C,G", [(171, 1), (77, 7), (5, 5), (4104, 27), (1, 1)])
def test_one_position_at_any_width(gpu, C, G, dt, act):
    """One row: a contiguous tensor whatever its width, with nothing that steps by its stride."""
    t = make(1, 1, C, dt)
    check(t, G, dt, act)
    y, _, _ = gn.groupnorm_fwd(t["x"], G, t["w"], t["b"], epilogue=act)
    out = torch.full((1, 1, C + 1), 7.0, dtype=DT[dt], device="cuda")
    gn.groupnorm_fwd(t["x"], G, t["w"], t["b"], epilogue=act, out=out[..., :C])
    assert torch.equal(out[..., :C], y) and (out[..., C] == 7).all()
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("w,b", [(False, False), (True, False), (False, True)])
def test_absent_parameters(gpu, w, b):
    check(make(2, 100, 96, "bf16"), 6, "bf16", "silu", w=w, b=b)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_mean_keeps_the_variance(gpu, dt):
    """Channels whose mean is far above their spread, and a first position far from the others: the
    variance must not lose its bits to the mean's square."""
    t = make(2, 777, 64, dt, spread=0.0)
    t["x"] += 200.0
    t["x"][:, 0] -= 3000.0
    t["x"] = t["x"].contiguous()
    check(t, 8, dt, "none")


@pytest.mark.gpu
def test_strided_and_spatial(gpu):
    t = make(2, 12 * 13, 64, "bf16", ld=104)
    check(t, 16, "bf16", "silu")
    u = make(2, 12 * 13, 64, "bf16")
    check(u, 16, "bf16", "silu", shape=(2, 12, 13, 64))


@pytest.mark.gpu
def test_in_place_and_unsaved(gpu):
    t = make(2, 500, 64, "bf16")
    y, _, _ = gn.groupnorm_fwd(t["x"], 8, t["w"], t["b"], epilogue="silu")
    x = t["x"].clone()
    out, mean, rstd = gn.groupnorm_fwd(x, 8, t["w"], t["b"], epilogue="silu", out=x, save_stats=False)
    assert out is x and mean is None and rstd is None and torch.equal(x, y)
    _, mean, rstd = gn.groupnorm_fwd(t["x"], 8, t["w"], t["b"])
    dx, dw, db = gn.groupnorm_bwd(t["x"], 8, t["w"], t["b"], mean, rstd, t["dy"])
    dx2, dw2, db2 = gn.groupnorm_bwd(t["x"], 8, t["w"], t["b"], mean, rstd, t["dy"], want_wgrad=False)
    assert torch.equal(dx, dx2) and dw2 is None and db2 is None


@pytest.mark.gpu
@pytest.mark.parametrize("N,S,C,G,dt", [(2, 200, 96, 6, "bf16"), (2, 5000, 512, 32, "bf16"), (1, 9001, 264, 3, "f32")])
def test_outputs_over_their_inputs(gpu, N, S, C, G, dt):
    """y over x and dx over dy, on images kept on chip and on images read twice: the same bits as apart."""
    t = make(N, S, C, dt)
    y, mean, rstd = gn.groupnorm_fwd(t["x"], G, t["w"], t["b"], epilogue="silu")
    x = t["x"].clone()
    gn.groupnorm_fwd(x, G, t["w"], t["b"], epilogue="silu", out=x)
    assert torch.equal(x, y)
    dx, dw, db = gn.groupnorm_bwd(t["x"], G, t["w"], t["b"], mean, rstd, t["dy"], epilogue="silu")
    code = gn.GN_BF16 if dt == "bf16" else gn.GN_F32
    n = gn.gn_groupnorm_bwd_workspace(N, S, C, G, code)
    ws, dw2, db2, dy = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(dw), torch.empty_like(db), t["dy"].clone()
    gn.check(gn.gn_groupnorm_bwd(t["x"].data_ptr(), t["w"].data_ptr(), t["b"].data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                 dy.data_ptr(), dy.data_ptr(), dw2.data_ptr(), db2.data_ptr(), ws.data_ptr(), n, N, S, C, G, C, C, C,
                                 gn.GN_EPI_SILU, code, torch.cuda.current_stream().cuda_stream))
    assert torch.equal(dy, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [512, 2048])
def test_offsets_past_32_bits(gpu, C):
    """Rows so far apart that the last ones lie beyond 2^31 elements (images kept on chip; read twice)."""
    S, ld = 2200, 1 << 20
    t = make(1, S, C, "bf16")
    y, mean, rstd = gn.groupnorm_fwd(t["x"], 32, t["w"], t["b"], epilogue="silu")
    dx, dw, db = gn.groupnorm_bwd(t["x"], 32, t["w"], t["b"], mean, rstd, t["dy"], epilogue="silu")
    far = [torch.empty(S * ld, dtype=torch.bfloat16, device="cuda").as_strided((1, S, C), (S * ld, ld, 1)) for _ in range(3)]
    far[0].copy_(t["x"])
    far[1].copy_(t["dy"])
    y2, mean2, rstd2 = gn.groupnorm_fwd(far[0], 32, t["w"], t["b"], epilogue="silu", out=far[2])
    assert torch.equal(y2, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    dx2, dw2, db2 = gn.groupnorm_bwd(far[0], 32, t["w"], t["b"], mean, rstd, far[1], epilogue="silu")
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    assert gpu.device_error() == 0


@pytest.mark.gpu
def test_padding_is_left_alone(gpu):
    """Bytes between the rows of a padded output, and rows behind the last image, keep what they held."""
    x = torch.randn(2, 9, 36, device="cuda").bfloat16()
    big = torch.full((4, 9, 48), 7.0, device="cuda", dtype=torch.bfloat16)
    xs = torch.zeros(2, 9, 40, device="cuda", dtype=torch.bfloat16)
    xs[..., :36] = x
    gn.groupnorm_fwd(xs[..., :36], 4, out=big[:2, :, :36])
    assert (big[2:] == 7).all() and (big[:2, :, 36:] == 7).all() and not (big[:2, :, :36] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N,S", [(0, 5), (3, 0)])
def test_empty(gpu, N, S):
    x = torch.zeros(N, S, 32, device="cuda", dtype=torch.bfloat16)
    y, _, _ = gn.groupnorm_fwd(x, 4)
    assert y.shape == x.shape
    st = torch.zeros(N, 4, device="cuda")
    dx, dw, db = gn.groupnorm_bwd(x, 4, None, None, st, st, x)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_statistics_of_no_positions_are_nan(gpu, dt):
    gen = torch.full((3, 4), 5.0, device="cuda")  # what the allocator hands out next is not NaN already
    del gen
    _, mean, rstd = gn.groupnorm_fwd(torch.zeros(3, 0, 32, device="cuda", dtype=DT[dt]), 4)
    assert mean.shape == rstd.shape == (3, 4) and torch.isnan(mean).all() and torch.isnan(rstd).all()


@pytest.mark.gpu
def test_nan_stays_in_its_group(gpu):
    x = torch.randn(2, 40, 32, device="cuda")
    x[0, 3, 5] = float("nan")
    x[1, 7, 30] = float("inf")
    y, mean, rstd = gn.groupnorm_fwd(x, 4)
    bad = torch.zeros(2, 40, 32, dtype=torch.bool, device="cuda")
    bad[0, :, 0:8] = True
    bad[1, :, 24:32] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N,S,C,G,dt", [(2, 3000, 320, 32, "bf16"), (4, 9000, 512, 32, "f32")])
def test_same_bits_every_run(gpu, N, S, C, G, dt):
    t = make(N, S, C, dt)
    run = lambda: (lambda y, m, r: (y, m, r) + gn.groupnorm_bwd(t["x"], G, t["w"], t["b"], m, r, t["dy"], epilogue="silu"))(  # noqa: E731
        *gn.groupnorm_fwd(t["x"], G, t["w"], t["b"], epilogue="silu"))
    a = run()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, run()))


@pytest.mark.gpu
def test_gradients_against_differences(gpu):
    """fp32: central differences of sum(y dy) along random directions of x, w and b. The difference
    quotient's own error (fp32 forward, second order in the step) is below 2 per cent of the
    derivative's typical size at these steps."""
    N, S, C, G = 2, 60, 48, 6
    t = make(N, S, C, "f32", spread=1.0)
    _, mean, rstd = gn.groupnorm_fwd(t["x"], G, t["w"], t["b"], epilogue="silu")
    grads = gn.groupnorm_bwd(t["x"], G, t["w"], t["b"], mean, rstd, t["dy"], epilogue="silu")
    f = lambda x, w, b: (gn.groupnorm_fwd(x, G, w, b, epilogue="silu")[0].double() * t["dy"].double()).sum()  # noqa: E731
    for k, name in enumerate("xwb"):
        base = [t["x"], t["w"], t["b"]]
        v = torch.randn(base[k].shape, device="cuda")
        h = 1e-2
        up, dn = list(base), list(base)
        up[k], dn[k] = base[k] + h * v, base[k] - h * v
        num = (f(*up) - f(*dn)) / (2 * h)
        ana = (grads[k].double() * v.double()).sum()
        size = grads[k].double().norm() * (v.double().norm() / v.numel() ** 0.5)
        assert (num - ana).abs() <= 0.02 * size, name


@pytest.mark.gpu
def test_captured_and_replayed_on_new_inputs(gpu):
    t = make(2, 2500, 320, "bf16")
    u = make(2, 2500, 320, "bf16", seed=5)
    run = lambda s: (lambda y, m, r: (y, m, r) + gn.groupnorm_bwd(s["x"], 32, s["w"], s["b"], m, r, s["dy"], epilogue="silu"))(  # noqa: E731
        *gn.groupnorm_fwd(s["x"], 32, s["w"], s["b"], epilogue="silu"))
    want = run(u)
    run(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(t)
    for k in ("x", "dy", "w", "b"):
        t[k].copy_(u[k])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_two_streams_at_once(gpu):
    ts = [make(2, 4000, 256, "bf16", seed=k) for k in range(2)]
    want = [gn.groupnorm_fwd(t["x"], 32, t["w"], t["b"])[0] for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, t in enumerate(ts):
            got[k].append(gn.groupnorm_fwd(t["x"], 32, t["w"], t["b"], stream=streams[k])[0])
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(y, want[k]) for y in got[k])


# ---------------------------------------------------------------- refusals (no GPU needed)

P = 1 << 20


def fwd(x=P, w=P, b=P, y=P, ws=P, nws=1 << 40, N=2, S=10, C=64, G=4, ldx=64, ldy=64, epi=0, dt=1):
    return gn.gn_groupnorm_fwd(x, w, b, y, None, None, ws, nws, N, S, C, G, ldx, ldy, 1e-5, epi, dt, None)


def bwd(x=P, mean=P, rstd=P, dy=P, dx=P, ws=P, nws=1 << 40, N=2, S=10, C=64, G=4, ldx=64, lddy=64, lddx=64, epi=0, dt=1):
    return gn.gn_groupnorm_bwd(x, None, None, mean, rstd, dy, dx, None, None, ws, nws, N, S, C, G, ldx, lddy, lddx, epi, dt, None)


# an image that is not kept on chip: the forward needs its workspace
BIG = dict(S=100000, C=512, G=32, ldx=512, ldy=512)


@pytest.mark.parametrize("call,kw,status", [
    (fwd, dict(dt=3), gn.GN_ERR_DTYPE), (fwd, dict(epi=7), gn.GN_ERR_DTYPE), (fwd, dict(G=5), gn.GN_ERR_SHAPE),
    (fwd, dict(G=0), gn.GN_ERR_SHAPE), (fwd, dict(C=0), gn.GN_ERR_SHAPE), (fwd, dict(N=-1), gn.GN_ERR_SHAPE),
    (fwd, dict(ldx=63), gn.GN_ERR_SHAPE), (fwd, dict(ldy=32), gn.GN_ERR_SHAPE), (fwd, dict(x=None), gn.GN_ERR_NULL),
    (fwd, dict(y=None), gn.GN_ERR_NULL), (fwd, dict(x=P + 8), gn.GN_ERR_ALIGN), (fwd, dict(ldx=65), gn.GN_ERR_ALIGN),
    (fwd, dict(BIG, ws=None), gn.GN_ERR_WORKSPACE), (fwd, dict(BIG, nws=8), gn.GN_ERR_WORKSPACE), (fwd, dict(BIG, ws=P + 4), gn.GN_ERR_ALIGN),
    (fwd, dict(N=0, x=None, ws=None), gn.GN_OK), (fwd, dict(S=0, x=None, ws=None), gn.GN_OK),
    (bwd, dict(mean=None), gn.GN_ERR_NULL), (bwd, dict(rstd=None), gn.GN_ERR_NULL), (bwd, dict(dy=None), gn.GN_ERR_NULL),
    (bwd, dict(lddx=60), gn.GN_ERR_SHAPE), (bwd, dict(lddy=68), gn.GN_ERR_ALIGN), (bwd, dict(nws=0), gn.GN_ERR_WORKSPACE),
    (bwd, dict(N=0), gn.GN_OK)])
def test_refusals(call, kw, status):
    gn.load()
    assert call(**kw) == status


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 171), (1, 1, 5), (1, 1, 64), (2, 3, 64), (2, 3, 77), (1, 1, 1), (3, 0, 77), (0, 4, 64)])
def test_row_strides_of_inputs_and_outputs(monkeypatch, shape, dt):
    """Every row stride that reaches the library is whole 16 bytes, an output's own where it has more than one row."""
    monkeypatch.setattr(gn, "_on_gpu", lambda t: True)
    x = gn.empty_rows(shape, DT[dt], "cpu")
    es = x.element_size()
    N, S, C, ld = gn._images(x)
    y, ldy = gn._like_rows(x)
    assert (N, S, C) == shape and y.shape == x.shape and y.dtype == x.dtype
    assert ld * es % 16 == 0 and ldy * es % 16 == 0 and ldy >= C
    if N * S > 1:
        assert gn._images(y)[3] == ldy and y.stride(-2) == ldy


def test_helper_refusals(monkeypatch):
    monkeypatch.setattr(gn, "_on_gpu", lambda t: True)
    x = torch.zeros(2, 10, 64, dtype=torch.bfloat16)
    st = torch.zeros(2, 4)
    for f in (lambda: gn.groupnorm_fwd(x[0, 0], 4), lambda: gn.groupnorm_fwd(x, 4, w=torch.zeros(63, dtype=torch.bfloat16)),
              lambda: gn.groupnorm_fwd(x, 4, w=torch.zeros(64)), lambda: gn.groupnorm_fwd(x.transpose(1, 2), 4),
              lambda: gn.groupnorm_fwd(x, 4, out=x[:1]), lambda: gn.groupnorm_fwd(x[:, ::2][:, :, :32].permute(1, 0, 2), 4),
              lambda: gn.groupnorm_bwd(x, 4, None, None, st[:1], st, x), lambda: gn.groupnorm_bwd(x, 4, None, None, st, st.double(), x),
              lambda: gn.groupnorm_bwd(x, 4, None, None, st, st, x.float())):
        with pytest.raises((ValueError, TypeError)):
            f()
