"""8-bit operands (norm_quant_fp8, quant_fp8, act_grad_quant_fp8) and their product (linear_fp8) against
their definitions in 64 bits.

Tolerances: codes stand for values v within half an e4m3 step, 2^-4 |v| or, below the smallest normal
code 2^-6, half of 2^-9 scales; plus 1e-5 of the magnitudes behind v for its fp32 evaluation (2e-5 on the
scale, which is amax / 448). A matrix quantised without a norm or an activation has the very codes and
scales of the fp32 definition. The product's fp32 sums: at most K + K / 128 roundings of 2^-24 of the sum
of |a||b|, plus half a step of the output, plus 2^-11 |z| for the approximate activations of bf16 outputs.
"""
import pytest
import torch

import transformer_norm_rope_b200 as gn

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def blocks(n):
    return -(-n // 128)


def padded(t, dtype, extra=0):
    """t in `dtype` on the GPU with rows on 16-byte boundaries (and `extra` more elements between them)"""
    es = torch.empty((), dtype=dtype).element_size()
    ld = (t.shape[-1] * es + 15) // 16 * 16 // es + extra
    base = torch.zeros(t.shape[:-1] + (ld,), dtype=torch.float32).to(dtype).cuda()
    base[..., :t.shape[-1]] = t.to(dtype).cuda()
    return base[..., :t.shape[-1]]


def over_448(t):
    return t / torch.full_like(t, 448.0)  # a true division: torch multiplies by the reciprocal of a Python number


def scale_of(v):
    """amax per run of 128 along the rows -> scales, in v's precision"""
    rows, cols = v.shape
    p = torch.zeros(rows, blocks(cols) * 128, dtype=v.dtype, device=v.device)
    p[:, :cols] = v
    return over_448(p.reshape(rows, -1, 128).abs().amax(2).clamp_min(2.0 ** -110))


def spread(s, cols):
    return s.repeat_interleave(128, 1)[:, :cols]


def check_codes(q, s, v, slack, what, blockwise=None):
    """q, s against the double values v (slack: fp32 evaluation error of v)"""
    ref = scale_of(v) if blockwise is None else blockwise
    sl = scale_of(slack) if blockwise is None else slack.max() / 448
    assert q.dtype == F8 and q.shape == v.shape and s.shape == ref.shape
    assert ((s.double() - ref).abs() <= 1e-6 * ref + sl).all(), f"{what}: scales"
    sx = spread(s.double(), v.shape[1]) if blockwise is None else s.double().repeat_interleave(128, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]
    got = q.double() * sx
    tol = 2.0 ** -4 * v.abs() + 2.0 ** -10 * sx + slack * (1 + 2.0 ** -4) + 1e-6 * v.abs()
    over = (got - v).abs() - tol
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} codes off, worst by {over.max():.3g}"


def codes32(v):
    """the fp32 definition by torch: bit-exact reference of a matrix quantised as it is"""
    s = scale_of(v.float())
    return (v.float() / spread(s, v.shape[1])).to(F8), s


def same_codes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- norm + quantise

ROWS = [(1, 5120), (3, 64), (5, 128), (7, 200), (2, 77), (33, 1000), (4, 1), (130, 1288), (2, 8192), (600, 384), (200, 2000), (5, 513), (160, 5120), (700, 5120), (650, 1291), (601, 8184)]


@pytest.mark.gpu
@pytest.mark.parametrize("norm,gemma", [("rms", False), ("rms", True), ("ln", False), ("none", False)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hidden", ROWS)
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
def test_norm_quant(gpu, rows, hidden, dt, norm, gemma, act):
    g = torch.Generator().manual_seed(rows * 10007 + hidden)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = padded(r(rows, hidden) * (0.5 + r(rows, 1).abs()) + 2 * r(rows, 1), DT[dt])
    w = (0.1 * r(hidden) + (0 if gemma else 1)).to(DT[dt]).cuda()
    b = (0.1 * r(hidden)).to(DT[dt]).cuda()
    eps = 1e-5
    q, s, mean, rstd = gn.norm_quant_fp8(x, None if norm == "none" else w, b if norm == "ln" else None, eps, norm=norm, gemma=gemma,
                                         epilogue=act)
    X = x.double()
    mu = X.mean(1, keepdim=True) if norm == "ln" else torch.zeros(rows, 1, dtype=torch.float64, device="cuda")
    rs = (((X - mu) ** 2).mean(1, keepdim=True) + eps) ** -0.5
    if norm == "ln":
        z = (X - mu) * rs * w.double() + b.double()
        mag = (X.abs() + mu.abs()) * rs * w.double().abs() + b.double().abs()
        tol = 4e-6 * (mu.abs() + 1 / rs)
        assert ((mean.double()[:, None] - mu).abs() <= tol).all()
    elif norm == "rms":
        z = X * rs * (1 + w.double() if gemma else w.double())
        mag = z.abs()
    else:
        z, mag = X, torch.zeros_like(X)
    if norm != "none":
        # a row of one value has (x - mu) = 0 exactly; elsewhere the variance's relative error is that of its sum
        assert ((rstd.double()[:, None] - rs).abs() <= 4e-6 * rs * (1 + (mu * rs).abs())).all()
    else:
        assert rstd is None
    if norm == "none" and act == "none":
        cq, cs = codes32(x)
        assert torch.equal(s, cs) and same_codes(q, cq)
    v = act64(z, act)
    slack = 1e-5 * (mag + (z.abs() if act != "none" else 0)) * (1 + (mu * rs).abs() if norm == "ln" else 1)
    check_codes(q, s, v, slack, "norm_quant")
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_quant_rows_whose_beginning_is_far_off(gpu, dt):
    """Statistics must not lose their bits to a first part of the row (or a mean) far from the rest."""
    x = torch.randn(640, 5120)
    x[::2, :256] += 500.0
    x[1::4] += 300.0
    x = x.to(DT[dt]).cuda()
    _, _, mean, rstd = gn.norm_quant_fp8(x, norm="ln", eps=1e-5)
    X = x.double()
    mu, rs = X.mean(1), (X.var(1, correction=0) + 1e-5) ** -0.5
    assert ((mean.double() - mu).abs() <= 4e-6 * (mu.abs() + 1 / rs)).all()
    assert ((rstd.double() - rs).abs() <= 1e-5 * rs).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0.0, 300.0])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hidden", [(1200, 5120), (1200, 2056), (1200, 4096)])
def test_norm_quant_means_are_rounded_once(gpu, rows, hidden, dt, shift):
    """LayerNorm's mean of rows with mean in [1, 2) and unit spread, also where the row's first part lies far off. Root
    mean square error over the rows, in 2^-24 (half an ulp of the mean; the last rounding alone leaves 0.58):
    * bf16 rows: x - K and its sums have few bits and are all but exact: 1, and 4 next to values of 300;
    * fp32 rows summed as x - K (up to 4096 wide): n independent roundings of partial sums p, sqrt(n) p / (sqrt 3 n): 0.4
      for p = 30, so 1; with four values of 301 in a partial sum that times 1206 / 30;
    * wider ones, summed as they are: 1, 2, 4 ... roundings of sums P, P / 2, P / 4 ...: sqrt(2 / 3) P / n, P / n = 1.5
      (256 x 301 / n next to 300), with the last rounding sqrt(0.58^2 + 1.22^2) = 1.35.
    (Roundings that are the same for all values of a row would not stay so small.)"""
    g = torch.Generator().manual_seed(rows + hidden)
    x = torch.randn(rows, hidden, generator=g) + 1.5
    if shift:  # first values up, the last down by as much: the mean stays
        x[:, :256] += shift
        x[:, -256:] -= shift
    x = padded(x, DT[dt])
    _, _, mean, _ = gn.norm_quant_fp8(x, norm="ln", eps=1e-5)
    mu = x.double().mean(1)
    err = (mean.double() - mu).square().mean().sqrt()
    if dt == "bf16":
        tol = 4 if shift else 1
    elif hidden <= 4096:
        tol = 1 + hidden ** -0.5 * 1206 / 3 ** 0.5 if shift else 1
    else:
        tol = 0.58 + (2 / 3) ** 0.5 * 256 * 301.5 / hidden if shift else 1.35
    assert err <= 2.0 ** -24 * tol, f"{err * 2 ** 24:.3g}, {tol:.3g} allowed"


@pytest.mark.gpu
def test_norm_quant_parameters_off_16_bytes(gpu):
    x = torch.randn(9, 520, device="cuda").bfloat16()
    w, b = (torch.randn(523, device="cuda").bfloat16() for _ in range(2))
    got = gn.norm_quant_fp8(x, w[3:], b[1:521], 1e-5, norm="ln", epilogue="silu")
    want = gn.norm_quant_fp8(x, w[3:].clone(), b[1:521].clone(), 1e-5, norm="ln", epilogue="silu")
    assert same_codes(got[0], want[0]) and all(torch.equal(p, q) for p, q in zip(got[1:], want[1:]))


# ---------------------------------------------------------------- matrices, both ways

MATS = [(1, 64), (128, 128), (129, 127), (4, 1000), (300, 77), (1000, 8), (255, 640), (1031, 300)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", MATS)
def test_quant_both_ways_has_the_definitions_codes(gpu, rows, cols, dt):
    g = torch.Generator().manual_seed(rows + cols)
    x = padded(torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g)), DT[dt], extra=16)
    q, s, qt, st = gn.quant_fp8(x, transposed=True)
    cq, cs = codes32(x)
    ct, cts = codes32(x.t())
    assert torch.equal(s, cs) and same_codes(q, cq), "by rows"
    assert torch.equal(st, cts) and same_codes(qt, ct), "transposed"
    q1, s1 = gn.quant_fp8(x)
    q2, s2 = gn.quant_fp8(x, by_rows=False, transposed=True)
    assert same_codes(q1, cq) and torch.equal(s1, cs) and same_codes(q2, ct) and torch.equal(s2, cts)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", MATS)
def test_quant_tiles_has_the_definitions_codes(gpu, rows, cols, dt):
    g = torch.Generator().manual_seed(rows + cols)
    x = padded(torch.randn(rows, cols, generator=g) * 0.02, DT[dt])
    q, s, qt, st = gn.quant_fp8(x, tile=True, transposed=True)
    R, Q = blocks(rows), blocks(cols)
    p = torch.zeros(R * 128, Q * 128, device="cuda")
    p[:rows, :cols] = x.float()
    cs = over_448(p.reshape(R, 128, Q, 128).abs().amax(3).amax(1).clamp_min(2.0 ** -110))
    cq = (p / cs.repeat_interleave(128, 0).repeat_interleave(128, 1)).to(F8)[:rows, :cols]
    assert torch.equal(s, cs) and same_codes(q, cq)
    assert torch.equal(st, cs.t()) and same_codes(qt, cq.t())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", MATS)
def test_activation_gradient(gpu, rows, cols, dt, act):
    g = torch.Generator().manual_seed(rows + cols)
    z = padded(1.5 * torch.randn(rows, cols, generator=g), DT[dt])
    dy = padded(1e-3 * torch.randn(rows, cols, generator=g), DT[dt], extra=8)
    q, s, qt, st, db = gn.act_grad_quant_fp8(z, dy, epilogue=act)
    zz = z.double().clone().requires_grad_(True)
    (dz,) = torch.autograd.grad((act64(zz, act) * dy.double()).sum(), zz)
    slack = 1e-5 * dy.double().abs() * (act != "none")
    check_codes(q, s, dz, slack, "dz")
    check_codes(qt, st, dz.t(), slack.t(), "dz transposed")
    assert ((db.double() - dz.sum(0)).abs() <= (4e-6 * dz.abs() + slack).sum(0) + 1e-30).all()
    _, _, _, _, none = gn.act_grad_quant_fp8(z, dy, epilogue=act, want_db=False)
    assert none is None


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", MATS)
def test_column_sums_of_a_matrix_as_it_is(gpu, rows, cols, dt, tile):
    """db without dy: the column sums of x itself, next to the codes that x has without them. Sums of up to 1031
    fp32 terms, slab by slab: 4e-6 of the magnitudes, as for the gradient."""
    g = torch.Generator().manual_seed(rows + cols)
    x = padded(torch.randn(rows, cols, generator=g), DT[dt], extra=16)
    want = gn.quant_fp8(x, tile=tile, transposed=True)
    r, c = (blocks(rows), blocks(cols)) if tile else (rows, cols)
    ldq, ldqt = (cols + 15) // 16 * 16, (rows + 15) // 16 * 16
    code = gn.GN_BF16 if dt == "bf16" else gn.GN_F32
    n = gn.gn_quant_fp8_workspace(rows, cols)
    for by_rows, transposed in ((True, True), (True, False), (False, True)):
        q, qt = (torch.zeros(a, b, dtype=torch.uint8, device="cuda") for a, b in ((rows, ldq), (cols, ldqt)))
        s, st = torch.zeros(r, blocks(cols), device="cuda"), torch.zeros(c, blocks(rows), device="cuda")
        ws = torch.full((n // 4,), float("nan"), device="cuda")
        db = torch.full((cols,), 7.0, device="cuda")
        gn.check(gn.gn_quant_fp8(x.data_ptr(), None, q.data_ptr() if by_rows else None, s.data_ptr(), qt.data_ptr() if transposed else None,
                                 st.data_ptr(), db.data_ptr(), ws.data_ptr(), n, rows, cols, x.stride(0) if rows > 1 else ldq, 0, ldq,
                                 blocks(cols), ldqt, blocks(rows), gn.GN_FP8_TILE if tile else gn.GN_FP8_VEC, 0, code,
                                 torch.cuda.current_stream().cuda_stream))
        X = x.double()
        assert ((db.double() - X.sum(0)).abs() <= 4e-6 * X.abs().sum(0)).all()
        if by_rows:
            assert same_codes(q.view(F8)[:, :cols], want[0]) and torch.equal(s, want[1])
        if transposed:
            assert same_codes(qt.view(F8)[:, :rows], want[2]) and torch.equal(st, want[3])
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_special_values(gpu, dt):
    """Zero blocks, the smallest and largest magnitudes, NaN and infinities: only their own blocks see them."""
    x = torch.randn(256, 384)
    x[0, :128] = 0
    x[1, 128:256] = 1e-38
    x[2, 256:] = 3e38
    x[3, 5] = float("nan")
    x[4, 130] = float("inf")
    x[5, 300] = -float("inf")
    x[6, :128] = 1e-40
    x = x.to(DT[dt]).cuda()
    for q, s in (gn.quant_fp8(x), gn.norm_quant_fp8(x, norm="none")[:2]):
        v = q.double() * spread(s.double(), 384)
        assert (v[0, :128] == 0).all() and torch.isfinite(s[0, 0])
        bad = torch.zeros(256, 384, dtype=torch.bool, device="cuda")
        bad[3, :128] = bad[4, 128:256] = bad[5, 256:] = True
        assert torch.isnan(v[bad]).all() and torch.isfinite(v[~bad]).all()
        assert torch.isnan(s[3, 0]) and torch.isnan(s[4, 1]) and torch.isnan(s[5, 2])
        for r, c in ((1, slice(128, 256)), (2, slice(256, 384))):
            assert ((v[r, c] - x[r, c].double()).abs() <= 2.0 ** -4 * x[r, c].double().abs() + 2.0 ** -10 * s[r, c.start // 128].double()).all()
    qt, st = gn.quant_fp8(x, by_rows=False, transposed=True)
    vt = qt.double() * spread(st.double(), 256)
    assert torch.isnan(vt[5, :128]).all() and torch.isfinite(vt[5, 128:]).all() and torch.isfinite(vt[6]).all()


@pytest.mark.gpu
def test_padding_is_left_alone(gpu):
    """Bytes of a code row past its width, and rows behind the last, keep what they held."""
    x = torch.randn(5, 77, device="cuda")
    xs = torch.zeros(5, 80, device="cuda")
    xs[:, :77] = x
    f = lambda *s: torch.full(s, 0x55, dtype=torch.uint8, device="cuda")  # noqa: E731
    q, qt, s, st = f(6, 96), f(78, 16), torch.full((6, 2), 7.0, device="cuda"), torch.full((78, 2), 7.0, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    gn.check(gn.gn_quant_fp8(xs.data_ptr(), None, q.data_ptr(), s.data_ptr(), qt.data_ptr(), st.data_ptr(), None, None, 0, 5, 77, 80,
                             0, 96, 2, 16, 2, gn.GN_FP8_VEC, 0, gn.GN_F32, stream))
    assert (q[5] == 0x55).all() and (q[:5, 77:] == 0x55).all() and (qt[77] == 0x55).all() and (qt[:77, 5:] == 0x55).all()
    assert (s[5] == 7).all() and (s[:5, 1:] == 7).all() and (st[77] == 7).all() and (st[:77, 1:] == 7).all()
    q.fill_(0x55)
    gn.check(gn.gn_norm_quant_fp8(xs.data_ptr(), None, None, q.data_ptr(), s.data_ptr(), None, None, 5, 77, 80, 96, 2, 1e-6,
                                  gn.GN_NORM_RMS, 0, 0, gn.GN_F32, stream))
    assert (q[5] == 0x55).all() and (q[:5, 77:] == 0x55).all() and (s[5] == 7).all() and (s[:5, 1:] == 7).all()


def far_rows(t, ld):
    """t on rows `ld` elements apart"""
    base = torch.empty(t.shape[0] * ld, dtype=torch.uint8 if t.dtype == F8 else t.dtype, device="cuda")
    v = base.as_strided(t.shape, (ld, 1))
    v.copy_(t.view(torch.uint8) if t.dtype == F8 else t)
    return base.view(F8).as_strided(t.shape, (ld, 1)) if t.dtype == F8 else v


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [384, 5120])
def test_quantiser_offsets_past_32_bits(gpu, hidden):
    x = torch.randn(2200, hidden, device="cuda").bfloat16()
    far = far_rows(x, 1 << 20)
    for f in (lambda v: gn.norm_quant_fp8(v, norm="ln"), lambda v: gn.norm_quant_fp8(v[2100:], norm="rms"), lambda v: gn.quant_fp8(v, transposed=True),
              lambda v: gn.quant_fp8(v, tile=True, transposed=True), lambda v: gn.act_grad_quant_fp8(v, v)):
        for a, b in zip(f(x), f(far)):
            assert a is None and b is None or (same_codes(a, b) if a.dtype == F8 else torch.equal(a, b))
    assert gpu.device_error() == 0


# ---------------------------------------------------------------- the product

def operands(M, N, K, b_rows, seed=0):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(M, K, generator=g) * (0.5 + torch.randn(M, 1, generator=g).abs())
    b = torch.randn(N, K, generator=g) / K ** 0.5
    aq, sa = codes32(a.cuda())
    if b_rows == 1:
        bq, sb = codes32(b.cuda())
    else:
        bq, sb = gn.quant_fp8(padded(b, torch.float32), tile=True)
    return padded8(aq), sa, padded8(bq), sb, (0.3 * torch.randn(N, generator=g)).cuda()


def padded8(q):
    base = torch.zeros(q.shape[0], (q.shape[1] + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    base[:, :q.shape[1]] = q.contiguous().view(torch.uint8)
    return base.view(F8)[:, :q.shape[1]]


def product64(aq, sa, bq, sb, d, act):
    M, K = aq.shape
    N = bq.shape[0]
    a = aq.double() * spread(sa.double(), K)
    sbx = sb.double() if sb.shape[0] == N else sb.double().repeat_interleave(128, 0)[:N]
    b = bq.double() * spread(sbx, K)
    z = a @ b.t() + (0 if d is None else d.double())
    tol = 2.0 ** -24 * (K + blocks(K) + 4) * (a.abs() @ b.abs().t() + (0 if d is None else d.double().abs()))
    return act64(z, act), z, tol


def check_product(y, ops, act, out):
    v, z, tol = product64(*ops, act)
    u = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
    tol = 1.2 * tol + u * v.abs() + (2.0 ** -11 * z.abs() if act != "none" else 0)  # an activation's slope is below 1.2
    assert torch.isfinite(y).all()
    over = (y.double() - v).abs() - tol
    assert (over <= 0).all(), f"{int((over > 0).sum())} of {over.numel()} off, worst by {over.max():.3g}"


# single tokens, fewer and more rows than a tile, contractions of one value, of part of a block and of
# odd lengths, widths that end inside a tile
PRODUCTS = [(1, 128, 128), (1, 5120, 5120), (2, 77, 300), (7, 1000, 1), (16, 256, 64), (17, 129, 127), (31, 513, 4093), (64, 640, 1280),
            (100, 8, 256), (128, 128, 384), (129, 257, 129), (200, 1288, 1000), (333, 300, 2049), (513, 770, 640), (1000, 1000, 1000),
            (2050, 260, 136), (2600, 1030, 520), (4100, 900, 129), (6000, 1290, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_linear(gpu, M, N, K, act):
    aq, sa, bq, sb, d = operands(M, N, K, 128)
    y = gn.linear_fp8(aq, sa, bq, sb, d, epilogue=act)
    assert y.dtype == torch.bfloat16 and y.shape == (M, N)
    check_product(y, (aq, sa, bq, sb, d), act, "bf16")
    if act == "none":
        check_product(gn.linear_fp8(aq, sa, bq, sb), (aq, sa, bq, sb, None), act, "bf16")
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_linear_row_scales_fp32(gpu, M, N, K):
    aq, sa, bq, sb, d = operands(M, N, K, 1)
    y = gn.linear_fp8(aq, sa, bq, sb, out_dtype=torch.float32)
    check_product(y, (aq, sa, bq, sb, None), "none", "f32")
    check_product(gn.linear_fp8(aq, sa, bq, sb, d), (aq, sa, bq, sb, d), "none", "bf16")
    first = y.clone()
    gn.linear_fp8(aq, sa, bq, sb, out=y, accumulate=True)
    assert ((y.double() - 2 * first.double()).abs() <= 2.0 ** -23 * y.double().abs()).all()
    aq, sa, bq, sb, d = operands(M, N, K, 128)
    check_product(gn.linear_fp8(aq, sa, bq, sb, d, out_dtype=torch.float32), (aq, sa, bq, sb, d), "none", "f32")
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,N", [(1, 256), (16, 130), (30, 130), (60, 130), (128, 130), (300, 140), (2048, 2048)])
def test_activations_keep_their_relative_precision(gpu, M, N, act):
    """One product of ones a value, scaled to z: the activation of known z from -12 to 12, its small values on the
    negative side included. Half a step of bf16; and for the evaluation z sigmoid(t) in fp32 with an exponential of
    -t, t = z or 2 k (z + c z^3): 2^-22 (|t| + 4) of the value, t's own roundings and the functions' two ulps. A
    sigmoid below 2^-126, the smallest normal number, is flushed to zero, and with it up to |z| 2^-126 of the value."""
    code = torch.zeros(max(M, N), 128).to(F8).cuda()
    code[:, 5] = torch.ones(()).to(F8).cuda()
    if N > 1000:  # z = sa sb
        sa, sb = torch.linspace(-12, 12, M, device="cuda")[:, None], torch.linspace(0.25, 1, blocks(N), device="cuda")[:, None]
        z = sa.double() * sb.double().repeat_interleave(128, 0)[:N].t()
        y = gn.linear_fp8(code[:M], sa, code[:N], sb, epilogue=act)
    else:  # z = sa + d
        sa, sb = torch.linspace(-6, 6, M, device="cuda")[:, None], torch.ones(blocks(N), 1, device="cuda")
        d = torch.linspace(-6, 6, N, device="cuda")
        z = (sa + d).double()  # one fp32 rounding, the kernel's own
        y = gn.linear_fp8(code[:M], sa, code[:N], sb, d, epilogue=act)
    t = z if act == "silu" else 2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)
    v = z * torch.sigmoid(t)
    tol = (2.0 ** -8 + 2.0 ** -22 * (t.abs() + 4)) * v.abs() + 2.0 ** -126 * (1 + z.abs())
    over = (y.double() - v).abs() - tol
    assert (over <= 0).all(), f"{int((over > 0).sum())} of {over.numel()} off; worst relative {((y.double() - v).abs() / v.abs())[v.abs() > 1e-30].max():.3g}"


@pytest.mark.gpu
def test_linear_strides_and_neighbours(gpu):
    """Operands, scales and outputs that are parts of larger tensors; what lies around the output stays."""
    M, N, K = 150, 300, 500
    aq, sa, bq, sb, d = operands(M, N, K, 128)
    A = torch.randint(0, 255, (M + 3, 640), dtype=torch.uint8, device="cuda")  # NaN codes among the neighbours
    A[:M, 16:16 + K] = aq.contiguous().view(torch.uint8)
    SA = torch.full((M + 2, 9), float("nan"), device="cuda")
    SA[:M, 2:2 + blocks(K)] = sa
    SB = torch.full((blocks(N) + 1, 7), float("nan"), device="cuda")
    SB[:blocks(N), 1:1 + blocks(K)] = sb
    big = torch.full((M + 5, 400), 9.0, dtype=torch.bfloat16, device="cuda")
    out = gn.linear_fp8(A.view(F8)[:M, 16:16 + K], SA[:M, 2:2 + blocks(K)], bq, SB[:blocks(N), 1:1 + blocks(K)], d, out=big[2:M + 2, 8:8 + N])
    assert torch.equal(out, gn.linear_fp8(aq, sa, bq, sb, d))
    big[2:M + 2, 8:8 + N] = 9.0
    assert (big == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,ld", [(40, 520, 640, 1 << 26), (3000, 2000, 640, 1 << 20)])
def test_linear_offsets_past_32_bits(gpu, M, N, K, ld):
    aq, sa, bq, sb, d = operands(M, N, K, 128)
    y = gn.linear_fp8(aq, sa, bq, sb, d)
    far = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda").as_strided((M, N), (ld, 1))
    assert torch.equal(gn.linear_fp8(far_rows(aq, ld), far_rows(sa, ld), bq, sb, d, out=far), y)
    assert gpu.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(4, 256, 512), (300, 520, 512), (3000, 2000, 512)])
def test_linear_nan_and_infinite_scales(gpu, M, N, K):
    """NaN codes or scales reach their own row (or weight block of columns) and nothing else."""
    aq, sa, bq, sb, d = operands(M, N, K, 128)
    y = gn.linear_fp8(aq, sa, bq, sb, d)
    sa2 = sa.clone()
    sa2[2, 1] = float("nan")
    y2 = gn.linear_fp8(aq, sa2, bq, sb, d)
    assert torch.isnan(y2[2]).all()
    keep = torch.arange(M, device="cuda") != 2
    assert torch.equal(y2[keep], y[keep])
    bq2 = bq.contiguous().view(torch.uint8).clone()
    bq2[5, 100] = 0x7f
    y3 = gn.linear_fp8(aq, sa, bq2.view(F8), sb, d)
    cols = torch.arange(N, device="cuda") != 5
    assert torch.isnan(y3[:, 5]).all() and torch.equal(y3[:, cols], y[:, cols])
    sb2 = sb.clone()
    sb2[1, 0] = float("inf")
    y4 = gn.linear_fp8(aq, sa, bq, sb2, d)
    assert not torch.isfinite(y4[:, 128:256]).any() and torch.equal(y4[:, :128], y[:, :128]) and torch.equal(y4[:, 256:], y[:, 256:])


@pytest.mark.gpu
def test_linear_empty(gpu):
    aq, sa, bq, sb, d = operands(4, 64, 256, 128)
    assert gn.linear_fp8(aq[:0], sa[:0], bq, sb, d).shape == (0, 64)
    assert gn.linear_fp8(aq, sa, bq[:0], sb[:0]).shape == (4, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,b_rows", [(1, 5120, 5120, 128), (48, 1000, 4000, 128), (600, 1300, 1500, 128), (700, 900, 3001, 1), (3000, 2000, 1500, 128), (3000, 2000, 1601, 1)])
def test_same_bits_every_run(gpu, M, N, K, b_rows):
    ops = operands(M, N, K, b_rows)
    dt = torch.float32 if b_rows == 1 else torch.bfloat16
    y = gn.linear_fp8(*ops, out_dtype=dt)
    for _ in range(4):
        assert torch.equal(y, gn.linear_fp8(*ops, out_dtype=dt))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 500, 5000])
def test_captured_and_replayed_on_new_inputs(gpu, M):
    N, K = 640, 1100
    W = padded(torch.randn(N, K), torch.bfloat16)
    xs = [padded(torch.randn(M, K), torch.bfloat16) for _ in range(2)]

    def run(x):
        wq, ws, wqt, wst = gn.quant_fp8(W, tile=True, transposed=True)
        q, s, _, rs = gn.norm_quant_fp8(x, norm="rms")
        y = gn.linear_fp8(q, s, wq, ws, epilogue="silu")
        dq, ds, dqt, dst, db = gn.act_grad_quant_fp8(y, y)
        dx = gn.linear_fp8(dq, ds, wqt, wst)
        xt, xts = gn.quant_fp8(x, by_rows=False, transposed=True)
        return y, dx, gn.linear_fp8(dqt, dst, xt, xts, out_dtype=torch.float32), db, rs

    want = run(xs[1])
    run(xs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(xs[0])
    xs[0].copy_(xs[1])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_two_streams_at_once(gpu):
    ops = [operands(300, 700, 900, 128, seed=k) for k in range(2)]
    want = [gn.linear_fp8(*o) for o in ops]
    streams = [torch.cuda.Stream() for _ in ops]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for k in range(2):
            got[k].append(gn.linear_fp8(*ops[k], stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(y, want[k]) for y in got[k])


# ---------------------------------------------------------------- refusals (no GPU needed)

P = 1 << 20


def nq(x=P, q=P, s=P, rows=4, hidden=256, ldx=256, ldq=256, lds=2, norm=0, epi=0, dt=1):
    return gn.gn_norm_quant_fp8(x, None, None, q, s, None, None, rows, hidden, ldx, ldq, lds, 1e-6, norm, 0, epi, dt, None)


def qu(x=P, dy=None, q=P, s=P, qt=None, st=None, db=None, ws=None, nws=0, rows=4, cols=256, ldx=256, lddy=256, ldq=256, lds=2, ldqt=16,
       ldst=1, block=0, epi=0, dt=1):
    return gn.gn_quant_fp8(x, dy, q, s, qt, st, db, ws, nws, rows, cols, ldx, lddy, ldq, lds, ldqt, ldst, block, epi, dt, None)


def li(A=P, sa=P, B=P, sb=P, d=None, y=P, M=4, N=256, K=256, lda=256, ldsa=2, ldb=256, ldsb=2, ldy=256, b_rows=128, acc=0, epi=0, out=1):
    return gn.gn_linear_fp8(A, sa, B, sb, d, y, M, N, K, lda, ldsa, ldb, ldsb, ldy, b_rows, acc, epi, out, None)


@pytest.mark.parametrize("call,kw,status", [
    (nq, dict(dt=2), gn.GN_ERR_DTYPE), (nq, dict(epi=3), gn.GN_ERR_DTYPE), (nq, dict(norm=4), gn.GN_ERR_SHAPE),
    (nq, dict(hidden=0), gn.GN_ERR_SHAPE), (nq, dict(rows=-1), gn.GN_ERR_SHAPE), (nq, dict(ldx=255), gn.GN_ERR_SHAPE),
    (nq, dict(ldq=128), gn.GN_ERR_SHAPE), (nq, dict(lds=1), gn.GN_ERR_SHAPE), (nq, dict(hidden=16400, ldx=16400, ldq=16400, lds=129), gn.GN_ERR_UNSUPPORTED),
    (nq, dict(x=None), gn.GN_ERR_NULL), (nq, dict(q=None), gn.GN_ERR_NULL), (nq, dict(s=None), gn.GN_ERR_NULL),
    (nq, dict(x=P + 2), gn.GN_ERR_ALIGN), (nq, dict(q=P + 8), gn.GN_ERR_ALIGN), (nq, dict(ldq=264), gn.GN_ERR_ALIGN), (nq, dict(ldx=257), gn.GN_ERR_ALIGN),
    (nq, dict(rows=0, x=None, q=None), gn.GN_OK),
    (qu, dict(dt=9), gn.GN_ERR_DTYPE), (qu, dict(block=2), gn.GN_ERR_SHAPE), (qu, dict(cols=0), gn.GN_ERR_SHAPE), (qu, dict(ldq=200), gn.GN_ERR_SHAPE),
    (qu, dict(qt=P, st=P, ldqt=3), gn.GN_ERR_SHAPE), (qu, dict(qt=P, st=P, ldst=0), gn.GN_ERR_SHAPE), (qu, dict(dy=P, block=1), gn.GN_ERR_UNSUPPORTED),
    (qu, dict(epi=1), gn.GN_ERR_UNSUPPORTED), (qu, dict(dy=P, lddy=100), gn.GN_ERR_SHAPE), (qu, dict(q=None), gn.GN_ERR_NULL),
    (qu, dict(s=None), gn.GN_ERR_NULL), (qu, dict(qt=P), gn.GN_ERR_NULL), (qu, dict(qt=P, st=P, ldqt=24), gn.GN_ERR_ALIGN),
    (qu, dict(dy=P + 4), gn.GN_ERR_ALIGN), (qu, dict(db=P), gn.GN_ERR_WORKSPACE), (qu, dict(db=P, ws=P, nws=16), gn.GN_ERR_WORKSPACE),
    (qu, dict(db=P, ws=P + 4, nws=1 << 20), gn.GN_ERR_ALIGN), (qu, dict(rows=8388481), gn.GN_ERR_SHAPE), (qu, dict(rows=0), gn.GN_OK),
    (li, dict(out=5), gn.GN_ERR_DTYPE), (li, dict(epi=4), gn.GN_ERR_DTYPE), (li, dict(K=0), gn.GN_ERR_SHAPE), (li, dict(M=-1), gn.GN_ERR_SHAPE),
    (li, dict(b_rows=64), gn.GN_ERR_SHAPE), (li, dict(lda=128), gn.GN_ERR_SHAPE), (li, dict(ldsa=1), gn.GN_ERR_SHAPE), (li, dict(ldsb=1), gn.GN_ERR_SHAPE),
    (li, dict(ldy=100), gn.GN_ERR_SHAPE), (li, dict(M=8388481), gn.GN_ERR_SHAPE), (li, dict(acc=1), gn.GN_ERR_UNSUPPORTED),
    (li, dict(out=0, epi=1), gn.GN_ERR_UNSUPPORTED), (li, dict(A=None), gn.GN_ERR_NULL), (li, dict(sb=None), gn.GN_ERR_NULL),
    (li, dict(y=None), gn.GN_ERR_NULL), (li, dict(A=P + 8), gn.GN_ERR_ALIGN), (li, dict(ldb=264), gn.GN_ERR_ALIGN), (li, dict(ldy=260), gn.GN_ERR_ALIGN),
    (li, dict(d=P + 4), gn.GN_ERR_ALIGN), (li, dict(sa=P + 2), gn.GN_ERR_ALIGN), (li, dict(M=0, A=None), gn.GN_OK), (li, dict(N=0), gn.GN_OK)])
def test_refusals(call, kw, status):
    gn.load()
    assert call(**kw) == status


def test_gradient_of_no_rows():
    """dy of an empty tensor is a null pointer: an activation asks for dy only where there are rows."""
    gn.load()
    assert qu(rows=0, epi=2) == gn.GN_OK and qu(rows=0, epi=2, x=None, q=None) == gn.GN_OK
    assert qu(rows=1, epi=2) == gn.GN_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
def test_activation_gradient_of_no_rows(gpu, act):
    z = torch.zeros(0, 200, dtype=torch.bfloat16, device="cuda")
    junk = torch.full((200,), 5.0, device="cuda")
    del junk
    q, s, qt, st, db = gn.act_grad_quant_fp8(z, z, epilogue=act)
    assert q.shape == (0, 200) and s.shape == (0, 2) and qt.shape == (200, 0) and st.shape == (200, 0) and (db == 0).all()


def test_helper_refusals(monkeypatch):
    monkeypatch.setattr(gn, "_on_gpu", lambda t: True)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    a, b = torch.zeros(4, 256).to(F8), torch.zeros(64, 256).to(F8)
    sa, sb = torch.zeros(4, 2), torch.zeros(1, 2)
    for f in (lambda: gn.norm_quant_fp8(x, torch.zeros(255, dtype=torch.bfloat16)), lambda: gn.norm_quant_fp8(x, torch.zeros(256)),
              lambda: gn.norm_quant_fp8(x.half()), lambda: gn.norm_quant_fp8(x.t()), lambda: gn.quant_fp8(x[None]),
              lambda: gn.quant_fp8(x, by_rows=False), lambda: gn.act_grad_quant_fp8(x, x[:2]), lambda: gn.act_grad_quant_fp8(x, x.float()),
              lambda: gn.act_grad_quant_fp8(x, None), lambda: gn.linear_fp8(x, sa, b, sb), lambda: gn.linear_fp8(a, sa, b[:, :128], sb),
              lambda: gn.linear_fp8(a, sa[:3], b, sb), lambda: gn.linear_fp8(a, sa, b, torch.zeros(2, 2)), lambda: gn.linear_fp8(a, sa.double(), b, sb),
              lambda: gn.linear_fp8(a, sa, b, sb, torch.zeros(63)), lambda: gn.linear_fp8(a, sa, b, sb, out=torch.zeros(4, 63)),
              lambda: gn.linear_fp8(a, torch.zeros(2, 4).t(), b, sb), lambda: gn.linear_fp8(a, sa, b, sb, accumulate=True, out_dtype=torch.float32),
              lambda: gn.linear_fp8(a, sa, b, sb, out=torch.zeros(4, 64), out_dtype=torch.bfloat16)):
        with pytest.raises((ValueError, TypeError)):
            f()


def test_stream_of_another_device_is_refused():
    class Tensor:
        is_cuda, device = True, torch.device("cuda", 1)

    class Stream:
        device = torch.device("cuda", 0)

    for f in (gn.groupnorm_fwd, gn.groupnorm_bwd, gn.norm_quant_fp8, gn.linear_fp8):
        with pytest.raises(ValueError, match="the stream is on"):
            f(Tensor(), stream=Stream())
