"""Cases of the GroupNorm, FP8 quantisation and FP8 product operators, for timing and comparison.

Five operators, each in a plain form (elementary torch operations in fp32, rounded once at the
end) and, where ``own`` is true, as the calls a program makes of ``transformer_norm_rope_b200``:

* ``groupnorm_fwd``: GroupNorm of channels-last images [N, S, C] (S = the flattened spatial
  positions) with an activation, and the saved statistics;
* ``groupnorm_bwd``: its backward from the saved statistics (dx, dw, db);
* ``norm_quant``: RMSNorm / LayerNorm of token rows, written in 8 bits (e4m3) with one fp32 scale
  for each 128 values of a row: the operand of the FP8 product behind the normalisation;
* ``quant``: 8-bit operands of the training products. "gradient": dz = dy act'(z) quantised along
  the channels (for dx) and, transposed, along the tokens (for dW), with the bias gradient;
  "both": a given matrix, both ways; "tile": a weight in 128 x 128 blocks, and transposed;
* ``linear``: y = act(A B^T + d) of two 8-bit operands with their block scales; B's scales one per
  128 x 128 block (a weight) or one per row and 128 values (a weight gradient, fp32 output).

A block's scale is amax / 448 (amax at least 2^-110); 448 is the largest e4m3 value.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -110
GELU_K = math.sqrt(2.0 / math.pi)
GELU_C = 0.044715
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the lowest resolution of an image network, one sample: latency counts; 10 channels a group
        dict(name="groupnorm_fwd small", op="groupnorm_fwd", N=1, S=63, C=320, G=32, dt="bf16", act="silu"),
        # the full resolution of an image decoder, a batch of four: memory-bound
        dict(name="groupnorm_fwd large", op="groupnorm_fwd", N=4, S=65536, C=512, G=32, dt="bf16", act="silu"),
        # the middle resolution of an image network in training; 20 channels a group
        dict(name="groupnorm_bwd middle", op="groupnorm_bwd", N=2, S=4096, C=640, G=32, dt="bf16", act="silu"),
        # a decoder's level in fp32 training, an odd picture size (127 x 129)
        dict(name="groupnorm_bwd fp32 odd", op="groupnorm_bwd", N=2, S=16383, C=256, G=32, dt="f32", act="gelu_tanh"),
        # one token through the norm in front of a projection
        dict(name="norm_quant one token", op="norm_quant", rows=1, hidden=5120, norm="rms", gemma=False, dt="bf16",
             act="none"),
        # a long video sequence through LayerNorm in front of a projection
        dict(name="norm_quant long", op="norm_quant", rows=32760, hidden=5120, norm="ln", gemma=False, dt="bf16",
             act="none"),
        # the gradient of a projection's pre-activation, a chunk of tokens of odd length
        dict(name="quant gradient", op="quant", form="gradient", rows=4093, cols=5120, dt="bf16", act="silu"),
        # a projection's weight after an optimiser step, for the forward and the input gradient
        dict(name="quant weight", op="quant", form="tile", rows=5120, cols=5120, dt="bf16", act="none"),
        # one token through a projection: the weight is read once
        dict(name="linear one token", op="linear", M=1, N=5120, K=5120, b_rows=128, act="silu", out="bf16"),
        # a short prompt through a projection onto an odd width
        dict(name="linear short", op="linear", M=333, N=1288, K=5120, b_rows=128, act="none", out="bf16"),
        # a long video sequence through a feed-forward projection
        dict(name="linear long", op="linear", M=32768, N=5120, K=5120, b_rows=128, act="gelu_tanh", out="bf16"),
        # a weight gradient over a chunk of tokens of odd length
        dict(name="linear weight gradient", op="linear", M=5120, N=5120, K=4093, b_rows=1, act="none", out="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["groupnorm_fwd", "groupnorm_bwd", "norm_quant", "quant", "linear", "linear"])
    if op.startswith("groupnorm"):
        G = rng.choice([1, 4, 8, 16, 32, 32])
        C = G * rng.randint(max(1, 32 // G), 1024 // G)
        N = rng.randint(1, 4)
        S = _log(rng, 1, min(65536, (2 ** 26 if op.endswith("fwd") else 2 ** 25) // (N * C)))
        return dict(op=op, N=N, S=S, C=C, G=G, dt=rng.choice(["bf16", "bf16", "f32"]),
                    act=rng.choice(["none", "silu", "gelu_tanh"]))
    if op == "norm_quant":
        hidden = _log(rng, 64, 8192)
        return dict(op=op, rows=_log(rng, 1, min(32768, 2 ** 27 // hidden)), hidden=hidden,
                    norm=rng.choice(["rms", "ln", "none"]), gemma=rng.random() < 0.3, dt=rng.choice(["bf16", "bf16", "f32"]),
                    act=rng.choice(["none", "none", "silu", "gelu_tanh"]))
    if op == "quant":
        form = rng.choice(["gradient", "both", "tile"])
        return dict(op=op, form=form, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192), dt=rng.choice(["bf16", "bf16", "f32"]),
                    act=rng.choice(["none", "silu", "gelu_tanh"]) if form == "gradient" else "none")
    if rng.random() < 0.3:
        return dict(op=op, M=_log(rng, 64, 5120), N=_log(rng, 64, 5120), K=_log(rng, 1, 8192), b_rows=1, act="none", out="f32")
    N, K = _log(rng, 64, 8192), _log(rng, 64, 8192)
    return dict(op=op, M=_log(rng, 1, 32768), N=N, K=K, b_rows=128, act=rng.choice(["none", "silu", "gelu_tanh"]), out="bf16")


# ---------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)


def _rows16(t, dtype):
    """t [..., cols] in `dtype`, its rows starting on 16-byte boundaries (a padded row stride where
    the width needs one), as a program lays out rows of an odd width."""
    es = torch.empty((), dtype=dtype).element_size()
    cols = t.shape[-1]
    ld = (cols * es + 15) // 16 * 16 // es
    if ld == cols:
        return t.to(dtype)
    base = torch.empty(t.shape[:-1] + (ld,), dtype=dtype, device=t.device)
    base[..., :cols] = t
    return base[..., :cols]


def _ceil(a, b):
    return -(-a // b)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    op = c["op"]
    if op.startswith("groupnorm"):
        N, S, C, G = c["N"], c["S"], c["C"], c["G"]
        dt = DTYPES[c["dt"]]
        x = _randn(gen, N, S, C) * (0.5 + 2.0 * _rand(gen, N, 1, C)) + 2.0 * _randn(gen, N, 1, C)
        st = dict(case=c, x=_rows16(x, dt), w=(1.0 + 0.1 * _randn(gen, C)).to(dt), b=(0.1 * _randn(gen, C)).to(dt), eps=1e-5)
        if op == "groupnorm_bwd":
            st["dy"] = _rows16(_randn(gen, N, S, C), dt)
            xs = st["x"].float().reshape(N, S, G, C // G)
            mean = xs.mean(dim=(1, 3), keepdim=True)
            st["rstd"] = torch.rsqrt((xs - mean).square().mean(dim=(1, 3)) + 1e-5)
            st["mean"] = mean.reshape(N, G).contiguous()
        return st
    if op == "norm_quant":
        rows, hidden, dt = c["rows"], c["hidden"], DTYPES[c["dt"]]
        x = _randn(gen, rows, hidden) * (0.5 + 2.5 * _rand(gen, rows, 1)) + (4.0 * _rand(gen, rows, 1) - 2.0)
        return dict(case=c, x=_rows16(x, dt), eps=1e-6 if c["norm"] == "rms" else 1e-5,
                    g=(0.1 * _randn(gen, hidden) + (0.0 if c["gemma"] else 1.0)).to(dt), beta=(0.1 * _randn(gen, hidden)).to(dt))
    if op == "quant":
        rows, cols, dt = c["rows"], c["cols"], DTYPES[c["dt"]]
        if c["form"] == "tile":
            return dict(case=c, x=_rows16(_randn(gen, rows, cols) / math.sqrt(cols), dt))
        st = dict(case=c, x=_rows16(_randn(gen, rows, cols), dt))
        if c["form"] == "gradient":
            st["dy"] = _rows16(_randn(gen, rows, cols) * torch.exp(_randn(gen, rows, 1)) * 1e-3, dt)
        return st
    M, N, K = c["M"], c["N"], c["K"]
    a = _randn(gen, M, K) * (0.5 + 2.0 * _rand(gen, M, 1))
    b = _randn(gen, N, K) / math.sqrt(K)
    aq, sa = _quant_rows(a)
    bq, sb = _quant_tiles(b) if c["b_rows"] == BLOCK else _quant_rows(b)
    d = 0.1 * _randn(gen, N) if c["out"] == "bf16" else None
    return dict(case=c, aq=_codes16(aq), sa=sa, bq=_codes16(bq), sb=sb, d=d)


def _codes16(q):
    cols = q.shape[1]
    if cols % 16 == 0:
        return q
    base = torch.zeros((q.shape[0], (cols + 15) // 16 * 16), dtype=torch.uint8, device=q.device)
    base[:, :cols] = q.view(torch.uint8)
    return base.view(torch.float8_e4m3fn)[:, :cols]


# ---------------------------------------------------------------- the operators in plain form

def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(GELU_K * (z + GELU_C * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu_tanh":
        t = torch.tanh(GELU_K * (z + GELU_C * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_K * (1.0 + 3.0 * GELU_C * z * z)
    return torch.ones_like(z)


def _scale(amax):
    """amax / 448; NaN for a block that holds a NaN or an infinity."""
    s = amax.clamp_min(AMAX_FLOOR) / E4M3_MAX
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, float("nan")))


def _pad(x, r, c):
    rows, cols = x.shape
    if rows % r == 0 and cols % c == 0:
        return x
    p = torch.zeros((_ceil(rows, r) * r, _ceil(cols, c) * c), dtype=x.dtype, device=x.device)
    p[:rows, :cols] = x
    return p


def _quant_rows(x):
    """e4m3 codes of x [rows, cols] fp32 and the scales [rows, ceil(cols / 128)]."""
    rows, cols = x.shape
    p = _pad(x, 1, BLOCK).reshape(rows, -1, BLOCK)
    s = _scale(p.abs().amax(dim=2))
    q = (p / s[:, :, None]).reshape(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    return q.contiguous(), s


def _quant_tiles(x):
    rows, cols = x.shape
    p = _pad(x, BLOCK, BLOCK)
    p = p.reshape(p.shape[0] // BLOCK, BLOCK, p.shape[1] // BLOCK, BLOCK)
    s = _scale(p.abs().amax(dim=3).amax(dim=1))
    q = (p / s[:, None, :, None]).reshape(p.shape[0] * BLOCK, -1)[:rows, :cols].to(torch.float8_e4m3fn)
    return q.contiguous(), s


def _plain_groupnorm_fwd(st):
    c = st["case"]
    N, S, C, G = c["N"], c["S"], c["C"], c["G"]
    x = st["x"].float().reshape(N, S, G, C // G)
    mean = x.mean(dim=(1, 3), keepdim=True)
    x = x - mean
    rstd = 1.0 / torch.sqrt((x * x).mean(dim=(1, 3), keepdim=True) + st["eps"])
    z = (x * rstd).reshape(N, S, C) * st["w"].float() + st["b"].float()
    return _act(z, c["act"]).to(st["x"].dtype), mean.reshape(N, G), rstd.reshape(N, G)


def _plain_groupnorm_bwd(st):
    c = st["case"]
    N, S, C, G = c["N"], c["S"], c["C"], c["G"]
    w, b = st["w"].float(), st["b"].float()
    xhat = ((st["x"].float().reshape(N, S, G, C // G) - st["mean"].reshape(N, 1, G, 1)) * st["rstd"].reshape(N, 1, G, 1))
    xhat = xhat.reshape(N, S, C)
    g = st["dy"].float() * _act_grad(xhat * w + b, c["act"])
    dw, db = (g * xhat).sum(dim=(0, 1)), g.sum(dim=(0, 1))
    gw = (g * w).reshape(N, S, G, C // G)
    xh = xhat.reshape(N, S, G, C // G)
    m1, m2 = gw.mean(dim=(1, 3), keepdim=True), (gw * xh).mean(dim=(1, 3), keepdim=True)
    dx = st["rstd"].reshape(N, 1, G, 1) * (gw - m1 - xh * m2)
    return dx.reshape(N, S, C).to(st["x"].dtype), dw, db


def _plain_norm_quant(st):
    c = st["case"]
    x, g = st["x"].float(), st["g"].float()
    stats = []
    if c["norm"] == "ln":
        mean = x.mean(dim=1, keepdim=True)
        x = x - mean
        rstd = 1.0 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + st["eps"])
        z = x * rstd * g + st["beta"].float()
        stats = [mean.reshape(-1), rstd.reshape(-1)]
    elif c["norm"] == "rms":
        rstd = 1.0 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + st["eps"])
        z = x * rstd * (1.0 + g if c["gemma"] else g)
        stats = [rstd.reshape(-1)]
    else:
        z = x
    q, s = _quant_rows(_act(z, c["act"]))
    return [q, s] + stats


def _plain_quant(st):
    c = st["case"]
    x = st["x"].float()
    if c["form"] == "tile":
        q, s = _quant_tiles(x)
        return q, s, q.t().contiguous(), s.t().contiguous()
    v = st["dy"].float() * _act_grad(x, c["act"]) if c["form"] == "gradient" else x
    q, s = _quant_rows(v)
    qt, s_t = _quant_rows(v.t().contiguous())
    return (q, s, qt, s_t, v.sum(dim=0)) if c["form"] == "gradient" else (q, s, qt, s_t)


def _spread(s, rows, cols, per):
    """scales [ceil(rows / per), ceil(cols / 128)] as one value per element of [rows, cols]"""
    if per > 1:
        s = s.repeat_interleave(per, dim=0)[:rows]
    return s.repeat_interleave(BLOCK, dim=1)[:, :cols]


def _plain_linear(st):
    c = st["case"]
    M, N, K = c["M"], c["N"], c["K"]
    a = st["aq"].float() * _spread(st["sa"], M, K, 1)
    b = st["bq"].float() * _spread(st["sb"], N, K, c["b_rows"])
    y = a @ b.t()
    if st["d"] is not None:
        y = y + st["d"]
    y = _act(y, c["act"])
    return y.to(torch.bfloat16) if c["out"] == "bf16" else y


PLAIN = {"groupnorm_fwd": _plain_groupnorm_fwd, "groupnorm_bwd": _plain_groupnorm_bwd, "norm_quant": _plain_norm_quant,
         "quant": _plain_quant, "linear": _plain_linear}


# ---------------------------------------------------------------- one pass

def _own_run(st):
    import transformer_norm_rope_b200 as gn

    c = st["case"]
    op = c["op"]
    if op == "groupnorm_fwd":
        return gn.groupnorm_fwd(st["x"], c["G"], st["w"], st["b"], st["eps"], epilogue=c["act"])
    if op == "groupnorm_bwd":
        return gn.groupnorm_bwd(st["x"], c["G"], st["w"], st["b"], st["mean"], st["rstd"], st["dy"], epilogue=c["act"])
    if op == "norm_quant":
        norm = c["norm"]
        q, s, mean, rstd = gn.norm_quant_fp8(st["x"], None if norm == "none" else st["g"], st["beta"] if norm == "ln" else None,
                                             st["eps"], norm=norm, gemma=c["gemma"], epilogue=c["act"])
        return [q, s] + ([mean, rstd] if norm == "ln" else [rstd] if norm == "rms" else [])
    if op == "quant":
        if c["form"] == "gradient":
            return gn.act_grad_quant_fp8(st["x"], st["dy"], epilogue=c["act"])
        return gn.quant_fp8(st["x"], tile=c["form"] == "tile", transposed=True)
    return gn.linear_fp8(st["aq"], st["sa"], st["bq"], st["sb"], st["d"], epilogue=c["act"], out_dtype=DTYPES[c["out"]])


def run(state):
    if own:
        return _own_run(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    op = c["op"]
    es = 2 if c.get("dt", c.get("out")) == "bf16" else 4
    if op.startswith("groupnorm"):
        n = c["N"] * c["S"] * c["C"]
        stats, params = 8 * c["N"] * c["G"], 2 * c["C"] * es
        if op == "groupnorm_fwd":
            return {"bytes": 2 * n * es + params + stats, "flops": 10 * n}
        return {"bytes": 3 * n * es + params + stats + 8 * c["C"], "flops": 30 * n}
    if op == "norm_quant":
        n = c["rows"] * c["hidden"]
        vectors = {"ln": 2, "rms": 1, "none": 0}[c["norm"]]
        scales = 4 * c["rows"] * _ceil(c["hidden"], BLOCK)
        return {"bytes": n * (es + 1) + scales + vectors * (c["hidden"] * es + 4 * c["rows"]), "flops": 10 * n}
    if op == "quant":
        n = c["rows"] * c["cols"]
        rb, cb = _ceil(c["rows"], BLOCK), _ceil(c["cols"], BLOCK)
        if c["form"] == "tile":
            return {"bytes": n * (es + 2) + 8 * rb * cb, "flops": 4 * n}
        grad = c["form"] == "gradient"
        return {"bytes": n * ((2 if grad else 1) * es + 2) + 4 * (c["rows"] * cb + c["cols"] * rb) + (4 * c["cols"] if grad else 0),
                "flops": (20 if grad else 6) * n}
    M, N, K = c["M"], c["N"], c["K"]
    kb = _ceil(K, BLOCK)
    return {"bytes": M * K + N * K + M * N * es + 4 * kb * (M + _ceil(N, c["b_rows"])) + (4 * N if c["out"] == "bf16" else 0),
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the same from the definitions, in 64 bits

def _exact_act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))  # (1 + tanh u) / 2 = sigmoid(2u)
    return z


def _exact_act_grad(z, act):
    with torch.enable_grad():
        v = z.detach().clone().requires_grad_(True)
        return torch.autograd.grad(_exact_act(v, act).sum(), v)[0]


def _e4m3(v):
    """The nearest e4m3 value (ties to the even mantissa), as a double: steps of 2^(e - 3) for 2^e <= |v| < 2^(e + 1),
    e at least -6."""
    m = v.abs()
    e = torch.floor(torch.log2(m.clamp_min(2.0 ** -6)))
    e = e + (torch.exp2(e + 1) <= m).double() - (torch.exp2(e) > m.clamp_min(2.0 ** -6)).double()
    step = torch.exp2(e - 3)
    return torch.sign(v) * torch.clamp(torch.round(m / step) * step, max=448.0)


def _exact_quant(v, down, across):
    """(values of the codes, scales) of the double matrix v in blocks of down x across."""
    rows, cols = v.shape
    R, Q = -(-rows // down), -(-cols // across)
    amax = torch.zeros((R, Q), dtype=torch.float64, device=v.device)
    for j in range(Q):
        top = v[:, j * across:(j + 1) * across].abs().amax(dim=1)
        if down > 1:
            top = torch.nn.functional.pad(top, (0, R * down - rows)).reshape(R, down).amax(dim=1)
        amax[:, j] = top
    s = torch.clamp(amax, min=2.0 ** -110) / 448.0
    held = s.float().double()  # the scale as it is held: the codes are of v over this value
    q = torch.empty_like(v)
    for j in range(Q):
        col = held[:, j].repeat_interleave(down)[:rows] if down > 1 else held[:, j]
        q[:, j * across:(j + 1) * across] = _e4m3(v[:, j * across:(j + 1) * across] / col[:, None])
    return q, s


def _exact_groups(t, N, S, G):
    return t.reshape(N, S, G, -1).permute(0, 2, 1, 3).reshape(N, G, -1)


def exact(case, seed):
    st = prepare(case, seed)
    c, op = st["case"], case["op"]
    if op.startswith("groupnorm"):
        N, S, C, G = c["N"], c["S"], c["C"], c["G"]
        w, b = st["w"].double(), st["b"].double()
        ys, means, rstds, dxs = [], [], [], []
        dw, db = torch.zeros(C, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
        for n in range(N):  # image by image: bounded memory
            x = st["x"][n].double()
            if op == "groupnorm_fwd":
                xg = _exact_groups(x, 1, S, G)[0]
                var, mu = torch.var_mean(xg, dim=1, correction=0)
                r = (var + st["eps"]) ** -0.5
                z = (x - mu.repeat_interleave(C // G)) * r.repeat_interleave(C // G) * w + b
                ys.append(_exact_act(z, c["act"]))
                means.append(mu)
                rstds.append(r)
            else:
                mu, r = (t[n].double().repeat_interleave(C // G) for t in (st["mean"], st["rstd"]))
                xhat = (x - mu) * r
                g = st["dy"][n].double() * _exact_act_grad(xhat * w + b, c["act"])
                dw += (g * xhat).sum(0)
                db += g.sum(0)
                p, q = _exact_groups(g * w, 1, S, G)[0].mean(1), _exact_groups(g * w * xhat, 1, S, G)[0].mean(1)
                dxs.append(r * (g * w - p.repeat_interleave(C // G) - xhat * q.repeat_interleave(C // G)))
        if op == "groupnorm_fwd":
            return torch.stack(ys), torch.stack(means), torch.stack(rstds)
        return torch.stack(dxs), dw, db
    if op == "norm_quant":
        x, g, stats = st["x"].double(), st["g"].double(), []
        if c["norm"] == "ln":
            var, mu = torch.var_mean(x, dim=1, correction=0)
            r = (var + st["eps"]) ** -0.5
            x = (x - mu[:, None]) * r[:, None] * g + st["beta"].double()
            stats = [mu, r]
        elif c["norm"] == "rms":
            r = (x.square().mean(dim=1) + st["eps"]) ** -0.5
            x = x * r[:, None] * (g + 1.0 if c["gemma"] else g)
            stats = [r]
        return list(_exact_quant(_exact_act(x, c["act"]), 1, 128)) + stats
    if op == "quant":
        x = st["x"].double()
        if c["form"] == "tile":
            q, s = _exact_quant(x, 128, 128)
            return q, s, q.t().contiguous(), s.t().contiguous()
        if c["form"] == "gradient":
            x = st["dy"].double() * _exact_act_grad(x, c["act"])
        q, s = _exact_quant(x, 1, 128)
        qt, s_t = _exact_quant(x.t().contiguous(), 1, 128)
        return (q, s, qt, s_t, x.sum(0)) if c["form"] == "gradient" else (q, s, qt, s_t)
    M, N, K = c["M"], c["N"], c["K"]
    y = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    for j in range(-(-K // 128)):  # block by block of the contraction
        cols = slice(128 * j, 128 * (j + 1))
        sb = st["sb"][:, j].double()
        if c["b_rows"] == 128:
            sb = sb.repeat_interleave(128)[:N]
        y.addmm_(st["aq"][:, cols].double() * st["sa"][:, j:j + 1].double(), (st["bq"][:, cols].double() * sb[:, None]).t())
    if st["d"] is not None:
        y += st["d"].double()
    return _exact_act(y, c["act"])
