"""GPU parity of the dense feed-forward operators against their definitions in 64 bits.

Tolerances.  u = 2^-24 (half a step of fp32), b = 2^-8 (half a step of bf16).
  * A dot product of exact terms summed in fp32 in any order is off by at most
    n u sum|terms| (first order); n + 8 covers the bias and the second order.
  * The activations are built from 1-ulp exponentials, reciprocals and erf: act(z) and act'(z)
    are off by at most 2^-20 (1 + |z|), and change by at most 1.13 per unit of z.
  * A stored bf16 value adds b |value|, and 2^-133 where it is subnormal.
  * dz is rounded to bf16 for dx where there is an activation: b sum|dz w|.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U, B, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -133
ACT_ERR, ACT_LIP = 2.0 ** -20, 1.13
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid"]
EPS = 1e-6


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import mxfp4_weight_moe_amd
    return mxfp4_weight_moe_amd


DEV = "cuda:0"


def say(*a):
    print(*a, flush=True)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def bf(*shape, g, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std + mean).to(torch.bfloat16)


def weights(rows, K, g, lo=115, hi=122):
    w = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(lo, hi, (rows, K // 32), generator=g, dtype=torch.uint8)
    return w, s


def decode(w, s):
    t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    v = torch.stack((t[(w & 15).long()], t[(w >> 4).long()]), -1).reshape(w.shape[0], -1, 32)
    p = torch.where(s == 255, torch.full(s.shape, math.nan, dtype=torch.float64),
                    torch.ldexp(torch.ones(s.shape, dtype=torch.float64), s.int() - 127))
    return (v * p[..., None]).flatten(1)


def act(z, kind):
    """(value, slope) in 64 bits."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0), (z > 0).double()
    if kind == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        p = torch.sigmoid(2 * k * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * 2 * k * (1 + 3 * 0.044715 * z * z)
    p = torch.sigmoid(z)
    return (p, p * (1 - p)) if kind == "sigmoid" else (z * p, p + z * p * (1 - p))


def within(got, want, tol, what):
    got, want, tol = got.double().cpu(), want.expand(got.shape), torch.as_tensor(tol).double().expand(got.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN at other places"
    fine = ~want.isnan()
    inf = fine & (want.isinf() | got.isinf())
    assert torch.equal(got[inf], want[inf]), f"{what}: Inf at other places"
    fine &= ~inf
    r = ((got - want).abs() / (tol + TINY))[fine]
    worst = float(r.max()) if r.numel() else 0.0
    assert worst <= 1, f"{what}: {int((r > 1).sum())} of {r.numel()} out of bound, worst {worst:.3g}"
    return worst


def cuda(*ts):
    return [t.to(DEV) if isinstance(t, torch.Tensor) else t for t in ts]


def z_of(x, w, s, bias):
    """z and the bound of its error."""
    W = decode(w, s)
    z = x.double() @ W.T
    size = x.double().abs() @ W.abs().T
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    return z, (x.shape[1] + 8) * U * size


def value_error(z, ez, a):
    return ACT_LIP * ez + ACT_ERR * (1 + z.abs())


# ------------------------------------------------------------------ linear

# streaming (few tokens, K < 128), thin tiles (9 to 128 tokens, 1, 2 and 4 parts of K in a
# workgroup, fewer stages than parts, over several workgroups), tiles of 64 (K % 128 != 0), 128 and
# 256 rows, split and whole K, odd rows and columns, K tails of 32, 64 and 96
LINEAR_SHAPES = [(1, 256, 64), (1, 32, 1), (2, 96, 7), (5, 512, 33), (16, 288, 16), (17, 2048, 40), (31, 256, 100),
                 (32, 160, 264), (33, 128, 8), (40, 32, 1), (64, 544, 130), (65, 256, 64), (77, 2048, 257),
                 (129, 96, 300), (300, 512, 520), (1025, 192, 264), (1300, 256, 65), (1100, 32, 512),
                 (128, 2048, 33), (97, 1024, 6200), (50, 2080, 70), (120, 1056, 64), (200, 2048, 129), (200, 2080, 65),
                 (130, 4096, 64), (4100, 544, 2100), (4200, 128, 2060), (4097, 1024, 2049),
                 (12, 384, 40), (16, 8192, 40), (9, 128, 4300), (13, 512, 4200), (24, 128, 300), (25, 16384, 70),
                 (48, 384, 33), (59, 8192, 100), (64, 128, 65), (90, 4096, 100), (3, 256, 4200), (3, 160, 9000),
                 (8, 16384, 24), (5, 384, 40), (7, 4224, 70)]


def linear_inputs(T, K, N, seed):
    g = gen(seed)
    return (bf(T, K, g=g), *weights(N, K, g), bf(N, g=g, std=0.5), bf(T, N, g=g))


def check_linear(y, z_got, x, w, s, bias, res, scale, kind):
    z, ez = z_of(x, w, s, bias)
    a, _ = act(z, kind)
    want, err = scale * a, abs(scale) * value_error(z, ez, a)
    if res is not None:
        want, err = want + res.double(), err + U * (want + res.double()).abs()
    worst = within(y, want, (1 + B) * err + B * want.abs(), "y")
    if z_got is not None:
        within(z_got, z, (1 + B) * ez + B * z.abs(), "z")
    return worst


@pytest.mark.parametrize("T,K,N", LINEAR_SHAPES)
def test_linear(mx, T, K, N):
    for i, (kind, has_bias, has_res, scale, save) in enumerate([
            ("none", False, False, 1.0, False), ("gelu_tanh", True, True, 0.5, True), ("silu", True, False, -2.0, False),
            ("none", False, True, 0.25, True)]):
        x, w, s, bias, res = linear_inputs(T, K, N, 100 * T + K + N + i)
        bias, res = bias if has_bias else None, res if has_res else None
        say("linear", T, K, N, kind, has_bias, has_res)
        r = mx.mx_linear_fused(*cuda(x, w, s), *cuda(bias, res), scale, kind, save_z=save)
        y, z = r if save else (r, None)
        say("   worst", check_linear(y, z, x, w, s, bias, res, scale, kind))


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("T", [3, 50])
def test_linear_activations(mx, T, kind):
    x, w, s, bias, res = linear_inputs(T, 256, 48, 7)
    x = (x * torch.linspace(0, 12, T)[:, None]).to(torch.bfloat16)  # pre-activations from 0 to beyond 30
    say("act", kind, T)
    y, z = mx.mx_linear_fused(*cuda(x, w, s, bias, res), 1.0, kind, save_z=True)
    check_linear(y, z, x, w, s, bias, res, 1.0, kind)


@pytest.mark.parametrize("T", [1, 20, 40, 100, 1030])
def test_linear_nan_inf_and_neighbours(mx, T):
    K, N = 288, 72
    x, w, s, bias, res = linear_inputs(T, K, N, 11)
    s[5, 3] = 255          # a NaN scale: column 5 alone
    x[T // 2, 17] = math.nan   # a NaN activation: its row alone
    if T > 2:
        x[0, K - 1] = math.inf
    say("nan", T)
    xd, wd, sd = cuda(x, w, s)
    out = torch.full((T + 3, N), 7.0, dtype=torch.bfloat16, device=DEV)
    y = mx.mx_linear_fused(xd, wd, sd, out=out[:T])
    z = x.double() @ decode(w, s).T
    size = (x.double().abs() @ decode(w, s).abs().T).nan_to_num(0, 0, 0)
    # Inf times a zero weight is NaN in the definition and on the GPU alike
    within(y, z, (K + 8) * U * 1.01 * size + B * z.abs().nan_to_num(0, 0, 0), "y")
    assert bool((out[T:] == 7).all()), "rows behind the last were written"


def test_linear_in_place_residual_and_repeat(mx):
    for T, K, N in ((4, 512, 64), (40, 2048, 64), (200, 256, 129), (1100, 256, 264)):
        x, w, s, bias, res = cuda(*linear_inputs(T, K, N, 21))
        say("in place", T)
        a = mx.mx_linear_fused(x, w, s, bias, res, 0.5, "relu")
        b = mx.mx_linear_fused(x, w, s, bias, res, 0.5, "relu")
        buf = res.clone()
        c = mx.mx_linear_fused(x, w, s, bias, buf, 0.5, "relu", out=buf)
        assert torch.equal(a, b) and torch.equal(a, c) and c.data_ptr() == buf.data_ptr()


# ------------------------------------------------------------------ linear, backward

def check_dx(dx, dz, edz, w, s, rounded, N):
    W = decode(w, s)
    want, size = dz @ W, dz.abs() @ W.abs()
    err = edz @ W.abs() + (N + 8) * U * size + (B * size if rounded else 0)
    return within(dx, want, (1 + B) * err + B * want.abs(), "dx")


BWD_SHAPES = [(1, 32, 1), (1, 256, 64), (3, 96, 7), (33, 128, 16), (64, 288, 130), (65, 160, 257), (100, 512, 520),
              (129, 544, 33), (700, 96, 72), (1025, 256, 264), (1100, 32, 100), (1030, 288, 65),
              (4, 128, 1000), (70, 256, 1090), (200, 544, 4160), (4100, 2112, 200), (4130, 2080, 64), (4100, 2176, 1)]


@pytest.mark.parametrize("T,K,N", BWD_SHAPES)
def test_linear_backward(mx, T, K, N):
    for kind, scale in (("none", 0.5), ("silu", 1.0), ("gelu", -2.0)):
        g = gen(T + K + N)
        w, s = weights(N, K, g)
        dy, z = bf(T, N, g=g), bf(T, N, g=g, std=1.5)
        say("linear backward", T, K, N, kind)
        dx, db = mx.mx_linear_fused_backward(*cuda(dy, w, s), None if kind == "none" else z.to(DEV), scale, kind)
        slope = act(z.double(), kind)[1]
        dz = scale * dy.double() * slope
        edz = abs(scale) * dy.double().abs() * ((ACT_ERR * (1 + z.double().abs()) if kind != "none" else 0) + 4 * U)
        say("   worst", check_dx(dx, dz, edz, w, s, kind != "none", N))
        within(db, dz.sum(0), edz.sum(0) + (T + 8) * U * dz.abs().sum(0), "dbias")
        only = mx.mx_linear_fused_backward(*cuda(dy, w, s), z.to(DEV), scale, kind, need_dx=False)
        assert only[0] is None and torch.equal(only[1], db)
        again = mx.mx_linear_fused_backward(*cuda(dy, w, s), z.to(DEV), scale, kind, need_dbias=False)
        assert again[1] is None and torch.equal(again[0], dx)


@pytest.mark.parametrize("kind", ["relu", "silu", "gelu", "gelu_tanh", "sigmoid"])
def test_far_values(mx, kind):
    """Where squares and cubes of z overflow, activations and slopes are their limits."""
    z = torch.tensor([[1e15, -1e15, 1e20, -1e20, 1e30, -1e30, 3e38, -3e38]]).bfloat16()
    N, K = 8, 32
    w = torch.zeros(N, K // 2, dtype=torch.uint8)
    s = torch.full((N, 1), 127, dtype=torch.uint8)
    dy = torch.arange(1.0, 9.0).reshape(1, N).bfloat16()
    pos = (z > 0).double()
    say("far values", kind)
    y = mx.mx_linear_fused(*cuda(torch.zeros(1, K, dtype=torch.bfloat16), w, s), bias=z[0].to(DEV), act=kind)
    assert torch.equal(y.double().cpu(), pos if kind == "sigmoid" else pos * z.double())
    db = mx.mx_linear_fused_backward(*cuda(dy, w, s, z), 1.0, kind, need_dx=False)[1]
    assert torch.equal(db.double().cpu(), (dy.double() * pos * (kind != "sigmoid"))[0])


def test_backward_nan_and_neighbours(mx):
    for T in (2, 70, 1030):
        g = gen(T)
        N, K = 72, 96
        w, s = weights(N, K, g)
        s[9, 1] = 255
        dy = bf(T, N, g=g)
        dy[T // 2, 3] = math.nan
        say("backward nan", T)
        dx, db = mx.mx_linear_fused_backward(*cuda(dy, w, s))
        W = decode(w, s)
        want = dy.double() @ W
        size = (dy.double().abs() @ W.abs()).nan_to_num(0)
        within(dx, want, (N + 8) * U * 1.01 * size + B * want.abs().nan_to_num(0), "dx")
        assert db.isnan().nonzero().flatten().tolist() == [3]


# ------------------------------------------------------------------ gate_up

GATED_SHAPES = [(1, 256, 64), (1, 32, 1), (3, 96, 7), (16, 288, 33), (17, 512, 16), (32, 160, 100), (33, 128, 8),
                (64, 544, 65), (65, 1024, 130), (130, 96, 257), (1025, 192, 136), (1100, 256, 33), (1030, 32, 264),
                (128, 2048, 72), (90, 1024, 3100), (200, 2048, 40), (4100, 288, 1050), (4097, 512, 1031),
                (12, 640, 24), (10, 256, 2100), (32, 16384, 20), (20, 128, 9), (60, 8192, 33), (41, 256, 100),
                (90, 4096, 60), (3, 256, 2100), (5, 16384, 17)]


@pytest.mark.parametrize("T,H,I", GATED_SHAPES)
def test_gate_up(mx, T, H, I):
    for kind, has_bias, save in (("silu", False, False), ("gelu_tanh", True, True), ("none", True, False)):
        g = gen(T + H + I)
        x, (w, s), bias = bf(T, H, g=g), weights(2 * I, H, g), bf(2 * I, g=g, std=0.5)
        bias = bias if has_bias else None
        say("gate_up", T, H, I, kind)
        r = mx.mx_gate_up(*cuda(x, w, s, bias), kind, save_z=save)
        h, z_got = r if save else (r, None)
        z, ez = z_of(x, w, s, bias)
        a = act(z[:, :I], kind)[0]
        want = a * z[:, I:]
        err = value_error(z[:, :I], ez[:, :I], a) * (z[:, I:].abs() + ez[:, I:]) + a.abs() * ez[:, I:] + U * want.abs()
        say("   worst", within(h, want, (1 + B) * err + B * want.abs(), "h"))
        if save:
            within(z_got, z, (1 + B) * ez + B * z.abs(), "z")


@pytest.mark.parametrize("kind", ACTS)
def test_gate_up_backward(mx, kind):
    for T, H, I in ((1, 32, 1), (5, 96, 33), (64, 288, 64), (130, 160, 65), (1030, 128, 72), (700, 512, 257)):
        g = gen(T + H + I)
        w, s = weights(2 * I, H, g)
        dh, z = bf(T, I, g=g), bf(T, 2 * I, g=g, std=1.5)
        say("gate_up backward", T, H, I, kind)
        dx, db = mx.mx_gate_up_backward(*cuda(dh, z, w, s), kind)
        gt, up, d = z[:, :I].double(), z[:, I:].double(), dh.double()
        a, slope = act(gt, kind)
        dz = torch.cat((d * up * slope, d * a), 1)
        e = ACT_ERR * (1 + gt.abs()) if kind != "none" else torch.zeros_like(gt)
        edz = torch.cat((d.abs() * up.abs() * e, d.abs() * e), 1) + 4 * U * dz.abs()
        say("   worst", check_dx(dx, dz, edz, w, s, True, 2 * I))
        within(db, dz.sum(0), edz.sum(0) + (T + 8) * U * dz.abs().sum(0), "dbias")
        assert torch.equal(mx.mx_gate_up_backward(*cuda(dh, z, w, s), kind, need_dx=False)[1], db)


def test_gradients_against_differences():
    """The gradient formulas used above against central differences of the forward's, in 64 bits."""
    g = gen(3)
    T, I = 5, 6
    z = torch.randn(T, 2 * I, generator=g, dtype=torch.float64)
    d = torch.randn(T, I, generator=g, dtype=torch.float64)
    dirn = torch.randn(T, 2 * I, generator=g, dtype=torch.float64)
    for kind in ACTS:
        f = lambda v: float((d * act(v[:, :I], kind)[0] * v[:, I:]).sum())  # noqa: B023, E731
        a, slope = act(z[:, :I], kind)
        grad = torch.cat((d * z[:, I:] * slope, d * a), 1)
        h = 1e-5
        assert abs((f(z + h * dirn) - f(z - h * dirn)) / (2 * h) - float((grad * dirn).sum())) < 1e-7
    x, b = torch.randn(T, 16, generator=g, dtype=torch.float64), torch.randn(T, 16, generator=g, dtype=torch.float64)
    wo, wi = torch.rand(16, generator=g, dtype=torch.float64) + 0.5, torch.rand(16, generator=g, dtype=torch.float64) + 0.5
    gate, c1, c2 = (torch.randn(T, 16, generator=g, dtype=torch.float64) for _ in range(3))
    args = [x, b, wo, gate, wi]

    def total(x, b, wo, gate, wi):
        y, xn = norm_forward(x, b, wo, gate, 0.7, wi)
        return float((c1 * y + c2 * xn).sum())

    y, _ = norm_forward(*args[:4], 0.7, wi)
    gr = norm_grads(c1, c2, y, b, wo, gate, 0.7, wi, "full")
    for i, name in enumerate(("dx", "db", "dw_post", "dgate", "dw_pre")):
        v = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + 1e-5 * v, args[i] - 1e-5 * v
        diff = (total(*hi) - total(*lo)) / 2e-5
        assert abs(diff - float((gr[name][0] * v).sum())) < 1e-6, name


# ------------------------------------------------------------------ norms

def rms(v):
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def norm_forward(x, b, w_post, gate, scale, w_pre):
    """(y, xn) in 64 bits, y not rounded."""
    y = x
    if b is not None:
        n = b if w_post is None else b * rms(b) * w_post
        y = x + scale * (n if gate is None else n * gate)
    return y, (None if w_pre is None else y * rms(y) * w_pre)


def norm_grads(dy, dxn, y, b, w_post, gate, scale, w_pre, mode):
    """{name: (gradient, sum of the sizes of its terms)} in 64 bits."""
    out = {}
    D = dy if dy is not None else torch.zeros_like(y)
    size = D.abs()
    if w_pre is not None:
        r, t = rms(y), dxn * w_pre
        out["dw_pre"] = ((dxn * y * r).sum(0), (dxn * y * r).abs().sum(0))
        D = D + r * (t - y * r * r * (t * y).mean(1, keepdim=True))
        size = size + r * (t.abs() + y.abs() * r * r * (t * y).abs().mean(1, keepdim=True))
    out["dx"] = (D, size)
    if b is None:
        return out
    q = rms(b) if w_post is not None else torch.ones_like(y[:, :1])
    w = w_post if w_post is not None else torch.ones_like(y[0])
    e, es = scale * D, abs(scale) * size
    if gate is not None:
        dg, ds = e * b * q * w, es * (b * q * w).abs()
        f = {"channel": lambda v: v.sum(0), "token": lambda v: v.sum(1, keepdim=True), "full": lambda v: v}[mode]
        out["dgate"] = (f(dg), f(ds))
        e, es = e * gate, es * gate.abs()
    if w_post is not None:
        out["dw_post"] = ((e * b * q).sum(0), (es * (b * q).abs()).sum(0))
        t, ts = e * w, es * w.abs()
        e = q * (t - b * q * q * (t * b).mean(1, keepdim=True))
        es = q * (ts + b.abs() * q * q * (ts * b.abs()).mean(1, keepdim=True))
    out["db"] = (e, es)
    return out


# every kernel width (one wave up to 1024 threads), rows that fill it and odd ones
# rows of a quarter and half a wave, of 1 to 16 waves, and more than one piece a thread; several
# rows a workgroup
NORM_SHAPES = [(1, 8), (3, 64), (5, 512), (2, 520), (33, 1000), (7, 2048), (4, 2056), (9, 4096), (600, 72), (3, 7168),
               (5, 8200), (2, 16384), (1030, 264), (2100, 40), (2050, 128), (701, 136), (1031, 256), (300, 1024),
               (260, 8704)]
NORM_KINDS = [("full", True, True), ("none", True, True), ("channel", True, True), ("token", True, False),
              ("token", False, True), ("channel", False, False), ("none", False, True), (None, False, True)]


def norm_inputs(T, H, kind, post, pre, seed):
    g = gen(seed)
    x, b = bf(T, H, g=g, std=2.0), bf(T, H, g=g, std=0.7)
    wo, wi = bf(H, g=g, std=0.1, mean=1.0), bf(H, g=g, std=0.1, mean=1.0)
    shape = {"full": (T, H), "channel": (H,), "token": (T, 1)}.get(kind)
    gate = bf(*shape, g=g, std=0.4, mean=0.5) if shape else None
    if T > 1:
        b[1] = 0  # a block that gives nothing: the norm divides by sqrt(eps)
    return x, (b if kind else None), (wo if post else None), gate, (wi if pre else None), bf(T, H, g=g), bf(T, H, g=g)


def dbl(t):
    return None if t is None else t.double()


@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_norm(mx, T, H):
    # a mean of H squares in fp32, then a reciprocal root and three products
    d = (H + 16) * U
    for kind, post, pre in NORM_KINDS:
        x, b, wo, gate, wi, _, _ = norm_inputs(T, H, kind, post, pre, T + H)
        say("norm", T, H, kind, post, pre)
        y, xn = mx.mx_norm_residual(*cuda(x, b), *cuda(wo, gate), 0.7, wi if wi is None else wi.to(DEV), EPS)
        want, _ = norm_forward(dbl(x), dbl(b), dbl(wo), dbl(gate), float(np.float32(0.7)), None)
        if b is not None:
            err = d * (want - x.double()).abs() + U * want.abs()
            within(y, want, (1 + B) * err + B * want.abs(), "y")
        if pre:
            yy = y.double().cpu()
            xw = yy * rms(yy) * wi.double()
            within(xn, xw, ((1 + B) * d + B) * xw.abs(), "xn")


@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_norm_backward(mx, T, H):
    # sums of H terms (means) and of T (parameter gradients), each on values off by a few u
    d = (2 * H + 64) * U
    for kind, post, pre in NORM_KINDS:
        y, b, wo, gate, wi, dy, dxn = norm_inputs(T, H, kind, post, pre, 3 * T + H)
        dy = None if (kind == "none" and pre) else dy
        dxn = dxn if pre else None
        say("norm backward", T, H, kind, post, pre)
        got = mx.mx_norm_residual_backward(*cuda(dy, dxn, y, b), *cuda(wo, gate), 0.7, wi if wi is None else wi.to(DEV), EPS)
        want = norm_grads(dbl(dy), dbl(dxn), dbl(y), dbl(b), dbl(wo), dbl(gate), float(np.float32(0.7)), dbl(wi), kind)
        assert {k for k, v in got.items() if v is not None} == set(want)
        for name, (v, size) in want.items():
            rounded = B if got[name].dtype == torch.bfloat16 else 0.0
            extra = (T + 16) * U if name.startswith("dw") or (name == "dgate" and kind == "channel") else 0.0
            within(got[name], v, (1 + rounded) * (d + extra) * size + rounded * v.abs(), name)


def test_norm_in_place_nan_and_neighbours(mx):
    T, H = 37, 520
    x, b, wo, gate, wi, dy, dxn = norm_inputs(T, H, "token", True, True, 5)
    x[3, 7], b[9, 0], x[20, 1] = math.nan, math.inf, math.inf
    xd, bd, wod, gd, wid = cuda(x, b, wo, gate, wi)
    say("norm in place")
    y, xn = mx.mx_norm_residual(xd, bd, wod, gd, 1.0, wid, EPS)
    buf = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device=DEV)
    buf[:T] = xd
    y2, xn2 = mx.mx_norm_residual(buf[:T], bd, wod, gd, 1.0, wid, EPS, out=buf[:T])
    assert torch.equal(y2.view(torch.int16), y.view(torch.int16)) and torch.equal(xn2.view(torch.int16), xn.view(torch.int16))
    assert bool((buf[T:] == 7).all())
    bad = {3, 9, 20}
    rows = [i for i in range(T) if bool((~xn[i].isfinite()).any())]
    assert set(rows) == bad, rows


# ------------------------------------------------------------------ together, streams, graphs

def block_inputs(T, H, I, seed):
    g = gen(seed)
    x = bf(T, H, g=g)
    wgu, sgu = weights(2 * I, H, g)
    wd, sd = weights(H, I, g)
    return cuda(x, wgu, sgu, wd, sd, bf(H, g=g, std=0.1, mean=1.0), bf(2 * I, g=g, std=0.3), bf(H, g=g, std=0.3),
                bf(H, g=g, std=0.1, mean=1.0), bf(T, 1, g=g, mean=0.5))


def check_block(mx, T, H, I):
    x, wgu, sgu, wd, sd, wi, bgu, bd, wo, gate = block_inputs(T, H, I, T + H)
    _, xn = mx.mx_norm_residual(x, w_pre=wi)
    h = mx.mx_gate_up(xn, wgu, sgu, bgu, "silu")
    plain = mx.mx_linear_fused(h, wd, sd, bd, x, 0.5)
    assert torch.equal(mx.mx_ffn_block(x, wgu, sgu, wd, sd, wi, bgu, bd, scale=0.5), plain)
    b = mx.mx_linear_fused(h, wd, sd, bd)
    y, _ = mx.mx_norm_residual(x, b, wo, gate, 0.5)
    assert torch.equal(mx.mx_ffn_block(x, wgu, sgu, wd, sd, wi, bgu, bd, "silu", wo, gate, 0.5), y)
    return plain


@pytest.mark.parametrize("T,H,I", [(1, 256, 64), (8, 1024, 512), (40, 512, 288), (200, 288, 96), (1100, 256, 160)])
def test_block_is_its_parts(mx, T, H, I):
    """The block's path against the separate calls (the same bits), and the whole of it against
    the definition with the same roundings between the calls."""
    say("block", T, H, I)
    plain = check_block(mx, T, H, I)
    x, wgu, sgu, wd, sd, wi, bgu, bd, _, _ = [t.cpu() for t in block_inputs(T, H, I, T + H)]
    _, xn = mx.mx_norm_residual(x.to(DEV), w_pre=wi.to(DEV))
    h = mx.mx_gate_up(*cuda(xn, wgu, sgu, bgu), "silu").cpu()
    z, ez = z_of(h, wd, sd, bd)
    want = x.double() + 0.5 * z
    within(plain, want, (1 + B) * (0.5 * ez + 2 * U * want.abs()) + B * want.abs(), "block")


def test_training_step_runs_together(mx):
    """Forward with saved pre-activations, then the whole backward: the input's gradient of a
    norm -> gate_up -> down -> norm block against the chain of definitions on the same values."""
    T, H, I = 70, 256, 96
    x, wgu, sgu, wd, sd, wi, bgu, bd, wo, gate = block_inputs(T, H, I, 9)
    dy = bf(T, H, g=gen(1)).to(DEV)
    say("training step")
    _, xn = mx.mx_norm_residual(x, w_pre=wi)
    h, z = mx.mx_gate_up(xn, wgu, sgu, bgu, "silu", save_z=True)
    b = mx.mx_linear_fused(h, wd, sd, bd)
    y, _ = mx.mx_norm_residual(x, b, wo, gate, 0.5)
    post = mx.mx_norm_residual_backward(dy, None, None, b, wo, gate, 0.5)
    dh, dbd = mx.mx_linear_fused_backward(post["db"], wd, sd)
    dxn, dbgu = mx.mx_gate_up_backward(dh, z, wgu, sgu, "silu")
    pre = mx.mx_norm_residual_backward(post["dx"], dxn, x, w_pre=wi)
    c = [dbl(t.cpu()) for t in (dy, b, wo, gate)]
    want = norm_grads(c[0], None, c[0], c[1], c[2], c[3], 0.5, None, "token")
    d = (2 * H + 64) * U
    within(post["db"], want["db"][0], (1 + B) * d * want["db"][1] + B * want["db"][0].abs(), "db")
    check_dx(dh.cpu(), post["db"].double().cpu(), torch.zeros(T, H, dtype=torch.float64), wd.cpu(), sd.cpu(), False, H)
    want = norm_grads(dbl(post["dx"].cpu()), dbl(dxn.cpu()), dbl(x.cpu()), None, None, None, 1.0, dbl(wi.cpu()), "none")
    within(pre["dx"], want["dx"][0], (1 + B) * d * want["dx"][1] + B * want["dx"][0].abs(), "dx")
    assert dbd.shape == (H,) and dbgu.shape == (2 * I,)


def every_call(mx, T, H, I, seed):
    """One pass through every operator: its outputs in a list."""
    x, wgu, sgu, wd, sd, wi, bgu, bd, wo, gate = block_inputs(T, H, I, seed)

    def run():
        y = mx.mx_ffn_block(x, wgu, sgu, wd, sd, wi, bgu, bd, "gelu", wo, gate, 0.5)
        h, z = mx.mx_gate_up(x, wgu, sgu, bgu, "silu", save_z=True)
        l, lz = mx.mx_linear_fused(h, wd, sd, bd, x, 0.5, "gelu_tanh", save_z=True)
        dh, dbd = mx.mx_linear_fused_backward(x, wd, sd, lz, 0.5, "gelu_tanh")
        dx, dbgu = mx.mx_gate_up_backward(h, z, wgu, sgu)
        n = mx.mx_norm_residual_backward(x, y, x, l, wo, gate, 0.5, wi)
        return [y, h, z, l, lz, dh, dbd, dx, dbgu] + [v for v in n.values() if v is not None]

    return run


@pytest.mark.parametrize("T", [3, 45, 150])
def test_graph_replays(mx, T):
    """Captured and replayed several times, with eager work between: every replay's outputs."""
    run = every_call(mx, T, 256, 96, T)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    say("graph", T)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    for k in range(4):
        for o in outs:
            o.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), k
        for a, b in zip(run(), want):  # eager calls between the replays
            assert torch.equal(a, b), k


def test_two_graphs_replayed_at_once(mx):
    """Each captured call owns its workspace: two graphs on two streams do not share one."""
    runs = [every_call(mx, T, 256, 96, T) for T in (45, 46)]
    wants = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(r())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    say("two graphs")
    for _ in range(3):
        for o in outs[0] + outs[1]:
            o.fill_(math.nan)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            for a, b in zip(o, w):
                assert torch.equal(a, b)


def test_streams(mx):
    """Calls on two streams at once, each waiting only for its own inputs."""
    run = every_call(mx, 45, 256, 96, 4)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    say("streams")
    for s in streams:
        with torch.cuda.stream(s):
            got.append(run())
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


def test_offsets_past_32_bits(mx):
    """Outputs, activations and weights of more than 4 GB: the last rows against the definition."""
    g = gen(6)
    dg = torch.Generator(device=DEV)
    dg.manual_seed(1)
    say("long activations")
    T, K, N = 70001, 128, 32800  # y has 4.6 GB
    x, (w, s) = bf(T, K, g=g), weights(N, K, g)
    xd, wd, sd = cuda(x, w, s)
    y = mx.mx_linear_fused(xd, wd, sd)
    rows = [0, 32769, 65536, T - 1]
    z, ez = z_of(x[rows], w, s, None)
    within(y[rows], z, (1 + B) * ez + B * z.abs(), "y")
    dx = mx.mx_linear_fused_backward(y, wd, sd, need_dbias=False)[0]
    dz = y[rows].double().cpu()
    check_dx(dx[rows].cpu(), dz, torch.zeros_like(dz), w, s, False, N)
    del y, dx
    say("many weights")
    T, K, N = 5, 2080, 1 << 22  # 4.4 GB of codes
    wd = torch.randint(0, 256, (N, K // 2), generator=dg, device=DEV, dtype=torch.uint8)
    sd = torch.full((N, K // 32), 118, dtype=torch.uint8, device=DEV)
    x = bf(T, K, g=g)
    for act_t in (T, 40):
        xx = bf(act_t, K, g=g)
        y = mx.mx_linear_fused(xx.to(DEV), wd, sd)
        last = slice(N - 70, N)
        z, ez = z_of(xx, wd[last].cpu(), sd[last].cpu(), None)
        within(y[:, last], z, (1 + B) * ez + B * z.abs(), "y")
    del wd, sd, y
    say("long norms")
    T, H = 300001, 8192
    x = torch.randn((T, H), generator=dg, device=DEV, dtype=torch.bfloat16)
    wi = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    xn = mx.mx_norm_residual(x, w_pre=wi)[1]
    rows = [0, 262144, T - 1]
    v = x[rows].double().cpu()
    want = v * rms(v)
    within(xn[rows], want, ((1 + B) * (H + 16) * U + B) * want.abs(), "xn")


def test_gate_up_scales_past_32_bits(mx):
    """Up rows whose scales begin 2 GB after the gate rows' (68 GB of codes)."""
    I, K = 1 << 21, 1 << 15
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of GPU memory")
    g = gen(8)
    wd = torch.zeros((2 * I, K // 2), dtype=torch.uint8, device=DEV)
    sd = torch.full((2 * I, K // 32), 118, dtype=torch.uint8, device=DEV)
    n = 70
    cols = torch.cat((torch.arange(I - n, I), torch.arange(n)))
    for r in (cols, I + cols):
        w, s = weights(len(cols), K, g)
        wd[r.to(DEV)], sd[r.to(DEV)] = cuda(w, s)
    both = torch.cat((cols, I + cols)).to(DEV)
    w, s = wd[both].cpu(), sd[both].cpu()
    for T in (3, 20, 40, 130):
        say("gate_up scales far apart", T)
        x = bf(T, K, g=g)
        h = mx.mx_gate_up(x.to(DEV), wd, sd, act="relu")[:, cols.to(DEV)]
        z, ez = z_of(x, w, s, None)
        m = len(cols)
        a, u = z[:, :m].clamp(min=0), z[:, m:]
        err = ez[:, :m] * u.abs() + ez[:, m:] * a + ez[:, :m] * ez[:, m:] + U * (a * u).abs()
        within(h, a * u, (1 + B) * err + B * (a * u).abs(), "h")


def test_most_tokens(mx):
    """T = 2^24, the limit: sampled rows against the definition, the bias gradient whole."""
    T, N = 1 << 24, 3
    rows = [0, 1 << 22, 3 << 22, T - 2, T - 1]
    for K in (32, 128):
        g = gen(K)
        dg = torch.Generator(device=DEV)
        dg.manual_seed(K)
        say("most tokens", K)
        x = torch.randn((T, K), generator=dg, device=DEV, dtype=torch.bfloat16)
        w, s = weights(2 * N, K, g)
        wd, sd = cuda(w, s)
        y = mx.mx_linear_fused(x, wd[:N], sd[:N].clone())
        xr = x[rows].cpu()
        z, ez = z_of(xr, w[:N], s[:N], None)
        within(y[rows], z, (1 + B) * ez + B * z.abs(), "y")
        h, zg = mx.mx_gate_up(x, wd, sd, act="relu", save_z=True)
        z, ez = z_of(xr, w, s, None)
        want, u = z[:, :N].clamp(min=0), z[:, N:]
        err = ez[:, :N] * u.abs() + ez[:, N:] * want + ez[:, :N] * ez[:, N:] + U * (want * u).abs()
        within(h[rows], want * u, (1 + B) * err + B * (want * u).abs(), "h")
        del x
        dx, db = mx.mx_linear_fused_backward(y, wd[:N], sd[:N].clone())
        dz = y[rows].double().cpu()
        check_dx(dx[rows].cpu(), dz, torch.zeros_like(dz), w[:N], s[:N], False, N)
        # 1024 strips of 2^14 rows: 2^11 + 8 + 1024 additions in a row at most
        yd = y.double()
        within(db, yd.sum(0).cpu(), (2 ** 12) * U * yd.abs().sum(0).cpu(), "dbias")
        del yd, dx
        dx, db = mx.mx_gate_up_backward(h, zg, wd, sd, act="relu")
        hr, zr = h[rows].double().cpu(), zg[rows].double().cpu()
        dz = torch.cat((hr * zr[:, N:] * (zr[:, :N] > 0), hr * zr[:, :N].clamp(min=0)), 1)
        check_dx(dx[rows].cpu(), dz, 4 * U * dz.abs(), w, s, True, 2 * N)
        del dx, db, y, h, zg
    say("most tokens, norm")
    x = torch.randn((T, 8), generator=dg, device=DEV, dtype=torch.bfloat16)
    one = torch.ones(8, dtype=torch.bfloat16, device=DEV)
    xn = mx.mx_norm_residual(x, w_pre=one)[1]
    v = x[rows].double().cpu()
    want = v * rms(v)
    within(xn[rows], want, ((1 + B) * 24 * U + B) * want.abs(), "xn")


@pytest.mark.parametrize("T", [3, 40, 200])
def test_longest_reduction(mx, T):
    """K = 2^20 forward, and N = 2^20 weight rows in the backward product."""
    K, N = 1 << 20, 33
    g = gen(T)
    x, (w, s) = bf(T, K, g=g), weights(N, K, g)
    say("longest reduction", T)
    y = mx.mx_linear_fused(*cuda(x, w, s))
    z, ez = z_of(x, w, s, None)
    within(y, z, (1 + B) * ez + B * z.abs(), "y")
    dy = bf(T, N, g=g)
    dx, db = mx.mx_linear_fused_backward(*cuda(dy, w, s))
    dz = dy.double()
    check_dx(dx, dz, torch.zeros_like(dz), w, s, False, N)
    within(db, dz.sum(0), (T + 8) * U * dz.abs().sum(0), "dbias")
    dy, (w, s) = bf(T, K, g=g), weights(K, 32, g)
    dx, db = mx.mx_linear_fused_backward(*cuda(dy, w, s))
    dz = dy.double()
    check_dx(dx, dz, torch.zeros_like(dz), w, s, False, K)
    within(db, dz.sum(0), (T + 8) * U * dz.abs().sum(0), "dbias")


def test_block_in_place(mx):
    T, H, I = 40, 256, 96
    x, wgu, sgu, wd, sd, wi, bgu, bd, wo, gate = block_inputs(T, H, I, 12)
    say("block in place")
    for post in (False, True):
        more = dict(w_post=wo, gate=gate) if post else {}
        want = mx.mx_ffn_block(x, wgu, sgu, wd, sd, wi, bgu, bd, **more)
        y = x.clone()
        mx.mx_ffn_block(y, wgu, sgu, wd, sd, wi, bgu, bd, out=y, **more)
        assert torch.equal(y, want)


def test_caller_workspace(mx):
    """A caller's workspace with any content, one byte short refused."""
    T, K, N = 40, 8192, 64
    x, w, s, bias, res = cuda(*linear_inputs(T, K, N, 2))
    need = mx.raw().mx_linear_fused_workspace_size(T, K, N)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    say("workspace", need)
    assert torch.equal(mx.mx_linear_fused(x, w, s, bias, ws=ws), mx.mx_linear_fused(x, w, s, bias))
    with pytest.raises(mx.MxError):
        mx.mx_linear_fused(x, w, s, bias, ws=ws[:-1])


def test_refusals(mx):
    x, w, s, bias, res = cuda(*linear_inputs(4, 64, 8, 2))
    for bad in (dict(bias=bias[:4]), dict(residual=res.t()), dict(act="swish"), dict(out=res[:2]), dict(bias=bias.float()),
                dict(scale=math.inf), dict(residual=res.cpu())):
        with pytest.raises((ValueError, TypeError)):
            mx.mx_linear_fused(x, w, s, **bad)
    for a in ((x[:, :32], w, s), (x, w[:, :16], s), (x, w, s[:, :1]), (x, w[:4], s), (x[:0], w, s), (x[0], w, s)):
        with pytest.raises((ValueError, TypeError)):
            mx.mx_linear_fused(*a)
    with pytest.raises(ValueError):
        mx.mx_linear_fused_backward(res, w, s, act="silu")
    with pytest.raises(ValueError):
        mx.mx_linear_fused_backward(res, w, s, need_dx=False, need_dbias=False)
    with pytest.raises(ValueError):
        mx.mx_gate_up(x, w[:7], s[:7])
    one = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(), dict(w_post=one), dict(w_pre=one, gate=one), dict(b=x, gate=one[:4]), dict(b=x, w_pre=one, eps=0.0),
                dict(b=x[:2]), dict(w_pre=one[:8])):
        with pytest.raises((ValueError, TypeError)):
            mx.mx_norm_residual(x, **bad)
    for bad in ((x, x, x), (x, None, None, None, one), (x, x, None, None, None, None, 1.0, one)):
        with pytest.raises((ValueError, TypeError)):
            mx.mx_norm_residual_backward(*bad)


# ------------------------------------------------------------------ what a call may do beside the cases above

@pytest.mark.parametrize("T,K,N", [(1, 32, 1), (3, 96, 7), (4, 128, 1000), (40, 64, 64), (70, 256, 1090), (130, 160, 65),
                                   (129, 96, 128), (4130, 2080, 70)])
def test_linear_backward_scales_without_activation(mx, T, K, N):
    """Without an activation dy goes into the product as it is, whatever N: the only rounding of dx
    is its own, also with a scale that is no power of two."""
    g = gen(T + N)
    w, s = weights(N, K, g)
    dy = bf(T, N, g=g)
    for scale in (float(np.float32(1 / 3)), float(np.float32(-1.4142))):
        say("scale without activation", T, K, N, scale)
        dx, db = mx.mx_linear_fused_backward(*cuda(dy, w, s), None, scale, "none")
        dz = scale * dy.double()
        edz = 4 * U * dz.abs()
        say("   worst", check_dx(dx, dz, edz, w, s, False, N))
        within(db, dz.sum(0), edz.sum(0) + (T + 8) * U * dz.abs().sum(0), "dbias")


def tail_errors(z, kind):
    """Bounds of the kernels' act(z) and act'(z) in fp32, relative in the tails: an exponential of a
    is off by |a| u for its rounded argument and 0.3 |a| u for the constant that makes it a power of
    two, beside a few u of its own; what lies below the smallest normal value may be 0."""
    z = z.double()
    a, d = act(z, kind)
    floor = 2.0 ** -126 * (1 + z.abs())
    if kind == "gelu":
        pdf = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        tail = 0.5 * torch.erfc(z.abs() / math.sqrt(2))
        et = tail * (1.3 * z * z / 2 + 0.7 * z * z / 2 + 16) * U + (z > 0) * U  # z^2 / 2 itself is rounded
        return z.abs() * et + U * a.abs() + floor, et + z.abs() * pdf * (z * z + 8) * U + U * d.abs() + floor
    if kind == "gelu_tanh":  # a logistic of A, whose six roundings count as its argument's
        k = 2 * math.sqrt(2 / math.pi)
        A, D, per = k * (z + 0.044715 * z ** 3), k * (1 + 3 * 0.044715 * z * z), 7.3
    else:
        A, D, per = z, torch.ones_like(z), 1.3
    p, q = torch.sigmoid(A), torch.sigmoid(-A)
    ep = q * (per * A.abs() + 3) * U + 4 * U  # of p, relative
    if kind == "sigmoid":
        return ep * p + floor, p * q * (2 * per * A.abs() + 12) * U + floor
    # the slope p + z p (1 - p) D, with 1 - p formed from p
    ed = ep * p + z.abs() * p * D * (q * (ep + 8 * U) + p * ep + U) + U * d.abs() + floor * (1 + D)
    return z.abs() * p * (ep + U) + floor, ed


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "sigmoid"])
def test_activation_tails(mx, kind):
    """Every bf16 pre-activation up to |z| = 13, given through the bias: the stored activation is
    exact to its rounding also where it is tiny, and so is the slope, which the bias gradient of one
    token gives in fp32."""
    z = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = z[(z.abs() <= 13) & (z.abs() >= 2.0 ** -10)]
    N, K = z.numel(), 32
    w = torch.zeros(N, K // 2, dtype=torch.uint8)
    s = torch.full((N, 1), 127, dtype=torch.uint8)
    say("tails", kind, N)
    ea, ed = tail_errors(z, kind)
    a, d = act(z.double(), kind)
    y = mx.mx_linear_fused(*cuda(torch.zeros(1, K, dtype=torch.bfloat16), w, s), bias=z.to(DEV), act=kind)
    say("   worst", within(y[0], a, (1 + B) * ea + B * a.abs(), "activation"))
    one = torch.ones(1, N, dtype=torch.bfloat16)
    db = mx.mx_linear_fused_backward(*cuda(one, w, s, z[None]), 1.0, kind, need_dx=False)[1]
    say("   worst", within(db, d, ed, "slope"))


@pytest.mark.parametrize("H", [64, 512, 7168, 8704])
def test_norm_smallest_eps(mx, H):
    """An eps whose root's reciprocal has no square in fp32: rows of zeros keep finite gradients."""
    T, eps = 3, float(np.float32(1e-40))
    x, b, wo, gate, wi, dy, dxn = norm_inputs(T, H, "channel", True, True, H)
    x[:], b[:] = 0, 0
    say("smallest eps", H)
    xd, bd, wod, gd, wid, dyd, dxnd = cuda(x, b, wo, gate, wi, dy, dxn)
    y, xn = mx.mx_norm_residual(xd, bd, wod, gd, 1.0, wid, eps)
    assert not bool(y.any()) and not bool(xn.any())
    got = mx.mx_norm_residual_backward(dyd, dxnd, xd, bd, wod, gd, 1.0, wid, eps)
    r = 1 / math.sqrt(eps)
    D = dbl(dy) + r * dbl(dxn) * dbl(wi)
    within(got["dx"], D, B * D.abs() + 16 * U * D.abs(), "dx")
    big = r * D * dbl(gate) * dbl(wo)  # of the order of 1e40, beyond bf16
    db = got["db"].double().cpu()
    assert not bool(db.isnan().any()) and torch.equal(torch.sign(db), torch.sign(big))
    for name in ("dgate", "dw_post", "dw_pre"):
        assert not bool(got[name].any()), name


@pytest.mark.parametrize("call", ["linear", "gate_up"])
def test_short_reduction_most_workgroups(mx, call):
    """K = 32 with so many tokens and rows that one axis of a grid could not hold the threads: sampled
    rows against the definition, the first and last columns."""
    T, K, N = 1 << 24, 32, (2056 if call == "linear" else 1032)
    if torch.cuda.mem_get_info()[0] < 4.2 * T * N:
        pytest.skip("needs 145 GB (linear) or 73 GB (gate_up) of GPU memory")
    g = gen(N)
    dg = torch.Generator(device=DEV)
    dg.manual_seed(N)
    say("most workgroups", call)
    x = torch.randn((T, K), generator=dg, device=DEV, dtype=torch.bfloat16)
    rows = [0, 31, 32, (1 << 20) - 1, 1 << 20, (1 << 23) + 5, T - 33, T - 1]
    xr = x[rows].cpu()
    if call == "linear":
        w, s = weights(N, K, g)
        y = torch.full((T, N), math.nan, dtype=torch.bfloat16, device=DEV)
        mx.mx_linear_fused(x, *cuda(w, s), out=y)
        z, ez = z_of(xr, w, s, None)
        within(y[rows], z, (1 + B) * ez + B * z.abs(), "y")
    else:
        w, s = weights(2 * N, K, g)
        y = torch.full((T, N), math.nan, dtype=torch.bfloat16, device=DEV)
        mx.mx_gate_up(x, *cuda(w, s), act="relu", out=y)
        z, ez = z_of(xr, w, s, None)
        a, u = z[:, :N].clamp(min=0), z[:, N:]
        err = ez[:, :N] * u.abs() + ez[:, N:] * a + ez[:, :N] * ez[:, N:] + U * (a * u).abs()
        within(y[rows], a * u, (1 + B) * err + B * (a * u).abs(), "h")
    for t0 in range(0, T, 1 << 21):  # no row was left out
        assert not bool(y[t0:t0 + (1 << 21), ::257].isnan().any()), t0


@pytest.mark.parametrize("T,H", [(5, 264), (40, 8704)])
@pytest.mark.parametrize("kind", ["channel", "token", "full"])
def test_norm_backward_leaves_out(mx, T, H, kind):
    """Every gradient beside dx can be left out; the others keep their bits."""
    y, b, wo, gate, wi, dy, dxn = cuda(*norm_inputs(T, H, kind, True, True, T + H))
    args = (dy, dxn, y, b, wo, gate, 0.7, wi, EPS)
    say("left out", T, H, kind)
    want = mx.mx_norm_residual_backward(*args)
    names = ("db", "dgate", "dw_post", "dw_pre")
    for off in [(n,) for n in names] + [names[:2], names[1:], names]:
        got = mx.mx_norm_residual_backward(*args, **{f"need_{n}": False for n in off})
        for n, v in want.items():
            assert got[n] is None if n in off else torch.equal(got[n], v), (off, n)


def test_training_step_every_gradient(mx):
    """The backward of norm -> gate_up -> down -> norm, every call's gradients against the definition on
    the values that the call before gave: bias and norm-weight gradients, the gate's, and gate_up's
    input gradient from the saved pre-activations, whose halves the forward laid out."""
    T, H, I = 70, 256, 96
    x, wgu, sgu, wd, sd, wi, bgu, bd, wo, gate = block_inputs(T, H, I, 9)
    dy = bf(T, H, g=gen(1)).to(DEV)
    say("training step, every gradient")
    _, xn = mx.mx_norm_residual(x, w_pre=wi)
    h, z = mx.mx_gate_up(xn, wgu, sgu, bgu, "silu", save_z=True)
    b = mx.mx_linear_fused(h, wd, sd, bd)
    post = mx.mx_norm_residual_backward(dy, None, None, b, wo, gate, 0.5)
    dh, dbd = mx.mx_linear_fused_backward(post["db"], wd, sd)
    dxn, dbgu = mx.mx_gate_up_backward(dh, z, wgu, sgu, "silu")
    pre = mx.mx_norm_residual_backward(post["dx"], dxn, x, w_pre=wi)
    d, over_t = (2 * H + 64) * U, (T + 16) * U

    def check(got, want, names):
        for name in names:
            v, size = want[name]
            rounded = B if got[name].dtype == torch.bfloat16 else 0.0
            within(got[name], v, (1 + rounded) * (d + over_t) * size + rounded * v.abs(), name)

    c = [dbl(t.cpu()) for t in (dy, b, wo, gate)]
    check(post, norm_grads(c[0], None, c[0], c[1], c[2], c[3], 0.5, None, "token"), ("dx", "db", "dgate", "dw_post"))
    db = dbl(post["db"].cpu())
    within(dbd, db.sum(0), (T + 8) * U * db.abs().sum(0), "dbd")
    # the saved pre-activations are the forward's, gate half first
    zw, ez = z_of(xn.cpu(), wgu.cpu(), sgu.cpu(), bgu.cpu())
    within(z, zw, (1 + B) * ez + B * zw.abs(), "z")
    dhc, zc = dbl(dh.cpu()), dbl(z.cpu())
    a, slope = act(zc[:, :I], "silu")
    dz = torch.cat((dhc * zc[:, I:] * slope, dhc * a), 1)
    e = ACT_ERR * (1 + zc[:, :I].abs())
    edz = torch.cat((dhc.abs() * zc[:, I:].abs() * e, dhc.abs() * e), 1) + 4 * U * dz.abs()
    check_dx(dxn.cpu(), dz, edz, wgu.cpu(), sgu.cpu(), True, 2 * I)
    within(dbgu, dz.sum(0), edz.sum(0) + (T + 8) * U * dz.abs().sum(0), "dbgu")
    want = norm_grads(dbl(post["dx"].cpu()), dbl(dxn.cpu()), dbl(x.cpu()), None, None, None, 1.0, dbl(wi.cpu()), "none")
    check(pre, want, ("dx", "dw_pre"))


@pytest.mark.parametrize("T,H,I", [(4100, 2112, 70), (4130, 2080, 33), (4097, 2176, 64)])
def test_gate_up_backward_wide_tiles(mx, T, H, I):
    """Sizes whose product takes tiles of 256 x 256, ragged in tokens, columns and weight rows."""
    g = gen(T + H + I)
    w, s = weights(2 * I, H, g)
    dh, z = bf(T, I, g=g), bf(T, 2 * I, g=g, std=1.5)
    say("gate_up backward, wide tiles", T, H, I)
    dx, db = mx.mx_gate_up_backward(*cuda(dh, z, w, s), "silu")
    gt, up, d = z[:, :I].double(), z[:, I:].double(), dh.double()
    a, slope = act(gt, "silu")
    dz = torch.cat((d * up * slope, d * a), 1)
    e = ACT_ERR * (1 + gt.abs())
    edz = torch.cat((d.abs() * up.abs() * e, d.abs() * e), 1) + 4 * U * dz.abs()
    say("   worst", check_dx(dx, dz, edz, w, s, True, 2 * I))
    within(db, dz.sum(0), edz.sum(0) + (T + 8) * U * dz.abs().sum(0), "dbias")


@pytest.mark.parametrize("T,H,I", [(2, 256, 64), (40, 288, 96), (300, 512, 160)])
def test_block_options(mx, T, H, I):
    """Every combination of the block's norms, gate and biases against the separate calls, into the first
    rows of a longer output."""
    x, wgu, sgu, wd, sd, wi, bgu, bd, wo, _ = block_inputs(T, H, I, T + H + 1)
    g = gen(H)
    gates = {None: None, "token": bf(T, 1, g=g), "channel": bf(H, g=g), "full": bf(T, H, g=g)}
    say("block options", T, H, I)
    for pre in (None, wi):
        for post in (None, wo):
            for kind, gate in gates.items():
                gate = None if gate is None else gate.to(DEV)
                for b1, b2 in ((None, None), (bgu, bd)):
                    xn = x if pre is None else mx.mx_norm_residual(x, w_pre=pre, eps=1e-5)[1]
                    h = mx.mx_gate_up(xn, wgu, sgu, b1, "relu")
                    if post is None and gate is None:
                        want = mx.mx_linear_fused(h, wd, sd, b2, x, -0.7)
                    else:
                        want, _ = mx.mx_norm_residual(x, mx.mx_linear_fused(h, wd, sd, b2), post, gate, -0.7, eps=1e-5)
                    buf = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device=DEV)
                    y = mx.mx_ffn_block(x, wgu, sgu, wd, sd, pre, b1, b2, "relu", post, gate, -0.7, 1e-5, out=buf[:T])
                    what = (pre is not None, post is not None, kind, b1 is not None)
                    assert torch.equal(y, want) and bool((buf[T:] == 7).all()), what


@pytest.mark.parametrize("T,K,N", [(1, 32, 1), (3, 96, 33), (20, 8192, 40), (70, 4096, 130), (200, 2048, 64),
                                   (1030, 288, 257), (4100, 2112, 66)])
def test_workspaces_are_large_enough(mx, T, K, N):
    """Every call with a workspace of exactly the size it asks for, inside a larger buffer: the bytes
    behind it stay as they were, and so do the results."""
    L, g = mx.raw(), gen(T + K + N)
    x, (w, s), dy = bf(T, K, g=g), weights(N, K, g), bf(T, N, g=g)
    w2, s2 = weights(2 * N, K, g)
    wd, sd = weights(K, 32, g)
    wgu, sgu = weights(64, K, g)
    x, w, s, dy, w2, s2, wd, sd, wgu, sgu = cuda(x, w, s, dy, w2, s2, wd, sd, wgu, sgu)
    z2 = bf(T, 2 * N, g=g).to(DEV)
    one = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    calls = [(L.mx_linear_fused_workspace_size(T, K, N), lambda ws: [mx.mx_linear_fused(x, w, s, ws=ws)]),
             (L.mx_linear_fused_backward_workspace_size(T, K, N),
              lambda ws: list(mx.mx_linear_fused_backward(dy, w, s, dy, 0.3, "silu", ws=ws))),
             (L.mx_linear_fused_backward_workspace_size(T, K, N),
              lambda ws: list(mx.mx_linear_fused_backward(dy, w, s, None, 0.3, ws=ws))),
             (L.mx_gate_up_workspace_size(T, K, N), lambda ws: [mx.mx_gate_up(x, w2, s2, ws=ws)]),
             (L.mx_gate_up_backward_workspace_size(T, K, N), lambda ws: list(mx.mx_gate_up_backward(dy, z2, w2, s2, ws=ws))),
             (L.mx_norm_residual_backward_workspace_size(T, K),
              lambda ws: list(mx.mx_norm_residual_backward(x, x, x, x, one, one, 1.0, one, ws=ws).values())),
             (L.mx_ffn_block_workspace_size(T, K, 32), lambda ws: [mx.mx_ffn_block(x, wgu, sgu, wd, sd, one, w_post=one, ws=ws)])]
    for i, (need, call) in enumerate(calls):
        say("workspace", i, T, K, N, need)
        buf = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        for a, b in zip(call(buf[:need]), call(None)):
            assert torch.equal(a, b), i
        assert bool((buf[need:] == 0x5A).all()), i


def test_two_threads_at_once(mx):
    """Two host threads, a stream each, the same tensors."""
    import threading
    run = every_call(mx, 45, 256, 96, 4)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i] = run()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    say("two threads")
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for o in got:
        for a, b in zip(o, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,K,N", [(2, 256, 40), (3, 288, 33), (20, 160, 40), (12, 512, 40), (40, 256, 40), (100, 640, 70),
                                   (50, 288, 33), (200, 288, 129), (200, 512, 130), (1100, 288, 520)])
def test_subnormal_weights_and_activations(mx, T, K, N):
    """Weights below bf16's and fp32's smallest normal value (scale bytes 0 to 3) with large
    activations, and subnormal activations with large scales, forward and backward."""
    for lo, hi, top in ((0, 4, 2.0 ** 100), (245, 250, 2.0 ** -130)):
        g = gen(T + K + N + lo)
        w, s = weights(N, K, g, lo, hi)
        x, dy = (bf(T, K, g=g).double() * top).bfloat16(), (bf(T, N, g=g).double() * top).bfloat16()
        say("subnormal", T, K, N, lo)
        y = mx.mx_linear_fused(*cuda(x, w, s))
        z, ez = z_of(x, w, s, None)
        say("   worst", within(y, z, (1 + B) * ez + B * z.abs(), "y"))
        dx, db = mx.mx_linear_fused_backward(*cuda(dy, w, s))
        dz = dy.double()
        say("   worst", check_dx(dx, dz, torch.zeros_like(dz), w, s, False, N))
        within(db, dz.sum(0), (T + 8) * U * dz.abs().sum(0), "dbias")


@pytest.mark.parametrize("T,H", [(7, 8), (9, 40), (6, 128), (5, 136), (3, 256), (6, 1024), (5, 8200)])
def test_norm_rows_do_not_mix(mx, T, H):
    """Rows with NaN and Inf leave every other row's outputs and gradients as they are, bit for bit, also
    where several rows share a wave."""
    y, b, wo, gate, wi, dy, dxn = norm_inputs(T, H, "token", True, True, T + H)
    say("rows", T, H)

    def run(y, b, gate, dy, dxn):
        y, b, gate, dy, dxn, o, i = cuda(y, b, gate, dy, dxn, wo, wi)
        f = mx.mx_norm_residual(y, b, o, gate, 0.7, i, EPS)
        r = mx.mx_norm_residual_backward(dy, dxn, y, b, o, gate, 0.7, i, EPS)
        return [t.cpu() for t in (*f, r["dx"], r["db"], r["dgate"])]

    want = run(y, b, gate, dy, dxn)
    bad = [T // 2, T - 1]
    y2, b2, g2, dy2 = y.clone(), b.clone(), gate.clone(), dy.clone()
    y2[bad[0], 0], b2[bad[0], H - 1], g2[bad[1]], dy2[bad[1], H // 2] = math.nan, math.inf, math.nan, -math.inf
    keep = [t for t in range(T) if t not in bad]
    for a, c in zip(run(y2, b2, g2, dy2, dxn), want):
        assert torch.equal(a[keep], c[keep])
        assert not bool(a[bad].isfinite().all(1).any())


def test_refuse_outputs_over_inputs(mx):
    """out over x, whole or in part, also where x is the residual too, and over part of what it may
    stand on as a whole: refused before anything runs."""
    T, K = 40, 64
    g = gen(1)
    w, s, w2, s2 = cuda(*weights(K, K, g), *weights(2 * K, K, g))
    buf = bf(2 * T, K, g=g).to(DEV)
    keep = buf.clone()
    x, shifted, beside = buf[:T], buf[1:T + 1], buf[T:]
    other = bf(T, K, g=g).to(DEV)
    say("out over x")
    for out in (x, shifted):
        with pytest.raises(ValueError, match="overlap"):
            mx.mx_linear_fused(x, w, s, residual=x, out=out)
        with pytest.raises(ValueError, match="overlap"):
            mx.mx_gate_up(x, w2, s2, out=out)
    for call in (lambda: mx.mx_linear_fused(other, w, s, residual=x, out=shifted),
                 lambda: mx.mx_norm_residual(x, other, out=shifted), lambda: mx.mx_norm_residual(other, x, out=shifted),
                 lambda: mx.mx_ffn_block(x, w2, s2, w, s, out=shifted)):
        with pytest.raises(ValueError, match="overlap"):
            call()
    assert torch.equal(buf, keep)
    want = mx.mx_gate_up(x, w2, s2)
    assert torch.equal(mx.mx_gate_up(x, w2, s2, out=beside), want)  # beside it is fine


@pytest.mark.parametrize("T,H", [(3, 72), (40, 2048), (5, 8704)])
def test_plain_residual(mx, T, H):
    """No norm and no gate: y = x + scale * b, and its gradients."""
    x, b, _, _, _, dy, _ = norm_inputs(T, H, "none", False, False, H)
    scale = float(np.float32(0.3))
    say("plain residual", T, H)
    y, xn = mx.mx_norm_residual(*cuda(x, b), scale=scale)
    want = x.double() + scale * b.double()
    assert xn is None
    within(y, want, (1 + B) * U * want.abs() + B * want.abs(), "y")
    got = mx.mx_norm_residual_backward(dy.to(DEV), None, None, b.to(DEV), scale=scale)
    assert {k for k, v in got.items() if v is not None} == {"dx", "db"} and torch.equal(got["dx"].cpu(), dy)
    want = scale * dy.double()
    within(got["db"], want, (1 + B) * U * want.abs() + B * want.abs(), "db")
