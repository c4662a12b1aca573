"""GPU parity of the microscaled operators against their definitions in 64 bits.

Tolerances.  u = 2^-24 (half a step of fp32), b = 2^-8 (half a step of bf16).
  * The quantizer alone: none, codes and scales are equal bit for bit.
  * A product: the scaled matrix instructions drop, within a group of 8 products, bits 14 binades below
    the largest, 7 * 2^-14 of the group's sum|products| at most, less than 2^-11; the fp32 sums of K
    terms add K u sum|products|.
  * Activations as in the other dense operators: act(z) is off by at most 2^-20 (1 + |z|) and changes by
    at most 1.13 per unit of z.
  * A value quantized from one that is off by `err`: the block's scale is that of an amax within err of
    the exact one, and the element within half a step, at the scale taken, of the value clamped to the
    type's range, plus err.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U, B, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -133
DROP = 2.0 ** -11
ACT_ERR, ACT_LIP = 2.0 ** -20, 1.13
EPS = 1e-6
DEV = "cuda:0"
FORMATS = ["mxfp8", "mxfp4"]


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import mxfp4_weight_moe_amd
    return mxfp4_weight_moe_amd


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


def cuda(*ts):
    return [t.to(DEV) if isinstance(t, torch.Tensor) else t for t in ts]


# ------------------------------------------------------------------ the formats

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127])


def table(fmt):
    return E4M3 if fmt == "mxfp8" else E2M1


def quantize_ref(x, fmt):
    """(element codes [rows, K], scale bytes) of an fp64 array by the definition."""
    grid, emax = table(fmt), 8 if fmt == "mxfp8" else 2
    rows, K = x.shape
    b = x.reshape(rows, K // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    top = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0)).max(-1))
    e = np.where(top > 0, np.frexp(top)[1] - 1, -1000)
    byte = np.clip(e - emax + 127, 0, 254)
    q = np.where(bad[..., None], 0.0, b) * 2.0 ** (127.0 - byte)[..., None]
    a = np.minimum(np.abs(q), grid[-1])
    lo = np.clip(np.searchsorted(grid, a, side="right") - 1, 0, len(grid) - 1)
    hi = np.minimum(lo + 1, len(grid) - 1)
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code | (np.signbit(q) * (128 if fmt == "mxfp8" else 8)).astype(np.int64)
    code = np.where(bad[..., None], 0x7F if fmt == "mxfp8" else 0, code)
    return code.reshape(rows, K).astype(np.uint8), np.where(bad, 255, byte).astype(np.uint8)


def elements(codes, fmt):
    """Element codes of a stored tensor."""
    c = codes.cpu().numpy()
    if fmt == "mxfp8":
        return c
    return np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1)


def values(codes, scales, fmt):
    """fp64 tensor of what codes and scales stand for."""
    c, s = elements(codes, fmt).astype(np.int64), scales.cpu().numpy().astype(np.float64)
    neg, mag = (128, 127) if fmt == "mxfp8" else (8, 7)
    grid = np.append(table(fmt), np.nan) if fmt == "mxfp8" else table(fmt)
    v = np.where(c & neg, -grid[c & mag], grid[c & mag])
    p = np.where(s == 255, np.nan, 2.0 ** (s - 127))
    return torch.from_numpy(v * np.repeat(p, 32, axis=-1))


def pack(code, fmt):
    return code if fmt == "mxfp8" else (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def activations(T, K, fmt, g, std=1.0):
    """A quantized tensor as (codes, scales) on the host."""
    code, byte = quantize_ref(bf(T, K, g=g, std=std).double().numpy(), fmt)
    return torch.from_numpy(pack(code, fmt)), torch.from_numpy(byte)


def decode(w, s):
    return values(w, s, "mxfp4")


def half_step(u, fmt):
    """Half the distance of elements around |u| (an array)."""
    man, low = (3, -6) if fmt == "mxfp8" else (1, 0)
    e = np.maximum(np.floor(np.log2(np.maximum(u, 1e-300))), low)
    return 2.0 ** (e - man - 1)


def check_codes(codes, scales, want, err, fmt, what):
    """Codes and scales of values within `err` of `want`."""
    emax, most = (8, 448.0) if fmt == "mxfp8" else (2, 6.0)
    want, err = want.double().numpy(), torch.as_tensor(err).double().expand(want.shape).numpy()
    got, byte = values(codes, scales, fmt).numpy(), scales.cpu().numpy().astype(np.int64)
    wb, eb = np.abs(want).reshape(*byte.shape, 32), err.reshape(*byte.shape, 32)
    lo, hi = np.maximum(wb - eb, 0).max(-1), (wb + eb).max(-1)
    floor = lambda v: np.where(v > 0, np.floor(np.log2(np.maximum(v, 1e-300))), -1000)  # noqa: E731
    assert ((byte >= np.clip(floor(lo) - emax + 127, 0, 254)) & (byte <= np.clip(floor(hi) - emax + 127, 0, 254))).all(), what
    s = np.repeat(2.0 ** (byte - 127.0), 32, axis=-1)
    clipped = np.clip(want, -most * s, most * s)
    tol = s * half_step((np.abs(clipped) + err) / s, fmt) + err
    r = np.abs(got - clipped) / (tol + 1e-300)
    assert r.max() <= 1 + 1e-9, f"{what}: {(r > 1).sum()} of {r.size} out of bound, worst {r.max():.4g}"
    return float(r.max())


def within(got, want, tol, what):
    got, want, tol = got.double().cpu(), want.expand(got.shape), torch.as_tensor(tol).double().expand(got.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN at other places"
    fine = ~want.isnan()
    r = ((got - want).abs() / (tol + TINY))[fine]
    worst = float(r.max()) if r.numel() else 0.0
    assert worst <= 1, f"{what}: {int((r > 1).sum())} of {r.numel()} out of bound, worst {worst:.3g}"
    return worst


# ------------------------------------------------------------------ quantizer

def hard_values(rows, K, g, f32):
    """Rows over the whole exponent range, with ties, zeros, subnormals, the largest and NaN and Inf."""
    x = torch.randn(rows, K, generator=g, dtype=torch.float64)
    x *= 2.0 ** torch.randint(-150 if f32 else -140, 125, (rows, K // 32), generator=g).repeat_interleave(32, 1).double()
    x = x.float() if f32 else x.bfloat16()
    x[0] = 0
    if rows > 1:
        x[1, ::2] = -0.0
    if rows > 2:  # ties of both types at every magnitude: multiples of an eighth and of 2^-10
        x[2] = torch.arange(K).to(x.dtype) / 8
    if rows > 3:
        x[3] = (torch.arange(K) % 64).to(x.dtype) * 2.0 ** -10
        x[3, ::32] = 448
    if rows > 4:
        x[4] = torch.finfo(x.dtype).max
        x[4, 1] = torch.finfo(x.dtype).tiny / 2
    if rows > 5:
        x[5, 3] = math.nan
        x[5, K - 1] = -math.inf
    if rows > 6:
        x[6] = 2.0 ** -126
        x[6, ::3] = torch.finfo(x.dtype).smallest_normal / 4
    return x


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (7, 160), (64, 544), (129, 7168)])
def test_quantize(mx, rows, K, fmt, f32):
    x = hard_values(rows, K, gen(rows + K), f32)
    say("quantize", rows, K, fmt, f32)
    codes, scales, vals = mx.mx_quantize(x.to(DEV), fmt, save_values=True)
    code, byte = quantize_ref(x.double().numpy(), fmt)
    assert np.array_equal(scales.cpu().numpy(), byte)
    assert np.array_equal(codes.cpu().numpy(), pack(code, fmt))
    # exact where bf16 has the value: an E4M3 element may be 2^-9, at the smallest scale 2^-136, and bf16's
    # last step is 2^-133
    exact = values(codes, scales, fmt)
    assert torch.equal(vals.double().cpu().nan_to_num(7777.0), exact.to(torch.bfloat16).double().nan_to_num(7777.0))
    assert torch.equal(exact.to(torch.bfloat16).double()[exact.abs() > 2.0 ** -121], exact[exact.abs() > 2.0 ** -121])
    again = mx.mx_quantize(x.to(DEV), fmt)
    assert torch.equal(again[0], codes) and torch.equal(again[1], scales)
    if fmt == "mxfp4":
        assert torch.equal(mx.mxfp4_dequantize(codes, scales).view(torch.int16)[~vals.isnan()], vals.view(torch.int16)[~vals.isnan()])
    elif not f32:
        c8, s8 = mx.mxfp8_quantize(x.to(DEV))
        assert torch.equal(c8, codes) and torch.equal(s8, scales)


def test_quantize_leading_dimensions_and_what_lies_behind(mx):
    x = bf(3, 5, 64, g=gen(1)).to(DEV)
    c, s = mx.mx_quantize(x, "mxfp4")
    assert c.shape == (3, 5, 32) and s.shape == (3, 5, 2)
    flat = mx.mx_quantize(x.reshape(15, 64), "mxfp4")
    assert torch.equal(c.reshape(15, 32), flat[0]) and torch.equal(s.reshape(15, 2), flat[1])
    one = mx.mx_quantize(x[0, 0], "mxfp8")
    assert one[0].shape == (64,) and one[1].shape == (2,)
    codes, scales = torch.full((400,), 9, dtype=torch.uint8, device=DEV), torch.full((64,), 9, dtype=torch.uint8, device=DEV)
    vals = torch.full((400,), 9.0, dtype=torch.bfloat16, device=DEV)
    st = mx.raw().mx_quantize(x.data_ptr(), 0, 0, codes.data_ptr(), scales.data_ptr(), vals.data_ptr(), 5, 64, None)
    torch.cuda.synchronize()
    assert st == 0
    assert (codes[320:] == 9).all() and (scales[10:] == 9).all() and (vals[320:] == 9).all()


def test_quantize_refusals(mx):
    x = bf(4, 64, g=gen(2)).to(DEV)
    for bad in (dict(fmt="mxfp6"), dict(fmt=None)):
        with pytest.raises(ValueError):
            mx.mx_quantize(x, **bad)
    with pytest.raises(ValueError):
        mx.mx_quantize(x[:, :48].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        mx.mx_quantize(x.t())
    with pytest.raises(ValueError):
        mx.mx_quantize(x[:0])
    with pytest.raises(TypeError):
        mx.mx_quantize(x.half())


# ------------------------------------------------------------------ norm

def norm_ref(x, b, wpost, gate, scale, wpre):
    """(y before rounding, its error, xn of y as stored, its error) in 64 bits."""
    unit = lambda v: v / (v.pow(2).mean(1, keepdim=True) + EPS).sqrt()  # noqa: E731
    y = x.double()
    if b is not None:
        n = b.double()
        n = n if wpost is None else unit(n) * wpost.double()
        y = y + scale * (n if gate is None else gate.double() * n)
    s = y.to(torch.bfloat16)
    return y, s


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H", [(1, 32), (3, 96), (5, 128), (2, 256), (9, 288), (4, 512), (3, 1024), (7, 2080), (33, 4096),
                                 (5, 7168), (2, 8192), (3, 8224), (2, 16384), (2100, 64)])
def test_norm(mx, T, H, fmt):
    g = gen(T + H)
    x, b, wo, wi = bf(T, H, g=g, std=2), bf(T, H, g=g), bf(H, g=g, mean=1, std=.1), bf(H, g=g, mean=1, std=.1)
    gates = dict(none=None, token=bf(T, 1, g=g), channel=bf(H, g=g), full=bf(T, H, g=g))
    for blk, post, kind, scale, keep in ((False, False, "none", 1.0, True), (True, True, "channel", 0.5, False),
                                         (True, False, "token", -1.0, True), (True, True, "full", 2.0, True),
                                         (True, True, "none", 1.0, False)):
        say("norm", T, H, fmt, blk, post, kind)
        args = cuda(x, b if blk else None, wo if post else None, gates[kind])
        y, codes, scales, xn = mx.mx_norm_residual_quantize(*args, scale, wi.to(DEV), EPS, fmt, save_xn=keep)
        y2, xn2 = mx.mx_norm_residual(*args, scale, wi.to(DEV), EPS)
        assert torch.equal(y, y2), "y is mx_norm_residual's"
        assert (xn is None) == (not keep) and (xn is None or torch.equal(xn, xn2)), "xn is mx_norm_residual's"
        yd = y.double().cpu()
        q = 1 / (yd.pow(2).mean(1, keepdim=True) + EPS).sqrt()
        want = yd * q * wi.double()
        # H + 8 roundings in the mean (its square root halves them), the inverse root and two products
        check_codes(codes, scales, want, want.abs() * ((H + 8) / 2 + 6) * U, fmt, "xn")


def test_norm_in_place_and_special_rows(mx):
    T, H = 6, 256
    g = gen(5)
    x, b, wi = bf(T, H, g=g), bf(T, H, g=g), bf(H, g=g)
    x[1] = 0
    b[1] = 0
    x[2, 7] = math.nan
    x[3, 40] = math.inf
    for fmt in FORMATS:
        xd, bd, wd = cuda(x, b, wi)
        y, c, s, xn = mx.mx_norm_residual_quantize(xd, bd, w_pre=wd, eps=EPS, fmt=fmt, save_xn=True)
        buf = xd.clone()
        y2, c2, s2, _ = mx.mx_norm_residual_quantize(buf, bd, w_pre=wd, eps=EPS, fmt=fmt, out=buf)
        assert y2.data_ptr() == buf.data_ptr() and torch.equal(y2.view(torch.int16), y.view(torch.int16))
        assert torch.equal(c, c2) and torch.equal(s, s2)
        assert (s[1] == 0).all() and (elements(c[1:2], fmt) & (127 if fmt == "mxfp8" else 7) == 0).all()
        assert (s[2] == 255).all()          # NaN through the whole row's norm
        assert s[3, 1] == 255               # Inf / Inf in its own block; the others of its row are 0
        assert (s[3, 2:] == 0).all() and bool(xn[2].isnan().all())
        fine = [0, 4, 5]
        yd = y.double().cpu()[fine]
        want = yd / (yd.pow(2).mean(1, keepdim=True) + EPS).sqrt() * wi.double()
        check_codes(c[fine], s[fine], want, want.abs() * ((H + 8) / 2 + 6) * U, fmt, "xn")


def test_norm_refusals(mx):
    g = gen(3)
    x, b, w = cuda(bf(4, 64, g=g), bf(4, 64, g=g), bf(64, g=g))
    for bad in (dict(w_pre=None), dict(w_pre=w, fmt="fp8"), dict(w_pre=w, out=x), dict(w_pre=w, w_post=w),
                dict(b=b, w_pre=w[:32].contiguous()), dict(b=b[:3].contiguous(), w_pre=w), dict(w_pre=w, eps=0.0),
                dict(b=b, w_pre=w, scale=math.inf)):
        with pytest.raises(ValueError):
            mx.mx_norm_residual_quantize(x, **bad)
    with pytest.raises(ValueError):  # H = 40
        mx.mx_norm_residual_quantize(x[:, :40].contiguous(), w_pre=w[:40].contiguous())
    with pytest.raises(ValueError, match="overlap"):
        big = torch.zeros(5, 64, dtype=torch.bfloat16, device=DEV)
        mx.mx_norm_residual_quantize(big[:4], b, w_pre=w, out=big[1:])


# ------------------------------------------------------------------ products

def act(z, kind):
    if kind == "none":
        return z
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if kind == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    p = torch.sigmoid(z)
    return p if kind == "sigmoid" else z * p


def z_of(a, sa, fmt, w, s, bias):
    x, W = values(a, sa, fmt), decode(w, s)
    z, size = x @ W.T, x.abs() @ W.abs().T
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    return z, (DROP + (x.shape[1] + 8) * U) * size


def value_error(z, ez):
    return ACT_LIP * ez + ACT_ERR * (1 + z.abs())


# streaming (up to 16 tokens, 32 where K % 512 != 0), thin tiles (17 to 64 tokens, 32 and 64 rows, fewer
# stages than waves), tiles of 64, 128 and 256 tokens by 64, 128 and 256 rows, K whole and split, tails of 32,
# 64 and 96, odd rows; K from one block on; scales that go to the LDS directly (K % 512 == 0) or through
# registers
SHAPES = [(1, 32, 1), (1, 256, 64), (2, 96, 7), (5, 512, 33), (16, 288, 16), (17, 2048, 40), (31, 160, 100), (32, 7168, 24),
          (33, 128, 8), (33, 32, 1), (40, 2048, 130), (64, 544, 130), (64, 4096, 64), (65, 256, 64), (77, 2048, 257),
          (100, 64, 300), (128, 1024, 260), (129, 96, 300), (200, 4192, 65), (300, 512, 520), (300, 2048, 1000),
          (1025, 192, 264), (130, 4096, 64), (97, 1120, 200), (4100, 544, 2100), (4097, 1024, 2049), (4200, 32, 2060),
          (4099, 640, 2080), (4200, 2560, 2300), (24, 512, 33), (17, 1024, 9000), (50, 512, 8300), (64, 2048, 100),
          (32, 16384, 33), (33, 4096, 70), (128, 2048, 7000), (100, 8192, 40), (40, 8192, 70), (60, 8192, 6000),
          (256, 4096, 2000), (1000, 1536, 1000)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_linear(mx, T, K, N, fmt):
    g = gen(T + K + N)
    a, sa = activations(T, K, fmt, g)
    (w, s), bias, res = weights(N, K, g), bf(N, g=g, std=0.5), bf(T, N, g=g)
    z, ez = z_of(a, sa, fmt, w, s, None)
    for kind, has_bias, has_res, scale, save in (("none", False, False, 1.0, False), ("gelu_tanh", True, True, 0.5, True),
                                                 ("silu", True, False, -2.0, False)):
        say("linear", T, K, N, fmt, kind)
        b, r = bias if has_bias else None, res if has_res else None
        out = mx.mx_linear_quantized(*cuda(a, sa, w, s, b, r), scale, kind, save_z=save)
        y, z_got = out if save else (out, None)
        zb = z if b is None else z + bias.double()
        eb = ez if b is None else ez + (K + 8) * U * bias.double().abs() + U * zb.abs()
        want, err = scale * act(zb, kind), abs(scale) * value_error(zb, eb)
        if r is not None:
            want, err = want + res.double(), err + U * (want + res.double()).abs()
        say("   worst", within(y, want, (1 + B) * err + B * want.abs(), "y"))
        if save:
            within(z_got, zb, (1 + B) * eb + B * zb.abs(), "z")


GATED_SHAPES = [(1, 32, 1), (1, 256, 64), (3, 96, 32), (16, 288, 33), (17, 512, 160), (32, 2048, 96), (33, 128, 8),
                (64, 544, 96), (65, 1024, 130), (77, 7168, 64), (130, 96, 257), (300, 2048, 512), (1025, 192, 136),
                (4100, 288, 1056), (4097, 512, 1031), (4100, 2048, 1088), (4200, 32, 1056),
                (24, 512, 32), (17, 2048, 100), (32, 7168, 64), (20, 512, 4160), (50, 1024, 96), (64, 4096, 33), (45, 512, 4128),
                (100, 2048, 2080), (50, 8192, 64), (128, 7168, 40)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H,I", GATED_SHAPES)
def test_gate_up(mx, T, H, I, fmt):
    g = gen(T + H + I)
    a, sa = activations(T, H, fmt, g)
    (w, s), bias = weights(2 * I, H, g), bf(2 * I, g=g, std=0.5)
    z0, e0 = z_of(a, sa, fmt, w, s, None)
    for kind, has_bias, out, save in (("silu", False, None, True), ("gelu", True, "mxfp8", False), ("silu", True, "mxfp4", True)):
        if out and I % 32:
            continue
        say("gate_up", T, H, I, fmt, kind, out)
        b = bias if has_bias else None
        got = mx.mx_gate_up_quantized(*cuda(a, sa, w, s, b), kind, out, save_z=save)
        z = z0 if b is None else z0 + bias.double()
        ez = e0 if b is None else e0 + (H + 8) * U * bias.double().abs() + U * z.abs()
        val = act(z[:, :I], kind)
        want = val * z[:, I:]
        err = value_error(z[:, :I], ez[:, :I]) * (z[:, I:].abs() + ez[:, I:]) + val.abs() * ez[:, I:] + U * want.abs()
        if out is None:
            h = got[0] if save else got
            within(h, want, (1 + B) * err + B * want.abs(), "h")
        else:
            check_codes(got[0], got[1], want, err, out, "h")
        if save:
            within(got[-1], z, (1 + B) * ez + B * z.abs(), "z")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 20, 40, 100, 4100])
def test_nan_and_neighbours(mx, T, fmt):
    """A NaN scale or element reaches its own row or column alone; rows behind the last stay."""
    K, N = 288, 2100 if T > 4000 else 72
    g = gen(T)
    a, sa = activations(T, K, fmt, g)
    w, s = weights(N, K, g)
    z, ez = z_of(a, sa, fmt, w, s, None)
    s[5, 3] = 255
    sa[T // 2, 8] = 255
    z[:, 5] = math.nan
    z[T // 2] = math.nan
    if fmt == "mxfp8" and T > 2:
        a[0, K - 1] = 0x7F
        z[0] = math.nan
    say("nan", T, fmt)
    out = torch.full((T + 3, N), 7.0, dtype=torch.bfloat16, device=DEV)
    y = mx.mx_linear_quantized(*cuda(a, sa, w, s), out=out[:T])
    within(y, z, ((1 + B) * ez + B * z.abs()).nan_to_num(0), "y")
    assert bool((out[T:] == 7).all()), "rows behind the last were written"


def test_extreme_scales(mx):
    """Scale bytes from both ends, products in and out of fp32's range, subnormal sums."""
    for T in (3, 50):
        K, N = 64, 40
        g = gen(T)
        a, _ = activations(T, K, "mxfp8", g)
        sa = torch.randint(0, 255, (T, K // 32), generator=g, dtype=torch.uint8)
        w, _ = weights(N, K, g)
        s = (254 - sa[0].int()).clamp(0, 254).to(torch.uint8).expand(N, K // 32).contiguous()
        x, W = values(a, sa, "mxfp8"), decode(w, s)
        z, size = x @ W.T, x.abs() @ W.abs().T
        y = mx.mx_linear_quantized(*cuda(a, sa, w, s)).double().cpu()
        fine = (size < 2.0 ** 120) & (size > 2.0 ** -90)
        say("extreme", T, int(fine.sum()))
        assert fine[0].all()
        tol = (1 + B) * (DROP + (K + 8) * U) * size + B * z.abs()
        assert ((y - z).abs() <= tol)[fine].all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_in_place_repeat_and_workspace(mx, fmt):
    for T, K, N in ((4, 512, 64), (40, 2048, 64), (200, 4096, 129), (1100, 256, 264), (4100, 544, 2100)):
        g = gen(T)
        a, sa, (w, s) = *activations(T, K, fmt, g), weights(N, K, g)
        a, sa, w, s, bias, res = cuda(a, sa, w, s, bf(N, g=g), bf(T, N, g=g))
        say("in place", T, fmt)
        one = mx.mx_linear_quantized(a, sa, w, s, bias, res, 0.5, "relu")
        need = mx.raw().mx_linear_quantized_workspace_size(T, K, N)
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)  # NaN in every float
        buf = res.clone()
        two = mx.mx_linear_quantized(a, sa, w, s, bias, buf, 0.5, "relu", out=buf, ws=ws[:need] if need else None)
        assert torch.equal(one, two) and two.data_ptr() == buf.data_ptr()
        assert bool((ws[need:] == 255).all())


def test_unaligned_scales(mx):
    """Scales may begin anywhere where K % 512 != 0."""
    for T in (9, 70, 4100):
        K, N = 544, 2100 if T > 4000 else 40
        g = gen(T)
        a, sa, (w, s) = *activations(T, K, "mxfp4", g), weights(N, K, g)
        a, sa, w, s = cuda(a, sa, w, s)
        one = mx.mx_linear_quantized(a, sa, w, s)
        pad = lambda t: torch.cat((t.new_zeros(3), t.flatten()))[3:].view(t.shape)  # noqa: E731
        sa2, s2 = pad(sa), pad(s)
        assert sa2.data_ptr() % 4 == 3
        assert torch.equal(one, mx.mx_linear_quantized(a, sa2, w, s2))


def test_offsets_beyond_32_bits(mx):
    """9 GB of activation codes, and 4.5 GB of weight codes: rows at the far end against the formula."""
    g = gen(3)
    K = 8192
    w, s = weights(64, K, g)
    T = (1 << 20) + 77
    dg = torch.Generator(device=DEV)
    dg.manual_seed(1)
    a = torch.randint(0, 120, (T, K), generator=dg, dtype=torch.uint8, device=DEV)
    sa = torch.randint(118, 124, (T, K // 32), generator=dg, dtype=torch.uint8, device=DEV)
    say("far tokens")
    y = mx.mx_linear_quantized(a, sa, *cuda(w, s))
    for at in (0, T // 2, T - 40):
        z, ez = z_of(a[at:at + 40], sa[at:at + 40], "mxfp8", w, s, None)
        within(y[at:at + 40], z, (1 + B) * ez + B * z.abs(), f"tokens from {at}")
    del a, sa, y
    N = (1 << 20) + 131
    w = torch.randint(0, 256, (N, K // 2), generator=dg, dtype=torch.uint8, device=DEV)
    s = torch.randint(115, 122, (N, K // 32), generator=dg, dtype=torch.uint8, device=DEV)
    for T in (3, 24, 70, 300):
        a, sa = activations(T, K, "mxfp4", g)
        say("far rows", T)
        y = mx.mx_linear_quantized(*cuda(a, sa), w, s)
        for at in (0, N // 2, N - 50):
            z, ez = z_of(a, sa, "mxfp4", w[at:at + 50], s[at:at + 50], None)
            within(y[:, at:at + 50], z, (1 + B) * ez + B * z.abs(), f"rows from {at}")


def test_quantize_beyond_32_bits_of_threads(mx):
    """More than 2^35 values: threads past 2^32, a launch's limit along x."""
    K = 1 << 15
    rows = (1 << 20) + 3
    x = torch.ones(rows, K, dtype=torch.bfloat16, device=DEV)
    x[-1] = torch.arange(K, device=DEV).to(torch.bfloat16) - 7
    codes, scales = mx.mx_quantize(x, "mxfp4")
    for at in (0, rows // 2, rows - 2):
        assert (codes[at] == 0x66).all() and (scales[at] == 125).all()  # 1 = 4 * 2^-2
    code, byte = quantize_ref(x[-1:].double().cpu().numpy(), "mxfp4")
    assert np.array_equal(codes[-1:].cpu().numpy(), pack(code, "mxfp4")) and np.array_equal(scales[-1:].cpu().numpy(), byte)


def test_product_refusals(mx):
    g = gen(1)
    a, sa, (w, s) = *activations(4, 64, "mxfp8", g), weights(32, 64, g)
    a, sa, w, s, bias = cuda(a, sa, w, s, bf(32, g=g))
    for bad in ((a[:, :48].contiguous(), sa, w, s), (a, sa[:, :1].contiguous(), w, s), (a, sa, w, s[:8].contiguous()),
                (a, sa[:3].contiguous(), w, s), (a[:0], sa[:0], w, s), (a, sa, w[0], s)):
        for call in (mx.mx_linear_quantized, mx.mx_gate_up_quantized):
            with pytest.raises(ValueError):
                call(*bad)
    for bad in (dict(act="swish"), dict(scale=math.nan), dict(bias=bias[:8].contiguous()), dict(residual=bias),
                dict(out=torch.empty(4, 31, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ValueError):
            mx.mx_linear_quantized(a, sa, w, s, **bad)
    for bad in (dict(fmt="mxfp6"), dict(act="swish"), dict(bias=bias[:8].contiguous())):
        with pytest.raises(ValueError):
            mx.mx_gate_up_quantized(a, sa, w, s, **bad)
    with pytest.raises(ValueError):  # I = 16
        mx.mx_gate_up_quantized(a, sa, w, s, fmt="mxfp8")
    with pytest.raises(ValueError, match="overlap"):
        mx.mx_linear_quantized(a, sa, w[:32].contiguous(), s[:32].contiguous(), out=a.view(torch.bfloat16))
    with pytest.raises(ValueError):
        mx.mx_gate_up_quantized(a, sa, w[:31].contiguous(), s[:31].contiguous())


# ------------------------------------------------------------------ together

def block(mx, x, p, fmt, save=False):
    """A feed-forward block on quantized activations, as a model runs it."""
    y0, c, s, _ = mx.mx_norm_residual_quantize(x, w_pre=p["wpre"], fmt=fmt)
    r = mx.mx_gate_up_quantized(c, s, p["wgu"], p["sgu"], fmt=fmt, save_z=save)
    b = mx.mx_linear_quantized(r[0], r[1], p["wd"], p["sd"])
    y, cn, sn, _ = mx.mx_norm_residual_quantize(x, b, w_post=p["wpost"], w_pre=p["wnext"], fmt=fmt)
    return (y, cn, sn, b) + tuple(r[2:]) if save else (y, cn, sn)


def params(H, I, g):
    (wgu, sgu), (wd, sd) = weights(2 * I, H, g), weights(H, I, g)
    p = dict(wgu=wgu, sgu=sgu, wd=wd, sd=sd, wpre=bf(H, g=g, mean=1, std=.1), wpost=bf(H, g=g, mean=1, std=.1),
             wnext=bf(H, g=g, mean=1, std=.1))
    return {k: v.to(DEV) for k, v in p.items()}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 24, 70, 600])
def test_block_against_bf16_block(mx, T, fmt):
    """The block's distance from the same block on bf16 activations is the formats': E4M3 rounds by 2^-4
    of a value at most, E2M1 by a quarter (more where it saturates); over many terms both are far smaller."""
    H, I = 512, 256
    g = gen(T)
    p, x = params(H, I, g), bf(T, H, g=g).to(DEV)
    say("block", T, fmt)
    y, cn, sn = block(mx, x, p, fmt)
    xn = mx.mx_norm_residual(x, w_pre=p["wpre"])[1]
    b = mx.mx_linear_fused(mx.mx_gate_up(xn, p["wgu"], p["sgu"]), p["wd"], p["sd"])
    ref, xn2 = mx.mx_norm_residual(x, b, w_post=p["wpost"], w_pre=p["wnext"])
    far = float((y - ref).float().norm() / (ref - x).float().norm())
    say("   far", far)
    assert far < (0.1 if fmt == "mxfp8" else 0.5)
    assert torch.equal(cn, mx.mx_norm_residual_quantize(y, w_pre=p["wnext"], fmt=fmt)[1])


@pytest.mark.parametrize("T", [3, 70])
def test_block_captured(mx, T):
    """The block in a graph, replayed on new inputs with eager work between, equals the eager one."""
    H, I = 512, 256
    g = gen(T)
    p, x = params(H, I, g), bf(T, H, g=g).to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(mx, x, p, "mxfp8")
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(mx, x, p, "mxfp8")
    for i in range(4):
        x.copy_(bf(T, H, g=g).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, block(mx, x, p, "mxfp8")):
            assert torch.equal(a, b), i


def test_block_on_another_stream(mx):
    H, I, T = 512, 256, 70
    g = gen(9)
    p, x = params(H, I, g), bf(T, H, g=g).to(DEV)
    want = block(mx, x, p, "mxfp4")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block(mx, x, p, "mxfp4")
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_straight_through_gradients(mx):
    """What a training step makes of the saved z: the gradients of the existing backward calls, against the
    formula with the quantized forward's own pre-activations."""
    H, I, T = 256, 96, 40
    g = gen(4)
    p, x = params(H, I, g), bf(T, H, g=g).to(DEV)
    y, _, _, b, z = block(mx, x, p, "mxfp8", save=True)
    db = bf(T, H, g=g).to(DEV)
    dh = mx.mx_linear_fused_backward(db, p["wd"], p["sd"], need_dbias=False)[0]
    dx, _ = mx.mx_gate_up_backward(dh, z, p["wgu"], p["sgu"], need_dbias=False)
    Wd, Wgu = decode(p["wd"], p["sd"]), decode(p["wgu"], p["sgu"])
    dh_want = db.double().cpu() @ Wd
    within(dh, dh_want, (H + 8) * U * (db.double().cpu().abs() @ Wd.abs()) + B * 1.01 * dh_want.abs(), "dh")
    zc, d = z.double().cpu(), dh.double().cpu()
    sg = torch.sigmoid(zc[:, :I])
    dz = torch.cat((d * zc[:, I:] * (sg * (1 + zc[:, :I] * (1 - sg))), d * zc[:, :I] * sg), 1)
    want, size = dz @ Wgu, dz.abs() @ Wgu.abs()
    e = ACT_ERR * (1 + zc[:, :I].abs())
    edz = torch.cat((d.abs() * zc[:, I:].abs() * e, d.abs() * e), 1) + 4 * U * dz.abs()
    err = edz @ Wgu.abs() + (2 * I + 8) * U * size + B * size
    within(dx, want, (1 + B) * err + B * want.abs(), "dx")


def test_outputs_over_weights_and_vectors(mx):
    """Weights, bias, gate and norm weights are read by other workgroups while outputs are written."""
    T, K, N = 64, 512, 64
    g = gen(61)
    a, sa = activations(T, K, "mxfp8", g)
    w, s = weights(N, K, g)
    a, sa, w, s = cuda(a, sa, w, s)
    out = w.view(-1)[: T * N * 2].view(torch.bfloat16).view(T, N)
    with pytest.raises(ValueError, match="weight codes"):
        mx.mx_linear_quantized(a, sa, w, s, out=out)
    room = torch.zeros(T * N * 2 + 4096, dtype=torch.uint8, device=DEV)
    out = room[: T * N * 2].view(torch.bfloat16).view(T, N)
    with pytest.raises(ValueError, match="weight scales"):
        mx.mx_linear_quantized(a, sa, w, room[64:64 + N * K // 32].view(N, K // 32), out=out)
    with pytest.raises(ValueError, match="bias"):
        mx.mx_linear_quantized(a, sa, w, s, room[128:128 + 2 * N].view(torch.bfloat16), out=out)
    H = 256
    x, b = cuda(bf(T, H, g=g), bf(T, H, g=g))
    room = torch.ones(2 * T * H, dtype=torch.bfloat16, device=DEV)
    out, ones = room[: T * H].view(T, H), torch.ones(H, dtype=torch.bfloat16, device=DEV)
    over = room[T * H - 8: T * H - 8 + H]
    for name, kw in (("w_post", dict(w_post=over, w_pre=ones)), ("w_pre", dict(w_pre=over)), ("gate", dict(w_pre=ones, gate=over)),
                     ("gate", dict(w_pre=ones, gate=room[T * H - 8:][: T].view(T, 1))),
                     ("gate", dict(w_pre=ones, gate=room[8: 8 + T * H].view(T, H)))):
        with pytest.raises(ValueError, match=name):
            mx.mx_norm_residual_quantize(x, b, out=out, **kw)
    want = mx.mx_norm_residual_quantize(x, b, gate=room[T * H:].view(T, H).clone(), w_pre=ones)
    got = mx.mx_norm_residual_quantize(x, b, gate=room[T * H:].view(T, H), w_pre=ones, out=out)
    assert all(torch.equal(p, q) for p, q in zip(want[:3], got[:3]))
    full = bf(T, H, g=g).to(DEV)
    want = mx.mx_norm_residual_quantize(x, b, gate=full, w_pre=ones)
    got = mx.mx_norm_residual_quantize(x, b, gate=full, w_pre=ones, out=full)  # each element read before it is written
    assert all(torch.equal(p, q) for p, q in zip(want[:3], got[:3]))
