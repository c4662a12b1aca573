"""GPU parity of routing by scores and its gradient against the definition in 64 bits.

Chosen experts are compared exactly, in order.  Tolerances, u = 2^-24:
  * a gate is one value of 64 bits rounded once, u relative (2 u), and with softmax scores over all
    experts has the sum of E exponentials below it, in fp32: a lane sums E / 16 of them, each off by
    (1.3 |x| + 2) u of itself where x e^-x is at most 0.37: (E / 16 + 24) u.
  * dlogits: the chosen values from 64 bits, a dense row's others -p c with c = sum dp p: the same
    (E / 16 + 24) u of |dp p| and of |p| sum|dp p|, and half a step of the stored type.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEV = "cuda:0"


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


def scores(l, kind):
    """Of fp64 logits; a row of nothing but -Inf has scores 0."""
    if kind == "sigmoid":
        return torch.sigmoid(l)
    return torch.where((l == -math.inf).all(1, keepdim=True), torch.zeros_like(l), torch.softmax(l, 1))


def ref(l, k, kind, bias, groups, kept, by, renorm, scale):
    """(ids, gates) by the definition; ties to the lower index by a stable sort."""
    T, E = l.shape
    l = l.double()
    p = scores(l, kind)
    low = lambda v: torch.where(v.isnan(), torch.full_like(v, -math.inf), v)  # noqa: E731
    key = low(p if bias is None else p + bias.double())
    order = low(l) if bias is None else key
    if groups > 1:
        per = key.reshape(T, groups, -1).sort(dim=-1, descending=True)[0]
        val = per[..., 0] if by == "max" or per.shape[-1] == 1 else low(per[..., 0] + per[..., 1])
        rank = val.sort(dim=-1, descending=True, stable=True)[1].argsort(-1)
        shut = (rank >= kept).repeat_interleave(E // groups, 1)
        # shut experts after all others, whatever their keys
        idx = (order.sort(dim=-1, descending=True, stable=True)[1])
        ids = torch.stack([i[~s[i]][:k] for i, s in zip(idx, shut)])
    else:
        ids = order.sort(dim=-1, descending=True, stable=True)[1][:, :k]
    g = p.gather(1, ids)
    if renorm:
        s = g.sum(1, keepdim=True)
        g = torch.where(s == 0, torch.zeros_like(g), g / s)
    return ids.int(), scale * g


def gate_tol(E, kind, renorm):
    return (2 if kind == "sigmoid" or renorm else E / 16 + 24) * U


def check(mx, l, k, kind="softmax", bias=None, groups=1, kept=1, by="top2", renorm=False, scale=1.0, what=""):
    ids, gates = mx.moe_route_scored(l.to(DEV), k, kind, None if bias is None else bias.to(DEV), groups, kept, by, renorm, scale)
    want_ids, want = ref(l, k, kind, bias, groups, kept, by, renorm, scale)
    ids, gates = ids.cpu(), gates.double().cpu()
    wrong = (ids != want_ids).any(1).nonzero().flatten()
    assert not len(wrong), f"{what}: {len(wrong)} rows, first {int(wrong[0])}: {ids[wrong[0]].tolist()} {want_ids[wrong[0]].tolist()}"
    assert torch.equal(gates.isnan(), want.isnan()), what
    r = ((gates - want).abs() / (gate_tol(l.shape[1], kind, renorm) * want.abs() + 2.0 ** -149))[~want.isnan()]
    assert not r.numel() or r.max() <= 1, f"{what}: gates off, worst {float(r.max()):.3g}"
    return ids


CASES = [  # E, k, groups, kept
    (1, 1, 1, 1), (2, 2, 1, 1), (8, 2, 1, 1), (17, 5, 1, 1), (64, 8, 1, 1), (100, 32, 1, 1), (256, 8, 1, 1), (257, 9, 1, 1),
    (384, 8, 1, 1), (512, 12, 1, 1), (1000, 16, 1, 1), (1024, 32, 1, 1), (33, 32, 1, 1), (40, 17, 1, 1),
    (256, 8, 8, 4), (256, 8, 8, 1), (160, 6, 8, 3), (384, 8, 8, 4), (64, 4, 64, 5), (12, 3, 4, 2), (512, 16, 32, 7), (96, 32, 3, 2),
    (1024, 32, 4, 2), (60, 7, 20, 3), (1024, 10, 64, 40)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E,k,groups,kept", CASES)
def test_route(mx, E, k, groups, kept, bf16):
    for i, (kind, has_bias, by, renorm, scale) in enumerate([
            ("softmax", False, "max", False, 1.0), ("sigmoid", True, "top2", True, 2.5), ("softmax", True, "top2", True, 1.0),
            ("sigmoid", False, "max", False, -0.5), ("softmax", False, "top2", True, 2.0), ("sigmoid", True, "max", True, 1.0)]):
        g = gen(E + k + i)
        T = (1, 33, 130)[i % 3]
        l = (torch.randn(T, E, generator=g) * 1.5).to(torch.bfloat16 if bf16 else torch.float32)
        bias = torch.randn(E, generator=g) * 0.05 if has_bias else None
        say("route", E, k, groups, kept, kind, by, bf16)
        check(mx, l, k, kind, bias, groups, kept, by, renorm, scale, f"{kind} {by}")


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 4097])
def test_route_tokens(mx, T, kind):
    g = gen(T)
    l = torch.randn(T, 256, generator=g) * 2
    bias = torch.randn(256, generator=g) * 0.1
    check(mx, l, 8, kind, bias, 8, 4, "top2", True, 2.5)
    check(mx, l, 8, kind)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_ties_and_near_ties(mx, kind):
    """Equal keys go to the lower id; keys that differ in the last bits keep their 64-bit order."""
    g = gen(1)
    E, T = 256, 64
    few = torch.randint(-3, 4, (T, E), generator=g).float() / 2
    zero = torch.zeros(T, E)
    near = 0.25 + torch.randint(-4, 5, (T, E), generator=g).float() * 2.0 ** -24
    wide = torch.randn(T, E, generator=g) * torch.tensor([2.0 ** (i % 40 - 20) for i in range(T)])[:, None]
    tiny = torch.randn(T, E, generator=g) * 2.0 ** -60
    for name, l in (("few", few), ("zero", zero), ("near", near), ("wide", wide), ("tiny", tiny)):
        for bias in (None, torch.zeros(E), torch.randint(-2, 3, (E,), generator=g).float() * 2.0 ** -25,
                     torch.randint(-1, 2, (E,), generator=g).float(), torch.randn(E, generator=g) * 1e-6,
                     torch.randn(E, generator=g) * 1e6):
            for groups, kept, by in ((1, 1, "max"), (8, 3, "top2"), (16, 5, "max")):
                say("ties", kind, name, groups)
                check(mx, l, 8, kind, bias, groups, kept, by, True, what=name)


def test_a_bias_that_cancels(mx):
    """Keys near zero, where a bias takes nearly all of a score away."""
    g = gen(8)
    l = torch.randn(200, 128, generator=g)
    l[:] = l[0] + torch.randn(200, 128, generator=g) * 1e-6
    check(mx, l, 8, "sigmoid", -torch.sigmoid(l[0]), 1, 1, what="sigmoid")
    check(mx, l, 8, "sigmoid", -torch.sigmoid(l[0]), 8, 4, what="groups")
    check(mx, l, 8, "softmax", -torch.softmax(l[0], 0), 1, 1, what="softmax")


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_masked_experts(mx, kind):
    """-Inf takes an expert out: score 0, chosen only when nothing else is left; a row of -Inf alone has
    gates 0 and the lowest ids."""
    g = gen(3)
    T, E, k = 40, 64, 6
    l = torch.randn(T, E, generator=g)
    for t in range(T):
        l[t, torch.randperm(E, generator=g)[: min(E, 2 * t)]] = -math.inf
    l[5] = -math.inf
    for bias in (None, torch.randn(E, generator=g) * 0.1):
        for renorm in (False, True):
            for groups, kept in ((1, 1), (8, 2)):
                ids = check(mx, l, k, kind, bias, groups, kept, "top2", renorm)
                assert all(len(set(r)) == k for r in ids.tolist())
    ids, gates = mx.moe_route_scored(l.to(DEV), k, kind, renormalize=True)
    assert ids[5].tolist() == list(range(k)) and (gates[5] == 0).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_nan_and_inf(mx, kind):
    """NaN sorts below all else; ids stay distinct and in range; other rows are as ever."""
    g = gen(4)
    T, E, k = 12, 96, 8
    l = torch.randn(T, E, generator=g)
    l[1, 7] = math.nan
    l[2] = math.nan
    l[3, 5] = math.inf
    l[4, 5:9] = math.inf
    l[5, :92] = math.nan
    l[6, ::2] = -math.nan
    for bias in (None, torch.randn(E, generator=g) * 0.1):
        for groups, kept in ((1, 1), (8, 3)):
            ids, gates = mx.moe_route_scored(l.to(DEV), k, kind, None if bias is None else bias.to(DEV), groups, kept)
            ids = ids.cpu()
            assert all(len(set(r)) == k and min(r) >= 0 and max(r) < E for r in ids.tolist())
            rest = [0, 7, 8, 9, 10, 11]
            want, gw = ref(l[rest], k, kind, bias, groups, kept, "top2", False, 1.0)
            assert torch.equal(ids[rest], want)
            assert ((gates.cpu()[rest].double() - gw).abs() <= gate_tol(E, kind, False) * gw).all()
            assert gates[2].isnan().all()
            if bias is None and groups == 1 and kind == "sigmoid":
                assert ids[5, :4].tolist() == l[5, 92:].sort(dim=-1, descending=True, stable=True)[1].add(92).tolist()
                assert gates[5, 4:].isnan().all() and not gates[5, :4].isnan().any()


def test_far_logits(mx):
    """Scores below fp32's range still renormalise; those below fp64's give 0."""
    l = torch.tensor([[-100.0, -101.0, -102.0, -300.0], [-800.0, -801.0, -802.0, -803.0], [90.0, 100.0, -100.0, 95.0]])
    ids, gates = mx.moe_route_scored(l.to(DEV), 2, "sigmoid", renormalize=True)
    assert ids.tolist() == [[0, 1], [0, 1], [1, 3]]
    assert abs(float(gates[0, 0]) - 1 / (1 + math.exp(-1))) < 1e-6 and gates[1].tolist() == [0.0, 0.0]
    assert gates[2].tolist() == [0.5, 0.5]


def test_matches_route_topk(mx):
    """Renormalised softmax scores without bias or groups are moe_route_topk's gates."""
    l = torch.randn(100, 256, generator=gen(5)).to(DEV)
    ids, gates = mx.moe_route_scored(l, 8, renormalize=True)
    ids2, gates2 = mx.moe_route_topk(l, 8)
    assert torch.equal(ids, ids2) and torch.allclose(gates, gates2, rtol=1e-6, atol=0)


def test_outputs_given_and_rows_behind(mx):
    l = torch.randn(5, 64, generator=gen(6)).to(DEV)
    ids = torch.full((7, 4), -7, dtype=torch.int32, device=DEV)
    gates = torch.full((7, 4), -7.0, device=DEV)
    a, b = mx.moe_route_scored(l, 4, ids=ids[:5], gates=gates[:5])
    assert a.data_ptr() == ids.data_ptr() and b.data_ptr() == gates.data_ptr()
    assert (ids[5:] == -7).all() and (gates[5:] == -7).all()
    want = mx.moe_route_scored(l, 4)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_refusals(mx):
    l = torch.randn(5, 64).to(DEV)
    bias = torch.zeros(64, device=DEV)
    for kw in (dict(top_k=0), dict(top_k=65), dict(top_k=33), dict(top_k=-1), dict(top_k=4, score="tanh"), dict(top_k=4, n_group=5),
               dict(top_k=4, n_group=8, topk_group=9), dict(top_k=9, n_group=8, topk_group=1), dict(top_k=4, group_score="sum"),
               dict(top_k=4, bias=bias[:8]), dict(top_k=4, scale=math.inf), dict(top_k=4, n_group=0)):
        with pytest.raises(ValueError):
            mx.moe_route_scored(l, **kw)
    for bad in (l.half(), l.double()):
        with pytest.raises(TypeError):
            mx.moe_route_scored(bad, 4)
    with pytest.raises(ValueError):
        mx.moe_route_scored(l.t(), 4)
    with pytest.raises(ValueError):
        mx.moe_route_scored(l[:0], 4)
    with pytest.raises(TypeError):
        mx.moe_route_scored(l, 4, bias=bias.bfloat16())
    with pytest.raises(ValueError):
        mx.moe_route_scored(torch.randn(2, 1025).to(DEV), 4)
    ids, gates = mx.moe_route_scored(l, 4)
    for bad in ((gates[:, :3].contiguous(), l, ids), (gates[:3], l, ids), (gates, l[:3], ids)):
        with pytest.raises(ValueError):
            mx.moe_route_scored_backward(*bad)
    with pytest.raises(ValueError):
        mx.moe_route_scored_backward(gates, l, ids, score="tanh")


# ------------------------------------------------------------------ gradient

def grad_ref(dg, l, ids, kind, renorm, scale):
    """(dlogits, the sizes that its error goes by) in 64 bits."""
    l, ids, c = l.double(), ids.long(), scale * dg.double()
    p = scores(l, kind)
    chosen = p.gather(1, ids)
    if renorm:
        s = chosen.sum(1, keepdim=True)
        c = torch.where(s == 0, torch.zeros_like(c), (c - (c * chosen).sum(1, keepdim=True) / s) / s)
    dp = torch.zeros_like(p).scatter(1, ids, c)
    if kind == "sigmoid":
        return dp * p * (1 - p), (dp * p).abs()
    return p * (dp - (dp * p).sum(1, keepdim=True)), (dp * p).abs() + p * (dp * p).abs().sum(1, keepdim=True)


def check_grad(got, dg, l, ids, kind, renorm, scale):
    want, size = grad_ref(dg, l, ids, kind, renorm, scale)
    half = 2.0 ** -8 if l.dtype == torch.bfloat16 else U
    tol = (l.shape[1] / 16 + 24) * U * size + half * 1.01 * want.abs() + 2.0 ** -133
    assert got.dtype == l.dtype and got.shape == l.shape
    r = ((got.double().cpu() - want).abs() / tol)
    assert r.max() <= 1, f"worst {float(r.max()):.3g} of {int((r > 1).sum())}"


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (5, 17, 5), (64, 256, 8), (33, 257, 9), (9, 384, 8), (7, 1000, 16),
                                   (6, 1024, 32), (700, 64, 6), (4, 60, 32)])
def test_backward(mx, T, E, k, bf16):
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            g = gen(T + E)
            l = (torch.randn(T, E, generator=g) * 1.5).to(torch.bfloat16 if bf16 else torch.float32)
            dg = torch.randn(T, k, generator=g)
            ids = mx.moe_route_scored(l.to(DEV), k, kind, renormalize=renorm, scale=2.5)[0]
            say("backward", T, E, k, kind, renorm, bf16)
            d = mx.moe_route_scored_backward(dg.to(DEV), l.to(DEV), ids, kind, renorm, 2.5)
            check_grad(d, dg, l, ids.cpu(), kind, renorm, 2.5)
            if kind == "sigmoid" or renorm:
                off = torch.ones_like(l, dtype=torch.bool).scatter(1, ids.cpu().long(), False)
                assert (d.cpu()[off] == 0).all()


def test_backward_masked_rows_and_skipped_ids(mx):
    g = gen(2)
    l = torch.randn(6, 32, generator=g)
    l[1] = -math.inf
    l[2, :30] = -math.inf
    dg = torch.randn(6, 4, generator=g)
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids = mx.moe_route_scored(l.to(DEV), 4, kind, renormalize=renorm)[0]
            d = mx.moe_route_scored_backward(dg.to(DEV), l.to(DEV), ids, kind, renorm).cpu()
            assert (d[1] == 0).all() and not d.isnan().any()
            check_grad(d, dg, l, ids.cpu(), kind, renorm, 1.0)
            # ids outside [0, E) are as if they were not there
            odd = ids.clone()
            odd[3, 1], odd[4, 2] = -1, 32
            d = mx.moe_route_scored_backward(dg.to(DEV), l.to(DEV), odd, kind, renorm).cpu()
            for t, j in ((3, 1), (4, 2)):
                keep = [i for i in range(4) if i != j]
                check_grad(d[t:t + 1], dg[t:t + 1, keep], l[t:t + 1], ids.cpu()[t:t + 1, keep], kind, renorm, 1.0)


def test_gradient_against_differences():
    """The gradient formula used above against central differences of the forward's, in 64 bits."""
    g = gen(7)
    l, dg = torch.randn(4, 12, generator=g, dtype=torch.float64), torch.randn(4, 3, generator=g, dtype=torch.float64)
    way = torch.randn(4, 12, generator=g, dtype=torch.float64)
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids = ref(l, 3, kind, None, 1, 1, "max", renorm, 1.7)[0]

            def loss(v):
                p = scores(v, kind).gather(1, ids.long())  # noqa: B023
                return float((dg * 1.7 * (p / p.sum(1, keepdim=True) if renorm else p)).sum())  # noqa: B023

            want = float((grad_ref(dg, l, ids, kind, renorm, 1.7)[0] * way).sum())
            h = 1e-5
            assert abs((loss(l + h * way) - loss(l - h * way)) / (2 * h) - want) < 1e-8


def test_backward_captured_with_an_eager_graph(mx):
    """Forward and backward inside torch.autograd.Function, captured while an eager run's results live."""

    class Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, l):
            ids, gates = mx.moe_route_scored(l, 4, "sigmoid", renormalize=True, scale=2.0)
            ctx.save_for_backward(l, ids)
            ctx.mark_non_differentiable(ids)
            return ids, gates

        @staticmethod
        def backward(ctx, _, dg):
            l, ids = ctx.saved_tensors
            return mx.moe_route_scored_backward(dg.contiguous(), l, ids, "sigmoid", True, 2.0)

    g = gen(1)
    l = torch.randn(50, 64, generator=g).to(DEV)
    dg = torch.randn(50, 4, generator=g).to(DEV)

    def step():
        x = l.detach().requires_grad_()
        ids, gates = Route.apply(x)
        return ids, gates, torch.autograd.grad(gates, x, dg)[0]

    eager = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        l.copy_(torch.randn(50, 64, generator=g).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), i
    assert all(t is not None for t in eager)


# ------------------------------------------------------------------ the layer behind it

def expert_weights(E, H, I, g):
    u8 = torch.uint8
    r = lambda *s, lo=0, hi=256: torch.randint(lo, hi, s, generator=g, dtype=u8).to(DEV)  # noqa: E731
    return r(E, 2 * I, H // 2), r(E, 2 * I, H // 32, lo=115, hi=120), r(E, H, I // 2), r(E, H, I // 32, lo=115, hi=120)


@pytest.mark.parametrize("act8", [False, True])
@pytest.mark.parametrize("T,E,k,I", [(1, 16, 4, 256), (7, 16, 4, 1024), (20, 16, 4, 256), (32, 32, 8, 1024), (40, 16, 4, 256),
                                     (256, 16, 4, 256), (24, 96, 8, 1024), (32, 64, 16, 256)])
def test_forward_routed(mx, T, E, k, I, act8):
    """With moe_route_topk's routing the layer is moe_mxfp4_forward bit for bit; with scored gates it is
    linear in them."""
    H = 1024
    g = gen(T + E)
    W = expert_weights(E, H, I, g)
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    l = torch.randn(T, E, generator=g).to(DEV)
    say("routed", T, E, k, I, act8)
    ids, gates = mx.moe_route_topk(l, k)
    want = mx.moe_mxfp4_forward(x, l, k, *W, act8=act8)
    for _ in range(2):
        assert torch.equal(mx.moe_mxfp4_forward_routed(x, ids, gates, *W, act8=act8), want)
    ids, gates = mx.moe_route_scored(l, k, "sigmoid", torch.randn(E, generator=g).to(DEV) * 0.1, 4, 2, renormalize=True, scale=2.0)
    one = mx.moe_mxfp4_forward_routed(x, ids, gates, *W, act8=act8)
    two = mx.moe_mxfp4_forward_routed(x, ids, 2 * gates, *W, act8=act8)
    assert torch.equal(two, 2 * one) and bool(one.isfinite().all())
    if not act8:
        sort = mx.moe_sort_by_expert(ids, E)
        h = mx.moe_gate_up_swiglu(x, W[0], W[1], sort, k)
        by_stages = mx.moe_down_combine(h, gates, W[2], W[3], sort, T, k)
        assert torch.equal(one, by_stages)


def test_router_of_a_moe_block(mx):
    """The path of a mixture-of-experts block: the norm hands the router bf16 and the shared expert 8 bits."""
    T, H, I, E, k = 24, 1024, 256, 32, 4
    g = gen(11)
    W = expert_weights(E, H, I, g)
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    wpre = torch.ones(H).bfloat16().to(DEV)
    wr = torch.randint(0, 256, (E, H // 2), generator=g, dtype=torch.uint8).to(DEV)
    sr = torch.randint(115, 120, (E, H // 32), generator=g, dtype=torch.uint8).to(DEV)
    _, codes, scales, xn = mx.mx_norm_residual_quantize(x, w_pre=wpre, save_xn=True)
    logits = mx.mx_linear(xn, wr, sr)
    bias = torch.zeros(E, device=DEV)
    ids, gates = mx.moe_route_scored(logits, k, "sigmoid", bias, 8, 4, renormalize=True, scale=2.5)
    want_ids, want = ref(logits.cpu(), k, "sigmoid", bias.cpu(), 8, 4, "top2", True, 2.5)
    assert torch.equal(ids.cpu(), want_ids)
    routed = mx.moe_mxfp4_forward_routed(xn, ids, gates, *W)
    h = mx.mx_gate_up_quantized(codes, scales, W[0][0], W[1][0], fmt="mxfp8")
    y = mx.mx_linear_quantized(*h, W[2][0], W[3][0], residual=routed)
    assert bool(y.isfinite().all()) and y.shape == (T, H)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_infinite_biases(mx, kind):
    """-Inf shuts an expert and +Inf forces it; a group with both sums to NaN and counts as the lowest."""
    g = gen(21)
    l = torch.randn(70, 64, generator=g)
    bias = torch.randn(64, generator=g) * 0.1
    shut = bias.clone()
    shut[::3] = -math.inf
    forced = bias.clone()
    forced[[5, 40]] = math.inf
    both = bias.clone()
    both[8:16] = -math.inf
    both[24:32] = -math.inf
    both[[9, 30]] = math.inf
    for name, b in (("shut", shut), ("forced", forced), ("both", both)):
        for groups, kept, by in ((1, 1, "max"), (8, 3, "top2"), (8, 6, "top2"), (8, 7, "top2"), (8, 3, "max")):
            say("infinite", kind, name, groups, kept, by)
            check(mx, l, 8, kind, b, groups, kept, by, True, what=name)


# ------------------------------------------------------------------ confident rows, NaN, scores that vanish

def grad_pairs(dg, l, ids, kind, renorm, scale):
    """(gradient of the chosen logits, the sizes that its error goes by, gradient of the others, their sizes):
    the same gradient with no difference of nearly equal values in it.  With q the chosen gates' weights and
    `rest` what the experts that are not chosen have, c_i - sum c_j q_j = sum (c_i - c_j) q_j + c_i rest."""
    l, ids, c = l.double(), ids.long(), scale * dg.double()
    mine = l.gather(1, ids)
    others = torch.ones_like(l, dtype=torch.bool).scatter(1, ids, False)
    slope, rest = torch.ones_like(mine), torch.zeros_like(c[:, :1])
    e_other = torch.zeros_like(l)
    if kind == "sigmoid":
        q, slope = torch.sigmoid(mine), torch.sigmoid(-mine)
        if not renorm:
            return c * q * slope, (c * q * slope).abs(), e_other, e_other
    else:
        top = l.max(1, keepdim=True)[0]
        e_other = torch.exp(l - top) * others
        q, rest = torch.exp(mine - top), e_other.sum(1, keepdim=True)
    total = q.sum(1, keepdim=True) if renorm else q.sum(1, keepdim=True) + rest
    q, rest, e_other = q / total, 0 * rest if renorm else rest / total, 0 * e_other if renorm else e_other / total
    diff = c[:, :, None] - c[:, None, :]
    pairs, size = (diff * q[:, None, :]).sum(2) + c * rest, (diff.abs() * q[:, None, :]).sum(2) + c.abs() * rest
    return (q * slope * pairs, q * slope * size, -e_other * (c * q).sum(1, keepdim=True),
            e_other * (c * q).abs().sum(1, keepdim=True))


def test_pairs_are_the_gradient():
    """grad_pairs against the definition p (dp - sum dp p) with 90 digits, on confident rows."""
    from decimal import Decimal, localcontext
    g = gen(31)
    E, k = 7, 3
    l = torch.randn(4, E, generator=g)
    l[1, 2] += 20
    l[2, 2] += 30
    l[2, 4] = l[2, 2]
    l[3, 0] += 60
    dg = torch.randn(4, k, generator=g)
    dg[2] = 1.0
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids = ref(l, k, kind, None, 1, 1, "max", renorm, 1.0)[0]
            got, size, other, other_size = grad_pairs(dg, l, ids, kind, renorm, 2.5)
            with localcontext() as ctx:
                ctx.prec = 90
                for t in range(4):
                    v = [Decimal(float(x)) for x in l[t]]
                    p = [1 / (1 + (-x).exp()) for x in v] if kind == "sigmoid" else [x.exp() for x in v]
                    if kind == "softmax":
                        z = sum(p)
                        p = [x / z for x in p]
                    c = [Decimal(2.5) * Decimal(float(x)) for x in dg[t]]
                    at = [int(i) for i in ids[t]]
                    if renorm:
                        s = sum(p[i] for i in at)
                        cp = sum(x * p[i] for x, i in zip(c, at)) / s
                        c = [(x - cp) / s for x in c]
                    dp = [Decimal(0)] * E
                    for x, i in zip(c, at):
                        dp[i] = x
                    if kind == "sigmoid":
                        d = [x * y * (1 - y) for x, y in zip(dp, p)]
                    else:
                        m = sum(x * y for x, y in zip(dp, p))
                        d = [y * (x - m) for x, y in zip(dp, p)]
                    for j, i in enumerate(at):
                        assert abs(Decimal(float(got[t, j])) - d[i]) <= Decimal(1e-12) * Decimal(float(size[t, j])) + Decimal(1e-80)
                    for i in set(range(E)) - set(at):
                        # renormalised, a logit that is not chosen has no gradient: 0 but for the 90 digits
                        tol = Decimal(1e-12) * Decimal(float(other_size[t, i])) + Decimal(1e-80)
                        assert abs(Decimal(float(other[t, i])) - d[i]) <= tol


def check_pairs(got, dg, l, ids, kind, renorm, scale, what=""):
    """Softmax over all experts: the others' exponentials, each off by 3 u, are summed in fp32, E / 16 of them and
    four steps: below r = (E / 16 + 24) u of their sum, which `rest` carries twice and the weights once; another
    expert's own is multiplied by a value rounded once and rounded.  The rest is 64-bit.  And half a step of the
    stored type, in bf16 after one of fp32; 2^-133 for what fp32 has no normal numbers for."""
    want, size, other, other_size = grad_pairs(dg, l, ids, kind, renorm, scale)
    l, half = l.double(), 2.0 ** -8 if l.dtype == torch.bfloat16 else U
    dense = kind == "softmax" and not renorm
    r = (l.shape[1] / 16 + 24) * U if dense else 2.0 ** -40
    got = got.double().cpu()
    tol = 3 * r * size + half * 1.01 * want.abs() + 2.0 ** -133
    worst = float(((got.gather(1, ids.long()) - want).abs() / tol).max())
    assert worst <= 1, f"{what}: chosen, worst {worst:.3g}"
    others = torch.ones_like(l, dtype=torch.bool).scatter(1, ids.long(), False)
    if not dense:
        assert (got[others] == 0).all(), what
    elif others.any():
        tol = (6 * U + 2 * r) * other_size + half * 1.01 * other.abs() + 2.0 ** -133
        worst = float(((got - other).abs() / tol)[others].max())
        assert worst <= 1, f"{what}: others, worst {worst:.3g}"


@pytest.mark.parametrize("kind,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("E,k", [(17, 5), (64, 1), (256, 8), (384, 8), (1000, 16), (1024, 32), (40, 32), (32, 32)])
def test_backward_of_confident_rows(mx, E, k, kind, renorm):
    """One expert, or two alike, 8 to 60 above all others: their gradients keep their digits, also where
    dgates are equal and what is left is the others' share alone."""
    for gap in (8, 12, 16, 20, 30, 60):
        for bf16 in (False, True):
            g = gen(E + k + gap)
            T = 24
            l = torch.randn(T, E, generator=g) * 0.5
            if kind == "sigmoid":
                l -= gap  # whose scores are next to 1 only for the best
            best = torch.randint(0, E, (T,), generator=g)
            l[torch.arange(T), best] = 1.0 if kind == "sigmoid" else gap + 2.0
            two = torch.randint(0, E, (T,), generator=g)
            l[torch.arange(T)[1::2], two[1::2]] = l[torch.arange(T)[1::2], best[1::2]]
            l = l.to(torch.bfloat16 if bf16 else torch.float32)
            dg = torch.randn(T, k, generator=g)
            dg[T // 2:] = 0.75
            ids = mx.moe_route_scored(l.to(DEV), k, kind, renormalize=renorm, scale=2.5)[0]
            d = mx.moe_route_scored_backward(dg.to(DEV), l.to(DEV), ids, kind, renorm, 2.5)
            check_pairs(d, dg, l, ids.cpu(), kind, renorm, 2.5, f"gap {gap} {bf16}")


def test_backward_of_vanishing_sigmoid_scores(mx):
    """Renormalised sigmoid scores near the end of 64 bits: 1 / sum p is near its other end, the gradient is not."""
    g = gen(43)
    l = -700 - 8 * torch.rand(20, 16, generator=g)
    dg = torch.randn(20, 4, generator=g) * 1e6
    ids, gates = mx.moe_route_scored(l.to(DEV), 4, "sigmoid", renormalize=True, scale=2.5)
    assert bool((gates[:, 0] > 0).all())
    d = mx.moe_route_scored_backward(dg.to(DEV), l.to(DEV), ids, "sigmoid", True, 2.5)
    assert bool(d.isfinite().all())
    check_pairs(d, dg, l, ids.cpu(), "sigmoid", True, 2.5)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E,k", [(32, 4), (384, 8), (96, 32), (1024, 3)])
def test_backward_of_nan_rows(mx, E, k, bf16):
    """A softmax row with a NaN logit has gates NaN and a gradient of NaN, whatever else is in the row and whether
    the NaN is chosen; a sigmoid row where the chosen logit (renormalised: any chosen one) is NaN.  Other rows are
    as they are without it."""
    g = gen(E)
    T = 9
    l = torch.randn(T, E, generator=g).to(torch.bfloat16 if bf16 else torch.float32)
    clean = l.clone()
    l[1] = math.nan
    l[2] = -math.inf
    l[2, E - 1] = math.nan   # not chosen: -Inf has the lower ids
    l[3] = -math.inf
    l[3, 0] = math.nan       # chosen
    l[5, E // 2] = math.nan  # behind all others, not chosen
    l[6, k:] = math.nan
    l[7, 1] = -math.nan
    bad = torch.tensor([False, True, True, True, False, True, True, True, False])
    dg = torch.randn(T, k, generator=g)
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            say("nan rows", E, k, kind, renorm)
            ids, gates = mx.moe_route_scored(l.to(DEV), k, kind, renormalize=renorm)
            d = mx.moe_route_scored_backward(dg.to(DEV), l.to(DEV), ids, kind, renorm).cpu()
            ids_clean = mx.moe_route_scored(clean.to(DEV), k, kind, renormalize=renorm)[0]
            want = mx.moe_route_scored_backward(dg.to(DEV), clean.to(DEV), ids_clean, kind, renorm).cpu()
            assert torch.equal(d[~bad], want[~bad])
            if kind == "softmax":
                assert gates.cpu()[bad].isnan().all()
                assert d[bad].isnan().all(), f"rows {(~d.isnan().all(1) & bad).nonzero().flatten().tolist()}"
            else:
                chosen = torch.zeros(T, E, dtype=torch.bool).scatter(1, ids.cpu().long(), True)
                hit = chosen & (l.isnan().logical_and(chosen).any(1, keepdim=True) if renorm else l.isnan())
                assert d[hit].isnan().all() and not d[~hit].isnan().any()


def test_backward_where_gates_are_0(mx):
    """A bias that chooses experts so far below the others that their scores are 0 in 64 bits: the gates are 0, and
    so is the gradient; a little nearer both are there."""
    E, k = 16, 4
    g = gen(41)
    l = torch.randn(3, E, generator=g)
    l[0, 4:] -= 800
    l[1, 4:] -= 300
    l[2, 4:] = -math.inf
    bias = torch.zeros(E)
    bias[:4] = -10.0
    dg = torch.randn(3, k, generator=g)
    for dtype in (torch.float32, torch.bfloat16):
        x = l.to(dtype)
        ids, gates = mx.moe_route_scored(x.to(DEV), k, "softmax", bias.to(DEV), renormalize=True)
        assert (ids.cpu() >= 4).all() and (gates[0] == 0).all() and (gates[2] == 0).all() and (gates[1] > 0).all()
        d = mx.moe_route_scored_backward(dg.to(DEV), x.to(DEV), ids, "softmax", True)
        assert (d[2] == 0).all() and (d[0] == 0).all(), d[0].tolist()
        check_pairs(d[1:2], dg[1:2], x[1:2], ids[1:2].cpu(), "softmax", True, 1.0)


# ------------------------------------------------------------------ gates

@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E,k", [(1, 1), (17, 5), (64, 8), (128, 8), (256, 8), (384, 8), (512, 12), (1000, 16), (1024, 32), (96, 32)])
def test_gates_are_rounded_once(mx, E, k, bf16):
    """Half a step of fp32 from the 64-bit value, for softmax over all experts as for the others, and the same bits
    whatever chooses the experts: without a bias, with one of zeros, with groups that are all there and with
    candidates that are decided again."""
    for spread in (0.01, 1.5, 6.0):
        g = gen(E + int(10 * spread))
        l = (torch.randn(130, E, generator=g) * spread).to(torch.bfloat16 if bf16 else torch.float32)
        for renorm in (False, True):
            ids, gates = mx.moe_route_scored(l.to(DEV), k, "softmax", renormalize=renorm)
            want = ref(l, k, "softmax", None, 1, 1, "max", renorm, 1.0)[1]
            off = ((gates.double().cpu() - want).abs() / (U * (1 + 2.0 ** -16) * want + 2.0 ** -150)).max()
            assert off <= 1, f"{spread} {renorm}: {float(off):.3g} half steps"
            zeros = torch.zeros(E, device=DEV)
            again = mx.moe_route_scored(l.to(DEV), k, "softmax", zeros, renormalize=renorm)
            assert torch.equal(again[0], ids) and torch.equal(again[1], gates), f"{spread} {renorm}"
            if E % 8 == 0:
                # the same experts again, by groups that keep them all in place: seven of eight, the last one shut out by a bias
                shut = zeros.clone()
                shut[E // 8 * 7:] = -100.0
                if k <= E // 8 * 7:
                    a = mx.moe_route_scored(l.to(DEV), k, "softmax", shut, renormalize=renorm)
                    b = mx.moe_route_scored(l.to(DEV), k, "softmax", shut, 8, 7, "max", renormalize=renorm)
                    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("act8", [False, True])
@pytest.mark.parametrize("T,E,k,I,H", [(32, 256, 16, 512, 1024), (17, 192, 16, 512, 2048), (32, 256, 9, 512, 1024), (33, 256, 16, 512, 1024),
                                       (16, 256, 16, 512, 1024), (12, 128, 4, 1024, 1024), (25, 200, 8, 768, 1024)])
def test_forward_routed_takes_every_plan(mx, T, E, k, I, H, act8):
    """Up to and beyond 256 slots and 32 tokens, where the layer's plans change: bit for bit moe_mxfp4_forward,
    again and again from the workspace that the call before left."""
    g = gen(T + E + k)
    W = expert_weights(E, H, I, g)
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    l = torch.randn(T, E, generator=g).to(DEV)
    say("plans", T, E, k, I, act8)
    ids, gates = mx.moe_route_topk(l, k)
    want = mx.moe_mxfp4_forward(x, l, k, *W, act8=act8)
    ws = mx.workspace(T, H, I, E, k, x.device)
    for _ in range(3):
        assert torch.equal(mx.moe_mxfp4_forward_routed(x, ids, gates, *W, act8=act8, ws=ws), want)


def test_outputs_over_what_is_read(mx):
    """An output over an input that other workgroups still read is refused: the bias as well as the logits; the
    layer's ids, gates, weights and workspace as well as x."""
    T, E, k = 64, 64, 4
    l = torch.randn(T, E, generator=gen(51)).to(DEV)
    room = torch.zeros(T * k + E, device=DEV)
    bias = room[T * k - 8: T * k - 8 + E]
    with pytest.raises(ValueError, match="bias"):
        mx.moe_route_scored(l, k, bias=bias, gates=room[:T * k].view(T, k))
    with pytest.raises(ValueError, match="bias"):
        mx.moe_route_scored(l, k, bias=bias, ids=room[:T * k].view(torch.int32).view(T, k))
    want = mx.moe_route_scored(l, k, bias=room[T * k:].clone())
    got = mx.moe_route_scored(l, k, bias=room[T * k:], gates=room[:T * k].view(T, k))  # side by side
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    H, I, E = 1024, 256, 16
    W = expert_weights(E, H, I, gen(52))
    x = torch.randn(T, H, generator=gen(53)).bfloat16().to(DEV)
    ids, gates = mx.moe_route_topk(torch.randn(T, E, generator=gen(54)).to(DEV), k)
    room = torch.zeros(T * H * 2, dtype=torch.uint8, device=DEV)
    out = room.view(torch.bfloat16).view(T, H)
    over = room[: T * k * 4]
    for name, args in (("gates", (x, ids, over.view(torch.float32).view(T, k), *W)),
                       ("ids", (x, over.view(torch.int32).view(T, k), gates, *W))):
        with pytest.raises(ValueError, match=name):
            mx.moe_mxfp4_forward_routed(*args, out=out)
    ws = mx.workspace(T, H, I, E, k, x.device)
    with pytest.raises(ValueError, match="workspace"):
        mx.moe_mxfp4_forward_routed(x, ids, gates, *W, out=ws[: T * H * 2].view(torch.bfloat16).view(T, H), ws=ws)
    with pytest.raises(ValueError, match="W_down"):
        mx.moe_mxfp4_forward_routed(x, ids, gates, *W, out=W[2].view(-1)[: T * H * 2].view(torch.bfloat16).view(T, H))


def test_layers_on_streams_at_once(mx):
    """The layer, behind a routing and as a whole, on four streams at once, each with a workspace of its own: no
    launch has the device to itself, and none waits for workgroups of its own that cannot start."""
    H, I, E, k = 1024, 1024, 96, 8
    W = expert_weights(E, H, I, gen(81))
    runs = []
    for T, act8, shared in ((24, False, 0), (32, True, 0), (32, False, 0), (20, False, 1)):
        g = gen(T + act8 + shared)
        x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
        l = torch.randn(T, E - shared, generator=g).to(DEV)

        def run(x=x, l=l, act8=act8, shared=shared):
            whole = mx.moe_mxfp4_forward(x, l, k, *W, act8=act8, n_shared=shared)
            if shared:
                return [whole]
            return [mx.moe_mxfp4_forward_routed(x, *mx.moe_route_topk(l, k), *W, act8=act8), whole]

        runs.append(run)
    wants = [[t.clone() for t in r()] for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    spaces = [mx.workspace(32, H, I, E, k + 1, DEV, stream=s) for s in streams]
    torch.cuda.synchronize()
    for i in range(5):
        say("streams", i)
        got = [[] for _ in runs]
        for _ in range(4):
            for s, r, o in zip(streams, runs, got):
                with torch.cuda.stream(s):
                    o.append(r())
        torch.cuda.synchronize()
        for o, w in zip(got, wants):
            for ys in o:
                for y, want in zip(ys, w):
                    assert torch.equal(y, want), i
        for ws in spaces:
            assert not ws[:mx.MX_WORKSPACE_CTL_BYTES].any()  # no wait gave up, nothing is left marked


def test_captured_layers_have_workspaces_of_their_own(mx):
    """The layer behind a routing, and the layer itself, captured without a workspace: two graphs replayed at once on
    two streams, eager calls beside them, and a graph whose sibling is gone give the eager results."""
    H, I, E, k = 1024, 1024, 96, 8
    W = expert_weights(E, H, I, gen(71))
    runs = []
    for T, act8 in ((24, False), (32, True), (4, False)):
        g = gen(T)
        x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
        l = torch.randn(T, E, generator=g).to(DEV)

        def run(x=x, l=l, act8=act8):
            ids, gates = mx.moe_route_scored(l, k, "sigmoid", renormalize=True)
            return mx.moe_mxfp4_forward_routed(x, ids, gates, *W, act8=act8), mx.moe_mxfp4_forward(x, l, k, *W, act8=act8)

        runs.append(run)
    wants = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    held = len(mx._ws_cache)
    graphs, outs = [], []
    for r in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(r())
        graphs.append(graph)
    assert len(mx._ws_cache) == held  # nothing of a graph's memory outlives it
    streams = [torch.cuda.Stream() for _ in graphs]
    say("three graphs")
    for i in range(4):
        if i == 3:
            graphs[0].reset()
        for s, graph, o in list(zip(streams, graphs, outs))[int(i == 3):]:
            for t in o:
                t.fill_(math.nan)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graph.replay()
        eager = runs[i % 3]()
        torch.cuda.synchronize()
        for o, w in list(zip(outs, wants))[int(i == 3):] + [(eager, wants[i % 3])]:
            for a, b in zip(o, w):
                assert torch.equal(a, b), i
