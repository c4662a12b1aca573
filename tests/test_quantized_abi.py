"""Refusals of the microscaled operators and of routing by scores: every call here fails a host-side
check, so nothing is enqueued and no pointer is followed."""
import ctypes

import pytest
import torch

m = pytest.importorskip("mxfp4_weight_moe_amd")

NULL, SHAPE, ALIGN, WORKSPACE, ARG = -1, -2, -3, -4, -7
P = ctypes.c_void_p
A = P(1 << 20)
MIS = P((1 << 20) + 1)
NAN, INF = float("nan"), float("inf")
BIG = 1 << 40


def quantize(x=A, kind=0, fmt=0, codes=A, scales=A, values=None, rows=4, K=64):
    return m.raw().mx_quantize(x, kind, fmt, codes, scales, values, rows, K, None)


def norm(x=A, b=A, wpost=A, gate=None, mode=0, scale=1.0, wpre=A, eps=1e-6, y=A, xn=None, fmt=0, codes=A, scales=A,
         T=4, H=64):
    return m.raw().mx_norm_residual_quantize(x, b, wpost, gate, mode, scale, wpre, eps, y, xn, fmt, codes, scales, T, H, None)


def linear(a=A, sa=A, fmt=0, w=A, s=A, bias=None, res=None, scale=1.0, act=0, y=A, z=None, T=64, K=256, N=64, ws=A, wb=BIG):
    return m.raw().mx_linear_quantized(a, sa, fmt, w, s, bias, res, scale, act, y, z, T, K, N, ws, wb, None)


def gate_up(a=A, sa=A, fmt=0, w=A, s=A, bias=None, act=2, h=A, hfmt=0, hc=None, hs=None, z=None, T=64, H=256, I=64, ws=A,
            wb=BIG):
    return m.raw().mx_gate_up_quantized(a, sa, fmt, w, s, bias, act, h, hfmt, hc, hs, z, T, H, I, ws, wb, None)


def gate_up_out(hc=A, hs=A, **kw):
    return gate_up(h=None, hc=hc, hs=hs, **kw)


def route(l=A, kind=1, bias=None, score=0, ng=1, tg=1, gs=0, renorm=0, scale=1.0, ids=A, gates=A, T=4, E=16, k=4):
    return m.raw().moe_route_scored(l, kind, bias, score, ng, tg, gs, renorm, scale, ids, gates, T, E, k, None)


def route_bwd(dg=A, l=A, kind=1, ids=A, score=0, renorm=0, scale=1.0, dl=A, T=4, E=16, k=4):
    return m.raw().moe_route_scored_backward(dg, l, kind, ids, score, renorm, scale, dl, T, E, k, None)


def routed(x=A, ids=A, gates=A, k=4, wgu=A, sgu=A, wd=A, sd=A, a8=0, y=A, T=4, H=1024, I=256, E=16, ws=A, wb=BIG):
    return m.raw().moe_mxfp4_forward_routed(x, ids, gates, k, wgu, sgu, wd, sd, a8, y, T, H, I, E, ws, wb, None)


@pytest.mark.parametrize("call,names", [
    (quantize, "x codes scales"), (norm, "x wpre y codes scales"), (linear, "a sa w s y"), (gate_up, "a sa w s h"),
    (gate_up_out, "a sa w s hc hs"), (route, "l ids gates"), (route_bwd, "dg l ids dl"),
    (routed, "x ids gates wgu sgu wd sd y")])
def test_null(call, names):
    for n in names.split():
        assert call(**{n: None}) == NULL, n


@pytest.mark.parametrize("call,K,N", [(linear, "K", "N"), (gate_up, "H", "I"), (gate_up_out, "H", "I")])
def test_product_sizes(call, K, N):
    for bad in (dict(T=0), dict(T=-1), dict(T=(1 << 24) + 1), {K: 0}, {K: 48}, {K: -32}, {K: (1 << 20) + 32}, {N: 0},
                {N: -1}, {N: (1 << 22) + 32}, {"T": 1 << 24, N: 1 << 18}, {"T": 1 << 24, K: 1 << 18}, {N: 1 << 62}):
        assert call(**bad) == SHAPE, bad
    assert gate_up_out(I=48) == SHAPE
    assert gate_up(I=48, ws=None, T=100, H=8224) == WORKSPACE  # bf16 takes any I


def test_other_sizes():
    for bad in (dict(rows=0), dict(rows=-1), dict(K=0), dict(K=48), dict(K=-32), dict(rows=1 << 40), dict(rows=1 << 62, K=1 << 32)):
        assert quantize(**bad) == SHAPE, bad
    for bad in (dict(T=0), dict(T=(1 << 24) + 1), dict(H=0), dict(H=40), dict(H=m.MX_NORM_MAX_H + 32)):
        assert norm(**bad) == SHAPE, bad
    for call in (route, route_bwd):
        for bad in (dict(T=0), dict(T=(1 << 24) + 1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(k=33, E=64),
                    dict(E=-1), dict(k=-1)):
            assert call(**bad) == SHAPE, bad
    for bad in (dict(ng=0), dict(ng=3), dict(ng=4, tg=5), dict(ng=4, tg=0), dict(ng=8, tg=1, k=3), dict(ng=128, tg=128, E=128),
                dict(ng=-1)):
        assert route(**bad) == SHAPE, bad
    for bad in (dict(T=257), dict(T=0), dict(k=17), dict(H=512), dict(I=128)):
        assert routed(**bad) == SHAPE, bad


def test_arguments():
    for call in (quantize, norm, linear, gate_up):
        for f in (-1, 2):
            assert call(fmt=f) == ARG
    assert quantize(kind=2) == ARG and quantize(kind=-1) == ARG
    for call in (linear, gate_up, gate_up_out):
        assert call(act=6) == ARG and call(act=-1) == ARG
    assert gate_up(hc=A) == ARG and gate_up(hs=A) == ARG  # h in both forms
    assert gate_up_out(hfmt=2) == ARG and gate_up_out(hfmt=-1) == ARG
    for v in (NAN, INF, -INF):
        for call in (linear, norm, route, route_bwd):
            assert call(scale=v) == ARG
    for v in (0.0, -1e-6, NAN, INF):
        assert norm(eps=v) == ARG
    assert norm(mode=1) == ARG and norm(gate=A) == ARG and norm(gate=A, mode=4) == ARG
    assert norm(b=None, y=None) == ARG                # w_post without b
    assert norm(b=None, wpost=None) == ARG            # y without b
    for call in (route, route_bwd):
        assert call(kind=2) == ARG and call(kind=-1) == ARG and call(score=2) == ARG and call(score=-1) == ARG
    assert route(gs=2) == ARG and route(gs=-1) == ARG


@pytest.mark.parametrize("call,names", [
    (quantize, "x codes values"), (norm, "x b wpost wpre y xn codes"), (linear, "a w bias res y z"),
    (gate_up, "a w bias h z"), (gate_up_out, "a w hc bias z"), (route, "l bias ids gates"), (route_bwd, "dg l ids dl"),
    (routed, "x ids gates wgu sgu wd sd y")])
def test_alignment(call, names):
    for n in names.split():
        assert call(**{n: MIS}) == ALIGN, n


def test_type_and_scale_alignment():
    two = P((1 << 20) + 2)
    assert route(l=two) == ALIGN and route_bwd(l=two) == ALIGN and route_bwd(dl=two) == ALIGN
    # scales: 16 bytes where rows of them are multiples of 16, else any address
    for call, K in ((linear, "K"), (gate_up, "H")):
        for n in ("sa", "s"):
            assert call(**{n: P((1 << 20) + 8), K: 8192}) == ALIGN
            assert call(**{n: MIS, K: 8224}, T=100, ws=None) == WORKSPACE
    assert norm(gate=P((1 << 20) + 8), mode=2) == ALIGN and norm(gate=MIS, mode=1) == ALIGN


def test_workspaces():
    L = m.raw()
    need = L.mx_linear_quantized_workspace_size(100, 8192, 64)
    assert need > 0
    for bad in (dict(wb=need - 1), dict(ws=None), dict(ws=P((1 << 20) + 128))):
        assert linear(T=100, K=8192, **bad) == WORKSPACE
    need = L.mx_gate_up_quantized_workspace_size(4, 256, 64)
    assert need > 0 and gate_up_out(T=4, wb=need - 1) == WORKSPACE and gate_up_out(T=4, ws=None) == WORKSPACE
    assert L.mx_linear_quantized_workspace_size(4, 7168, 4096) == 0
    assert L.mx_linear_quantized_workspace_size(64, 48, 64) == 0
    assert L.mx_gate_up_quantized_workspace_size(64, 256, 0) == 0
    assert L.mx_gate_up_quantized_workspace_size(0, 256, 64) == 0
    assert routed(ws=None) == WORKSPACE and routed(wb=16) == WORKSPACE


def test_binding_refuses_host_tensors_and_wrong_types():
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    x, c, s = torch.zeros(4, 64, dtype=bf), torch.zeros(4, 64, dtype=u8), torch.zeros(4, 2, dtype=u8)
    w, ws = torch.zeros(8, 32, dtype=u8), torch.zeros(8, 2, dtype=u8)
    l, ids, g = torch.zeros(4, 16), torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2)
    for call in (lambda: m.mx_quantize(x), lambda: m.mx_norm_residual_quantize(x, w_pre=x[0]),
                 lambda: m.mx_linear_quantized(c, s, w, ws), lambda: m.mx_gate_up_quantized(c, s, w, ws),
                 lambda: m.moe_route_scored(l, 2), lambda: m.moe_route_scored_backward(g, l, ids),
                 lambda: m.moe_mxfp4_forward_routed(x, ids, g, w[None], ws[None], w[None], ws[None])):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: m.mx_quantize(x.half()), lambda: m.mx_quantize(None), lambda: m.mx_norm_residual_quantize(x.float()),
                 lambda: m.mx_linear_quantized(c.int(), s, w, ws), lambda: m.moe_route_scored(l.half(), 2),
                 lambda: m.moe_route_scored_backward(g, l.double(), ids)):
        with pytest.raises((TypeError, ValueError)):
            call()
