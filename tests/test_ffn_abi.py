"""Refusals of the dense feed-forward operators: every call here fails a host-side check, so
nothing is enqueued and no pointer is followed."""
import ctypes
import os
import subprocess

import pytest
import torch

m = pytest.importorskip("mxfp4_weight_moe_amd")

NULL, SHAPE, ALIGN, WORKSPACE, ARG = -1, -2, -3, -4, -7
P = ctypes.c_void_p
A = P(1 << 20)
MIS = P((1 << 20) + 2)
NAN, INF = float("nan"), float("inf")
BIG = 1 << 40


def linear(x=A, w=A, s=A, bias=None, res=None, scale=1.0, act=0, y=A, z=None, T=64, K=256, N=64, ws=A, wb=BIG):
    return m.raw().mx_linear_fused(x, w, s, bias, res, scale, act, y, z, T, K, N, ws, wb, None)


def linear_bwd(dy=A, z=A, w=A, s=A, scale=1.0, act=2, dx=A, db=A, T=64, K=256, N=64, ws=A, wb=BIG):
    return m.raw().mx_linear_fused_backward(dy, z, w, s, scale, act, dx, db, T, K, N, ws, wb, None)


def gate_up(x=A, w=A, s=A, bias=None, act=2, h=A, z=None, T=64, H=256, I=64, ws=A, wb=BIG):
    return m.raw().mx_gate_up(x, w, s, bias, act, h, z, T, H, I, ws, wb, None)


def gate_up_bwd(dh=A, z=A, w=A, s=A, act=2, dx=A, db=A, T=64, H=256, I=64, ws=A, wb=BIG):
    return m.raw().mx_gate_up_backward(dh, z, w, s, act, dx, db, T, H, I, ws, wb, None)


def norm(x=A, b=A, wpost=A, gate=None, mode=0, scale=1.0, wpre=A, eps=1e-6, y=A, xn=A, T=4, H=64):
    return m.raw().mx_norm_residual(x, b, wpost, gate, mode, scale, wpre, eps, y, xn, T, H, None)


def norm_bwd(dy=A, dxn=A, y=A, b=A, wpost=A, gate=None, mode=0, scale=1.0, wpre=A, eps=1e-6, dx=A, db=A, dg=None,
             dwpost=A, dwpre=A, T=4, H=64, ws=A, wb=BIG):
    return m.raw().mx_norm_residual_backward(dy, dxn, y, b, wpost, gate, mode, scale, wpre, eps, dx, db, dg, dwpost,
                                             dwpre, T, H, ws, wb, None)


def block(x=A, wpre=A, wgu=A, sgu=A, bgu=None, act=2, wd=A, sd=A, bd=None, wpost=A, gate=None, mode=0, scale=1.0,
          eps=1e-6, y=A, T=4, H=64, I=64, ws=A, wb=BIG):
    return m.raw().mx_ffn_block(x, wpre, wgu, sgu, bgu, act, wd, sd, bd, wpost, gate, mode, scale, eps, y, T, H, I, ws,
                                wb, None)


@pytest.mark.parametrize("call,names", [(linear, "x w s y"), (gate_up, "x w s h"), (linear_bwd, "dy z w s"),
                                        (gate_up_bwd, "dh z w s"), (norm, "x y xn"), (norm_bwd, "dxn y dx"),
                                        (block, "x wgu sgu wd sd y")])
def test_null(call, names):
    for n in names.split():
        assert call(**{n: None}) == NULL, n


def test_null_combinations():
    assert linear_bwd(dx=None, db=None) == NULL
    assert gate_up_bwd(dx=None, db=None) == NULL
    assert norm(b=None, wpost=None, y=None, wpre=None, xn=None) == NULL
    assert norm_bwd(dy=None, wpre=None, dxn=None, dwpre=None) == NULL


@pytest.mark.parametrize("call,K,N", [(linear, "K", "N"), (linear_bwd, "K", "N"), (gate_up, "H", "I"),
                                      (gate_up_bwd, "H", "I"), (block, "H", "I")])
def test_sizes(call, K, N):
    for bad in (dict(T=0), dict(T=-1), dict(T=(1 << 24) + 1), {K: 0}, {K: 48}, {K: -32}, {K: (1 << 20) + 32}, {N: 0},
                {N: -1}, {N: (1 << 22) + 32}, {"T": 1 << 24, N: 1 << 18}, {"T": 1 << 24, K: 1 << 18},
                {N: 1 << 62}):
        assert call(**bad) == SHAPE, bad


def test_norm_sizes():
    for call in (norm, norm_bwd):
        for bad in (dict(T=0), dict(T=(1 << 24) + 1), dict(H=0), dict(H=12), dict(H=m.MX_NORM_MAX_H + 8)):
            assert call(**bad) == SHAPE, bad
    assert block(I=48) == SHAPE
    assert block(H=m.MX_NORM_MAX_H + 32) == SHAPE


def test_arguments():
    for call in (linear, linear_bwd, gate_up, gate_up_bwd, block):
        assert call(act=6) == ARG
        assert call(act=-1) == ARG
    for call in (linear, linear_bwd, norm, norm_bwd, block):
        for v in (NAN, INF, -INF):
            assert call(scale=v) == ARG
    for call in (norm, norm_bwd, block):
        for v in (0.0, -1e-6, NAN, INF):
            assert call(eps=v) == ARG
        assert call(mode=1) == ARG          # a mode without a gate
        assert call(gate=A) == ARG          # a gate without a mode
        assert call(gate=A, mode=4) == ARG
        assert call(gate=A, mode=-1) == ARG
    assert norm(b=None, y=None) == ARG                      # w_post without b
    assert norm(b=None, wpost=None) == ARG                  # y without b
    assert norm(wpre=None) == ARG                           # xn without w_pre
    assert norm_bwd(b=None, wpost=None, dwpost=None) == ARG  # db without b
    assert norm_bwd(wpost=None) == ARG                      # dw_post without w_post
    assert norm_bwd(dg=A) == ARG                            # dgate without a gate
    assert norm_bwd(wpre=None, dwpre=None) == ARG           # dxn without w_pre


@pytest.mark.parametrize("call,names", [
    (linear, "x w s bias res y z"), (linear_bwd, "dy z w dx db"), (gate_up, "x w s bias h z"),
    (gate_up_bwd, "dh z w dx db"), (norm, "x b wpost wpre y xn"),
    (norm_bwd, "dy dxn y b wpost wpre dx db dwpost dwpre"), (block, "x wpre wgu bgu wd bd wpost y")])
def test_alignment(call, names):
    for n in names.split():
        assert call(**{n: MIS}) == ALIGN, n
    if call in (norm, norm_bwd, block):
        assert call(gate=MIS, mode=2) == ALIGN
        assert call(gate=P((1 << 20) + 1), mode=1) == ALIGN


@pytest.mark.parametrize("call,K", [(linear, "K"), (gate_up, "H")])
def test_scale_alignment(call, K):
    """8 bytes where K % 256 == 0, 4 where K % 128 == 0, else any: what passes is refused for its workspace."""
    for k, off, want in ((8192, 4, ALIGN), (8192, 8, WORKSPACE), (8320, 2, ALIGN), (8320, 4, WORKSPACE),
                         (8224, 1, WORKSPACE)):
        assert call(**{K: k}, s=P((1 << 20) + off), ws=None) == want, (k, off)
    assert linear_bwd(s=P((1 << 20) + 1), K=2048, ws=None) == WORKSPACE


def test_workspaces():
    L = m.raw()
    need = L.mx_linear_fused_workspace_size(64, 8192, 64)
    assert need > 0 and linear(K=8192, wb=need - 1) == WORKSPACE
    assert linear(K=8192, ws=None, wb=need) == WORKSPACE
    assert linear(K=8192, ws=P((1 << 20) + 128), wb=need) == WORKSPACE
    for call, size in ((linear_bwd, L.mx_linear_fused_backward_workspace_size(64, 256, 64)),
                       (gate_up_bwd, L.mx_gate_up_backward_workspace_size(64, 256, 64)),
                       (norm_bwd, L.mx_norm_residual_backward_workspace_size(4, 64)),
                       (block, L.mx_ffn_block_workspace_size(4, 64, 64))):
        assert size > 0
        assert call(wb=size - 1) == WORKSPACE
        assert call(ws=None) == WORKSPACE
        assert call(ws=P((1 << 20) + 16)) == WORKSPACE
    need = L.mx_gate_up_workspace_size(64, 8192, 64)
    assert need > 0 and gate_up(H=8192, wb=need - 1) == WORKSPACE
    # a decode step streams the weights and needs none
    assert L.mx_linear_fused_workspace_size(4, 7168, 4096) == 0
    assert L.mx_gate_up_workspace_size(4, 7168, 2048) == 0
    # sizes that the call rejects
    assert L.mx_linear_fused_workspace_size(64, 48, 64) == 0
    assert L.mx_linear_fused_backward_workspace_size(0, 256, 64) == 0
    assert L.mx_gate_up_workspace_size(64, 256, 0) == 0
    assert L.mx_gate_up_backward_workspace_size(64, 256, 1 << 62) == 0
    assert L.mx_norm_residual_backward_workspace_size(4, 12) == 0
    assert L.mx_ffn_block_workspace_size(4, 64, 48) == 0


def test_status_of_a_bad_argument():
    assert m.status_string(ARG) != m.status_string(12345)
    with pytest.raises(ValueError):
        m._raise(ARG, "mx_norm_residual")


def test_binding_refuses_host_tensors_and_wrong_types():
    bf, u8 = torch.bfloat16, torch.uint8
    x, w, s = torch.zeros(4, 64, dtype=bf), torch.zeros(8, 32, dtype=u8), torch.zeros(8, 2, dtype=u8)
    with pytest.raises(ValueError, match="GPU"):
        m.mx_linear_fused(x, w, s)
    with pytest.raises(ValueError, match="GPU"):
        m.mx_gate_up(x, w, s)
    with pytest.raises(ValueError, match="GPU"):
        m.mx_norm_residual(x, w_pre=torch.ones(64, dtype=bf))
    with pytest.raises(ValueError, match="GPU"):
        m.mx_linear_fused_backward(x, w, s)
    with pytest.raises(ValueError, match="GPU"):
        m.mx_norm_residual_backward(x, None, None, b=x)
    with pytest.raises(TypeError):
        m.mx_linear_fused(x.float(), w, s)
    with pytest.raises(TypeError):
        m.mx_gate_up(None, w, s)
    with pytest.raises(TypeError):
        m.mx_norm_residual_backward(None, None, None)


def test_stream_grid_at_the_limits(tmp_path):
    """The streaming launch within the grid limits of HIP (fewer than 2^32 threads along x, 65535
    workgroups along y and z) wherever the calls' sizes are allowed, and over every token."""
    src = tmp_path / "grid.cpp"
    csrc = os.path.join(os.path.dirname(m.__file__), "csrc")
    src.write_text(f'#include "{csrc}/mx_grid.hpp"\nextern "C" void grid(int64_t T, int64_t rows, int64_t cols, uint32_t* o) '
                   "{ const auto g = mx::stream_grid(T, rows, cols); o[0] = g.items, o[1] = g.y, o[2] = g.z; }\n")
    so = tmp_path / "grid.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    grid = ctypes.CDLL(str(so)).grid
    grid.argtypes = [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_uint32)]
    out = (ctypes.c_uint32 * 3)()
    tokens = sorted({min(max(t + d, 1), 1 << 24) for e in range(25) for t in (1 << e, 3 << max(e - 1, 0)) for d in (-1, 0, 1)})
    for cols, most in ((16, 1 << 22), (8, 1 << 21)):  # a linear layer's rows, one half of gate_up's
        for rows in (1, cols - 1, cols, cols + 1, 1024, 2056, most - 1, most):
            for T in tokens:
                grid(T, rows, cols, out)
                x, y, z = out
                assert x == -(-rows // cols) and 1 <= y <= 65535 and 1 <= z <= 65535, (T, rows, cols)
                # more than one group of tokens has one wave a workgroup (K < 128), one group up to 8
                assert x * (64 if T > 32 else 512) < 1 << 32
                assert (y * z - y) * 32 < T <= y * z * 32 < 1 << 31, (T, y, z)
