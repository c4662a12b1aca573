"""The dense feed-forward operators around MXFP4 weights, as measured cases.

Three operators, forward and backward:
  linear   y = residual + scale * act(x W^T + bias)      W in MXFP4, frozen
  gate_up  h = act(x Wg^T + bg) * (x Wu^T + bu)          both projections in MXFP4, frozen
  norm     y = x + scale * gate * rms_norm(b) and xn = rms_norm(y): the norms after and before a block

Where `own` is false, run() computes the plain form in 32 bits with elementary torch
operations, rounded once at the end; where it is true, it calls this library.  exact() is
the definition in 64 bits, written apart from the plain form.

Sizes: hidden size 7168 and intermediate size 2048 with steps of 1 to 128 tokens are this
repository's workloads; 4096 and 8192 tokens are prompts and training batches of generic length.
"""
import math

import torch

own = False

EPS = 1e-6
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid")
# Work of one multiply-add against one byte, for bounding what draw() may cost.
MOST_PRODUCT = 4096 * 7168 * 4096


# ------------------------------------------------------------------ cases

def _linear(name, T, K, N, act="none", bias=False, residual=False, scale=1.0, save_z=False):
    return dict(name=name, op="linear", T=T, K=K, N=N, act=act, bias=bias, residual=residual, scale=scale, save_z=save_z)


def _linear_bwd(name, T, K, N, act="none", scale=1.0, bias=True):
    return dict(name=name, op="linear_bwd", T=T, K=K, N=N, act=act, scale=scale, bias=bias)


def _gate_up(name, T, H, I, act="silu", bias=False, save_z=False):
    return dict(name=name, op="gate_up", T=T, H=H, I=I, act=act, bias=bias, save_z=save_z)


def _gate_up_bwd(name, T, H, I, act="silu", bias=False):
    return dict(name=name, op="gate_up_bwd", T=T, H=H, I=I, act=act, bias=bias)


def _norm(name, T, H, block=True, post=True, gate="none", scale=1.0, pre=True):
    return dict(name=name, op="norm", T=T, H=H, block=block, post=post, gate=gate, scale=scale, pre=pre)


def _norm_bwd(name, T, H, block=True, post=True, gate="none", scale=1.0, pre=True):
    return dict(name=name, op="norm_bwd", T=T, H=H, block=block, post=post, gate=gate, scale=scale, pre=pre)


def listed():
    return [
        # one decoded token through a small square projection with bias and activation: latency
        _linear("linear_t1", 1, 2048, 2048, act="gelu_tanh", bias=True),
        # a verify step of 4 positions: the projection back into the residual stream
        _linear("linear_t4_residual", 4, 7168, 4096, residual=True),
        # a ragged decode batch through the down projection of one dense block
        _linear("linear_t77_down", 77, 2048, 7168, bias=True, residual=True, scale=0.5),
        # a prompt of 4096 tokens, every part of the epilogue
        _linear("linear_t4096", 4096, 7168, 4096, act="gelu", bias=True, residual=True),
        # gradients of that projection's input and bias in a training step with frozen weights
        _linear_bwd("linear_bwd_t2048", 2048, 7168, 4096, act="gelu", bias=True),
        # a decode step of 8 requests through the gated block
        _gate_up("gate_up_t8", 8, 7168, 2048),
        # 32 requests x 4 verify positions
        _gate_up("gate_up_t128", 128, 7168, 2048),
        # the training forward of 4096 tokens, which also keeps both pre-activations
        _gate_up("gate_up_train_t4096", 4096, 7168, 2048, save_z=True),
        # its backward
        _gate_up_bwd("gate_up_bwd_t4096", 4096, 7168, 2048, bias=True),
        # the norms between two blocks in a decode step of 32 tokens
        _norm("norm_t32", 32, 7168, gate="token"),
        # the same for two prompts of 4096 tokens, with a scale per channel
        _norm("norm_t8192", 8192, 7168, gate="channel", scale=0.5),
        # their backward in training, with all parameter gradients
        _norm_bwd("norm_bwd_t4096", 4096, 7168, gate="channel", scale=0.5),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear_bwd", "gate_up", "gate_up_bwd", "norm", "norm_bwd"))
    act = rng.choice(ACTS)
    if op.startswith("norm"):
        block = rng.random() < 0.8
        return dict(op=op, T=_spread(rng, 1, 4096), H=8 * _spread(rng, 8, 896), block=block,
                    post=block and rng.random() < 0.7,
                    gate=rng.choice(("none", "token", "channel", "full")) if block else "none",
                    scale=rng.choice((1.0, 0.5, 1.4142135)) if block else 1.0, pre=not block or rng.random() < 0.7)
    K = 32 * _spread(rng, 8, 256)
    N = _spread(rng, 64, 4096)
    T = min(_spread(rng, 1, 4096), MOST_PRODUCT // (K * N))
    if op == "linear":
        return dict(op=op, T=T, K=K, N=N, act=act, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    scale=rng.choice((1.0, 0.25)), save_z=rng.random() < 0.3)
    if op == "linear_bwd":
        return dict(op=op, T=T, K=K, N=N, act=act, scale=rng.choice((1.0, 0.25)), bias=rng.random() < 0.5)
    I = max(32, N // 2)
    if op == "gate_up":
        return dict(op=op, T=T, H=K, I=I, act=act, bias=rng.random() < 0.5, save_z=rng.random() < 0.5)
    return dict(op=op, T=T, H=K, I=I, act=act, bias=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def prepare(case, seed):
    """Inputs of one pass.  Activations are N(0, 1) values in bf16; codes are uniform over all
    16; block scales are 2^-12 .. 2^-6, which puts the pre-activations at order one, where the
    activations curve."""
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(torch.bfloat16)

    def weights(rows, K):
        w = torch.randint(0, 256, (rows, K // 2), generator=g, device=dev, dtype=torch.uint8)
        s = torch.randint(115, 122, (rows, K // 32), generator=g, device=dev, dtype=torch.int16).to(torch.uint8)
        return w, s

    op, st = case["op"], dict(case)
    if op in ("linear", "linear_bwd"):
        T, K, N = case["T"], case["K"], case["N"]
        st["w"], st["s"] = weights(N, K)
        if op == "linear":
            st["x"] = normal(T, K)
            st["b"] = normal(N, std=0.5) if case["bias"] else None
            st["r"] = normal(T, N) if case["residual"] else None
        else:
            st["dy"] = normal(T, N)
            st["z"] = normal(T, N, std=1.5) if case["act"] != "none" else None
    elif op in ("gate_up", "gate_up_bwd"):
        T, H, I = case["T"], case["H"], case["I"]
        st["w"], st["s"] = weights(2 * I, H)
        if op == "gate_up":
            st["x"] = normal(T, H)
            st["b"] = normal(2 * I, std=0.5) if case["bias"] else None
        else:
            st["dh"] = normal(T, I)
            st["z"] = normal(T, 2 * I, std=1.5)
    else:
        T, H = case["T"], case["H"]
        st["x"] = normal(T, H, std=2.0)
        st["blk"] = normal(T, H, std=0.7) if case["block"] else None
        st["wpost"] = normal(H, std=0.1, mean=1.0) if case["post"] else None
        st["wpre"] = normal(H, std=0.1, mean=1.0) if case["pre"] else None
        shape = {"none": None, "token": (T, 1), "channel": (H,), "full": (T, H)}[case["gate"]]
        st["g"] = normal(*shape, std=0.3, mean=0.5) if shape else None
        if op == "norm_bwd":
            st["dy"] = normal(T, H)
            st["dxn"] = normal(T, H) if case["pre"] else None
    return st


# ------------------------------------------------------------------ plain form (32 bits)

def _dequantize(w, s):
    """fp32 [rows, K] of MXFP4 codes and scales."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         dtype=torch.float32, device=w.device)
    rows, half = w.shape
    v = torch.stack((table[(w & 15).int()], table[(w >> 4).int()]), dim=-1).reshape(rows, half // 16, 32)
    scale = (s.int() << 23).view(torch.float32)
    return (v * scale[..., None]).reshape(rows, 2 * half)


def _act(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if kind == "sigmoid":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 - p)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.7071067811865476)) + z * 0.3989422804014327 * torch.exp(-0.5 * z * z)
    if kind == "gelu_tanh":
        t = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.7978845608028654 * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _bf(v):
    return v.to(torch.bfloat16)


def _plain_linear(st):
    z = st["x"].float() @ _dequantize(st["w"], st["s"]).t()
    if st["b"] is not None:
        z = z + st["b"].float()
    y = st["scale"] * _act(z, st["act"])
    if st["r"] is not None:
        y = st["r"].float() + y
    return (_bf(y), _bf(z)) if st["save_z"] else _bf(y)


def _plain_linear_bwd(st):
    dz = st["scale"] * st["dy"].float()
    if st["z"] is not None:
        dz = dz * _act_slope(st["z"].float(), st["act"])
    dx = _bf(dz @ _dequantize(st["w"], st["s"]))
    return (dx, dz.sum(0)) if st["bias"] else (dx,)


def _plain_gate_up(st):
    I = st["I"]
    z = st["x"].float() @ _dequantize(st["w"], st["s"]).t()
    if st["b"] is not None:
        z = z + st["b"].float()
    h = _act(z[:, :I], st["act"]) * z[:, I:]
    return (_bf(h), _bf(z)) if st["save_z"] else _bf(h)


def _plain_gate_up_bwd(st):
    I = st["I"]
    z, dh = st["z"].float(), st["dh"].float()
    dz = torch.cat((dh * z[:, I:] * _act_slope(z[:, :I], st["act"]), dh * _act(z[:, :I], st["act"])), dim=1)
    dx = _bf(dz @ _dequantize(st["w"], st["s"]))
    return (dx, dz.sum(0)) if st["bias"] else (dx,)


def _plain_norm(st):
    y = x = st["x"]
    if st["blk"] is not None:
        n = st["blk"].float()
        if st["wpost"] is not None:
            n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + EPS) * st["wpost"].float()
        if st["g"] is not None:
            n = n * st["g"].float()
        y = _bf(x.float() + st["scale"] * n)
    if st["wpre"] is None:
        return (y,)
    f = y.float()
    xn = _bf(f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * st["wpre"].float())
    return (y, xn) if st["blk"] is not None else (xn,)


def _plain_norm_bwd(st):
    """In the backward pass st["x"] is y, what the forward wrote into the residual stream."""
    H, out = st["H"], {}
    d = st["dy"].float()
    if st["wpre"] is not None:
        f, dxn = st["x"].float(), st["dxn"].float()
        r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
        t = dxn * st["wpre"].float()
        out["dw_pre"] = (dxn * f * r).sum(0)
        d = d + r * (t - f * r * r * (t * f).sum(-1, keepdim=True) / H)
    out["dx"] = _bf(d)
    if st["blk"] is None:
        return out
    b, e = st["blk"].float(), st["scale"] * d
    n = b
    if st["wpost"] is not None:
        q = torch.rsqrt((b * b).mean(-1, keepdim=True) + EPS)
        n = b * q * st["wpost"].float()
    if st["g"] is not None:
        kind = st["gate"]
        dg = e * n
        out["dgate"] = dg.sum(0) if kind == "channel" else dg.sum(1, keepdim=True) if kind == "token" else _bf(dg)
        e = e * st["g"].float()
    if st["wpost"] is not None:
        out["dw_post"] = (e * b * q).sum(0)
        t = e * st["wpost"].float()
        e = q * (t - b * q * q * (t * b).sum(-1, keepdim=True) / H)
    out["db"] = _bf(e)
    return out


PLAIN = dict(linear=_plain_linear, linear_bwd=_plain_linear_bwd, gate_up=_plain_gate_up, gate_up_bwd=_plain_gate_up_bwd,
             norm=_plain_norm, norm_bwd=_plain_norm_bwd)


# ------------------------------------------------------------------ this library's calls

def _own(st):
    import mxfp4_weight_moe_amd as mx

    op = st["op"]
    if op == "linear":
        return mx.mx_linear_fused(st["x"], st["w"], st["s"], bias=st["b"], residual=st["r"], scale=st["scale"],
                                  act=st["act"], save_z=st["save_z"])
    if op == "linear_bwd":
        dx, db = mx.mx_linear_fused_backward(st["dy"], st["w"], st["s"], z=st["z"], scale=st["scale"], act=st["act"],
                                             need_dbias=st["bias"])
        return (dx, db) if st["bias"] else (dx,)
    if op == "gate_up":
        return mx.mx_gate_up(st["x"], st["w"], st["s"], bias=st["b"], act=st["act"], save_z=st["save_z"])
    if op == "gate_up_bwd":
        dx, db = mx.mx_gate_up_backward(st["dh"], st["z"], st["w"], st["s"], act=st["act"], need_dbias=st["bias"])
        return (dx, db) if st["bias"] else (dx,)
    if op == "norm":
        y, xn = mx.mx_norm_residual(st["x"], st["blk"], w_post=st["wpost"], gate=st["g"], scale=st["scale"],
                                    w_pre=st["wpre"], eps=EPS)
        return (xn,) if st["blk"] is None else (y,) if xn is None else (y, xn)
    d = mx.mx_norm_residual_backward(st["dy"], st["dxn"], st["x"], st["blk"], w_post=st["wpost"], gate=st["g"],
                                     scale=st["scale"], w_pre=st["wpre"], eps=EPS)
    return {k: v for k, v in d.items() if v is not None}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, T = case["op"], case["T"]
    if op.startswith("norm"):
        H = case["H"]
        n = T * H
        small = H * (int(case["post"]) + int(case["pre"]))
        gate = {"none": 0, "token": T, "channel": H, "full": n}[case["gate"]]
        if op == "norm":
            arrays = 1 + 2 * int(case["block"]) + int(case["pre"])
            return {"bytes": 2 * (arrays * n + small + gate), "flops": n * (4 * int(case["post"]) + 4 * int(case["pre"]) + 3)}
        # dy, dx, and per norm: dxn and y; b and db (b once for both of its uses)
        arrays = 2 + 2 * int(case["pre"]) + 2 * int(case["block"])
        return {"bytes": 2 * (arrays * n + small + gate) + 4 * small + (2 if case["gate"] == "full" else 4) * gate,
                "flops": n * (12 * int(case["post"]) + 12 * int(case["pre"]) + 6)}
    if op.startswith("linear"):
        K, rows, out = case["K"], case["N"], case["N"]
    else:
        K, rows, out = case["H"], 2 * case["I"], case["I"]
    weights = rows * (K // 2 + K // 32)
    product = 2 * T * K * rows
    bias = rows * (4 if op.endswith("bwd") else 2) * int(case["bias"])
    if op.endswith("bwd"):
        kept = rows if op == "gate_up_bwd" or case["act"] != "none" else 0
        return {"bytes": weights + bias + 2 * T * (out + kept + K), "flops": product}
    extra = out * int(case.get("residual", False)) + rows * int(case["save_z"])
    return {"bytes": weights + bias + 2 * T * (K + out + extra), "flops": product}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_weights(w, s):
    """Per code: sign, two exponent bits, one mantissa bit; the block's scale is 2^(byte - 127)."""
    c = torch.stack((w.long() % 16, w.long() // 16), dim=2).flatten(1)
    e, m = (c // 2) % 4, (c % 2).double()
    size = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.pow(torch.full_like(m, 2.0), (e - 1).double()))
    value = torch.where(c >= 8, -size, size)
    power = torch.pow(torch.full(s.shape, 2.0, dtype=torch.float64, device=s.device), s.double() - 127)
    return value * power.repeat_interleave(32, dim=1)


def _exact_act(z, kind):
    """(act(z), act'(z))."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros_like(z))
    if kind in ("silu", "sigmoid"):
        p = torch.sigmoid(z)
        return (p, p * (1 - p)) if kind == "sigmoid" else (z * p, p + z * p * (1 - p))
    if kind == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    # (1 + tanh v) / 2 is the logistic function of 2 v
    p = torch.sigmoid(2 * a * (z + 0.044715 * z ** 3))
    return z * p, p + z * p * (1 - p) * 2 * a * (1 + 0.134145 * z ** 2)


def _exact_norm_grad(d, v, w):
    """Gradient of w * v / sqrt(mean v^2 + eps) into v, and the terms of the gradient into w."""
    rms = (v.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    unit = v / rms
    dw = d * unit
    return (d * w - unit * (dw * w).mean(1, keepdim=True)) / rms, dw


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    q = {k: v.double() if isinstance(v, torch.Tensor) and v.dtype == torch.bfloat16 else v for k, v in st.items()}
    if not op.startswith("norm"):
        W = _exact_weights(q["w"], q["s"])
        if op in ("linear", "gate_up"):
            z = torch.matmul(q["x"], W.T)
            if q["b"] is not None:
                z = z + q["b"]
            if op == "linear":
                y = q["scale"] * _exact_act(z, q["act"])[0] + (0 if q["r"] is None else q["r"])
            else:
                gate, up = z.chunk(2, dim=1)
                y = up * _exact_act(gate, q["act"])[0]
            return (y, z) if q["save_z"] else y
        if op == "linear_bwd":
            dz = q["dy"] * q["scale"] * (1 if q["z"] is None else _exact_act(q["z"], q["act"])[1])
        else:
            gate, up = q["z"].chunk(2, dim=1)
            a, slope = _exact_act(gate, q["act"])
            dz = torch.hstack((q["dh"] * up * slope, q["dh"] * a))
        dx = torch.matmul(dz, W)
        return (dx, dz.sum(dim=0)) if case["bias"] else (dx,)

    unit = lambda v: v / (v.pow(2).mean(1, keepdim=True) + EPS).sqrt()  # noqa: E731
    if op == "norm":
        y = q["x"]
        if q["blk"] is not None:
            n = q["blk"] if q["wpost"] is None else unit(q["blk"]) * q["wpost"]
            y = y + q["scale"] * (n if q["g"] is None else q["g"] * n)
        if q["wpre"] is None:
            return (y,)
        if q["blk"] is None:
            return (unit(y) * q["wpre"],)
        # the second norm's input is y as it is stored
        return (y, unit(y.to(torch.bfloat16).double()) * q["wpre"])
    out = {}
    d = q["dy"]
    if q["wpre"] is not None:
        more, dw = _exact_norm_grad(q["dxn"], q["x"], q["wpre"])
        d = d + more
        out["dw_pre"] = dw.sum(dim=0)
    out["dx"] = d
    if q["blk"] is None:
        return out
    d = d * q["scale"]
    n = q["blk"] if q["wpost"] is None else unit(q["blk"]) * q["wpost"]
    if q["g"] is not None:
        dg = d * n
        out["dgate"] = {"channel": lambda: dg.sum(dim=0), "token": lambda: dg.sum(dim=1, keepdim=True), "full": lambda: dg}[case["gate"]]()
        d = d * q["g"]
    if q["wpost"] is not None:
        d, dw = _exact_norm_grad(d, q["blk"], q["wpost"])
        out["dw_post"] = dw.sum(dim=0)
    out["db"] = d
    return out
