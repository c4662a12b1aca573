"""Operators of microscaled activations and of expert routing, as measured cases.

  route      ids, gates: softmax or sigmoid scores, a bias for balance, groups, top-k, renormalised gates
  route_bwd  its gradient into the router's logits
  quantize   rows of bf16 or fp32 to MXFP8 or MXFP4
  norm_q     the norms and residual around a block, the next block's input in MXFP8 or MXFP4
  linear_q   y = residual + scale * act(x W^T + bias), x in MXFP8 or MXFP4, W in MXFP4
  gate_up_q  h = act(x Wg^T + bg) * (x Wu^T + bu), x as above, h in bf16, MXFP8 or MXFP4

Where `own` is false, run() computes the plain form in 32 bits (the router's order and its gradient in 64) with
elementary torch operations, rounded once at the end; where it is true, it calls this library.
exact() is the definition in 64 bits, written apart from the plain form.

MXFP8 comes back as its E4M3 elements and E8M0 scales in torch's types of that name.  MXFP4, which
packs two values in a byte, comes back as bf16 values.

Sizes: hidden size 7168, intermediate size 2048, 256 and 384 experts of which 8 are chosen and steps
of 1 to 128 tokens are this repository's workloads; 300, 4096, 8192 and 16384 tokens are prompts and
training batches of generic length.
"""
import math

import torch

own = False

EPS = 1e-6
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid")
FORMATS = ("mxfp8", "mxfp4")
# Work of one multiply-add, for bounding what draw() may cost.
MOST_PRODUCT = 4096 * 7168 * 4096


# ------------------------------------------------------------------ cases

def _route(name, T, E, k, score, bias=False, groups=1, kept=1, by="top2", renorm=False, scale=1.0, dtype="fp32"):
    return dict(name=name, op="route", T=T, E=E, k=k, score=score, bias=bias, groups=groups, kept=kept, by=by,
                renorm=renorm, scale=scale, dtype=dtype)


def _route_bwd(name, T, E, k, score, renorm=False, scale=1.0, dtype="fp32"):
    return dict(name=name, op="route_bwd", T=T, E=E, k=k, score=score, renorm=renorm, scale=scale, dtype=dtype)


def _quantize(name, rows, K, fmt, dtype="bf16"):
    return dict(name=name, op="quantize", rows=rows, K=K, fmt=fmt, dtype=dtype)


def _norm_q(name, T, H, fmt, block=True, post=True, gate="none", scale=1.0, keep=False):
    return dict(name=name, op="norm_q", T=T, H=H, fmt=fmt, block=block, post=post, gate=gate, scale=scale, keep=keep)


def _linear_q(name, T, K, N, fmt, act="none", bias=False, residual=False, scale=1.0, save_z=False):
    return dict(name=name, op="linear_q", T=T, K=K, N=N, fmt=fmt, act=act, bias=bias, residual=residual, scale=scale,
                save_z=save_z)


def _gate_up_q(name, T, H, I, fmt, out, act="silu", bias=False, save_z=False):
    return dict(name=name, op="gate_up_q", T=T, H=H, I=I, fmt=fmt, out=out, act=act, bias=bias, save_z=save_z)


def listed():
    return [
        # a decode batch of 32 tokens, sigmoid scores with a balance bias, 4 of 8 groups: latency
        _route("route_t32_groups", 32, 256, 8, "sigmoid", bias=True, groups=8, kept=4, renorm=True, scale=2.5),
        # a training batch over 384 experts, softmax scores
        _route("route_t16384", 16384, 384, 8, "softmax"),
        # the gradient of that routing: every expert's logit has one, through the softmax
        _route_bwd("route_bwd_t8192", 8192, 256, 8, "softmax"),
        # the activations of a verify step of 4 positions, ahead of a product: latency
        _quantize("quantize_t4", 4, 7168, "mxfp8"),
        # the gate_up weights of four experts, from bf16 into this library's format
        _quantize("quantize_weights", 16384, 7168, "mxfp4"),
        # the norms between two blocks in a decode step, the next block's input in 8 bits
        _norm_q("norm_q_t16", 16, 7168, "mxfp8"),
        # the same for two prompts of 4096 tokens, with a scale per channel; the router reads the
        # norm's output before it is quantised
        _norm_q("norm_q_t8192", 8192, 7168, "mxfp8", gate="channel", scale=0.5, keep=True),
        # one decoded token through a projection with bias and activation
        _linear_q("linear_q_t1", 1, 7168, 2048, "mxfp8", act="gelu_tanh", bias=True),
        # a ragged prompt of 300 tokens through a down projection, back into the residual stream
        _linear_q("linear_q_t300_down", 300, 2048, 7168, "mxfp8", residual=True),
        # a prompt of 4096 tokens, both sides in 4 bits, the whole epilogue
        _linear_q("linear_q_t4096", 4096, 7168, 4096, "mxfp4", act="gelu", bias=True, residual=True),
        # a decode step of 24 tokens through the gated block, ready for the down projection
        _gate_up_q("gate_up_q_t24", 24, 7168, 2048, "mxfp8", "mxfp8"),
        # the same for a prompt of 4096 tokens
        _gate_up_q("gate_up_q_t4096", 4096, 7168, 2048, "mxfp8", "mxfp8"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route", "route_bwd", "quantize", "norm_q", "linear_q", "linear_q", "gate_up_q", "gate_up_q"))
    fmt, act, dtype = rng.choice(FORMATS), rng.choice(ACTS), rng.choice(("fp32", "bf16"))
    if op.startswith("route"):
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * _spread(rng, 8 if groups == 1 else 4, 512 // groups)
        kept = rng.randint(1, groups)
        k = min(_spread(rng, 1, 16), E // groups * kept)
        T, score = _spread(rng, 1, 16384), rng.choice(("softmax", "sigmoid"))
        renorm, scale = rng.random() < 0.5, rng.choice((1.0, 2.5))
        if op == "route_bwd":
            # one renormalised gate is 1 whatever its logit: two at least
            return dict(op=op, T=min(T, 8192 * 256 // E), E=E, k=max(2, k), score=score, renorm=renorm, scale=scale, dtype=dtype)
        return dict(op=op, T=min(T, 16384 * 384 // E), E=E, k=k, score=score, bias=rng.random() < 0.5, groups=groups,
                    kept=kept, by=rng.choice(("top2", "max")), renorm=renorm, scale=scale, dtype=dtype)
    if op == "quantize":
        return dict(op=op, rows=_spread(rng, 1, 8192), K=32 * _spread(rng, 1, 224), fmt=fmt, dtype=dtype)
    if op == "norm_q":
        block = rng.random() < 0.8
        return dict(op=op, T=_spread(rng, 1, 4096), H=32 * _spread(rng, 2, 224), fmt="mxfp8", block=block,
                    post=block and rng.random() < 0.7,
                    gate=rng.choice(("none", "token", "channel", "full")) if block else "none",
                    scale=rng.choice((1.0, 0.5, 1.4142135)) if block else 1.0, keep=rng.random() < 0.5)
    K = 32 * _spread(rng, 8, 256)
    N = _spread(rng, 64, 4096)
    T = min(_spread(rng, 1, 4096), MOST_PRODUCT // (K * N))
    if op == "linear_q":
        return dict(op=op, T=T, K=K, N=N, fmt=fmt, act=act, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    scale=rng.choice((1.0, 0.25)), save_z=rng.random() < 0.3)
    out = rng.choice(("bf16", "mxfp8", "mxfp8"))
    I = max(32, N // 2)
    return dict(op=op, T=T, H=K, I=I if out == "bf16" else I // 32 * 32, fmt=fmt, out=out, act=act, bias=rng.random() < 0.5,
                save_z=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def prepare(case, seed):
    """Inputs of one pass.  Activations are N(0, 1) values; those that a product takes are
    quantised here, as the call before it leaves them.  Weight codes are uniform over all 16,
    block scales 2^-12 .. 2^-6, which puts the pre-activations at order one.  Router logits are
    N(0, 1.5), the balance bias N(0, 0.05)."""
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 23)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype)

    def weights(rows, K):
        w = torch.randint(0, 256, (rows, K // 2), generator=g, device=dev, dtype=torch.uint8)
        s = torch.randint(115, 122, (rows, K // 32), generator=g, device=dev, dtype=torch.int16).to(torch.uint8)
        return w, s

    op, st = case["op"], dict(case)
    kind = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    if op.startswith("route"):
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = normal(T, E, std=1.5, dtype=kind)
        if op == "route":
            st["b"] = normal(E, std=0.05, dtype=torch.float32) if case["bias"] else None
        else:
            # what the forward call chose: the k largest logits in descending order
            st["ids"] = torch.sort(st["logits"], dim=1, descending=True, stable=True)[1][:, :k].int().contiguous()
            st["dgates"] = normal(T, k, dtype=torch.float32)
    elif op == "quantize":
        st["x"] = normal(case["rows"], case["K"], dtype=kind)
    elif op == "norm_q":
        T, H = case["T"], case["H"]
        st["x"] = normal(T, H, std=2.0)
        st["blk"] = normal(T, H, std=0.7) if case["block"] else None
        st["wpost"] = normal(H, std=0.1, mean=1.0) if case["post"] else None
        st["wpre"] = normal(H, std=0.1, mean=1.0)
        shape = {"none": None, "token": (T, 1), "channel": (H,), "full": (T, H)}[case["gate"]]
        st["g"] = normal(*shape, std=0.3, mean=0.5) if shape else None
    else:
        T, K = case["T"], case["K"] if op == "linear_q" else case["H"]
        rows = case["N"] if op == "linear_q" else 2 * case["I"]
        st["a"], st["as"] = _pack(*_blocks(normal(T, K).float(), case["fmt"]), case["fmt"])
        st["w"], st["s"] = weights(rows, K)
        st["bias"] = normal(rows, std=0.5) if case["bias"] else None
        st["r"] = normal(T, rows) if case.get("residual") else None
    return st


# ------------------------------------------------------------------ plain form (32 bits)

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _power(byte):
    """fp32 2^(byte - 127), exact (torch's powers are not everywhere)."""
    return torch.where(byte == 0, 1 << 22, byte.int() << 23).int().view(torch.float32)


def _blocks(v, fmt):
    """(elements, scale bytes) of fp32 rows: the scale of 32 values is the power of two that puts
    their largest into the element type's last binade."""
    rows, K = v.shape
    b = v.reshape(rows, K // 32, 32)
    top = b.abs().amax(-1)
    e = torch.frexp(top)[1] - 1
    byte = torch.where(top > 0, (e - (8 if fmt == "mxfp8" else 2) + 127).clamp(0, 254), torch.zeros_like(e))
    q = b * _power(254 - byte)[..., None]
    if fmt == "mxfp8":
        q = q.clamp(-448, 448).to(E4M3)
    else:
        a = q.abs().clamp(max=6)
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = torch.copysign(torch.round(a / step) * step, q)
    return q.reshape(rows, K), byte.to(torch.uint8)


def _pack(q, byte, fmt):
    """Elements and scale bytes as this library stores them."""
    if fmt == "mxfp8":
        return q.view(torch.uint8), byte
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte


def _values(codes, byte, fmt):
    """fp32 values of stored elements and scale bytes."""
    scale = _power(byte)
    if fmt == "mxfp8":
        v = codes.view(E4M3).float()
    else:
        table = torch.tensor(E2M1, dtype=torch.float32, device=codes.device)
        v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), dim=-1)
    return (v.reshape(*byte.shape, 32) * scale[..., None]).reshape(byte.shape[0], -1)


def _answer(q, byte, fmt):
    """What a call's MXFP8 output is here: its elements and scales; of MXFP4 its values."""
    if fmt == "mxfp8":
        return q, byte.view(E8M0)
    scale = _power(byte)
    return ((q.reshape(*byte.shape, 32) * scale[..., None]).reshape(q.shape).to(torch.bfloat16),)


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


def _scores(l, kind):
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_route(st):
    l, E, k = st["logits"], st["E"], st["k"]
    p = _scores(l.double(), st["score"])
    key = p + st["b"].double() if st["b"] is not None else p
    # without a bias the order is that of the logits, which the scores keep
    order = key if st["b"] is not None else l.double()
    if st["groups"] > 1:
        shape = (l.shape[0], st["groups"], E // st["groups"])
        best = torch.sort(key.reshape(shape), dim=-1, descending=True)[0]
        group = best[..., 0] if st["by"] == "max" or shape[2] == 1 else best[..., 0] + best[..., 1]
        rank = torch.sort(group, dim=-1, descending=True, stable=True)[1]
        open_ = torch.zeros_like(group).scatter(1, rank[:, :st["kept"]], 1.0)
        order = torch.where(open_[..., None] > 0, order.reshape(shape), -math.inf).reshape(l.shape)
    ids = torch.sort(order, dim=-1, descending=True, stable=True)[1][:, :k]
    g = p.gather(1, ids)
    if st["renorm"]:
        g = g / g.sum(-1, keepdim=True)
    return ids.int(), (st["scale"] * g).float()


def _plain_route_bwd(st):
    # in 64 bits: what is left of differences of nearly equal values
    l, ids, dg = st["logits"].double(), st["ids"].long(), st["scale"] * st["dgates"].double()
    p = _scores(l, st["score"])
    chosen = p.gather(1, ids)
    if st["renorm"]:
        total = chosen.sum(-1, keepdim=True)
        dg = (dg - (dg * chosen).sum(-1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter(1, ids, dg)
    if st["score"] == "sigmoid":
        d = dp * p * (1 - p)
    else:
        d = p * (dp - (dp * p).sum(-1, keepdim=True))
    return d.to(st["logits"].dtype)


def _plain_quantize(st):
    return _answer(*_blocks(st["x"].float(), st["fmt"]), st["fmt"])


def _plain_norm_q(st):
    y = st["x"]
    if st["blk"] is not None:
        n = st["blk"].float()
        if st["wpost"] is not None:
            n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + EPS) * st["wpost"].float()
        if st["g"] is not None:
            n = n * st["g"].float()
        y = (y.float() + st["scale"] * n).to(torch.bfloat16)
    f = y.float()
    xn = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * st["wpre"].float()
    out = _answer(*_blocks(xn, st["fmt"]), st["fmt"])
    return out + ((y,) if st["blk"] is not None else ()) + ((xn.to(torch.bfloat16),) if st["keep"] else ())


def _plain_product(st):
    z = _values(st["a"], st["as"], st["fmt"]) @ _values(st["w"], st["s"], "mxfp4").t()
    return z if st["bias"] is None else z + st["bias"].float()


def _plain_linear_q(st):
    z = _plain_product(st)
    y = st["scale"] * _act(z, st["act"])
    if st["r"] is not None:
        y = st["r"].float() + y
    return (y.to(torch.bfloat16), z.to(torch.bfloat16)) if st["save_z"] else (y.to(torch.bfloat16),)


def _plain_gate_up_q(st):
    z, I = _plain_product(st), st["I"]
    h = _act(z[:, :I], st["act"]) * z[:, I:]
    out = (h.to(torch.bfloat16),) if st["out"] == "bf16" else _answer(*_blocks(h, st["out"]), st["out"])
    return out + ((z.to(torch.bfloat16),) if st["save_z"] else ())


PLAIN = dict(route=_plain_route, route_bwd=_plain_route_bwd, quantize=_plain_quantize, norm_q=_plain_norm_q,
             linear_q=_plain_linear_q, gate_up_q=_plain_gate_up_q)


# ------------------------------------------------------------------ this library's calls

def _own(st):
    import mxfp4_weight_moe_amd as mx

    op = st["op"]
    if op == "route":
        return mx.moe_route_scored(st["logits"], st["k"], score=st["score"], bias=st["b"], n_group=st["groups"],
                                   topk_group=st["kept"], group_score=st["by"], renormalize=st["renorm"], scale=st["scale"])
    if op == "route_bwd":
        return mx.moe_route_scored_backward(st["dgates"], st["logits"], st["ids"], score=st["score"],
                                            renormalize=st["renorm"], scale=st["scale"])
    if op == "quantize":
        if st["fmt"] == "mxfp4":
            return (mx.mx_quantize(st["x"], "mxfp4", save_values=True)[2],)
        codes, scales = mx.mx_quantize(st["x"], "mxfp8")
        return codes.view(E4M3), scales.view(E8M0)
    if op == "norm_q":
        y, codes, scales, xn = mx.mx_norm_residual_quantize(
            st["x"], st["blk"], w_post=st["wpost"], gate=st["g"], scale=st["scale"], w_pre=st["wpre"], eps=EPS,
            fmt=st["fmt"], save_xn=st["keep"])
        return (codes.view(E4M3), scales.view(E8M0)) + ((y,) if st["blk"] is not None else ()) + ((xn,) if st["keep"] else ())
    if op == "linear_q":
        out = mx.mx_linear_quantized(st["a"], st["as"], st["w"], st["s"], bias=st["bias"], residual=st["r"],
                                     scale=st["scale"], act=st["act"], save_z=st["save_z"])
        return out if st["save_z"] else (out,)
    out = mx.mx_gate_up_quantized(st["a"], st["as"], st["w"], st["s"], bias=st["bias"], act=st["act"],
                                  fmt=None if st["out"] == "bf16" else st["out"], save_z=st["save_z"])
    if st["out"] == "bf16":
        return out if st["save_z"] else (out,)
    return (out[0].view(E4M3), out[1].view(E8M0)) + tuple(out[2:])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def _stored(n, fmt):
    """Bytes of n values."""
    return n * 2 if fmt == "bf16" else (n if fmt == "mxfp8" else n // 2) + n // 32


def work(case):
    op = case["op"]
    if op.startswith("route"):
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "fp32" else 2
        if op == "route":
            return {"bytes": T * E * size + T * k * 8 + 4 * E * int(case["bias"]), "flops": T * E * 8}
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * E * size + (T * E if dense else T * k) * size + T * k * 8, "flops": T * E * 8}
    if op == "quantize":
        n = case["rows"] * case["K"]
        out = _stored(n, case["fmt"]) + (2 * n if case["fmt"] == "mxfp4" else 0)
        return {"bytes": n * (4 if case["dtype"] == "fp32" else 2) + out, "flops": 3 * n}
    T = case["T"]
    if op == "norm_q":
        H = case["H"]
        n = T * H
        gate = {"none": 0, "token": T, "channel": H, "full": n}[case["gate"]]
        arrays = 1 + 2 * int(case["block"]) + int(case["keep"])
        return {"bytes": 2 * (arrays * n + H * (1 + int(case["post"])) + gate) + _stored(n, case["fmt"]),
                "flops": n * (4 * int(case["post"]) + 10)}
    K = case["K"] if op == "linear_q" else case["H"]
    rows, out = (case["N"], case["N"]) if op == "linear_q" else (2 * case["I"], case["I"])
    extra = out * int(case.get("residual", False)) + rows * int(case["save_z"])
    return {"bytes": rows * (K // 2 + K // 32) + 2 * rows * int(case["bias"]) + _stored(T * K, case["fmt"]) +
                     _stored(T * out, case.get("out", "bf16")) + 2 * T * extra,
            "flops": 2 * T * K * rows}


# ------------------------------------------------------------------ the definition in 64 bits

def _pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_decode(codes, byte, fmt):
    """Sign, exponent and mantissa bits of each element, times 2^(byte - 127)."""
    c = codes.long()
    if fmt == "mxfp8":
        bits, bias, man = c, 7, 3
    else:
        bits, bias, man = torch.stack((c % 16, c // 16), dim=2).flatten(1), 1, 1
    m = (bits % 2 ** man).double() / 2 ** man
    width = 7 if fmt == "mxfp8" else 3
    e = bits // 2 ** man % 2 ** (width - man)
    size = torch.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * _pow2(e - bias))
    value = torch.where(bits // 2 ** width % 2 == 1, -size, size)
    return value * _pow2(byte.long() - 127).repeat_interleave(32, dim=1)


def _exact_quantize(v, fmt):
    """(element values, scales) of rows in 64 bits: nearest element, halves to the even one."""
    last, man, low, most = (8, 3, -6, 448.0) if fmt == "mxfp8" else (2, 1, 0, 6.0)
    blocks = v.unflatten(1, (-1, 32))
    top = blocks.abs().max(dim=2).values
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - last
    scale = _pow2(torch.where(top > 0, e, torch.full_like(e, -127.0)).clamp(min=-127))
    u = blocks / scale[..., None]
    size = u.abs().clamp(max=most)
    binade = torch.floor(torch.log2(size.clamp(min=1e-300))).clamp(min=low)
    step = _pow2(binade - man)
    q = (torch.sign(u) * torch.round(size / step) * step).clamp(-most, most)
    return q.flatten(1), scale


def _exact_answer(v, fmt):
    q, scale = _exact_quantize(v, fmt)
    return (q, scale) if fmt == "mxfp8" else (q * scale.repeat_interleave(32, dim=1),)


def _exact_act(z, kind):
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "sigmoid":
        return torch.sigmoid(z)
    if kind == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if kind == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def _exact_route(case, st):
    """Chosen one by one: the largest left, the lowest index among equals."""
    l = st["logits"].double()
    T, E = l.shape
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)
    key = score if st["b"] is None else score + st["b"].double()

    def first_best(v):
        best = v.max(dim=1, keepdim=True).values
        place = torch.arange(v.shape[1], device=v.device).expand_as(v)
        return torch.where(v == best, place, torch.full_like(place, v.shape[1])).min(dim=1, keepdim=True).values

    left = (l if st["b"] is None else key).clone()
    if case["groups"] > 1:
        per = key.unflatten(1, (case["groups"], -1))
        two = per.topk(1 if case["by"] == "max" or per.shape[2] == 1 else 2, dim=2).values.sum(dim=2)
        closed = torch.ones_like(two, dtype=torch.bool)
        for _ in range(case["kept"]):
            at = first_best(two)
            closed.scatter_(1, at, False)
            two.scatter_(1, at, -math.inf)
        left.masked_fill_(closed.repeat_interleave(E // case["groups"], dim=1), -math.inf)
    ids = []
    for _ in range(case["k"]):
        at = first_best(left)
        ids.append(at)
        left.scatter_(1, at, -math.inf)
    ids = torch.cat(ids, dim=1)
    g = torch.take_along_dim(score, ids, dim=1)
    if case["renorm"]:
        g = g / g.sum(dim=1, keepdim=True)
    return ids.int(), case["scale"] * g


def _exact_route_bwd(case, st):
    """By the chain of Jacobians' products with vectors, per kind of score."""
    l, ids = st["logits"].double(), st["ids"].long()
    dg = case["scale"] * st["dgates"].double()
    if case["score"] == "softmax" and case["renorm"]:
        # a softmax over the chosen logits
        q = torch.softmax(torch.take_along_dim(l, ids, dim=1), dim=1)
        return torch.zeros_like(l).scatter_(1, ids, q * dg - q * (q * dg).sum(dim=1, keepdim=True))
    if case["score"] == "softmax":
        p = torch.softmax(l, dim=1)
        into = torch.zeros_like(l).scatter_(1, ids, dg)
        return p * into - p * (p * into).sum(dim=1, keepdim=True)
    s = torch.sigmoid(torch.take_along_dim(l, ids, dim=1))
    if case["renorm"]:
        total = s.sum(dim=1, keepdim=True)
        dg = dg / total - (dg * s).sum(dim=1, keepdim=True) / total ** 2
    slope = s * torch.sigmoid(-torch.take_along_dim(l, ids, dim=1))
    return torch.zeros_like(l).scatter_(1, ids, dg * slope)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "route_bwd":
        return _exact_route_bwd(case, st)
    if op == "quantize":
        return _exact_answer(st["x"].double(), case["fmt"])
    if op == "norm_q":
        unit = lambda v: v / (v.pow(2).mean(1, keepdim=True) + EPS).sqrt()  # noqa: E731
        y = st["x"].double()
        if st["blk"] is not None:
            n = st["blk"].double()
            n = n if st["wpost"] is None else unit(n) * st["wpost"].double()
            y = y + case["scale"] * (n if st["g"] is None else st["g"].double() * n)
        # the second norm's input is y as it is stored
        xn = unit(y.to(torch.bfloat16).double()) * st["wpre"].double()
        return _exact_answer(xn, case["fmt"]) + ((y,) if st["blk"] is not None else ()) + ((xn,) if case["keep"] else ())
    z = torch.matmul(_exact_decode(st["a"], st["as"], case["fmt"]), _exact_decode(st["w"], st["s"], "mxfp4").T)
    if st["bias"] is not None:
        z = z + st["bias"].double()
    if op == "linear_q":
        y = case["scale"] * _exact_act(z, case["act"]) + (0 if st["r"] is None else st["r"].double())
        return (y, z) if case["save_z"] else (y,)
    gate, up = z.chunk(2, dim=1)
    h = up * _exact_act(gate, case["act"])
    out = (h,) if case["out"] == "bf16" else _exact_answer(h, case["out"])
    return out + ((z,) if case["save_z"] else ())
