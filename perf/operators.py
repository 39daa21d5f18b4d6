"""Cases of the gated feed-forward operators: forward, backward, their FP4 form, and the products beside them.

Five operators, for operands as ``include/tcgemm.h`` lays them out (A is M x K; weights are N x K):

  gated       D = act(A Bg^T) * (A Bu^T), for training with both products kept in 16 bits
  backward    from dD and the kept products: the gradients of A, Bg and Bu
  trans       D = alpha op(A) op(B) + beta C with operands stored K x M or K x N (the products
              of a linear layer's backward pass)
  quantize    rows of 32-element blocks to E2M1 codes and UE8M0 scales, with the values they stand for
  gated_e2m1  activations quantised, then the gated block with both operands in FP4

``prepare`` makes inputs on the GPU from the seed; rows are padded to a multiple of eight
elements, as the library asks, so odd sizes come as slices of wider buffers.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # E2M1 magnitudes by code


def listed():
    return [
        # decoding: 16 sequences, one token each; N = 2 * 14336 weight rows stream once
        dict(name="gated_decode_16", op="gated", type="bf16", m=16, n=14336, k=4096, act="silu", save=False),
        # decoding: a single token through a small block, where latency counts
        dict(name="gated_token_1", op="gated", type="f16", m=1, n=4096, k=1024, act="gelu_tanh", save=False),
        # a short prompt through a block of odd width
        dict(name="gated_ragged", op="gated", type="f16", m=777, n=2743, k=1000, act="gelu", save=False),
        # a training step's forward pass over 8192 tokens, products kept for the backward pass
        dict(name="gated_train_8192", op="gated", type="bf16", m=8192, n=14336, k=4096, act="silu", save=True),
        # the same step's backward pass
        dict(name="backward_train_8192", op="backward", type="bf16", m=8192, n=14336, k=4096, act="silu"),
        # fine-tuning of a small block of odd sizes
        dict(name="backward_ragged", op="backward", type="f16", m=1000, n=1367, k=1000, act="gelu"),
        # gradient of the down projection's weights over 8192 tokens: both operands token-major
        dict(name="trans_weight_grad", op="trans", type="bf16", m=4096, n=14336, k=8192, ta=True, tb=True, c=False,
             out="bf16"),
        # gradient of a small projection's input, accumulated onto another branch's
        dict(name="trans_input_grad", op="trans", type="f16", m=1000, n=1367, k=1000, ta=False, tb=True, c=True,
             out="f32"),
        # a long prompt's activations before an FP4 down projection
        dict(name="quantize_8192", op="quantize", type="bf16", m=8192, k=14336),
        # one decoding step's activations
        dict(name="quantize_decode_16", op="quantize", type="f32", m=16, k=4096),
        # decoding with FP4 weights and activations
        dict(name="gated_e2m1_decode_16", op="gated_e2m1", type="bf16", m=16, n=14336, k=4096, act="silu"),
        # a long prompt with FP4 weights and activations
        dict(name="gated_e2m1_8192", op="gated_e2m1", type="bf16", m=8192, n=14336, k=4096, act="silu"),
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; half of them multiples of 64, the rest as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 128 and rng.random() < 0.5:
        v = v // 64 * 64
    v += v == 3072
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("gated", "backward", "trans", "quantize", "gated_e2m1"))
    m, n, k = _size(rng, 1, 8192), _size(rng, 64, 14336), _size(rng, 64, 4096)
    t = rng.choice(("bf16", "f16"))
    if op == "gated":
        return dict(op=op, type=t, m=m, n=n, k=k, act=rng.choice(ACTS), save=rng.random() < 0.5)
    if op == "backward":
        return dict(op=op, type=t, m=m, n=n, k=k, act=rng.choice(ACTS))
    if op == "trans":
        ta, tb = rng.choice(((False, True), (True, True), (True, False)))
        c = rng.random() < 0.5
        # float32 results for short sums, as a gradient added onto float32 gradients
        return dict(op=op, type=t, m=m, n=n, k=k, ta=ta, tb=tb, c=c, out="f32" if k <= 1024 else t)
    k = max(32, k // 32 * 32)
    if op == "quantize":
        return dict(op=op, type=rng.choice(("bf16", "f16", "f32")), m=m, k=max(32, n // 32 * 32))
    return dict(op=op, type=t, m=m, n=n, k=k, act=rng.choice(ACTS))


# ---------------------------------------------------------------- inputs

def _pad8(cols):
    return (cols + 7) // 8 * 8


def _normal(gen, rows, cols, dtype, scale=1.0):
    x = torch.empty((rows, _pad8(cols)), dtype=torch.float32, device=DEV)
    x.normal_(0.0, scale, generator=gen)
    return x.to(dtype)[:, :cols]


def _activations(gen, rows, cols, dtype):
    """Near-normal rows with a few wide channels and some empty (padding) rows, as activations are."""
    x = torch.empty((rows, _pad8(cols)), dtype=torch.float32, device=DEV).normal_(0.0, 1.0, generator=gen)
    wide = torch.randint(0, cols, (max(1, cols // 256),), generator=gen, device=DEV)
    x[:, wide] *= 24.0
    if rows >= 16:
        x[rows // 3] = 0.0
    return x.to(dtype)[:, :cols]


def _empty(rows, cols, dtype):
    """An output matrix whose rows are a multiple of 16 bytes apart."""
    return torch.empty((rows, _pad8(cols)), dtype=dtype, device=DEV)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, dt = case["op"], TYPES[case["type"]]
    m, n, k = case["m"], case.get("n", 0), case["k"]
    s = dict(case)
    if op == "gated":
        s["a"] = _normal(gen, m, k, dt)
        s["bg"], s["bu"] = _normal(gen, n, k, dt, 0.02), _normal(gen, n, k, dt, 0.02)
        s["d"] = _empty(m, n, dt)
        if case["save"]:
            s["g"], s["u"] = _empty(m, n, dt), _empty(m, n, dt)
    elif op == "backward":
        spread = 0.02 * math.sqrt(k)  # of A Bg^T and A Bu^T
        s["a"] = _normal(gen, m, k, dt)
        s["bg"], s["bu"] = _normal(gen, n, k, dt, 0.02), _normal(gen, n, k, dt, 0.02)
        s["g"], s["u"] = _normal(gen, m, n, dt, spread), _normal(gen, m, n, dt, spread)
        s["dd"] = _normal(gen, m, n, dt)
        s["dg"], s["du"] = _empty(m, n, dt), _empty(m, n, dt)
        s["da"], s["dbg"], s["dbu"] = _empty(m, k, dt), _empty(n, k, dt), _empty(n, k, dt)
    elif op == "trans":
        s["a"] = _normal(gen, k, m, dt) if case["ta"] else _normal(gen, m, k, dt)
        s["b"] = _normal(gen, k, n, dt, 0.02) if case["tb"] else _normal(gen, n, k, dt, 0.02)
        s["c"] = _normal(gen, m, n, torch.float32) if case["c"] else None
        s["d"] = _empty(m, n, TYPES[case["out"]])
    elif op == "quantize":
        s["x"] = _activations(gen, m, k, dt)
        s["y"] = _empty(m, k, dt)
    else:
        s["x"] = _activations(gen, m, k, dt)
        s["bgq"], s["bgs"], _ = _quantize(_normal(gen, n, k, torch.float32, 0.02))
        s["buq"], s["bus"], _ = _quantize(_normal(gen, n, k, torch.float32, 0.02))
        s["bgs"], s["bus"] = _pitched(s["bgs"]), _pitched(s["bus"])
        s["d"] = _empty(m, n, dt)
    return s


def _pitched(scales):
    """Scale rows at a pitch of 16 bytes, as a model's loader lays them out once."""
    rows, cols = scales.shape
    wide = torch.zeros((rows, (cols + 15) // 16 * 16), dtype=torch.uint8, device=DEV)
    wide[:, :cols] = scales
    return wide[:, :cols]


# ---------------------------------------------------------------- plain forms

def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))
    if name == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g))
    return 1.0 / (1.0 + torch.exp(-g))


def _act_slope(name, g):
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return p * (1.0 + g * (1.0 - p))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)
    if name == "relu":
        return (g > 0).to(g.dtype)
    p = 1.0 / (1.0 + torch.exp(-g))
    return p * (1.0 - p)


def _power(s):
    """2^(s - 127) for integers s in [0, 254], exactly, from the bits of a float32."""
    return torch.where(s > 0, s.int() << 23, torch.full_like(s, 1 << 22, dtype=torch.int32)).view(torch.float32)


def _quantize(x):
    """float32 rows -> (packed codes, scales K/32 x M, values): the scale is 2^(floor(log2(max)) - 2), codes
    round to nearest, ties to the even code, and stop at 6."""
    m, k = x.shape
    b = x.reshape(m, k // 32, 32)
    top = b.abs().amax(dim=2)
    _, e = torch.frexp(top)
    s = torch.where(top > 0, torch.clamp(e - 1 - 2 + 127, 0, 254), torch.zeros_like(e))
    y = b * _power(254 - s)[:, :, None]
    z = y.abs()
    code = ((z > 0.25).to(torch.uint8) + (z >= 0.75) + (z > 1.25) + (z >= 1.75) + (z > 2.5) + (z >= 3.5) + (z > 5.0))
    levels = torch.tensor(LEVELS, dtype=torch.float32, device=x.device)
    minus = torch.signbit(y)
    v = torch.where(minus, -levels[code.long()], levels[code.long()])
    values = (v * _power(s)[:, :, None]).reshape(m, k)
    code = (code + 8 * minus.to(torch.uint8)).reshape(m, k // 2, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), s.t().to(torch.uint8).contiguous(), values


def _values(codes, scales):
    """float32 values of packed codes (rows x K/2) and scales (K/32 x rows)."""
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float32, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], -1)
    v = levels[c.long()].reshape(codes.shape[0], -1, 32)
    return (v * _power(scales.t().int())[:, :, None]).reshape(codes.shape[0], -1)


def _plain(s):
    op, dt = s["op"], TYPES[s["type"]]
    if op == "gated":
        a = s["a"].float()
        g, u = a @ s["bg"].float().t(), a @ s["bu"].float().t()
        out = {"d": (_act(s["act"], g) * u).to(dt)}
        if s["save"]:
            out["g"], out["u"] = g.to(dt), u.to(dt)
        return out
    if op == "backward":
        a, g, u, dd = s["a"].float(), s["g"].float(), s["u"].float(), s["dd"].float()
        dg, du = dd * u * _act_slope(s["act"], g), dd * _act(s["act"], g)
        return {"da": (dg @ s["bg"].float() + du @ s["bu"].float()).to(dt),
                "dbg": (dg.t() @ a).to(dt), "dbu": (du.t() @ a).to(dt)}
    if op == "trans":
        a = s["a"].float().t() if s["ta"] else s["a"].float()
        b = s["b"].float() if s["tb"] else s["b"].float().t()
        d = 0.5 * (a @ b)
        return {"d": (d + s["c"] if s["c"] is not None else d).to(TYPES[s["out"]])}
    q, sc, v = _quantize(s["x"].float())
    if op == "quantize":
        return {"values": v.to(dt), "codes": q, "scales": sc}
    g, u = v @ _values(s["bgq"], s["bgs"]).t(), v @ _values(s["buq"], s["bus"]).t()
    return {"d": (_act(s["act"], g) * u).to(dt)}


# ---------------------------------------------------------------- the framework's operators

def _own(s):
    from tensor_core_gemm_02_gb300 import binding as tc

    op = s["op"]
    out = {"bf16": tc.OUT_BF16, "f16": tc.OUT_F16, "f32": tc.OUT_F32}
    if op == "gated":
        tc.gemm_gated(s["a"], s["bg"], s["bu"], s["d"], G=s.get("g"), U=s.get("u"), act=s["act"], out=out[s["type"]])
        return {"d": s["d"], "g": s["g"], "u": s["u"]} if s["save"] else {"d": s["d"]}
    if op == "backward":
        tc.gemm_gated_backward(s["dd"], s["g"], s["u"], s["a"], s["bg"], s["bu"], dG=s["dg"], dU=s["du"],
                               dA=s["da"], dBg=s["dbg"], dBu=s["dbu"], act=s["act"], out=out[s["type"]])
        return {"da": s["da"], "dbg": s["dbg"], "dbu": s["dbu"]}
    if op == "trans":
        tc.gemm_trans(s["a"], s["b"], s["c"], s["d"], trans_a=s["ta"], trans_b=s["tb"], alpha=0.5, beta=1.0,
                      out=out[s["out"]])
        return {"d": s["d"]}
    if op == "quantize":
        q, sc = tc.gemm_quantize_e2m1(s["x"], Y=s["y"])
        return {"values": s["y"], "codes": q, "scales": sc}
    q, sc = tc.gemm_quantize_e2m1(s["x"])
    tc.gemm_gated_e2m1(q, sc, s["bgq"], s["bgs"], s["buq"], s["bus"], s["d"], act=s["act"], out=out[s["type"]])
    return {"d": s["d"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits

def _act64(name, g):
    """The activations from their definitions, differentiable, in 64 bits."""
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu":
        return g * torch.special.ndtr(g)
    if name == "gelu_tanh":
        return g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))
    if name == "relu":
        return torch.relu(g)
    return torch.sigmoid(g)


def _nearest64(x):
    """The quantiser from its definition: for each element the nearest of the eight magnitudes, the even code
    where two are equally near."""
    m, k = x.shape
    b = x.reshape(m, k // 32, 32)
    top = b.abs().amax(dim=2, keepdim=True)
    e = (top.view(torch.int64) >> 52) - 1023  # floor(log2(top)); an empty block's scale is the smallest
    scale = ((torch.clamp(e - 2, -127, 127) + 1023) << 52).view(torch.float64)
    z = (b / scale).abs().clamp(max=6.0)
    best, at = (z - LEVELS[0]).abs(), torch.zeros_like(z)
    for c in range(1, 8):
        d = (z - LEVELS[c]).abs()
        take = (d < best) | ((d == best) & (c % 2 == 0))
        best, at = torch.where(take, d, best), torch.where(take, torch.full_like(z, LEVELS[c]), at)
    return (torch.copysign(at, b) * scale).reshape(m, k)


def _decode64(codes, scales):
    """FP4 weights from the fields of their codes (sign, two exponent bits with bias 1, one mantissa bit)."""
    c = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.int32, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
    exponent, half = (c // 2) % 4, (c % 2).double() / 2
    v = torch.where(exponent == 0, half, (1.0 + half) * (1 << exponent).double() / 2)
    v = torch.where(c >= 8, -v, v)
    return v * ((scales.t().long() - 127 + 1023) << 52).view(torch.float64).repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated":
        a = s["a"].double()
        g, u = torch.mm(a, s["bg"].double().t()), torch.mm(a, s["bu"].double().t())
        out = {"d": _act64(case["act"], g) * u}
        if case["save"]:
            out["g"], out["u"] = g, u
        return out
    if op == "backward":
        g = s["g"].double().requires_grad_()
        u = s["u"].double().requires_grad_()
        dg, du = torch.autograd.grad(_act64(case["act"], g) * u, (g, u), s["dd"].double())
        a = s["a"].double()
        return {"da": torch.addmm(torch.mm(dg, s["bg"].double()), du, s["bu"].double()),
                "dbg": torch.mm(dg.t(), a), "dbu": torch.mm(du.t(), a)}
    if op == "trans":
        a, b = s["a"].double(), s["b"].double()
        d = torch.einsum("%s,%s->mn" % ("km" if case["ta"] else "mk", "kn" if case["tb"] else "nk"), a, b) / 2
        return {"d": d if s["c"] is None else d + s["c"].double()}
    v = _nearest64(s["x"].double())
    if op == "quantize":
        return {"values": v, "codes": None, "scales": None}
    wg, wu = _decode64(s["bgq"], s["bgs"]), _decode64(s["buq"], s["bus"])
    return {"d": _act64(case["act"], torch.mm(v, wg.t())) * torch.mm(v, wu.t())}


# ---------------------------------------------------------------- work

def work(case):
    op, e = case["op"], 4 if case["type"] == "f32" else 2
    m, n, k = case["m"], case.get("n", 0), case["k"]
    if op == "gated":
        return {"bytes": e * (m * k + 2 * n * k + m * n * (3 if case["save"] else 1)), "flops": 4.0 * m * n * k}
    if op == "backward":  # A, both weights, G, U and dD once; the three gradients
        return {"bytes": e * (2 * m * k + 4 * n * k + 3 * m * n), "flops": 8.0 * m * n * k}
    if op == "trans":
        w = 4 if case["out"] == "f32" else 2
        return {"bytes": e * (m * k + n * k) + m * n * (w + (4 if case["c"] else 0)), "flops": 2.0 * m * n * k}
    if op == "quantize":  # read, values, codes, scales; a product by the scale and a rounding each
        return {"bytes": m * k * (2 * e + 0.5 + 1 / 32), "flops": 3.0 * m * k}
    # activations in 16 bits, weights at 4.25 bits an element, D
    return {"bytes": e * m * k + 2 * n * k * (0.5 + 1 / 32) + e * m * n, "flops": 4.0 * m * n * k}
