"""Cases of the operators for layers of experts: rows grouped by expert, the grouped products and their gradients,
and the orthogonalised update of a stack of weights.

Four operators, for operands as ``include/tcgemm.h`` lays them out:

  group_rows   expert ids -> offsets of each expert's rows and the rows in that order (a stable counting sort)
  grouped      D[i] = A[i] B_e^T for the rows i of group e, the rows gathered through an index or not; B_e stored
               N x K, or K x N (the gradient of the input)
  weights      dB_e = dD_e^T A_e, the gradients of the groups' weights, each a sum over its rows
  orthogonalize  X / |X| and some steps of X <- a X + (b X X^T + c (X X^T)^2) X, for a stack of matrices

Groups are as uneven as a router leaves them (``_counts``): some are empty, and rows behind the last group belong
to none and keep what they hold.  ``prepare`` makes inputs on the GPU from the seed; rows are padded to a multiple
of eight elements, as the library asks, so odd sizes come as slices of wider buffers.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
COEFS = (3.4445, -4.7750, 2.0315)  # of the polynomial's terms X, (X X^T) X and (X X^T)^2 X
STEPS = 5
EPS = 1e-7


def listed():
    return [
        # decoding: 16 sequences, one token each, two of eight experts a token; their weights stream once
        dict(name="grouped_decode_16", op="grouped", type="bf16", out="bf16", e=8, m=32, n=14336, k=4096, choices=2,
             trans=False, skew=0.5, empty=0, behind=0),
        # decoding: one token through two of 64 small experts, where latency counts
        dict(name="grouped_token_1", op="grouped", type="f16", out="f32", e=64, m=2, n=2816, k=1024, choices=2,
             trans=False, skew=0.0, empty=62, behind=0),
        # a short prompt in a padded batch through experts of odd width, some of them empty
        dict(name="grouped_ragged", op="grouped", type="f16", out="f16", e=11, m=777, n=2743, k=1000, choices=0,
             trans=False, skew=1.0, empty=2, behind=23),
        # a training step's forward pass: 8192 tokens, two of eight experts each
        dict(name="grouped_train_16384", op="grouped", type="bf16", out="bf16", e=8, m=16384, n=14336, k=4096,
             choices=0, trans=False, skew=0.3, empty=0, behind=0),
        # the same step's gradient of the input
        dict(name="grouped_input_grad_16384", op="grouped", type="bf16", out="bf16", e=8, m=16384, n=4096, k=14336,
             choices=0, trans=True, skew=0.3, empty=0, behind=0),
        # and of the weights
        dict(name="weights_train_16384", op="weights", type="bf16", out="bf16", e=8, m=16384, n=14336, k=4096,
             skew=0.3, empty=0, behind=0),
        # fine-tuning of small experts of odd sizes, one without a row
        dict(name="weights_ragged", op="weights", type="f16", out="f32", e=5, m=1000, n=1367, k=1000, skew=1.0,
             empty=1, behind=24),
        # the training step's tokens by expert
        dict(name="group_rows_16384", op="group_rows", e=64, m=16384, choices=2, skew=0.5, empty=0, behind=100),
        # a decoding step's
        dict(name="group_rows_decode_16", op="group_rows", e=8, m=32, choices=2, skew=0.5, empty=0, behind=0),
        # the update of one small projection, held in float32
        dict(name="orthogonalize_2816", op="orthogonalize", type="f32", e=1, m=2816, n=1024),
        # the updates of a stack of small experts of odd sizes
        dict(name="orthogonalize_ragged", op="orthogonalize", type="f16", e=8, m=1000, n=1367),
        # the updates of two large projections
        dict(name="orthogonalize_14336", op="orthogonalize", type="bf16", e=2, m=4096, n=14336),
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; half of them multiples of 64, the rest as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 128 and rng.random() < 0.5:
        v = v // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("grouped", "grouped", "weights", "group_rows", "orthogonalize"))
    t = rng.choice(("bf16", "f16"))
    if op == "orthogonalize":
        m, n = _size(rng, 16, 8192), _size(rng, 16, 4096)
        e = max(1, min(_size(rng, 1, 16), 2 * 4096 * 14336 // (m * n)))
        return dict(op=op, type=rng.choice(("bf16", "f16", "f32")), e=e, m=m, n=n)
    e, m = _size(rng, 1, 64), _size(rng, 1, 16384)
    skew = rng.choice((0.0, 0.3, 1.0))
    empty = rng.choice((0, 0, e // 3))
    behind = rng.choice((0, 0, m // 8))
    if op == "group_rows":
        choices = rng.choice((1, 2, 4))
        return dict(op=op, e=4 * e, m=m * choices, choices=choices, skew=skew, empty=empty, behind=behind)
    n, k = _size(rng, 64, 14336), _size(rng, 64, 4096)
    e = max(1, min(e, 8 * 14336 * 4096 // (n * k)))
    empty = min(empty, e // 3)
    # float32 results for short sums, as a gradient added onto float32 gradients
    if op == "weights":
        return dict(op=op, type=t, out="f32" if n * k < 1 << 22 else t, e=e, m=m, n=n, k=k, skew=skew, empty=empty,
                    behind=behind)
    trans = rng.random() < 0.4
    if trans:
        n, k = k, n
    choices = 0 if trans else rng.choice((0, 1, 2))
    return dict(op=op, type=t, out="f32" if k <= 1024 else t, e=e, m=m, n=n, k=k, choices=choices, trans=trans,
                skew=skew, empty=empty, behind=0 if choices else behind)


def _counts(case):
    """Rows of each group, largest first: m - behind of them, shared out as (1 + i)^-skew over the groups but the
    last `empty` ones."""
    live = case["e"] - case["empty"]
    rows = case["m"] - case["behind"]
    share = [(1.0 + i) ** -case["skew"] for i in range(live)]
    total = sum(share)
    counts = [int(rows * s / total) for s in share]
    for i in range(rows - sum(counts)):
        counts[i % live] += 1
    return counts + [0] * case["empty"]


# ---------------------------------------------------------------- inputs

def _pad8(cols):
    return (cols + 7) // 8 * 8


def _normal(gen, shape, dtype, scale=1.0):
    x = torch.empty((*shape[:-1], _pad8(shape[-1])), dtype=torch.float32, device=DEV)
    x.normal_(0.0, scale, generator=gen)
    return x.to(dtype)[..., :shape[-1]]


def _stack(gen, e, n, k, dtype, scale):
    """e matrices, made one by one (their float32 values need not exist at once)."""
    x = torch.empty((e, n, _pad8(k)), dtype=dtype, device=DEV)
    for i in range(e):
        x[i] = torch.empty((n, _pad8(k)), dtype=torch.float32, device=DEV).normal_(0.0, scale, generator=gen)
    return x[:, :, :k]


def _ids(gen, case):
    """Expert ids as a router gives them: each expert as often as its count says, in any order; -1 for the
    assignments that were dropped (as many as lie behind the last group)."""
    perm = torch.randperm(case["e"], generator=gen, device=DEV)
    per = torch.tensor(_counts(case), device=DEV)[perm]
    ids = torch.repeat_interleave(torch.arange(case["e"], device=DEV), per)
    ids = torch.cat((ids, torch.full((case["behind"],), -1, device=DEV)))
    ids = ids[torch.randperm(case["m"], generator=gen, device=DEV)]
    return per, ids.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, e, m = case["op"], case["e"], case["m"]
    s = dict(case)
    if op == "orthogonalize":
        # a momentum: some strong directions over noise
        n, dt = case["n"], TYPES[case["type"]]
        rank = max(1, min(m, n) // 16)
        s["x"] = torch.empty((e, m, _pad8(n)), dtype=dt, device=DEV)
        for i in range(e):
            x = torch.empty((m, _pad8(n)), dtype=torch.float32, device=DEV).normal_(0.0, 1.0, generator=gen)
            u = torch.empty((m, rank), device=DEV).normal_(0.0, 1.0, generator=gen)
            v = torch.empty((rank, _pad8(n)), device=DEV).normal_(0.0, 1.0, generator=gen)
            s["x"][i] = 0.01 * (x + (u * torch.linspace(2.0, 0.1, rank, device=DEV)) @ v)
        s["x"] = s["x"][:, :, :n]
        s["y"] = torch.zeros((e, m, _pad8(n)), dtype=dt, device=DEV)[:, :, :n]
        return s
    per, ids = _ids(gen, case)
    if op == "group_rows":
        s["ids"] = ids.reshape(-1, case["choices"])
        return s
    # the offsets, where a kernel finds them and where the plain form's slices need them
    s["bounds"] = [0] + torch.cumsum(per, 0).tolist()
    s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device=DEV)
    n, k, dt, out = case["n"], case["k"], TYPES[case["type"]], TYPES[case["out"]]
    if op == "weights":
        s["dd"], s["a"] = _normal(gen, (m, n), dt), _normal(gen, (m, k), dt)
        s["db"] = torch.zeros((e, n, _pad8(k)), dtype=out, device=DEV)[:, :, :k]
        return s
    choices = case["choices"]
    s["a"] = _normal(gen, (m // choices if choices else m, k), dt)
    s["idx"] = None
    if choices:
        s["idx"] = (torch.argsort(ids, stable=True) // choices).to(torch.int32)
        s["idx"] = s["idx"].clamp_(max=s["a"].shape[0] - 1) if s["a"].shape[0] else s["idx"]
    s["b"] = _stack(gen, e, k, n, dt, 0.02) if case["trans"] else _stack(gen, e, n, k, dt, 0.02)
    s["d"] = torch.zeros((m, _pad8(n)), dtype=out, device=DEV)[:, :n]
    return s


# ---------------------------------------------------------------- plain forms

def _plain(s):
    op = s["op"]
    if op == "group_rows":
        ids = s["ids"].reshape(-1)
        key = torch.where((ids >= 0) & (ids < s["e"]), ids, torch.full_like(ids, s["e"]))
        order = torch.sort(key, stable=True).indices
        ends = (key[:, None] == torch.arange(s["e"], device=key.device, dtype=key.dtype)).sum(dim=0).cumsum(dim=0)
        return {"offsets": torch.cat((torch.zeros_like(ends[:1]), ends)).to(torch.int32),
                "order": order.to(torch.int32),
                "rows": torch.div(order, s["choices"], rounding_mode="floor").to(torch.int32)}
    if op == "orthogonalize":
        a, b, c = COEFS
        x = s["x"].float()
        flip = x.shape[1] > x.shape[2]
        if flip:
            x = x.transpose(1, 2)
        x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
        for _ in range(STEPS):
            g = x @ x.transpose(1, 2)
            x = a * x + (b * g + c * (g @ g)) @ x
        s["y"].copy_(x.transpose(1, 2) if flip else x)
        return {"y": s["y"]}
    lo_hi = list(zip(s["bounds"][:-1], s["bounds"][1:]))
    if op == "weights":
        for i, (lo, hi) in enumerate(lo_hi):
            s["db"][i] = s["dd"][lo:hi].float().t() @ s["a"][lo:hi].float()
        return {"db": s["db"]}
    a = s["a"] if s["idx"] is None else s["a"][s["idx"].long()]
    for i, (lo, hi) in enumerate(lo_hi):
        if lo < hi:
            b = s["b"][i].float()
            s["d"][lo:hi] = a[lo:hi].float() @ (b if s["trans"] else b.t())
    return {"d": s["d"]}


# ---------------------------------------------------------------- the framework's operators

def _own(s):
    from tensor_core_gemm_02_gb300 import binding as tc

    op = s["op"]
    out = {"bf16": tc.OUT_BF16, "f16": tc.OUT_F16, "f32": tc.OUT_F32}
    if op == "group_rows":
        offsets, order, rows = tc.gemm_group_rows(s["ids"], s["e"])
        return {"offsets": offsets, "order": order, "rows": rows}
    if op == "orthogonalize":
        tc.gemm_orthogonalize(s["x"], s["y"], steps=STEPS, coefs=COEFS, eps=EPS)
        return {"y": s["y"]}
    if op == "weights":
        tc.gemm_grouped_weights(s["dd"], s["a"], s["offsets"], s["db"], out=out[s["out"]])
        return {"db": s["db"]}
    tc.gemm_grouped(s["a"], s["b"], s["offsets"], s["d"], idx=s["idx"], trans_b=s["trans"], out=out[s["out"]])
    return {"d": s["d"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "group_rows":
        # each id's place: the ids below it, and the equal ones before it
        order, offsets = [], [0]
        flat = s["ids"].flatten().tolist()
        groups = [[] for _ in range(case["e"] + 1)]
        for at, i in enumerate(flat):
            groups[i if 0 <= i < case["e"] else -1].append(at)
        for group in groups:
            order += group
            offsets.append(len(order))
        whole = lambda v: torch.tensor(v, dtype=torch.float64, device=DEV)  # noqa: E731
        return {"offsets": whole(offsets[:-1]), "order": whole(order), "rows": whole([at // case["choices"] for at in order])}
    if op == "orthogonalize":
        # every iterate is P X0 with P a polynomial in X0 X0^T (or X0 P): P is carried, and P^2 X0 X0^T, the
        # iterate's own product with itself
        ca, cb, cc = COEFS
        y = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
        for i in range(case["e"]):
            x = s["x"][i].double()
            x = x / (torch.linalg.vector_norm(x) + EPS)
            left = x.shape[0] <= x.shape[1]
            g = torch.einsum("ik,jk->ij" if left else "ki,kj->ij", x, x)
            p = torch.eye(g.shape[0], dtype=torch.float64, device=DEV)
            for _ in range(STEPS):
                q = torch.addmm(cb * g, g, g, alpha=cc)
                q.diagonal().add_(ca)
                p = q.mm(p)
                g = q.mm(g).mm(q)
            y[i] = p.mm(x) if left else x.mm(p)
        return {"y": y}
    starts = [0]
    for c in s["offsets"].diff().tolist():
        starts.append(starts[-1] + c)
    if op == "weights":
        db = torch.empty(s["db"].shape, dtype=torch.float64, device=DEV)
        for i in range(case["e"]):
            rows = slice(starts[i], starts[i + 1])
            db[i] = torch.einsum("rn,rk->nk", s["dd"][rows].double(), s["a"][rows].double())
        return {"db": db}
    d = torch.zeros(s["d"].shape, dtype=torch.float64, device=DEV)
    for i in range(case["e"]):
        if starts[i] == starts[i + 1]:
            continue
        r = torch.arange(starts[i], starts[i + 1], device=DEV)
        a = s["a"].index_select(0, r if s["idx"] is None else s["idx"].index_select(0, r).long()).double()
        d[starts[i]:starts[i + 1]] = torch.einsum("rk,kn->rn" if case["trans"] else "rk,nk->rn", a, s["b"][i].double())
    return {"d": d}


# ---------------------------------------------------------------- work

def work(case):
    op, e, m = case["op"], case["e"], case["m"]
    if op == "group_rows":  # ids in, order and rows out, the offsets; a count and a place for each
        return {"bytes": 12.0 * m + 4 * (e + 1), "flops": 2.0 * m}
    if op == "orthogonalize":
        n = case["n"]
        s, l = min(m, n), max(m, n)
        # X X^T and its square are symmetric: half of each; then the product with X
        step = s * (s + 1.0) * l + s * (s + 1.0) * s + 2.0 * s * s * l
        return {"bytes": 2.0 * e * m * n * (4 if case["type"] == "f32" else 2), "flops": STEPS * e * step}
    n, k, rows = case["n"], case["k"], case["m"] - case["behind"]
    w = 4 if case["out"] == "f32" else 2
    if op == "weights":
        return {"bytes": 2.0 * rows * (n + k) + w * e * n * k, "flops": 2.0 * rows * n * k}
    live = sum(1 for c in _counts(case) if c)
    a = rows // case["choices"] if case["choices"] else rows
    return {"bytes": 2.0 * (a * k + live * n * k) + w * rows * n, "flops": 2.0 * rows * n * k}
