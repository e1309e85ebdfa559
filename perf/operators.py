"""Cases of the router and MXFP4 operators: inputs, plain forms, what each has to move and compute, and 64-bit results.

Five operators around the routed expert step:

* ``router``: top-k of the router's logits, the routing weights and the row's log-sum-exp (serving).
* ``router_train``: the same with the balance loss, the z-loss and the per-expert counts, and the gradient of the
  logits from the gradients of the routing weights and of both losses (one training pass).
* ``quant``: rows or weights rounded to MXFP4 and read back.
* ``product``: one grouped projection, MXFP4 rows times MXFP4 expert weights.
* ``up``: the grouped gate/up projection of MXFP4 token rows read through the dispatch order, with SwiGLU.

MXFP4 (OCP Microscaling Formats v1.0): blocks of 32 values along the contraction share one power of two, kept as a
byte (exponent + 127); each value is a 4-bit float, sign, two exponent bits and one mantissa bit, of magnitude 0, 0.5,
1, 1.5, 2, 3, 4 or 6. The block's exponent is floor(log2(largest magnitude)) - 2, values round to nearest even and
saturate at 6. Rows are packed two values a byte, the even one in the low half; a row of K values takes
16 * ceil(K / 32) bytes, and its scale bytes 16 * ceil(K / 512) (zeros behind the last block).
"""

import math

import torch

own = False

BLOCK = 32
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64


def listed():
    return [
        # the router of a decode step of four sequences: latency alone
        dict(name="router_decode", op="router", T=4, E=128, k=8, dtype="bf16", renorm=True, pad=0, lowest=0),
        # the router of a prefill batch, float32 logits
        dict(name="router_prefill", op="router", T=8192, E=64, k=8, dtype="f32", renorm=True, pad=0, lowest=0),
        # a training step of a padded batch: the last rows are padding, masked for every expert
        dict(name="router_train_4k", op="router_train", T=4096, E=128, k=8, dtype="bf16", renorm=True, pad=200, lowest=0),
        # a long training batch, an odd number of tokens and of experts, three experts masked by the type's lowest value
        dict(name="router_train_64k", op="router_train", T=65537, E=100, k=6, dtype="f32", renorm=False, pad=1, lowest=3),
        # a decode step's token rows
        dict(name="quant_decode", op="quant", rows=32, K=2048, E=1, layout="rows"),
        # a prefill batch's permuted rows
        dict(name="quant_prefill", op="quant", rows=65536, K=2048, E=1, layout="rows"),
        # the down projection's weights of sixteen experts, stored with the contraction outermost
        dict(name="quant_weights", op="quant", rows=2880, K=2880, E=16, layout="in_out"),
        # the down projection of a decode step: four tokens, eight experts each
        dict(name="product_decode", op="product", M=32, spare=0, E=128, K=768, N=2048, load="spread"),
        # ragged rows, the contraction ends inside a block, the columns inside a tile; rows behind the last stay
        dict(name="product_ragged", op="product", M=4091, spare=5, E=8, K=392, N=520, load="zipf"),
        # the down projection of a skewed prefill batch
        dict(name="product_prefill", op="product", M=65536, spare=0, E=64, K=768, N=2048, load="zipf"),
        # the gate/up projection of a decode step
        dict(name="up_decode", op="up", T=4, k=8, E=128, d=2048, h=768, load="spread", drop=0),
        # the gate/up projection of a skewed prefill batch, one slot in twenty dropped
        dict(name="up_prefill", op="up", T=8192, k=8, E=64, d=2048, h=768, load="zipf", drop=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "router_train", "quant", "product", "product", "up", "up"])
    if op.startswith("router"):
        E = _log(rng, 4, 512)
        T = _log(rng, 1, min(70000, 6500000 // E))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 12)), dtype=rng.choice(["bf16", "f32"]),
                    renorm=rng.random() < 0.6, pad=rng.choice([0, 0, T // 10]), lowest=rng.choice([0, 0, min(2, E - 1)]))
    if op == "quant":
        K = 8 * _log(rng, 1, 1000)
        if rng.random() < 0.7:
            return dict(op=op, rows=_log(rng, 1, min(70000, 130000000 // K)), K=K, E=1, layout="rows")
        N = 8 * _log(rng, 1, 600)
        return dict(op=op, rows=N, K=K, E=rng.randint(1, max(1, min(32, 130000000 // (N * K)))), layout="in_out")
    load = rng.choice(["spread", "zipf"])
    if op == "product":
        K, N = 8 * _log(rng, 4, 400), 8 * _log(rng, 4, 400)
        E = _log(rng, 1, min(256, 600000000 // (K * N)))
        M = _log(rng, 1, min(65536, 100000000000 // (K * N)))
        return dict(op=op, M=M, spare=rng.choice([0, 0, 7]), E=E, K=K, N=N, load=load)
    d, h = 8 * _log(rng, 4, 360), 8 * _log(rng, 4, 200)
    E = _log(rng, 1, min(256, 600000000 // (2 * d * h)))
    k = rng.randint(1, min(E, 8))
    T = max(1, _log(rng, 1, min(65536, 200000000000 // (2 * d * h))) // k)
    return dict(op=op, T=T, k=k, E=E, d=d, h=h, load=load, drop=rng.choice([0, 0, 5]))


# ------------------------------------------------------------------------------------------------ inputs

def _row_bytes(K):
    return 16 * (-(-K // BLOCK))


def _scale_bytes(K):
    return 16 * (-(-K // (16 * BLOCK)))


def _blocks(x):
    """float32 values of x [..., K] in blocks [..., ceil(K / 32), 32], zeros behind the last."""
    K = x.shape[-1]
    f = torch.nn.functional.pad(x.float(), (0, -K % BLOCK))
    return f.reshape(*f.shape[:-1], -1, BLOCK)


def _round_blocks(f):
    """(magnitudes on the 4-bit grid, signs, exponents) of blocks [..., n, 32]."""
    top = f.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    y = torch.ldexp(f.abs(), -e)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    return (torch.round(y / step) * step).clamp(max=6.0), torch.signbit(f), e


def _pack(x):
    """MXFP4 rows of x [..., K]: packed values and scale bytes."""
    K = x.shape[-1]
    r, neg, e = _round_blocks(_blocks(x))
    code = torch.where(r <= 2, 2 * r, torch.where(r < 4, 5.0, torch.where(r < 6, 6.0, 7.0))).to(torch.uint8)
    code = code | (neg.to(torch.uint8) << 3)
    code = code.reshape(*x.shape[:-1], -1, 2)
    q = code[..., 0] | (code[..., 1] << 4)
    s = (e.squeeze(-1) + 127).to(torch.uint8)
    return q.contiguous(), torch.nn.functional.pad(s, (0, _scale_bytes(K) - s.shape[-1])).contiguous()


def _normal(g, shape, sigma):
    """bf16 normals, drawn a part at a time."""
    out = torch.empty(shape, dtype=BF16, device="cuda")
    flat = out.view(-1)
    part = 1 << 26
    for lo in range(0, flat.numel(), part):
        n = min(part, flat.numel() - lo)
        flat[lo:lo + n] = torch.randn(n, generator=g, device="cuda") * sigma
    return out


def _activations(g, shape):
    """Rows whose columns differ in size, as activations' do: a few columns are eight times the rest."""
    x = _normal(g, shape, 1.0)
    loud = torch.rand(shape[-1], generator=g, device="cuda") < 0.01
    return torch.where(loud, x * 8, x)


def _pack_many(x):
    """_pack of [E, N, K], one expert at a time."""
    parts = [_pack(w) for w in x]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def _expert_ids(g, case, n, E):
    """n expert ids: spread evenly, or skewed as a router's with some experts left out."""
    if case["load"] == "spread":
        ids = torch.arange(n, device="cuda") % E
        order = torch.randperm(E, generator=g, device="cuda")
        return order[ids][torch.randperm(n, generator=g, device="cuda")]
    used = max(1, E * 15 // 16)
    p = torch.arange(1, used + 1, device="cuda", dtype=F64) ** -1.2
    edges = torch.cumsum(p / p.sum(), 0).float()
    rank = torch.searchsorted(edges, torch.rand(n, generator=g, device="cuda")).clamp(max=used - 1)
    return torch.randperm(E, generator=g, device="cuda")[rank]


def _offsets(counts):
    return torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op in ("router", "router_train"):
        T, E, k = case["T"], case["E"], case["k"]
        dt = BF16 if case["dtype"] == "bf16" else F32
        x = (torch.randn((T, E), generator=g, device="cuda") * 1.5).to(dt)
        if case["lowest"]:
            x[:, torch.randperm(E, generator=g, device="cuda")[:case["lowest"]]] = torch.finfo(dt).min
        if case["pad"]:
            x[T - case["pad"]:] = -math.inf
        s.update(logits=x, ids=torch.empty((T, k), dtype=torch.int32, device="cuda"),
                 w=torch.empty((T, k), dtype=F32, device="cuda"), lse=torch.empty((T,), dtype=F32, device="cuda"))
        if op == "router_train":
            s.update(d_w=torch.randn((T, k), generator=g, device="cuda") / T, d_logits=torch.empty_like(x),
                     d_losses=torch.tensor([0.01, 0.001], device="cuda"))
        return s
    if op == "quant":
        shape = (case["rows"], case["K"]) if case["layout"] == "rows" else (case["E"], case["K"], case["rows"])
        x = _activations(g, shape) if case["layout"] == "rows" else _normal(g, shape, 0.02)
        lead = (case["rows"],) if case["layout"] == "rows" else (case["E"], case["rows"])
        s.update(x=x, q=torch.empty(lead + (_row_bytes(case["K"]),), dtype=torch.uint8, device="cuda"),
                 scales=torch.empty(lead + (_scale_bytes(case["K"]),), dtype=torch.uint8, device="cuda"),
                 out=torch.empty(lead + (case["K"],), dtype=BF16, device="cuda"))
        return s
    E = case["E"]
    if op == "product":
        M = case["M"]
        counts = torch.bincount(_expert_ids(g, case, M, E), minlength=E)
        s["x"] = _pack(_activations(g, (M + case["spare"], case["K"])))
        s["w"] = _pack_many(_normal(g, (E, case["N"], case["K"]), 0.02))
        s["out"] = torch.zeros((M + case["spare"], case["N"]), dtype=BF16, device="cuda")
    else:
        T, k = case["T"], case["k"]
        ids = _expert_ids(g, case, T * k, E)
        ids[torch.rand(T * k, generator=g, device="cuda") < case["drop"] / 100] = E
        counts = torch.bincount(ids, minlength=E + 1)[:E]
        # the dispatch order as the permutation writes it: slots sorted by expert, the dropped ones behind
        s["perm"] = torch.sort(ids, stable=True)[1].to(torch.int32)
        s["x"] = _pack(_activations(g, (T, case["d"])))
        s["w"] = _pack_many(_normal(g, (E, 2 * case["h"], case["d"]), 0.02))
        s["out"] = torch.zeros((T * k, case["h"]), dtype=BF16, device="cuda")
    s["offsets"] = _offsets(counts)
    s["bounds"] = s["offsets"].tolist()  # the plain form's plan: its loop over experts needs the counts on the host
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _route(x, k, renorm):
    f = x.float()
    m = f.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    top, ids = torch.sort(f, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    kept = top > -math.inf
    total = torch.exp(f - m).sum(1, keepdim=True)
    part = torch.exp(top - m)
    denom = part.sum(1, keepdim=True) if renorm else total
    w = part / torch.where(denom > 0, denom, torch.ones_like(denom))
    return torch.where(kept, ids, -1).to(torch.int32), w, (m + torch.log(total)).squeeze(1)


def _route_train(s):
    x, k, E = s["logits"], s["k"], s["E"]
    ids, w, lse = _route(x, k, s["renorm"])
    kept = ids >= 0
    live = lse > -math.inf
    tokens = live.sum()
    n = tokens.clamp(min=1).float()
    p = torch.where(live[:, None], torch.exp(x.float() - lse[:, None]), 0.0)
    counts = torch.bincount(torch.where(kept, ids, E).reshape(-1).long(), minlength=E + 1)[:E]
    share = counts.float() / counts.sum().clamp(min=1)
    mean = (p.double().sum(0) / n).float()
    z = (torch.where(live, lse, 0.0).double() ** 2).sum() / n
    losses = torch.stack([E * (share.double() * mean).sum(), z]).float()
    c = s["d_losses"][0] * E * share / n
    dz = 2 * s["d_losses"][1] * torch.where(live, lse, 0.0) / n
    d = p * (c - (p * c).sum(1, keepdim=True) + dz[:, None])
    gw = torch.where(kept, s["d_w"] * w, 0.0)
    if s["renorm"]:
        part = gw - w * gw.sum(1, keepdim=True)
    else:
        part = gw
        d = d - p * gw.sum(1, keepdim=True)
    d = d.scatter_add(1, ids.clamp(min=0).long(), torch.where(kept, part, 0.0))
    return dict(ids=ids, w=w, lse=lse, counts=counts.to(torch.int32), tokens=tokens.to(torch.int32).reshape(1),
                prob_mean=mean, losses=losses, d_logits=d.to(x.dtype))


def _quant(s):
    x = s["x"].transpose(1, 2) if s["layout"] == "in_out" else s["x"]
    f = _blocks(x)
    r, neg, e = _round_blocks(f)
    v = torch.ldexp(torch.where(neg, -r, r), e)
    v = torch.where(f.isfinite().all(-1, keepdim=True), v, math.nan)
    return v.reshape(*x.shape[:-1], -1)[..., :x.shape[-1]].to(BF16)


GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _values(q, scales, K):
    """float32 values of packed rows."""
    grid = torch.tensor(GRID, device=q.device)
    code = torch.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1, BLOCK)
    v = torch.ldexp(grid[code.int()], scales[..., :code.shape[-2], None].int() - 127)
    return v.reshape(*q.shape[:-1], -1)[..., :K]


def _experts(bounds):
    return [(e, bounds[e], bounds[e + 1]) for e in range(len(bounds) - 1) if bounds[e + 1] > bounds[e]]


def _product(s):
    # the groups are ragged: a padded batch would multiply several times the rows, so one product an expert
    x = _values(*s["x"], s["K"])
    for e, lo, hi in _experts(s["bounds"]):
        s["out"][lo:hi] = (x[lo:hi] @ _values(s["w"][0][e], s["w"][1][e], s["K"]).T).to(BF16)
    return s["out"]


def _up(s):
    x = _values(*s["x"], s["d"])
    rows = s["perm"].long() // s["k"]
    for e, lo, hi in _experts(s["bounds"]):
        u = x[rows[lo:hi]] @ _values(s["w"][0][e], s["w"][1][e], s["d"]).T
        g, u = u[:, :s["h"]], u[:, s["h"]:]
        s["out"][lo:hi] = (g / (1 + torch.exp(-g)) * u).to(BF16)
    return s["out"]


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    s = state
    op = s["op"]
    if own:
        import ragged_grouped_gemm_histogram_amd as moe

        if op == "router":
            r = moe.moe_router_topk(s["logits"], s["k"], renormalize=s["renorm"], expert_ids=s["ids"],
                                    routing_w=s["w"], lse=s["lse"])
            return dict(ids=r.expert_ids, w=r.routing_w, lse=r.lse)
        if op == "router_train":
            r = moe.moe_router_topk_losses(s["logits"], s["k"], renormalize=s["renorm"], expert_ids=s["ids"],
                                           routing_w=s["w"], lse=s["lse"])
            d = moe.moe_router_backward(s["logits"], r, s["d_w"], s["d_losses"], d_logits=s["d_logits"])
            return dict(ids=r.expert_ids, w=r.routing_w, lse=r.lse, counts=r.counts, tokens=r.tokens,
                        prob_mean=r.prob_mean, losses=r.losses, d_logits=d)
        if op == "quant":
            if s["layout"] == "in_out":
                m = moe.moe_mxfp4_quantize_weights(s["x"], "in_out", q=s["q"], scales=s["scales"])
            else:
                m = moe.moe_mxfp4_quantize(s["x"], q=s["q"], scales=s["scales"])
            return moe.moe_mxfp4_dequantize(m, x=s["out"])
        if op == "product":
            return moe.moe_grouped_projection_mxfp4(moe.Mxfp4(*s["x"], s["K"]), s["offsets"],
                                                    moe.Mxfp4(*s["w"], s["K"]), y=s["out"])
        return moe.moe_gemm_up_swiglu_mxfp4(moe.Mxfp4(*s["x"], s["d"]), s["offsets"], moe.Mxfp4(*s["w"], s["d"]),
                                            perm=s["perm"], k=s["k"], h_buf=s["out"])
    if op == "router":
        ids, w, lse = _route(s["logits"], s["k"], s["renorm"])
        return dict(ids=ids, w=w, lse=lse)
    if op == "router_train":
        return _route_train(s)
    return {"quant": _quant, "product": _product, "up": _up}[op](s)


# ------------------------------------------------------------------------------------------------ what a pass needs

def _experts_used(case, n):
    """Experts that get rows, on average over the inputs: those whose weights have to be read."""
    E = case["E"]
    if case["load"] == "spread":
        return min(E, n)
    used = max(1, E * 15 // 16)
    total = sum(r ** -1.2 for r in range(1, used + 1))
    return sum(1 - (1 - r ** -1.2 / total) ** n for r in range(1, used + 1))


def work(case):
    op = case["op"]
    if op in ("router", "router_train"):
        T, E, k = case["T"], case["E"], case["k"]
        logits = T * E * (2 if case["dtype"] == "bf16" else 4)
        out = T * k * 8 + T * 4
        if op == "router":
            return dict(bytes=logits + out, flops=T * E * 4)
        # the logits once, their gradient once, the gradients of the weights and losses in, the statistics out
        return dict(bytes=2 * logits + out + T * k * 4 + 8 + E * 8 + 12, flops=T * E * 14)
    if op == "quant":
        n = case["rows"] * case["K"] * case["E"]
        return dict(bytes=4 * n, flops=4 * n)
    if op == "product":
        M, K, N = case["M"], case["K"], case["N"]
        packed = _row_bytes(K) + -(-K // BLOCK)
        return dict(bytes=M * packed + _experts_used(case, M) * N * packed + M * N * 2 + 4 * case["E"] + 4,
                    flops=2 * M * K * N)
    T, k, d, h = case["T"], case["k"], case["d"], case["h"]
    M = T * k * (100 - case["drop"]) // 100
    packed = _row_bytes(d) + -(-d // BLOCK)
    return dict(bytes=min(T, M) * packed + _experts_used(case, M) * 2 * h * packed + M * h * 2 + 4 * M + 4 * case["E"] + 4,
                flops=4 * M * d * h + 5 * M * h)


# ------------------------------------------------------------------------------------------------ 64 bits

def _exact_values(q, scales, K):
    """float64 values of packed rows, from the bits: magnitude (1 + m/2) 2^(x-1), or m/2 where the exponent bits x are 0."""
    nib = torch.empty(*q.shape, 2, dtype=torch.int64, device=q.device)
    nib[..., 0] = q.long() % 16
    nib[..., 1] = q.long() // 16
    nib = nib.reshape(*q.shape[:-1], -1)[..., :K]
    m, ex, sign = (nib % 2).double(), nib // 2 % 4, 1.0 - 2.0 * (nib // 8).double()
    mag = torch.where(ex == 0, m / 2, (1 + m / 2) * torch.pow(2.0, (ex - 1).double()))
    scale = torch.pow(2.0, scales.double() - 127)
    return sign * mag * torch.repeat_interleave(scale, BLOCK, -1)[..., :K]


def _exact_router(s, train):
    x, k, E = s["logits"].double(), s["k"], s["E"]
    T = x.shape[0]
    lse = torch.logsumexp(x, 1)
    p = torch.softmax(x, 1).nan_to_num(0.0)
    # the k largest, the lowest index first among equals: rank by (value, -index)
    rank = torch.argsort(-x, dim=1, stable=True)
    ids = rank[:, :k]
    keep = torch.gather(x, 1, ids) != -math.inf
    pk = torch.gather(p, 1, ids) * keep
    w = pk / pk.sum(1, keepdim=True).clamp(min=1e-300) if s["renorm"] else pk
    out = dict(ids=torch.where(keep, ids, -1).to(torch.int32), w=w, lse=lse)
    if not train:
        return out
    live = ~torch.isinf(lse)
    n = max(1, int(live.sum()))
    onehot = torch.zeros((T, E), dtype=F64, device=x.device).scatter_(1, ids, keep.double())
    counts = onehot.sum(0)
    f = counts / max(1.0, float(counts.sum()))
    mean = p.sum(0) / n
    lz = torch.where(live, lse, torch.zeros_like(lse))
    db, dz = (float(v) for v in s["d_losses"].double())
    # dL/dp of the balance loss is the same for every token; softmax's Jacobian is diag(p) - p p^T
    a = (db * E * f / n).expand(T, E)
    g = s["d_w"].double() * keep
    if s["renorm"]:
        # softmax over the chosen experts alone
        chosen = torch.zeros((T, E), dtype=F64, device=x.device).scatter_(1, ids, w * (g - (g * w).sum(1, keepdim=True)))
    else:
        a = a + torch.zeros((T, E), dtype=F64, device=x.device).scatter_(1, ids, g)
        chosen = torch.zeros((), dtype=F64, device=x.device)
    d = p * a - p * (p * a).sum(1, keepdim=True) + chosen + p * (2 * dz * lz / n)[:, None]
    out.update(counts=counts.to(torch.int32), tokens=live.sum().to(torch.int32).reshape(1), prob_mean=mean,
               losses=torch.stack([E * (f * mean).sum(), (lz ** 2).sum() / n]), d_logits=d)
    return out


def _exact_quant(s):
    x = s["x"].double()
    if s["layout"] == "in_out":
        x = x.permute(0, 2, 1)
    grid = torch.tensor(GRID[:8], dtype=F64, device=x.device)
    out = torch.empty(x.shape, dtype=F64, device=x.device)
    K = x.shape[-1]
    for lo in range(0, K, BLOCK):
        b = x[..., lo:lo + BLOCK]
        top = b.abs().amax(-1, keepdim=True)
        # the power of two at or below the largest magnitude, found among the powers of two themselves
        e = torch.floor(torch.log2(torch.where(top > 0, top, 2.0 ** -133)))
        e = torch.where(torch.pow(2.0, e) > top, e - 1, e)
        e = torch.where(torch.pow(2.0, e + 1) <= top, e + 1, e)
        scale = torch.pow(2.0, (e - 2).clamp(min=-127.0))
        y = b.abs() / scale
        # the nearest grid value; halfway between two neighbours the one whose code is even
        near = torch.zeros_like(y)
        for c in range(7):
            mid = (grid[c] + grid[c + 1]) / 2
            up = y > mid if c % 2 == 0 else y >= mid
            near = torch.where(up, grid[c + 1], near)
        out[..., lo:lo + BLOCK] = torch.copysign(near, b) * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("router", "router_train"):
        return _exact_router(s, op == "router_train")
    if op == "quant":
        return _exact_quant(s)
    out = torch.zeros(s["out"].shape, dtype=F64, device="cuda")
    K = case["K"] if op == "product" else case["d"]
    x = _exact_values(*s["x"], K)
    off = s["offsets"].tolist()
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        w = _exact_values(s["w"][0][e], s["w"][1][e], K)
        if op == "product":
            out[lo:hi] = torch.matmul(x[lo:hi], w.transpose(0, 1))
        else:
            r = torch.matmul(x[torch.div(s["perm"][lo:hi].long(), case["k"], rounding_mode="floor")], w.transpose(0, 1))
            gate, val = r[:, :case["h"]], r[:, case["h"]:]
            out[lo:hi] = gate * torch.sigmoid(gate) * val
    return out
