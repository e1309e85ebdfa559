"""Cases of the operators around the experts: inputs, plain forms, what each has to move and compute, and 64-bit results.

* ``norm``: what stands before and after a block on the residual stream. Before: n = RMSNorm(r) w. After, for the
  block's output y: r' = a r + b gate RMSNorm(y) w_post and, for the block behind it, n = RMSNorm(r') w_next, of one
  read; both norms, the gate (a number a token or a channel) and the scales a and b may be left out.
* ``norm_back``: the gradients of all of these from those of r' and n.
* ``adamw``: one AdamW step over a list of tensors, moments in 32 bits or in 8, with or without 32-bit copies of the
  parameters.
* ``int4``: one grouped projection of bf16 rows by 4-bit expert weights with group scales; ``int4_up``: the grouped
  gate/up projection of token rows read through the dispatch order, with SwiGLU.

Moments in 8 bits share a power of two per 32 consecutive values, kept as a byte (exponent + 127; 255: the block holds
an infinity or a NaN and reads as NaN). The first moment's values are float8 e4m3, scaled so that the block's largest is
in [128, 256), rounded to nearest even. The second's are codes c of (1 + (c % 8) / 8) 2^(c // 8), 0 for c = 0, scaled so
that the largest has c // 8 = 30; what is above zero gets at least code 1. Given a seed, they are rounded up or down at
random in proportion, as are bf16 parameters without a 32-bit copy; the random bits of a value are a hash of seed, step
and place. The tensors' moments lie in one buffer, each tensor from a multiple of 32 on.

4-bit weights: w = s (q - z), q packed two a byte, the even one in the low half, rows of 16 * ceil(K / 32) bytes; s
(bf16) and z (a byte; 8 where there is none) for each group of consecutive values of the contraction, [E, groups, N].
"""

import math

import torch

own = False

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
EPS = 1e-6


def listed():
    return [
        # between two blocks of a decode step of four sequences: latency alone
        dict(name="norm_decode", op="norm", T=4, d=2048, stream="bf16", weights="bf16", branch=True, post=False,
             gate="none", next=True, a=1.0, b=1.0),
        # between two blocks of a prefill batch: norms on both sides, a shared expert's gate for each token
        dict(name="norm_prefill", op="norm", T=8192, d=2048, stream="bf16", weights="bf16", branch=True, post=True,
             gate="token", next=True, a=1.0, b=1.0),
        # the norm before a block in a short odd training batch, its gradient joined with the stream's
        dict(name="norm_back_before", op="norm_back", T=1025, d=392, stream="bf16", weights="f32", branch=False,
             post=False, gate="none", next=True, a=1.0, b=1.0),
        # a training batch on a stream in 32 bits, learned scales for each channel
        dict(name="norm_back_f32", op="norm_back", T=8191, d=2880, stream="f32", weights="bf16", branch=True, post=True,
             gate="channel", next=True, a=0.9, b=0.5),
        # router and norm weights of a layer, all in 32 bits
        dict(name="adamw_small", op="adamw", sizes="router", p="f32", g="f32", bits=32, master=False, seed=-1),
        # sixteen experts of 2880 x 2880, bf16 with 32-bit copies
        dict(name="adamw_experts", op="adamw", sizes="experts:16,2880,2880", p="bf16", g="bf16", bits=32, master=True,
             seed=-1),
        # sixty-four experts of 2048 x 768, bf16 alone, moments in 8 bits, rounded at random
        dict(name="adamw8_experts", op="adamw", sizes="experts:64,2048,768", p="bf16", g="bf16", bits=8, master=False,
             seed=11),
        # tensors of many sizes, one value to a million, odd ones among them
        dict(name="adamw8_ragged", op="adamw", sizes="ragged:30,1000003", p="bf16", g="f32", bits=8, master=True, seed=-1),
        # the down projection of a decode step: four tokens, eight experts each
        dict(name="int4_decode", op="int4", M=32, spare=0, E=128, K=768, N=2048, group=128, zeros=True, load="spread"),
        # ragged rows, the contraction ends inside a group, the columns inside a tile; rows behind the last stay
        dict(name="int4_ragged", op="int4", M=61, spare=3, E=8, K=392, N=520, group=32, zeros=True, load="zipf"),
        # the gate/up projection of a decode step
        dict(name="int4_up_decode", op="int4_up", T=4, k=8, E=128, d=2048, h=768, group=64, zeros=False, load="spread",
             drop=0),
        # the gate/up projection of a wide decode batch, skewed, one slot in twenty dropped
        dict(name="int4_up_batch", op="int4_up", T=256, k=8, E=64, d=2048, h=768, group=128, zeros=True, load="zipf",
             drop=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "adamw", "int4", "int4_up"])
    if op.startswith("norm"):
        d = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, min(60000, 23000000 // d))
        branch = rng.random() < 0.7
        return dict(op=op, T=T, d=d, stream=rng.choice(["bf16", "f32"]), weights=rng.choice(["bf16", "f32"]),
                    branch=branch, post=branch and rng.random() < 0.5,
                    gate=rng.choice(["none", "token", "channel"]) if branch else "none",
                    next=not branch or rng.random() < 0.7, a=rng.choice([1.0, 0.9]) if branch else 1.0,
                    b=rng.choice([1.0, 0.22]) if branch else 1.0)
    if op == "adamw":
        bits = rng.choice([8, 32])
        p = rng.choice(["bf16", "bf16", "f32"])
        kind = rng.choice(["router", "experts", "ragged"])
        if kind == "experts":
            d, h = 8 * _log(rng, 8, 360), 8 * _log(rng, 8, 360)
            kind = "experts:%d,%d,%d" % (_log(rng, 1, min(128, 390000000 // (3 * d * h))), d, h)
        elif kind == "ragged":
            kind = "ragged:%d,%d" % (rng.randint(1, 30), _log(rng, 1000, 3000000))
        return dict(op=op, sizes=kind, p=p, g=p if kind.startswith("e") else rng.choice(["bf16", "f32"]), bits=bits,
                    master=p == "bf16" and rng.random() < 0.5, seed=rng.choice([-1, 5]))
    load, group, zeros = rng.choice(["spread", "zipf"]), rng.choice([32, 64, 128]), rng.random() < 0.5
    if op == "int4":
        K, N = 8 * _log(rng, 4, 400), 8 * _log(rng, 4, 400)
        E = _log(rng, 1, min(128, 400000000 // (K * N)))
        return dict(op=op, M=_log(rng, 1, min(2048, 6000000000 // (K * N))), spare=rng.choice([0, 0, 7]), E=E, K=K, N=N,
                    group=group, zeros=zeros, load=load)
    d, h = 8 * _log(rng, 4, 360), 8 * _log(rng, 4, 200)
    E = _log(rng, 1, min(128, 400000000 // (2 * d * h)))
    k = rng.randint(1, min(E, 8))
    T = max(1, _log(rng, 1, min(2048, 6000000000 // (2 * d * h))) // k)
    return dict(op=op, T=T, k=k, E=E, d=d, h=h, group=group, zeros=zeros, load=load, drop=rng.choice([0, 0, 5]))


# ------------------------------------------------------------------------------------------------ inputs

def _dt(name):
    return BF16 if name == "bf16" else F32


def _normal(g, shape, sigma, dtype=BF16):
    """Normals, drawn a part at a time."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    part = 1 << 26
    for lo in range(0, flat.numel(), part):
        n = min(part, flat.numel() - lo)
        flat[lo:lo + n] = torch.randn(n, generator=g, device="cuda") * sigma
    return out


def _activations(g, shape, dtype=BF16):
    """Rows whose columns differ in size, as activations' do: a few columns are eight times the rest."""
    x = _normal(g, shape, 1.0, dtype)
    loud = torch.rand(shape[-1], generator=g, device="cuda") < 0.01
    return torch.where(loud, x * 8, x)


def _shapes(text):
    kind, _, rest = text.partition(":")
    if kind == "router":
        return [(128, 2048), (2048,), (2048,), (2048,)]
    n = [int(v) for v in rest.split(",")]
    if kind == "experts":
        return [(n[0], 2 * n[2], n[1]), (n[0], n[2], n[1])]
    # `n[0]` sizes spread over the logarithm from one value to n[1], with a tensor of n[1] itself
    u = torch.rand(n[0] - 1, generator=torch.Generator().manual_seed(n[1]), dtype=F64)
    return [(max(1, round(n[1] ** v)),) for v in u.tolist()] + [(n[1],)]


def _starts(sizes):
    """Where each tensor's moments begin, and how many values the buffer holds."""
    at, n = [], 0
    for s in sizes:
        at.append(n)
        n += -(-s // 32) * 32
    return at, n


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


def _int4(g, E, N, K, group, zeros):
    """Random expert weights rounded to 4 bits, one expert at a time: packed values, scales, zeros."""
    G = -(-K // group)
    q = torch.empty((E, N, 16 * (-(-K // 32))), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, G, N), dtype=BF16, device="cuda")
    z = torch.empty((E, G, N), dtype=torch.uint8, device="cuda") if zeros else None
    for e in range(E):
        w = torch.nn.functional.pad(torch.randn((N, K), generator=g, device="cuda") * 0.02, (0, G * group - K))
        w = w.view(N, G, group)
        if zeros:
            lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
            sc = ((hi - lo) / 15).to(BF16)
            zp = torch.round(-lo / sc.float()).clamp(0, 15)
            z[e] = zp.T.to(torch.uint8)
        else:
            sc = (w.abs().amax(2) / 7).to(BF16)
            zp = torch.full_like(sc, 8, dtype=F32)
        c = (torch.round(w / sc.float()[..., None]) + zp[..., None]).clamp(0, 15).to(torch.uint8).view(N, -1)[:, :K]
        c = torch.nn.functional.pad(c, (0, q.shape[2] * 2 - K)).view(N, -1, 2)
        q[e] = c[..., 0] | (c[..., 1] << 4)
        s[e] = sc.T
    return q, s, z


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op in ("norm", "norm_back"):
        T, d, st, wt = case["T"], case["d"], _dt(case["stream"]), _dt(case["weights"])
        s["r"] = _activations(g, (T, d), st)  # for norm_back the stream behind the block, as the forward wrote it
        s["y"] = _normal(g, (T, d), 0.3) if case["branch"] else None
        s["w_post"] = 1 + _normal(g, (d,), 0.2, wt) if case["post"] else None
        s["w_next"] = 1 + _normal(g, (d,), 0.2, wt) if case["next"] else None
        gates = {"none": lambda: None, "token": lambda: torch.sigmoid(torch.randn((T, 1), generator=g, device="cuda")),
                 "channel": lambda: _normal(g, (d,), 0.5, wt)}
        s["gate_w"] = gates[case["gate"]]()
        if op == "norm":
            s["out"] = torch.empty_like(s["r"]) if case["branch"] else None
            s["n"] = torch.empty((T, d), dtype=BF16, device="cuda") if case["next"] else None
        else:
            s["dr"] = _normal(g, (T, d), 1.0 / T, st)
            s["dn"] = _normal(g, (T, d), 1.0 / T) if case["next"] else None
        return s
    if op == "adamw":
        shapes = _shapes(case["sizes"])
        sizes = [math.prod(v) for v in shapes]
        s["at"], n = _starts(sizes)
        s["params"] = [_normal(g, v, 0.02, _dt(case["p"])) for v in shapes]
        s["grads"] = [_normal(g, v, 1e-3, _dt(case["g"])) for v in shapes]
        m, v = _normal(g, (n,), 3e-4, F32), _normal(g, (n,), 1e-3, F32).square_()
        for lo, size in zip(s["at"], sizes):  # nothing between the tensors
            hi = lo + -(-size // 32) * 32
            m[lo + size:hi], v[lo + size:hi] = 0, 0
        s["m"], s["v"] = (m, v) if case["bits"] == 32 else (_to_e4m3(m), _to_e5m3(v, None))
        s["master"] = None
        if case["master"]:
            s["master"] = torch.zeros(n, device="cuda")
            for p, lo in zip(s["params"], s["at"]):
                s["master"][lo:lo + p.numel()] = p.reshape(-1).float() + torch.randn(
                    p.numel(), generator=g, device="cuda") * 1e-5
        s["step"] = 1000
        s["adam"] = None
        return s
    E = case["E"]
    if op == "int4":
        M = case["M"]
        counts = torch.bincount(_expert_ids(g, case, M, E), minlength=E)
        s["x"] = _activations(g, (M + case["spare"], case["K"]))
        s["w"] = _int4(g, E, case["N"], case["K"], case["group"], case["zeros"])
        s["out"] = torch.zeros((M + case["spare"], case["N"]), dtype=BF16, device="cuda")
    else:
        T, k = case["T"], case["k"]
        ids = _expert_ids(g, case, T * k, E)
        ids[torch.rand(T * k, generator=g, device="cuda") < case["drop"] / 100] = E
        counts = torch.bincount(ids, minlength=E + 1)[:E]
        # the dispatch order as the permutation writes it: slots sorted by expert, the dropped ones behind
        s["perm"] = torch.sort(ids, stable=True)[1].to(torch.int32)
        s["x"] = _activations(g, (T, case["d"]))
        s["w"] = _int4(g, E, 2 * case["h"], case["d"], case["group"], case["zeros"])
        s["out"] = torch.zeros((T * k, case["h"]), dtype=BF16, device="cuda")
    s["offsets"] = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)).to(torch.int32)
    s["bounds"] = s["offsets"].tolist()  # the plain form's plan: its loop over experts needs the counts on the host
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _rms(x):
    return 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)


def _weight(w):
    return 1.0 if w is None else w.float()


def _norm(s):
    r = s["r"].float()
    if s["branch"]:
        u = s["y"].float()
        if s["post"]:
            u = u * _rms(u) * _weight(s["w_post"])
        r = s["a"] * r + s["b"] * _weight(s["gate_w"]) * u
    out = dict(r=r.to(s["r"].dtype)) if s["branch"] else {}
    if s["next"]:
        out["n"] = (r * _rms(r) * _weight(s["w_next"])).to(BF16)
    return out


def _norm_grad(x, w, dn):
    """Gradients of x and w through n = x rms(x) w."""
    rs = _rms(x)
    xh, h = x * rs, dn * _weight(w)
    return rs * (h - xh * (h * xh).mean(1, keepdim=True)), (dn * xh).sum(0, dtype=F64).float()


def _norm_back(s):
    out = {}
    r, d = s["r"].float(), s["dr"].float()
    if s["next"]:
        dx, out["w_next"] = _norm_grad(r, s["w_next"], s["dn"].float())
        d = d + dx
    if s["branch"]:
        y, gate = s["y"].float(), _weight(s["gate_w"])
        u = y * _rms(y) * _weight(s["w_post"]) if s["post"] else y
        if s["gate"] == "token":
            out["gate"] = s["b"] * (d * u).sum(1, keepdim=True)
        if s["gate"] == "channel":
            out["gate"] = s["b"] * (d * u).sum(0, dtype=F64).float()
        du = s["b"] * gate * d
        if s["post"]:
            du, out["w_post"] = _norm_grad(y, s["w_post"], du)
        out["y"] = du.to(BF16)
    out["r"] = (s["a"] * d).to(s["r"].dtype)
    return out


def _scale_bytes(x, top):
    """The scale byte of each block of 32: its largest magnitude's exponent field less `top`, at least 1; 255 where
    something is not finite."""
    b = x.view(-1, 32)
    field = (b.abs().amax(1).view(torch.int32) >> 23)
    return torch.where(b.isfinite().all(1), (field - top).clamp(min=1), 255).to(torch.uint8)


def _power(byte):
    """2^(byte - 127) for bytes 1 to 254."""
    return (byte.int() << 23).view(F32)


def _to_e4m3(m):
    s = _scale_bytes(m, 7)
    bad = s == 255
    y = m.view(-1, 32) * _power(254 - torch.where(bad, 1, s).int())[:, None]
    y = torch.where(bad[:, None], 0.0, y)
    step = _power((y.abs().view(torch.int32) >> 23).clamp(min=121) - 3)  # e4m3: exponents from -6, three bits
    r = torch.copysign(torch.round(y.abs() / step) * step, y)
    return r.to(torch.float8_e4m3fn).view(torch.uint8).view(-1), s


def _of_e4m3(m):
    q, s = m
    v = q.view(torch.float8_e4m3fn).float().view(-1, 32) * _power(torch.where(s == 255, 1, s))[:, None]
    return torch.where((s == 255)[:, None], math.nan, v).view(-1)


def _to_e5m3(v, bits):
    """Codes and scale bytes; `bits`: 16 random bits a value, or None for rounding to nearest even."""
    s = _scale_bytes(v, 30)
    i = v.view(torch.int32).long().view(-1, 32) - (s.long() << 23)[:, None]
    c = (i + ((1 << 19) - 1 + ((i >> 20) & 1)) if bits is None else i + (bits.view(-1, 32) << 4)) >> 20
    c = torch.where(v.view(-1, 32) > 0, c.clamp(min=1), 0)
    return torch.where((s == 255)[:, None], 0, c).to(torch.uint8).view(-1), s


def _of_e5m3(v):
    q, s = v
    c = q.view(-1, 32).int()
    x = ((c << 20) + (s.int() << 23)[:, None]).view(F32)
    return torch.where((s == 255)[:, None], math.nan, torch.where(c == 0, 0.0, x)).view(-1)


def _mix(h):
    """A hash of 32-bit values kept in 64 bits."""
    h = ((h ^ (h >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random_bits(seed, step, n):
    key = _mix(seed ^ _mix(step))
    i = torch.arange(n, device="cuda")
    return _mix(((i & 0xFFFFFFFF) + (i >> 32) * 0x9E3779B1 + key) & 0xFFFFFFFF)


def _round_random(p, bits):
    """bf16 of p, the 16 dropped bits added to a random number of as many bits; a NaN stays one."""
    i = (p.view(torch.int32).long() & 0xFFFFFFFF) + bits
    r = ((i >> 16) << 16).to(torch.int32).view(F32)
    return torch.where(p.isfinite(), r, p).to(BF16)


LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.1


def _adamw(s):
    s["step"] += 1
    t = s["step"]
    m, v = (s["m"], s["v"]) if s["bits"] == 32 else (_of_e4m3(s["m"]), _of_e5m3(s["v"]))
    n = m.numel()
    g, p = torch.zeros(n, device="cuda"), s["master"]
    p = torch.zeros(n, device="cuda") if p is None else p
    for q, d, lo in zip(s["params"], s["grads"], s["at"]):
        g[lo:lo + q.numel()] = d.reshape(-1)
        if s["master"] is None:
            p[lo:lo + q.numel()] = q.reshape(-1)
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    p = p * (1 - LR * DECAY) - m / (torch.sqrt(v) / math.sqrt(1 - BETA2 ** t) + ADAM_EPS) * (LR / (1 - BETA1 ** t))
    bits = _random_bits(s["seed"], t, n) if s["seed"] >= 0 else None
    low = p if bits is None or s["p"] == "f32" or s["master"] is not None else _round_random(p, bits & 0xFFFF)
    for q, lo in zip(s["params"], s["at"]):
        q.copy_(low[lo:lo + q.numel()].view(q.shape))
    if s["master"] is not None:
        s["master"].copy_(p)
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        for old, new in zip((*s["m"], *s["v"]), (*_to_e4m3(m), *_to_e5m3(v, None if bits is None else bits >> 16))):
            old.copy_(new)


def _adamw_out(s):
    out = dict(params=s["params"], master=s["master"])
    if s["bits"] == 32:
        return dict(out, m=s["m"], v=s["v"])
    # what the codes stand for; three bits of mantissa and a power of two fit bf16
    return dict(out, m=_of_e4m3(s["m"]).to(BF16), v=_of_e5m3(s["v"]).to(BF16))


def _values(q, sc, z, K, group):
    """float32 weights [N, K] of one expert."""
    c = torch.stack([q & 15, q >> 4], -1).view(q.shape[0], -1)[:, :K].float()
    at = torch.arange(K, device=q.device) // group
    return (c - (8.0 if z is None else z.float().T[:, at])) * sc.float().T[:, at]


def _experts(bounds):
    return [(e, bounds[e], bounds[e + 1]) for e in range(len(bounds) - 1) if bounds[e + 1] > bounds[e]]


def _int4_product(s):
    # the groups are ragged: a padded batch would multiply several times the rows, so one product an expert
    up = s["op"] == "int4_up"
    x, (q, sc, z) = s["x"].float(), s["w"]
    K = x.shape[1]
    for e, lo, hi in _experts(s["bounds"]):
        rows = x[s["perm"][lo:hi].long() // s["k"]] if up else x[lo:hi]
        r = rows @ _values(q[e], sc[e], None if z is None else z[e], K, s["group"]).T
        if up:
            g, u = r[:, :s["h"]], r[:, s["h"]:]
            r = g / (1 + torch.exp(-g)) * u
        s["out"][lo:hi] = r.to(BF16)
    return s["out"]


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    s = state
    op = s["op"]
    if own:
        import ragged_grouped_gemm_histogram_amd as moe

        if op == "norm":
            if not s["branch"]:
                return dict(n=moe.moe_rmsnorm(s["r"], s["w_next"], eps=EPS, y=s["n"]))
            r, n = moe.moe_residual_norm(s["y"], s["r"], post_norm=s["post"], w_post=s["w_post"], gate=s["gate_w"],
                                         residual_scale=s["a"], branch_scale=s["b"], next_norm=s["next"],
                                         w_next=s["w_next"], eps=EPS, r_out=s["out"], n_out=s["n"])
            return dict(r=r, n=n) if s["next"] else dict(r=r)
        if op == "norm_back":
            if not s["branch"]:
                dx, dw = moe.moe_rmsnorm_backward(s["dn"], s["r"], s["w_next"], eps=EPS, dx_add=s["dr"])
                return dict(r=dx, w_next=dw)
            b = moe.moe_residual_norm_backward(s["dr"], s["dn"], s["y"], s["r"], post_norm=s["post"], w_post=s["w_post"],
                                               gate=s["gate_w"], residual_scale=s["a"], branch_scale=s["b"],
                                               next_norm=s["next"], w_next=s["w_next"], eps=EPS)
            out = dict(r=b.d_r, y=b.d_y, gate=b.d_gate, w_post=b.d_w_post, w_next=b.d_w_next)
            return {k: v for k, v in out.items() if v is not None}
        if op == "adamw":
            if s["adam"] is None:  # the optimizer's state, which a program makes once
                moments = (s["m"], s["v"]) if s["bits"] == 32 else (moe.Blocks8(*s["m"]), moe.Blocks8(*s["v"]))
                s["adam"] = moe.AdamW(s["params"], *moments, master=s["master"])
            s["step"] += 1
            moe.moe_adamw_step(s["adam"], s["grads"], lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=DECAY,
                               step=s["step"], seed=s["seed"] if s["seed"] >= 0 else None)
            if s["bits"] == 32:
                return _adamw_out(s)
            m, v = moe.moe_adamw_moments(s["adam"])
            return dict(params=s["params"], master=s["master"], m=m, v=v)
        w = moe.Int4(*s["w"], s["K"] if op == "int4" else s["d"], s["group"])
        if op == "int4":
            return moe.moe_grouped_projection_int4(s["x"], s["offsets"], w, y=s["out"])
        return moe.moe_gemm_up_swiglu_int4(s["x"], s["offsets"], w, perm=s["perm"], k=s["k"], h_buf=s["out"])
    if op == "norm":
        return _norm(s)
    if op == "norm_back":
        return _norm_back(s)
    if op == "adamw":
        _adamw(s)
        return _adamw_out(s)
    return _int4_product(s)


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
    if op in ("norm", "norm_back"):
        n, st = case["T"] * case["d"], 2 if case["stream"] == "bf16" else 4
        if op == "norm":
            moved = st + (2 + st if case["branch"] else 0) + (2 if case["next"] else 0)
        else:
            moved = 3 * st + (4 if case["branch"] else 0) + (2 if case["next"] else 0)
        return dict(bytes=n * moved + 16 * case["d"], flops=n * (12 if op == "norm" else 30))
    if op == "adamw":
        shapes = _shapes(case["sizes"])
        n = sum(math.prod(v) for v in shapes)
        p, g = (2 if case[k] == "bf16" else 4 for k in ("p", "g"))
        moments = 16 if case["bits"] == 32 else 4 + 4 / 32
        out = 0 if case["bits"] == 32 else 4 + 2 + 2 / 32  # the moments' values: read once more and written as bf16
        return dict(bytes=int(n * (g + (p + 8 if case["master"] else 2 * p) + moments + out)), flops=n * 16)
    up = op == "int4_up"
    K, N = (case["d"], 2 * case["h"]) if up else (case["K"], case["N"])
    M = case["T"] * case["k"] * (100 - case["drop"]) // 100 if up else case["M"]
    rows = min(case["T"], M) if up else M
    groups = -(-K // case["group"]) * (3 if case["zeros"] else 2)
    return dict(bytes=int(rows * K * 2 + _experts_used(case, M) * N * (K / 2 + groups) + M * N * (1 if up else 2)
                          + (4 * M if up else 0) + 4 * case["E"] + 4), flops=2 * M * K * N)


# ------------------------------------------------------------------------------------------------ 64 bits

def _exact_forward(r, y, w_post, w_next, gate, a, b, post, nxt):
    def unit(x):
        return x / (x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS).sqrt()

    if y is not None:
        u = unit(y) if post else y
        u = u * w_post if w_post is not None else u
        u = u * gate if gate is not None else u
        r = a * r + b * u
    n = None
    if nxt:
        n = unit(r) * w_next
    return r, n


def _exact_norm(s, back):
    def leaf(x):
        return None if x is None else x.double().requires_grad_(back)

    r, y, wp, wn, gate = (leaf(s[k]) for k in ("r", "y", "w_post", "w_next", "gate_w"))
    if not back:
        out, n = _exact_forward(r, y, wp, wn, gate, s["a"], s["b"], s["post"], s["next"])
        full = dict(r=out if s["branch"] else None, n=n)
        return {k: v for k, v in full.items() if v is not None}
    # the stream behind the block is an input: its norm's part first, then the block's with all of its gradient
    d = s["dr"].double()
    out = {}
    if s["next"]:
        _, n = _exact_forward(r, None, None, wn, None, 1, 1, False, True)
        dr, out["w_next"] = torch.autograd.grad((n * s["dn"].double()).sum(), (r, wn))
        d = d + dr
    if s["branch"]:
        r0 = torch.zeros_like(d)
        res, _ = _exact_forward(r0, y, wp, None, gate, s["a"], s["b"], s["post"], False)
        asked = {k: v for k, v in (("y", y), ("w_post", wp), ("gate", gate)) if v is not None}
        out.update(zip(asked, torch.autograd.grad((res * d).sum(), list(asked.values()))))
    out["r"] = d * s["a"]
    return out


def _exact_scale(byte):
    return torch.repeat_interleave(torch.where(byte == 255, math.nan, torch.pow(2.0, byte.double() - 127)), 32)


def _exact_adamw(s):
    t = s["step"] + 1
    if s["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        (mq, ms), (vq, vs) = s["m"], s["v"]
        m = mq.view(torch.float8_e4m3fn).to(F64) * _exact_scale(ms)
        c = vq.long()
        v = (c > 0) * (1 + (c % 8).double() / 8) * torch.pow(2.0, (c // 8).double()) * _exact_scale(vs)
    params = []
    master = None if s["master"] is None else s["master"].double()
    for q, d, lo in zip(s["params"], s["grads"], s["at"]):
        at = slice(lo, lo + q.numel())
        g = d.reshape(-1).double()
        p = q.reshape(-1).double() if master is None else master[at]
        m[at] += (1 - BETA1) * (g - m[at])
        v[at] += (1 - BETA2) * (g * g - v[at])
        m_hat, v_hat = m[at] / (1 - BETA1 ** t), v[at] / (1 - BETA2 ** t)
        p = p - LR * DECAY * p - LR * m_hat / (v_hat.sqrt() + ADAM_EPS)
        if master is not None:
            master[at] = p
        params.append(p.view(q.shape))
    if s["bits"] == 8:
        # rounded at random there is no one value; and of bf16 gradients 0.9 m + 0.1 g falls midway between two codes in
        # one value of a hundred, where the last bit of the constants decides
        m = v = None
    return dict(params=params, master=master, m=m, v=v)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_back"):
        return _exact_norm(s, op == "norm_back")
    if op == "adamw":
        return _exact_adamw(s)
    out = torch.zeros(s["out"].shape, dtype=F64, device="cuda")
    x, (q, sc, z) = s["x"].double(), s["w"]
    K, group = x.shape[1], case["group"]
    off = s["offsets"].tolist()
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        w = torch.empty((q.shape[1], 2 * q.shape[2]), dtype=F64, device="cuda")
        w[:, 0::2] = q[e] % 16
        w[:, 1::2] = torch.div(q[e], 16, rounding_mode="floor")
        w = w[:, :K].contiguous()
        for j in range(sc.shape[1]):
            part = w[:, j * group:(j + 1) * group]
            part -= 8.0 if z is None else z[e, j].double()[:, None]
            part *= sc[e, j].double()[:, None]
        if op == "int4":
            out[lo:hi] = torch.matmul(x[lo:hi], w.transpose(0, 1))
        else:
            token = torch.div(s["perm"][lo:hi].long(), case["k"], rounding_mode="floor")
            r = torch.matmul(x[token], w.transpose(0, 1))
            gate, val = r[:, :case["h"]], r[:, case["h"]:]
            out[lo:hi] = gate * torch.sigmoid(gate) * val
    return out
