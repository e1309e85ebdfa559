"""Router and MXFP4 calls where indexes pass 2^31, workgroups run through many tiles, or two streams work at once.

Every result of a row depends on that row alone (and on its expert), in the same order of operations whatever else the
call holds, so a large call's rows equal, bit for bit, those of a small call on a copy of them. The small calls are held
to the 64-bit reference elsewhere.
"""

import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def random_mxfp4(g, shape, K):
    """Random codes and scale bytes of mixed sizes: [..., rows] of K values."""
    q = torch.randint(0, 256, (*shape, moe.mxfp4_row_bytes(K)), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.randint(118, 126, (*shape, moe.mxfp4_scale_bytes(K)), generator=g, device=DEV, dtype=torch.uint8)
    return moe.Mxfp4(q, s, K)


def rows_of(m, idx):
    return moe.Mxfp4(m.q[idx].contiguous(), m.scales[idx].contiguous(), m.width)


def offsets_of(counts):
    return torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32, device=DEV)


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def picked(n, rows, g):
    idx = torch.randint(0, rows, (n,), generator=g, device=DEV)
    return torch.unique(torch.cat([idx, torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device=DEV)]))


@pytest.mark.timeout(300)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_router_more_than_2_31_logits(dtype):
    E, k = 1024, 2
    T = 2 ** 21 + 5
    say(f"[gpu] router T={T} E={E} {dtype}")
    g = generator(1)
    x = torch.empty((T, E), dtype=dtype, device=DEV).normal_(generator=g)
    r = moe.moe_router_topk_losses(x, k)
    plain = moe.moe_router_topk(x, k)
    dw, dl = torch.randn((T, k), generator=g, device=DEV), torch.tensor([0.5, 0.25], device=DEV)
    d = moe.moe_router_backward(x, r, dw, dl)
    assert r.tokens.item() == T and torch.equal(r.counts.long(), torch.bincount(r.expert_ids.reshape(-1), minlength=E))
    idx = picked(500, T, g)
    xs = x[idx].contiguous()
    s = moe.moe_router_topk(xs, k)
    for f in ("expert_ids", "routing_w", "lse"):
        assert torch.equal(getattr(r, f)[idx], getattr(s, f)) and torch.equal(getattr(plain, f)[idx], getattr(s, f))
    s.counts, s.tokens = r.counts, r.tokens
    assert torch.equal(d[idx], moe.moe_router_backward(xs, s, dw[idx].contiguous(), dl))


@pytest.mark.timeout(300)
def test_quantise_more_than_2_31_values():
    K = 2048
    R = 2 ** 20 + 7
    say(f"[gpu] quantise {R} x {K}")
    g = generator(2)
    x = torch.empty((R, K), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    m = moe.moe_mxfp4_quantize(x)
    back = moe.moe_mxfp4_dequantize(m)
    idx = picked(500, R, g)
    s = moe.moe_mxfp4_quantize(x[idx].contiguous())
    assert torch.equal(m.q[idx], s.q) and torch.equal(m.scales[idx], s.scales)
    assert torch.equal(back[idx], moe.moe_mxfp4_dequantize(s))
    del x, m, back
    E, n = 9, 16384
    w = torch.empty((E, n, n), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    for layout in ("in_out", "out_in"):
        m = moe.moe_mxfp4_quantize_weights(w, layout)
        s = moe.moe_mxfp4_quantize_weights(w[E - 1:], layout)
        assert torch.equal(m.q[E - 1:], s.q) and torch.equal(m.scales[E - 1:], s.scales)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("rows", [40, 3000])
def test_products_with_weights_past_4_gib(rows):
    """72 experts of 65536 rows of 2048 values (4.8 GB): only the first and the last have rows."""
    E, N, K = 72, 65536, 2048
    say(f"[gpu] mxfp4 products, {rows} rows, 4.8 GB of weights")
    g = generator(3)
    w = random_mxfp4(g, (E, N), K)
    x = random_mxfp4(g, (rows,), K)
    first = rows // 3
    off = offsets_of([first, *[0] * (E - 2), rows - first])
    ends = moe.Mxfp4(w.q[[0, E - 1]], w.scales[[0, E - 1]], K)
    # (the small call takes the same kernel: rows per expert below 32, or far above, in both)
    pair = offsets_of([first, rows - first])
    y = moe.moe_grouped_projection_mxfp4(x, off, w)
    assert y.isfinite().all() and y.any()
    assert torch.equal(y, moe.moe_grouped_projection_mxfp4(x, pair, ends))
    assert torch.equal(moe.moe_gemm_up_swiglu_mxfp4(x, off, w), moe.moe_gemm_up_swiglu_mxfp4(x, pair, ends))


@pytest.mark.timeout(300)
def test_gathered_tokens_past_2_gib():
    """Token rows that 32-bit offsets from the first one do not reach are read all the same."""
    K, h, E = 8192, 64, 2
    T = 2 ** 31 // moe.mxfp4_row_bytes(K) + 301
    say(f"[gpu] mxfp4 gate/up gathered from {T} tokens of {K}")
    g = generator(4)
    x = random_mxfp4(g, (T,), K)
    w = random_mxfp4(g, (E, 2 * h), K)
    perm = torch.randperm(T, generator=g, device=DEV).int()
    cut = T // 3
    off = offsets_of([cut, T - cut])
    out = moe.moe_gemm_up_swiglu_mxfp4(x, off, w, perm=perm, k=1)
    fused = moe.moe_gemm_up_swiglu_mxfp4_q(x, off, w, perm=perm, k=1)
    for lo, hi, e in ((0, cut, 0), (cut, T, 1)):
        far = perm[lo:hi].topk(10)[1] + lo  # the last tokens
        p = torch.cat([far, torch.tensor([lo, hi - 1], device=DEV)])
        small = moe.moe_gemm_up_swiglu_mxfp4(rows_of(x, perm[p].long()), offsets_of([len(p)]),
                                             moe.Mxfp4(w.q[e:e + 1], w.scales[e:e + 1], K))
        assert torch.equal(out[p], small)
        q = moe.moe_mxfp4_quantize(small)
        assert torch.equal(fused.q[p], q.q) and torch.equal(fused.scales[p], q.scales)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("K", [512, 520])
def test_more_tiles_than_a_workgroup_lists_at_once(K):
    """Over 64 tiles of 256 x 256 a workgroup (the coordinates are worked out 64 at a time)."""
    N, counts = 16384, [20000, 0, 700, 46200]
    M = sum(counts)
    assert sum(-(-c // 256) for c in counts) * (N // 256) > 64 * torch.cuda.get_device_properties(0).multi_processor_count
    say(f"[gpu] mxfp4 products, {M} x {N} x {K}")
    g = generator(5)
    E = len(counts)
    x, w = random_mxfp4(g, (M,), K), random_mxfp4(g, (E, N), K)
    off = offsets_of(counts)
    y = moe.moe_grouped_projection_mxfp4(x, off, w)
    perm = torch.randperm(M, generator=g, device=DEV).int()
    up = moe.moe_gemm_up_swiglu_mxfp4(x, off, w, perm=perm, k=1)
    fused = moe.moe_gemm_up_swiglu_mxfp4_q(x, off, w, perm=perm, k=1)
    q = moe.moe_mxfp4_quantize(up)
    assert torch.equal(fused.q, q.q) and torch.equal(fused.scales, q.scales)
    lo = 0
    for e, c in enumerate(counts):
        one = moe.Mxfp4(w.q[e:e + 1], w.scales[e:e + 1], K)
        for a in range(lo, lo + c, 16384):
            b = min(a + 16384, lo + c)
            n = offsets_of([b - a])
            assert torch.equal(y[a:b], moe.moe_grouped_projection_mxfp4(rows_of(x, slice(a, b)), n, one)), (e, a)
            rows = rows_of(x, perm[a:b].long())
            assert torch.equal(up[a:b], moe.moe_gemm_up_swiglu_mxfp4(rows, n, one)), (e, a)
        lo += c


def test_two_streams_at_once():
    """Two layers on two streams, each with its own buffers, give what one after the other gives."""
    say("[gpu] router and mxfp4 step on two streams")
    T, k, E, d, h = 2048, 4, 32, 520, 264
    g = generator(6)
    layers = []
    for _ in range(2):
        w = [torch.randn((E, *s), generator=g, device=DEV).mul_(0.1).bfloat16() for s in ((2 * h, d), (h, d))]
        layers.append((torch.randn((T, d), generator=g, device=DEV).bfloat16(), torch.randn((T, E), generator=g, device=DEV),
                       moe.moe_mxfp4_quantize_weights(w[0], "out_in"), moe.moe_mxfp4_quantize_weights(w[1], "in_out")))

    def step(x, logits, w_ug, w_down):
        r = moe.moe_router_topk_losses(logits, k)
        y, _ = moe.moe_expert_forward_mxfp4(x, r.expert_ids, r.routing_w, w_ug, w_down)
        d_logits = moe.moe_router_backward(logits, r, torch.ones_like(r.routing_w), torch.ones(2, device=DEV))
        return y, r.losses, r.counts, d_logits

    want = [step(*a) for a in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*layers[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@pytest.mark.parametrize("renormalize", [True, False])
def test_router_gradient_of_experts_chosen_twice(renormalize):
    """Ids from elsewhere may name an expert more than once, or none: its slots' parts are added up.

    Every term is a product of fp32 numbers below 4 in size with at most k + 3 roundings behind it, and each row adds at
    most 2 k + 2 of them: (4 k + 8) u of the terms' sizes, beside the weights' own softmax of 2^-18."""
    say("[gpu] router gradient of repeated ids")
    T, E, k = 200, 24, 6
    g = generator(8)
    x = torch.randn((T, E), generator=g, device=DEV)
    r = moe.moe_router_topk(x, k, renormalize=renormalize)
    r.expert_ids = torch.randint(-1, 3, (T, k), generator=g, device=DEV, dtype=torch.int32)
    r.expert_ids[0] = 5
    r.expert_ids[1] = -1
    r.routing_w = torch.rand((T, k), generator=g, device=DEV)
    dw = torch.randn((T, k), generator=g, device=DEV)
    first, again = moe.moe_router_backward(x, r, dw), moe.moe_router_backward(x, r, dw)
    assert torch.equal(first, again)
    on = (r.expert_ids >= 0).double()
    w, d, p = r.routing_w.double() * on, dw.double(), torch.softmax(x.double(), 1)
    total = (w * d).sum(1, keepdim=True)
    slot = w * ((d - total) if renormalize else d)
    want = torch.zeros((T, E), dtype=torch.float64, device=DEV)
    size = torch.zeros_like(want)
    for j in range(k):
        want.scatter_add_(1, r.expert_ids[:, j:j + 1].clamp(min=0).long(), slot[:, j:j + 1])
        size.scatter_add_(1, r.expert_ids[:, j:j + 1].clamp(min=0).long(), w[:, j:j + 1] * (d[:, j:j + 1].abs() + (w * d.abs()).sum(1, keepdim=True)))
    if not renormalize:
        want -= p * total
        size += p * (w * d.abs()).sum(1, keepdim=True)
    assert ((first.double() - want).abs() <= size * ((4 * k + 8) * 2.0 ** -24 + 2.0 ** -18)).all()


def test_two_captured_layers_replayed_in_turn():
    """Router, MXFP4 step and router gradient of two layers, a graph each: every replay, in any order and with new
    inputs and eager work between, equals the eager calls."""
    say("[gpu] two captured router and mxfp4 layers")
    T, k, E, d, h = 640, 4, 16, 264, 136
    g = generator(9)
    layers = []
    for _ in range(2):
        w = [torch.randn((E, *s), generator=g, device=DEV).mul_(0.1).bfloat16() for s in ((2 * h, d), (h, d))]
        layers.append((torch.randn((T, d), generator=g, device=DEV).bfloat16(), torch.randn((T, E), generator=g, device=DEV),
                       torch.randn((T, k), generator=g, device=DEV),
                       moe.moe_mxfp4_quantize_weights(w[0], "out_in"), moe.moe_mxfp4_quantize_weights(w[1], "in_out")))
    dl = torch.tensor([0.01, 0.001], device=DEV)

    def step(x, logits, dw, w_ug, w_down):
        r = moe.moe_router_topk_losses(logits, k)
        y, _ = moe.moe_expert_forward_mxfp4(x, r.expert_ids, r.routing_w, w_ug, w_down)
        return y, r.losses, r.counts, moe.moe_router_backward(logits, r, dw, dl)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(s):
        for layer in layers:
            step(*layer)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                outs.append(step(*layer))
            graphs.append(graph)
    torch.cuda.current_stream().wait_stream(s)
    for rep, order in enumerate(([0, 1], [1, 0], [1, 1, 0], [0, 0, 1])):
        for x, logits, *_ in layers:
            x.copy_(torch.randn((T, d), generator=g, device=DEV))
            logits.copy_(torch.randn((T, E), generator=g, device=DEV))
        logits[rep::7] = -float("inf")
        want = [[t.clone() for t in step(*layer)] for layer in layers]
        torch.cuda.synchronize()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i])), (rep, i)
