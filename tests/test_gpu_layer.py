"""A routed layer on the residual stream: forward, backward and optimizer steps together, as a training loop runs them."""

import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def weights(T, d, h, E, stream=F32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype, sigma=1.0, mean=0.0):
        return (mean + sigma * torch.randn(shape, generator=g, device="cuda")).to(dtype)

    return dict(r=normal((T, d), stream), w_norm=normal((d,), F32, 0.1, 1.0), w_router=normal((E, d), BF16, d ** -0.5),
                w_ug=normal((E, 2 * h, d), BF16, d ** -0.5), w_down=normal((E, h, d), BF16, h ** -0.5),
                w_post=normal((d,), F32, 0.1, 1.0), w_next=normal((d,), F32, 0.1, 1.0), gate=normal((d,), F32, 0.2, 1.0))


KW = dict(post_norm=True, residual_scale=0.9, branch_scale=0.5, next_norm=True)


def forward(w, k):
    return moe.moe_layer_forward(w["r"], w["w_norm"], w["w_router"], w["w_ug"], w["w_down"], k, w_post=w["w_post"],
                                 gate=w["gate"], w_next=w["w_next"], **KW)


def unit(x, eps=1e-6):
    return x * torch.rsqrt(x.pow(2).mean(1, keepdim=True) + eps)


def reference(w, ids, k):
    """The same layer in 64 bits on the chosen experts, and its leaves."""
    p = {n: t.double().cpu().requires_grad_() for n, t in w.items()}
    n = unit(p["r"]) * p["w_norm"]
    logits = n @ p["w_router"].T
    prob = torch.softmax(logits, 1)
    chosen = torch.gather(prob, 1, ids.long().cpu())
    wt = chosen / chosen.sum(1, keepdim=True)
    y = torch.zeros_like(n)
    h = w["w_down"].shape[1]
    for e in range(w["w_ug"].shape[0]):
        t, j = (ids.cpu() == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        u = n[t] @ p["w_ug"][e].T
        y = y.index_add(0, t, wt[t, j, None] * ((torch.nn.functional.silu(u[:, :h]) * u[:, h:]) @ p["w_down"][e]))
    r = 0.9 * p["r"] + 0.5 * p["gate"] * unit(y) * p["w_post"]
    return r, unit(r) * p["w_next"], logits, prob, p


@pytest.mark.parametrize("stream", [F32, BF16])
def test_gradients_of_the_whole_layer(stream):
    """Against 64-bit autograd with the same experts chosen. Between input and result stand at most 12 roundings to bf16
    (n, logits, x_perm's products U, H, Y and y forward, as many gradients backward), each at most 2^-8 of its rows'
    size; the 2-norm of what they add up to stays within 12 2^-8 of the gradient's, twice that where two such paths meet."""
    T, d, h, E, k = 96, 128, 64, 8, 2
    w = weights(T, d, h, E, stream)
    f = forward(w, k)
    g = torch.Generator(device="cuda").manual_seed(1)
    dr, dn = (torch.randn((T, d), generator=g, device="cuda") for _ in range(2))
    dr, dn = dr.to(stream), dn.to(BF16)
    dl = torch.tensor([0.02, 0.001], device="cuda")
    got = moe.moe_layer_backward(dr, f, w["w_norm"], w["w_router"], w["w_ug"], w["w_down"], d_n_out=dn, d_losses=dl)
    r, n, logits, prob, p = reference(w, f.routed.expert_ids, k)
    counts = torch.bincount(f.routed.expert_ids.flatten().cpu().long(), minlength=E).double()
    losses = E * (counts / counts.sum() * prob.mean(0)).sum() * 0.02 + torch.logsumexp(logits, 1).pow(2).mean() * 0.001
    ((r * dr.double().cpu()).sum() + (n * dn.double().cpu()).sum() + losses).backward()
    names = dict(dr="r", dw_norm="w_norm", dw_router="w_router", dw_ug="w_ug", dw_down="w_down", dw_post="w_post",
                 dw_next="w_next", d_gate="gate")
    for name, (a, b) in dict(r=(f.r_out, r), n=(f.n_out, n)).items():
        assert float((a.double().cpu() - b.detach()).norm() / b.detach().norm()) < 12 * 2.0 ** -8, name
    for name, leaf in names.items():
        want = p[leaf].grad
        off = float((got[name].double().cpu() - want).norm() / want.norm())
        assert off < 24 * 2.0 ** -8, (name, off)


def test_a_layer_without_rows():
    w = weights(0, 128, 64, 8, BF16, 3)
    f = forward(w, 2)
    assert f.r_out.shape == f.n_out.shape == (0, 128)
    g = moe.moe_layer_backward(w["r"], f, w["w_norm"], w["w_router"], w["w_ug"], w["w_down"], d_n_out=w["r"])
    assert g["dr"].shape == (0, 128)
    for name in ("dw_norm", "dw_router", "dw_ug", "dw_down", "dw_post", "dw_next"):
        assert not g[name].any(), name  # sums over no rows


def test_the_layer_is_its_calls():
    T, d, h, E, k = 40, 256, 128, 16, 4
    w = weights(T, d, h, E, BF16, 2)
    f = forward(w, k)
    n = moe.moe_rmsnorm(w["r"], w["w_norm"])
    rows = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    logits = moe.moe_grouped_projection(n, rows, w["w_router"][None], "out_in")
    routed = moe.moe_router_topk(logits, k)
    y, *_ = moe.moe_expert_forward(n, routed.expert_ids, routed.routing_w, w["w_ug"], w["w_down"])
    r, nn = moe.moe_residual_norm(y, w["r"], w_post=w["w_post"], gate=w["gate"], w_next=w["w_next"], **KW)
    assert torch.equal(f.r_out, r) and torch.equal(f.n_out, nn)
    assert torch.equal(f.routed.expert_ids, routed.expert_ids)


@pytest.mark.parametrize("bits,master,seed", [(32, True, None), (8, False, 3), (8, True, None)])
def test_training_steps(bits, master, seed):
    """Two layers, three steps: forward, backward, one AdamW call for everything that is learned; the second run repeats the
    first bit for bit, and one replayed from a graph does too."""
    T, d, h, E, k, steps = 64, 128, 64, 8, 2, 3
    names = ("w_norm", "w_router", "w_ug", "w_down", "w_post", "w_next", "gate")

    def run(captured):
        layers = [weights(T, d, h, E, BF16, s) for s in (3, 4)]
        params = [w[n] for w in layers for n in names]
        state = moe.moe_adamw_state(params, bits=bits, master=master)
        x = torch.empty((T, d), dtype=BF16, device="cuda")
        step = torch.zeros(1, dtype=torch.int32, device="cuda")
        dl = torch.tensor([0.01, 0.001], device="cuda")
        clip = torch.ones(1, device="cuda")

        def one():
            step.add_(1)
            layers[0]["r"] = x
            f0 = forward(layers[0], k)
            layers[1]["r"] = f0.r_out
            f1 = forward(layers[1], k)
            g = [None, None]
            zero = torch.zeros_like(f1.n_out)
            args = [(w["w_norm"], w["w_router"], w["w_ug"], w["w_down"]) for w in layers]
            g[1] = moe.moe_layer_backward(f1.r_out, f1, *args[1], d_n_out=zero, d_losses=dl)
            g[0] = moe.moe_layer_backward(g[1]["dr"], f0, *args[0], d_n_out=zero, d_losses=dl)
            grads = [t for v in g for t in (v["dw_norm"], v["dw_router"], v["dw_ug"], v["dw_down"], v["dw_post"],
                                            v["dw_next"], v["d_gate"])]
            moe.moe_adamw_step(state, grads, lr=1e-2, step=step, grad_scale=clip, seed=seed)

        inputs = [torch.randn((T, d), generator=torch.Generator().manual_seed(s)).to(BF16).cuda() for s in range(steps)]
        graph = None
        if captured:
            x.copy_(inputs[0])
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one()
        for v in inputs:
            x.copy_(v)
            one() if graph is None else graph.replay()
            torch.cuda.synchronize()
        return params, state

    first, state = run(False)
    before = [weights(T, d, h, E, BF16, s)[n] for s in (3, 4) for n in names]
    for p, q in zip(first, before):
        assert torch.isfinite(p).all() and not torch.equal(p, q)
    for again, other in (run(False), run(True)):
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert all(torch.equal(a, b) for a, b in zip(moe.moe_adamw_moments(state), moe.moe_adamw_moments(other)))


def test_decode_on_4_bit_experts():
    """norm, router, 4-bit experts, norm: against the bf16 path on the weights read back. Both round n, H and Y to bf16 and
    the bf16 path U besides: 8 roundings in all, each at most 2^-8, between the two."""
    T, d, h, E, k = 4, 256, 128, 16, 4
    w = weights(T, d, h, E, BF16, 5)
    u4 = moe.moe_int4_quantize_weights(w["w_ug"], "out_in", group=64)
    d4 = moe.moe_int4_quantize_weights(w["w_down"], "in_out", group=32, symmetric=True)
    n = moe.moe_rmsnorm(w["r"], w["w_norm"])
    rows = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    routed = moe.moe_router_topk(moe.moe_grouped_projection(n, rows, w["w_router"][None], "out_in"), k)
    y4, p = moe.moe_expert_forward_int4(n, routed.expert_ids, routed.routing_w, u4, d4)
    back_ug, back_d = moe.moe_int4_dequantize_weights(u4), moe.moe_int4_dequantize_weights(d4)
    y, *_ = moe.moe_expert_forward(n, routed.expert_ids, routed.routing_w, back_ug, back_d.transpose(1, 2).contiguous())
    assert float((y4.double() - y.double()).norm() / y.double().norm()) < 8 * 2.0 ** -8
    r, nn = moe.moe_residual_norm(y4, w["r"], w_next=w["w_next"])
    assert torch.isfinite(r).all() and torch.isfinite(nn).all()
