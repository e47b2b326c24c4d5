"""The operators around a block's products run together, as examples/fp8_block.py uses them: against torch's autograd on
the values that the FP8 codes stand for, in captured graphs, and on several streams at once."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import fp8_block as ex  # noqa: E402
import fp8_block_scaled_amd as gfg  # noqa: E402
from oracle import layers_oracle as lo  # noqa: E402

pytestmark = pytest.mark.gpu


class Quantized(torch.autograd.Function):
    """x W^T of the values after quantizing, in 64 bits, with the layer's own definition of its gradients."""

    @staticmethod
    def forward(ctx, x, w, w8):
        ctx.save_for_backward(x, w8)
        x8 = torch.from_numpy(lo.through_fp8(x.float().numpy()))
        return x8 @ w8.t()

    @staticmethod
    def backward(ctx, dy):
        x, w8 = ctx.saved_tensors
        dx, dw, _ = lo.linear_backward(dy.float().numpy(), x.float().numpy(), w8.numpy())
        return torch.from_numpy(dx), torch.from_numpy(dw), None


def reference(block, y, r, dout, dm, dweights):
    """Losses and gradients of the same block from torch's autograd in 64 bits on the CPU, every rounding to bf16 left out
    but for the quantizers' inputs."""
    d = lambda t: t.detach().double().cpu()  # noqa: E731
    leaf = {n: d(t).requires_grad_(True) for n, t in (("y", y), ("r", r), ("norm", block.norm), ("post", block.post), ("gate", block.gate))}
    w = {n: d(getattr(block, n).w).requires_grad_(True) for n in ("router", "w1", "w2")}
    w8 = {n: gfg_values(getattr(block, n)) for n in w}
    round16 = lambda t: t + (t.detach().to(torch.bfloat16).double() - t.detach())  # noqa: E731
    rstd = lambda t: torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    out = leaf["r"] + leaf["gate"] * leaf["y"] * rstd(leaf["y"]) * leaf["post"]
    n = round16(out * rstd(out) * leaf["norm"])
    logits = round16(Quantized.apply(n, w["router"], w8["router"]))
    ids = d(block.choose(logits.detach().to(torch.bfloat16).cuda())[0]).long()
    p = torch.softmax(logits, 1)
    weights = p.gather(1, ids)
    weights = weights / weights.sum(1, keepdim=True)
    f = torch.bincount(ids.flatten(), minlength=p.shape[1]).double() * p.shape[1] / ids.numel()
    loss = ex.ALPHA * (f * p.mean(0)).sum()
    gu = round16(Quantized.apply(n, w["w1"], w8["w1"]))
    g, u = gu.chunk(2, -1)
    m = Quantized.apply(round16(torch.nn.functional.silu(g) * u), w["w2"], w8["w2"])
    ((out * d(dout)).sum() + (m * d(dm)).sum() + (weights * d(dweights)).sum() + loss).backward()
    return out.detach(), m.detach(), weights.detach(), loss.detach(), ids, {**{n: t.grad for n, t in leaf.items()}, **{n: t.grad for n, t in w.items()}}


def gfg_values(linear):
    from oracle import fp8_oracle as o
    return torch.from_numpy(o.dequantize_weight(linear.q.view(torch.uint8).cpu().numpy()[None], linear.s.cpu().numpy()[None])[0])


@pytest.mark.parametrize("T", [1, 33, 200])
def test_training_step(T):
    """Outputs are rounded to bf16 (2^-8 each) between the operators, up to six times in a chain, and such a change of a
    quantizer's input moves its codes by up to half a step of theirs (2^-4) where it crosses a border, which 2^-8 of the
    values in 2^-4 wide steps do at 1 in 16: 2^-4 / 4 = 2^-6 of the norm a quantizer, three of them in a chain."""
    torch.manual_seed(T)
    E, k, H, I = 16, 3, 272, 144
    block = ex.random_block(E, k, H, I, seed=T)
    y, r, dout, dm = (torch.randn(T, H, device="cuda").to(torch.bfloat16) for _ in range(4))
    dweights = torch.randn(T, k, device="cuda")
    out, m, weights, loss, saved = block.forward(y, r)
    dy, dr = block.backward(dout, dm, dweights, saved)
    r_out, r_m, r_w, r_loss, r_ids, grads = reference(block, y, r, dout, dm, dweights)
    assert torch.equal(saved[5].cpu().long(), r_ids)
    near = lambda a, b, tol: float((a.double().cpu() - b).norm()) <= tol * float(b.norm())  # noqa: E731
    assert near(out, r_out, 2.0 ** -8) and near(m, r_m, 3 * 2.0 ** -6) and near(weights, r_w, 2.0 ** -6)
    assert abs(float(loss) - float(r_loss)) <= 2.0 ** -6 * float(r_loss)
    got = dict(y=dy, r=dr, norm=block.norm_grad, post=block.post_grad, gate=block.gate_grad, router=block.router.grad, w1=block.w1.grad, w2=block.w2.grad)
    for n, g in got.items():
        assert near(g, grads[n], 3 * 2.0 ** -6), (n, float((g.double().cpu() - grads[n]).norm() / grads[n].norm()))
    once = {n: got[n].clone() for n in ("norm", "post", "gate", "router", "w1", "w2")}
    block.backward(dout, dm, dweights, saved)              # gradients are added to
    for n, g in once.items():
        assert torch.allclose(got[n], 2 * g, rtol=2.0 ** -20, atol=0)


@pytest.mark.parametrize("T", [1, 16, 40])
def test_serving(T):
    """The 8-bit rows and the 16-bit rows give the same block, to the quantizer's half steps."""
    torch.manual_seed(T)
    block = ex.random_block(16, 2, 256, 128, seed=T, with_experts=True)
    y, r = (torch.randn(T, 256, device="cuda").to(torch.bfloat16) for _ in range(2))
    out, m = block.serve(y, r)
    t_out, t_m, weights, _, saved = block.forward(y, r)
    experts = gfg.moe_fp8_layer(saved[3], saved[5], weights, *block.experts, torch.empty_like(y))
    assert torch.equal(out, t_out)
    want = t_m.float() + experts.float()
    # (the serving path norms the stored sum again for the experts: its rows differ by a bf16 rounding, and a choice may)
    assert float((m.float() - want).norm()) <= 0.1 * float(want.norm())


def step(block, y, r, dout, dm, dweights):
    out, m, weights, loss, saved = block.forward(y, r)
    dy, dr = block.backward(dout, dm, dweights, saved)
    return out, m, weights, loss, dy, dr


def test_graph_replays_match_eager():
    """Everything is captured, replayed with eager work and synchronizations in between, and every replay is the eager
    result bit for bit (the gradients that are added to are cleared in the graph)."""
    torch.manual_seed(1)
    T, E, k, H, I = 70, 16, 3, 272, 144
    block = ex.random_block(E, k, H, I)
    ins = [torch.randn(T, H, device="cuda").to(torch.bfloat16) for _ in range(4)] + [torch.randn(T, k, device="cuda")]
    grads = [block.w1.grad, block.w2.grad, block.router.grad, block.norm_grad, block.post_grad, block.gate_grad]

    def run():
        for g in grads:
            g.zero_()
        for w in (block.w1, block.w2, block.router):
            w.quantize()
        return step(block, *ins)

    want = [t.clone() for t in run()] + [g.clone() for g in grads]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for _ in range(4):
        for t in outs:
            t.zero_()
        for g in grads:
            g.fill_(7.0)
        torch.randn(256, 256, device="cuda").square().sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(list(outs) + grads, want))


def test_streams_with_their_own_workspaces():
    """Calls in flight at once on several streams, each with its own workspace, are the calls run alone."""
    torch.manual_seed(2)
    M, N, K, E, k = 300, 528, 1040, 64, 4
    dev = "cuda"
    q, s, qt, st = gfg.fp8_quantize_weight_device(torch.randn(N, K, device=dev), transposed=True)
    sets = []
    for i in range(3):
        x, dy = torch.randn(M, K, device=dev, dtype=torch.bfloat16), torch.randn(M, N, device=dev, dtype=torch.bfloat16)
        l, ids = torch.randn(M, E, device=dev), torch.randint(0, E, (M, k), device=dev, dtype=torch.int32)
        w = torch.rand(K, device=dev)
        stats = torch.empty(2, M, device=dev)
        out, _, _ = gfg.residual_norm(x, x, w, post_weight=w, gate=w, stats=stats)
        ws = torch.empty(16 << 20, dtype=torch.uint8, device=dev)

        def call(stream=None, x=x, dy=dy, l=l, ids=ids, w=w, out=out, stats=stats, ws=ws):
            with torch.cuda.stream(stream or torch.cuda.current_stream()):
                y, dx, dw, db = (torch.empty(*n, device=dev, dtype=t) for n, t in
                                 (((M, N), torch.bfloat16), ((M, K), torch.bfloat16), ((N, K), torch.float32), ((N,), torch.float32)))
                gr, gy, gw, gp, gg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w), torch.empty_like(w)
            gfg.fp8_linear(x, q, s, y, workspace=ws, stream=stream)
            gfg.fp8_linear_backward(dy, x, qt, st, dx=dx, dw=dw, dbias=db, workspace=ws, stream=stream)
            loss, counts, factors = gfg.moe_balance_loss(l, ids, z=0.1, workspace=ws, stream=stream)
            gfg.residual_norm_backward(x, x, out, x, stats, w, post_weight=w, gate=w, dresidual=gr, dy=gy, dweight=gw, dpost_weight=gp,
                                       dgate=gg, workspace=ws, stream=stream)
            return y, dx, dw, db, loss, counts, factors, gr, gy, gw, gp, gg

        sets.append(call)
    want = [[t.clone() for t in call()] for call in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [call(st_) for call, st_ in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_example_runs(capsys):
    ex.main()
    assert "4096 tokens" in capsys.readouterr().out
