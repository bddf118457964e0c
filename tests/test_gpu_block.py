"""GPU: the operators together (the example model), in HIP graphs, and at sizes whose offsets pass 32 bits."""
import os
import sys

import pytest
import torch

from tests import block_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ss():
    import selective_state_space_softplus_amd as ss

    return ss


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import head_block

    return head_block


def say(msg):
    print(f"[case] {msg}", flush=True)


def test_example_decodes_what_it_prefills(ss, example):
    """Prefill then steps against one pass over all tokens, fp32: two orders of the same sums, through two blocks and
    their projections (each relative 1e-5 at most, a few dozen of them)."""
    say("example decode")
    torch.manual_seed(0)
    model = example.HeadModel(d_model=48, heads=3, head_dim=16, state=24, dtype=F32).to(DEV)
    tokens = torch.randint(0, 32, (3, 40), device=DEV)
    with torch.no_grad():
        whole, states = model(tokens)
        _, run = model(tokens[:, :33])
        for k in range(33, 40):
            logits = model.step(tokens[:, k], run)
            assert ref.rel(logits, whole[:, k].cpu().to(F64)) < 1e-3, k
        for a, b in zip(run, states):
            assert ref.rel(a, b.cpu().to(F64)) < 1e-3


def test_example_gradients(ss, example):
    """Every parameter's gradient of the example model (fp32) against the same model with the operators' 64-bit forms on
    the CPU; the projections' fp32 rounding and the sums over tokens stay below 1e-4 of each gradient's norm."""
    say("example gradients")
    torch.manual_seed(1)
    model = example.HeadModel(d_model=32, heads=2, head_dim=12, state=8, dtype=F32).to(DEV)
    tokens = torch.randint(0, 32, (2, 70), device=DEV)
    logits, _ = model(tokens)
    (logits * torch.sin(torch.arange(logits.numel(), device=DEV, dtype=F32)).view_as(logits)).sum().backward()

    w = {k: v.detach().cpu().to(F64).requires_grad_(True) for k, v in model.named_parameters()}
    h, r = w["embed.weight"][tokens.cpu()], None
    for i, blk in enumerate(model.blocks):
        p = f"blocks.{i}."
        out, r = ref.residual_norm(h, w[p + "norm"], residual=r)
        z, x, B, C, dt = blk.split(out @ w[p + "in_proj.weight"].T)
        y, _ = ref.head_scan(x, dt, w[p + "A_log"], B, C, w[p + "D"], w[p + "dt_bias"])
        h = ref.gated_norm(y.flatten(-2), z, w[p + "gate"]) @ w[p + "out_proj.weight"].T
    out, _ = ref.residual_norm(h, w["norm"], residual=r)
    want = out @ w["embed.weight"].T
    (want * torch.sin(torch.arange(want.numel(), dtype=F32)).to(F64).view_as(want)).sum().backward()
    assert ref.rel(logits, want) < 1e-4
    for k, v in model.named_parameters():
        assert ref.rel(v.grad, w[k].grad) < 1e-4, k


def test_example_learns(ss, example):
    say("example training")
    torch.manual_seed(0)
    losses = example.train(example.HeadModel().to(DEV), steps=200)
    assert all(x == x for x in losses)
    assert sum(losses[-5:]) / 5 < 0.8 * losses[0], losses


def test_graph_replays(ss):
    """Forward, backward and the decode step captured once and replayed with new inputs; eager calls of other sizes,
    which grow the cached workspace, run between the replays."""
    say("graph replays")
    gen = torch.Generator(device=DEV).manual_seed(2)

    def make():
        n = lambda *s, dt=BF16: torch.randn(*s, generator=gen, device=DEV).to(dt)  # noqa: E731
        return dict(x=n(1, 700, 4, 64), delta=n(1, 700, 4), B=n(1, 700, 1, 64), C=n(1, 700, 1, 64), dy=n(1, 700, 4, 64),
                    z=n(1, 700, 256), state=n(1, 4, 64, 64, dt=F32))

    A_log, D, w = torch.zeros(4, device=DEV), torch.ones(4, device=DEV), torch.ones(256, device=DEV)

    def run(t):
        y, last = ss.head_scan_fwd(t["x"], t["delta"], A_log, t["B"], t["C"], D, return_last_state=True)
        g = ss.head_scan_bwd(t["x"], t["delta"], A_log, t["B"], t["C"], D, t["dy"])
        o, r = ss.residual_norm_fwd(y.flatten(-2), w, residual=t["z"])
        q = ss.gated_norm_fwd(o, t["z"], w)
        gq = ss.gated_norm_bwd(q, o, t["z"], w)
        s = t["state"].clone()
        ys = ss.head_state_update(s, *(t[k][:, 0].contiguous() for k in ("x", "delta")), A_log,
                                  *(t[k][:, 0].contiguous() for k in ("B", "C")), D)
        return [y, last, *g.values(), o, r, q, *gq.values(), s, ys]

    held = make()
    run(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(held)
    for k in range(3):
        new = make()
        big = make()
        big = {n: (v.repeat(4, *([1] * (v.dim() - 1)))) for n, v in big.items()}
        run(big)
        for n in held:
            held[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, run(new))):
            assert torch.equal(a, b), (k, i)


def test_offsets_past_32_bits(ss):
    """x, y and their gradients of more than 2^32 bytes and 2^31 elements: the last heads of the last steps against the
    same heads alone (the same arithmetic; bf16, so equal up to the order of sums over heads: heads are apart here)."""
    b, L, H, P, N = 1, 33000, 1024, 64, 16
    say(f"large offsets {b} {L} {H} {P} {N}")
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty(b, L, H, P, dtype=BF16, device=DEV).normal_(generator=gen)
    assert x.numel() > 2 ** 31
    delta = torch.empty(b, L, H, dtype=BF16, device=DEV).normal_(generator=gen)
    B = torch.empty(b, L, 1, N, dtype=BF16, device=DEV).normal_(generator=gen)
    C = torch.empty(b, L, 1, N, dtype=BF16, device=DEV).normal_(generator=gen)
    A_log, D = torch.zeros(H, device=DEV), torch.ones(H, device=DEV)
    bias = torch.full((H,), -3.0, device=DEV)
    y, last = ss.head_scan_fwd(x, delta, A_log, B, C, D, delta_bias=bias, return_last_state=True)
    few = slice(H - 2, H)
    xs, ds = x[:, :, few], delta[:, :, few]        # views with the large strides
    ys, ls = ss.head_scan_fwd(xs, ds, A_log[few], B, C, D[few], delta_bias=bias[few], return_last_state=True)
    assert ref.rel(y[:, -200:, few], ys[:, -200:].cpu().to(F64)) < 3 * 2.0 ** -9
    assert ref.rel(last[:, few], ls.cpu().to(F64)) < 1e-5
    dy = x                                         # any values do
    g = ss.head_scan_bwd(x, delta, A_log, B, C, D, dy, delta_bias=bias)
    gs = ss.head_scan_bwd(xs, ds, A_log[few], B, C, D[few], dy[:, :, few].contiguous(), delta_bias=bias[few])
    assert ref.rel(g["dx"][:, -200:, few], gs["dx"][:, -200:].cpu().to(F64)) < 3 * 2.0 ** -9
    assert ref.rel(g["ddelta"][:, -200:, few], gs["ddelta"][:, -200:].cpu().to(F64)) < 3 * 2.0 ** -9
    assert ref.rel(g["dD"][few], gs["dD"].cpu().to(F64)) < 1e-5
    del y, g, last
    rows = y2 = x.view(L, H * P)
    w = torch.ones(H * P // 8, device=DEV)
    out = ss.gated_norm_fwd(rows, y2, torch.ones(H * P, device=DEV), groups=8)
    want = ss.gated_norm_fwd(rows[-3:, -w.numel():].contiguous(), y2[-3:, -w.numel():].contiguous(), w)
    assert torch.equal(out[-3:, -w.numel():], want)
