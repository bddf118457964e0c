"""GPU: the head-wise scan, its gradient and its decode step against the 64-bit step-by-step form.

Tolerances (2-norm of the error over that of the result):
  outputs stored in bf16: their own rounding, and one rounded operand in the products that they sum.  A bf16 rounding is
    at most 2^-8 of an element, 2^-9 in the root mean square, so the two together are sqrt(2) * 2^-9 over many
    elements and at most 2^-8 of a result that is one product: 3 * 2^-9 = 5.9e-3 bounds both;
  fp32 outputs: decays are exp2 of differences of running sums, whose rounding is 2^-24 of sums of up to 64 steps'
    logs (tens here), and sums of a few thousand products: 1e-5 covers 100 units of 2^-24 and their square-root growth.
A sum with heavy cancellation (the gradients of A_log and of the bias) is measured against the sum of its terms' sizes
per head, to the same figure.
"""
import pytest
import torch

from tests import block_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DEV = "cuda:0"
TOL = {BF16: 3 * 2.0 ** -9, F32: 1e-5}


@pytest.fixture(scope="module")
def ss():
    import selective_state_space_softplus_amd as ss

    return ss


def say(msg):
    print(f"[case] {msg}", flush=True)


def inputs(b, L, H, P, N, G, dtype, seed, packed=False, state=True):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, dt=dtype, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(dt).to(DEV)

    t = dict(delta=normal(b, L, H), A_log=torch.log(1 + 15 * torch.rand(H, generator=g)).to(DEV), D=normal(H, dt=F32),
             bias=normal(H, dt=F32, scale=0.5) - 3)
    if packed:
        row = normal(b, L, H * P + 2 * G * N + 8)[..., 8:]
        t["x"] = row[..., :H * P].unflatten(-1, (H, P))
        t["B"] = row[..., H * P:H * P + G * N].unflatten(-1, (G, N))
        t["C"] = row[..., H * P + G * N:].unflatten(-1, (G, N))
    else:
        t["x"], t["B"], t["C"] = normal(b, L, H, P), normal(b, L, G, N), normal(b, L, G, N)
    t["h0"] = normal(b, H, P, N, dt=F32, scale=0.5) if state else None
    t["dy"] = normal(b, L, H, P)
    t["dlast"] = normal(b, H, P, N, dt=F32, scale=0.5) if state else None
    return t


NAMES = ("x", "delta", "A_log", "B", "C", "D", "bias", "h0")

SHAPES = [
    # b, L, H, P, N, G: one token; one channel; ends inside a tile; groups; several slabs; segments of the sequence
    (1, 1, 1, 1, 1, 1), (2, 1, 4, 64, 128, 2), (1, 64, 2, 64, 64, 1), (2, 63, 3, 33, 40, 3), (1, 65, 4, 16, 16, 2),
    (1, 130, 2, 80, 31, 1), (1, 200, 2, 128, 100, 1), (2, 129, 6, 64, 128, 3), (1, 1000, 2, 64, 128, 1),
    (1, 1343, 3, 17, 9, 1), (3, 257, 2, 200, 64, 2),
]


def check_fwd(ss, t, dtype, softplus=True, bias=True):
    kw = dict(delta_bias=t["bias"] if bias else None, delta_softplus=softplus, initial_state=t["h0"])
    y, last = ss.head_scan_fwd(t["x"], t["delta"], t["A_log"], t["B"], t["C"], t["D"], return_last_state=True, **kw)
    w = {k: ref.wide(t[k]) for k in NAMES}
    yr, lr = ref.head_scan(*(w[k] for k in NAMES[:6]), w["bias"] if bias else None, softplus, w["h0"])
    assert ref.rel(y, yr) < TOL[dtype]
    assert ref.rel(last, lr) < TOL[F32]
    return y, last


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(ss, shape, dtype):
    say(f"head scan fwd {shape} {dtype}")
    t = inputs(*shape, dtype, seed=sum(shape), state=shape[1] % 2 == 0)
    check_fwd(ss, t, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_views_of_one_projection(ss, dtype):
    """x, B and C side by side in a token's row, and a row offset that leaves them unaligned for vector loads."""
    for shape in ((2, 150, 4, 32, 64, 2), (1, 99, 3, 20, 12, 1), (1, 70, 2, 33, 7, 1)):
        say(f"head scan views {shape} {dtype}")
        t = inputs(*shape, dtype, seed=5, packed=True)
        assert not t["x"].is_contiguous()
        check_fwd(ss, t, dtype)


def test_forward_plain_step_sizes(ss):
    """No softplus: the step is delta + bias itself (positive, zero and slightly negative here); and no bias."""
    say("head scan without softplus")
    t = inputs(2, 100, 2, 24, 16, 1, F32, seed=3)
    t["delta"] = t["delta"].abs() * 0.1
    t["delta"][:, ::7] = 0
    check_fwd(ss, t, F32, softplus=False, bias=False)
    t["bias"] = torch.full_like(t["bias"], -0.01)
    check_fwd(ss, t, F32, softplus=False)
    check_fwd(ss, t, F32, bias=False)


def test_forward_large_steps(ss):
    """Steps that wipe the state (decays of exp(-1000)) between ordinary ones."""
    say("head scan with wiping steps")
    t = inputs(1, 150, 2, 16, 16, 1, F32, seed=4)
    t["delta"][:, 20::31] = 200.0
    check_fwd(ss, t, F32)


def test_split_sequence_continues_the_state(ss):
    """A sequence in two parts, the state carried over in place, against one call."""
    say("head scan in two parts")
    t = inputs(1, 500, 2, 64, 64, 1, F32, seed=6)
    y, last = check_fwd(ss, t, F32)
    state = t["h0"].clone()
    parts = []
    for lo, hi in ((0, 203), (203, 500)):
        a = {k: t[k][:, lo:hi] for k in ("x", "delta", "B", "C")}
        yp, out = ss.head_scan_fwd(a["x"], a["delta"], t["A_log"], a["B"], a["C"], t["D"], delta_bias=t["bias"],
                                   initial_state=state, last_state=state, return_last_state=True)
        assert out.data_ptr() == state.data_ptr()
        parts.append(yp)
    assert ref.rel(torch.cat(parts, 1), y.cpu().to(F64)) < TOL[F32]
    assert ref.rel(state, last.cpu().to(F64)) < TOL[F32]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_inputs_stay_causal(ss, dtype, bad):
    """An infinite or NaN x, B, C or delta changes nothing before its step, nor in other heads or channels it does not
    reach: those outputs are the same bit for bit."""
    say(f"head scan non-finite {bad} {dtype}")
    t = inputs(1, 150, 2, 20, 16, 2, dtype, seed=8)
    args = lambda q: (q["x"], q["delta"], q["A_log"], q["B"], q["C"], q["D"])  # noqa: E731
    base, last = ss.head_scan_fwd(*args(t), delta_bias=t["bias"], initial_state=t["h0"], return_last_state=True)
    at = 77
    for name in ("x", "B", "C", "delta"):
        q = dict(t, **{name: t[name].clone()})
        if name == "delta":
            q[name][0, at, 0] = bad
        else:
            q[name][0, at, 0, 3] = bad
        y, after = ss.head_scan_fwd(*args(q), delta_bias=t["bias"], initial_state=t["h0"], return_last_state=True)
        assert ref.rel(y[:, :at], base[:, :at].cpu().to(F64)) < TOL[dtype], name
        assert torch.isfinite(y[:, :at].float()).all(), name
        assert torch.isfinite(y[:, :, 1].float()).all() and torch.isfinite(after[:, 1]).all(), name
        if name == "x":
            others = [c for c in range(20) if c != 3]
            assert torch.isfinite(y[:, :, 0, others].float()).all()
            assert not torch.isfinite(y[:, at, 0, 3].float()).any()
            assert not torch.isfinite(after[0, 0, 3]).any()
        if name == "C":
            assert torch.isfinite(after).all() and torch.isfinite(y[:, at + 1:].float()).all()
            assert not torch.isfinite(y[:, at, 0].float()).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_non_finite_x_across_segments(ss, dtype):
    """The same in segments of several chunks: a NaN x in the first step, at a segment's last step and in between
    reaches its own channel alone, from its step on, and the others keep their values."""
    say(f"head scan non-finite in long segments {dtype}")
    t = inputs(4, 827, 40, 9, 16, 2, dtype, seed=21)
    for at in (0, 319, 500):
        x = t["x"].clone()
        x[1, at, 7, 3] = float("nan")
        y, last = ss.head_scan_fwd(x, t["delta"], t["A_log"], t["B"], t["C"], t["D"], t["bias"],
                                   initial_state=t["h0"], return_last_state=True)
        w = {k: ref.wide(t[k]) for k in NAMES}
        yr, lr = ref.head_scan(*(w[k] for k in NAMES[:6]), w["bias"], True, w["h0"])
        reached = torch.zeros(y.shape, dtype=torch.bool)
        reached[1, at:, 7, 3] = True
        assert torch.equal(torch.isnan(y.float()).cpu(), reached), at
        assert torch.isnan(last[1, 7, 3]).all() and torch.isnan(last).sum() == 16, at
        y, last = y.cpu(), last.cpu()
        assert ref.rel(y[~reached], yr.cpu()[~reached]) < TOL[dtype], at
        left = ~torch.isnan(last)
        assert ref.rel(last[left], lr.cpu()[left]) < TOL[F32], at


def grads(ss, t, bias=True, softplus=True):
    return ss.head_scan_bwd(t["x"], t["delta"], t["A_log"], t["B"], t["C"], t["D"], t["dy"],
                            delta_bias=t["bias"] if bias else None, delta_softplus=softplus, initial_state=t["h0"],
                            dlast_state=t["dlast"])


def check_bwd(ss, t, dtype, bias=True, softplus=True):
    g = grads(ss, t, bias, softplus)
    w = {k: ref.wide(t[k], True) for k in NAMES}
    if not bias:
        w["bias"] = None
    y, last = ref.head_scan(*(w[k] for k in NAMES[:6]), w["bias"], softplus, w["h0"])
    loss = (y * ref.wide(t["dy"])).sum()
    if t["dlast"] is not None:
        loss = loss + (last * ref.wide(t["dlast"])).sum()
    loss.backward()
    pairs = dict(dx="x", ddelta="delta", dA_log="A_log", dB="B", dC="C", dD="D", ddelta_bias="bias",
                 dinitial_state="h0")
    for name, of in pairs.items():
        if w[of] is None:
            assert name not in g
            continue
        want = w[of].grad
        assert torch.isfinite(g[name].float()).all(), name
        if name in ("dA_log", "ddelta_bias", "dD"):
            # Sums over rows and time with terms of both signs: measured against the terms' sizes.
            terms = {"dD": (ref.wide(t["dy"]) * ref.wide(t["x"])).norm(),
                     "ddelta_bias": w["delta"].grad.norm(), "dA_log": w["delta"].grad.norm()}[name]
            err = (g[name].cpu().to(F64) - want).norm().item() / max(want.norm().item(), terms.item())
            assert err < TOL[F32], (name, err)
        elif name == "dinitial_state":
            assert ref.rel(g[name], want) < TOL[F32], name
        else:
            err = ref.rel(g[name], want)
            assert err < TOL[dtype], (name, err)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(ss, shape, dtype):
    say(f"head scan bwd {shape} {dtype}")
    check_bwd(ss, inputs(*shape, dtype, seed=1 + sum(shape), state=shape[1] % 2 == 1), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(8, 827, 40, 8, 8, 1), (4, 827, 40, 9, 16, 2), (2, 827, 40, 8, 8, 1),
                                   (3, 1500, 42, 16, 8, 2), (2, 700, 100, 8, 8, 4)])
def test_segments_of_several_chunks(ss, shape, dtype):
    """Many heads: few segments of several chunks each, whose first pass is cut at other bounds than theirs."""
    say(f"head scan segments {shape} {dtype}")
    t = inputs(*shape, dtype, seed=sum(shape))
    check_fwd(ss, t, dtype)
    check_bwd(ss, t, dtype)


def test_backward_views_and_plain_steps(ss):
    say("head scan bwd views, no softplus, no bias")
    t = inputs(2, 100, 4, 24, 16, 2, F32, seed=13, packed=True)
    check_bwd(ss, t, F32)
    t["delta"] = t["delta"].abs() * 0.1
    check_bwd(ss, t, F32, bias=False, softplus=False)


def test_backward_against_differences(ss):
    """The gradient along random directions against central differences of the forward (fp32).

    With a step e the difference's own error is e^2 times the third derivative plus 2^-24 / e times the sum of the
    outputs' sizes; at e = 2^-6 both stay below 1e-2 of the derivative's scale, |grad| |direction|.
    """
    say("head scan bwd differences")
    t = inputs(1, 90, 2, 16, 16, 1, F32, seed=21)
    g = grads(ss, t)
    names = dict(x="dx", delta="ddelta", A_log="dA_log", B="dB", C="dC", D="dD", bias="ddelta_bias",
                 h0="dinitial_state")

    def loss(q):
        y, last = ss.head_scan_fwd(q["x"], q["delta"], q["A_log"], q["B"], q["C"], q["D"], delta_bias=q["bias"],
                                   initial_state=q["h0"], return_last_state=True)
        return (y.double() * t["dy"].double()).sum() + (last.double() * t["dlast"].double()).sum()

    e = 2.0 ** -6
    gen = torch.Generator().manual_seed(1)
    for k, name in names.items():
        d = torch.randn(t[k].shape, generator=gen).to(DEV)
        up, down = (loss(dict(t, **{k: t[k] + s * e * d})) for s in (1, -1))
        want = ((up - down) / (2 * e)).item()
        got = (g[name].double() * d.double()).sum().item()
        scale = g[name].double().norm().item() * d.double().norm().item() / d.numel() ** 0.5
        assert abs(got - want) < 1e-2 * max(abs(want), scale), (k, got, want)


def test_autograd_and_run_to_run(ss):
    """The differentiable form gives the same gradients, and every call the same bits."""
    say("head scan autograd")
    t = inputs(2, 300, 4, 64, 64, 2, BF16, seed=31)
    w = {k: t[k].clone().requires_grad_(True) for k in NAMES}
    y, last = ss.head_scan(*(w[k] for k in NAMES[:6]), delta_bias=w["bias"], initial_state=w["h0"],
                           return_last_state=True)
    torch.autograd.backward([y, last], [t["dy"], t["dlast"]])
    g = grads(ss, t)
    for k, name in (("x", "dx"), ("delta", "ddelta"), ("A_log", "dA_log"), ("B", "dB"), ("C", "dC"), ("D", "dD"),
                    ("bias", "ddelta_bias"), ("h0", "dinitial_state")):
        assert torch.equal(w[k].grad, g[name]), name
    y2, last2 = ss.head_scan_fwd(*(t[k] for k in NAMES[:6]), delta_bias=t["bias"], initial_state=t["h0"],
                                 return_last_state=True)
    assert torch.equal(y, y2) and torch.equal(last, last2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (3, 4, 33, 31, 2), (2, 6, 64, 128, 3), (5, 2, 16, 16, 1),
                                   (1, 3, 7, 6, 3), (4, 80, 64, 128, 8)])
def test_decode_step(ss, shape, dtype):
    """A step against the 64-bit one, and against a one-token scan."""
    b, H, P, N, G = shape
    say(f"head step {shape} {dtype}")
    t = inputs(b, 1, H, P, N, G, dtype, seed=sum(shape))
    state = t["h0"].clone()
    y = ss.head_state_update(state, t["x"][:, 0], t["delta"][:, 0], t["A_log"], t["B"][:, 0], t["C"][:, 0], t["D"],
                             dt_bias=t["bias"])
    w = {k: ref.wide(t[k]) for k in NAMES}
    yr, lr = ref.head_scan(*(w[k] for k in NAMES[:6]), w["bias"], True, w["h0"])
    assert ref.rel(y, yr[:, 0]) < TOL[dtype]
    assert ref.rel(state, lr) < TOL[F32]


def test_steps_follow_a_prefill(ss):
    """A prompt by the scan and the next tokens by steps, against one scan over all of them."""
    say("head scan prefill then steps")
    t = inputs(2, 75, 4, 32, 48, 2, F32, seed=17, state=False)
    y, last = check_fwd(ss, t, F32)
    first = {k: t[k][:, :70] for k in ("x", "delta", "B", "C")}
    _, state = ss.head_scan_fwd(first["x"], first["delta"], t["A_log"], first["B"], first["C"], t["D"],
                                delta_bias=t["bias"], return_last_state=True)
    for k in range(70, 75):
        yk = ss.head_state_update(state, t["x"][:, k].contiguous(), t["delta"][:, k].contiguous(), t["A_log"],
                                  t["B"][:, k].contiguous(), t["C"][:, k].contiguous(), t["D"], dt_bias=t["bias"])
        assert ref.rel(yk, y[:, k].cpu().to(F64)) < 2 * TOL[F32]
    assert ref.rel(state, last.cpu().to(F64)) < 2 * TOL[F32]


def test_empty_sizes(ss):
    say("head scan empty sizes")
    t = inputs(2, 4, 2, 8, 8, 1, F32, seed=1)
    none = {k: t[k][:, :0] for k in ("x", "delta", "B", "C")}
    y, last = ss.head_scan_fwd(none["x"], none["delta"], t["A_log"], none["B"], none["C"], t["D"],
                               initial_state=t["h0"], return_last_state=True)
    assert y.shape == (2, 0, 2, 8) and torch.equal(last, t["h0"])
    g = ss.head_scan_bwd(none["x"], none["delta"], t["A_log"], none["B"], none["C"], t["D"], t["dy"][:, :0],
                         initial_state=t["h0"], dlast_state=t["dlast"])
    assert torch.equal(g["dinitial_state"], t["dlast"]) and not g["dA_log"].any()


def test_another_stream(ss):
    """Work goes on the caller's current stream, and its workspace with it."""
    say("head scan on another stream")
    t = inputs(1, 700, 2, 64, 64, 1, BF16, seed=9)
    args = (t["x"], t["delta"], t["A_log"], t["B"], t["C"], t["D"])
    want = ss.head_scan_fwd(*args, delta_bias=t["bias"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = ss.head_scan_fwd(*args, delta_bias=t["bias"])
    side.synchronize()
    assert torch.equal(got, want)


def test_refusals(ss):
    say("head scan refusals")
    t = inputs(1, 8, 4, 8, 8, 2, F32, seed=1)
    args = [t["x"], t["delta"], t["A_log"], t["B"], t["C"], t["D"]]

    def swap(i, v):
        return args[:i] + [v] + args[i + 1:]

    with pytest.raises(TypeError):
        ss.head_scan_fwd(*swap(0, t["x"].half()))
    with pytest.raises(TypeError):
        ss.head_scan_fwd(*swap(3, t["B"].to(BF16)))
    with pytest.raises(ValueError):
        ss.head_scan_fwd(*swap(1, t["delta"][:, :4]))
    with pytest.raises(ValueError):
        ss.head_scan_fwd(*swap(0, t["x"].transpose(2, 3).contiguous().transpose(2, 3)))
    with pytest.raises(ValueError):
        ss.head_scan_fwd(*swap(0, t["x"].cpu()))
    with pytest.raises(ValueError):
        ss.head_scan_fwd(t["x"][:, :, :3], t["delta"][:, :, :3], t["A_log"][:3], t["B"], t["C"], t["D"][:3])
    with pytest.raises(ss.SSError) as e:
        big = torch.zeros(1, 8, 2, 129, device=DEV)
        ss.head_scan_fwd(t["x"], t["delta"], t["A_log"], big, big, t["D"])
    assert e.value.code == -4
    with pytest.raises(ss.SSError) as e:
        ss.head_scan_fwd(*args, out=t["x"])
    assert e.value.code == -7
    with pytest.raises(ss.SSError) as e:
        ss.head_scan_bwd(*args, t["dy"], workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == -5
    with pytest.raises(ValueError):
        ss.head_state_update(t["h0"], t["x"][:, 0], t["delta"][:, 0], t["A_log"], t["B"][:, 0, :, :4].contiguous(),
                             t["C"][:, 0], t["D"])
