"""GPU: the residual norm and the gated norm, forward and backward, against their 64-bit forms.

Tolerances (2-norm of the error over that of the result): bf16 outputs carry one rounding, at most 2^-8 of each
element (half a unit of an 8-bit significand); fp32 ones the sums' rounding (a few units of 2^-24 times the square root of at most 16384 terms over 64 lanes)
and that of the hardware reciprocal, square root and exponential (about 2^-23 each): 4e-6.
"""
import pytest
import torch

from tests import block_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DEV = "cuda:0"
TOL = {BF16: 2.0 ** -8 + 4e-6, F32: 4e-6}


@pytest.fixture(scope="module")
def ss():
    import selective_state_space_softplus_amd as ss

    return ss


def say(msg):
    print(f"[case] {msg}", flush=True)


def make(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *shape, dt=F32, scale=1.0, mean=0.0: \
        (torch.randn(*shape, generator=g) * scale + mean).to(dt).to(DEV)


# rows, d: one channel; a row in a wave (odd, vectors, two vectors), in a workgroup (each width), and the widest
SIZES = [(1, 1), (5, 7), (130, 64), (9, 500), (33, 1000), (7, 1536), (4100, 96), (3, 2048), (11, 2561), (5, 4096),
         (6, 5120), (2, 8192), (2, 8193), (1, 16384)]


@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("size", SIZES)
def test_residual_norm(ss, size, types):
    rows, d = size
    dt, rt = types
    say(f"residual norm {size} {types}")
    normal = make(rows + d)
    for residual, scale in ((True, True), (True, False), (False, True), (False, False)):
        x, w = normal(rows, d, dt=dt), normal(d, scale=0.2, mean=1.0)
        res = normal(rows, d, dt=rt, scale=2.0) if residual else None
        sc = normal(d, scale=0.1, mean=0.5) if scale else None
        dout, dres = normal(rows, d, dt=dt), normal(rows, d, dt=rt)
        out, r = ss.residual_norm_fwd(x, w, residual=res, scale=sc, residual_dtype=rt)
        assert r.dtype == rt and out.dtype == dt
        t = [ref.wide(v, True) for v in (x, w, res, sc)]
        # The stored residual stream is what is normalised, in both directions.
        want_r = (t[0] if sc is None else t[0] * t[3]) + (0 if res is None else t[2])
        assert ref.rel(r, want_r) < TOL[rt]
        stream = want_r + (ref.wide(r) - want_r.detach())
        want = stream / torch.sqrt((stream * stream).mean(-1, keepdim=True) + 1e-5) * t[1]
        assert ref.rel(out, want) < TOL[dt]
        for with_dres in (True, False):
            for v in t:
                if v is not None:
                    v.grad = None
            torch.autograd.backward([want] + ([stream] if with_dres else []),
                                    [ref.wide(dout)] + ([ref.wide(dres)] if with_dres else []), retain_graph=True)
            g = ss.residual_norm_bwd(dout, r, w, dresidual_out=dres if with_dres else None, x=x, scale=sc)
            assert ref.rel(g["dx"], t[0].grad) < TOL[dt] or (d == 1 and not with_dres)
            assert ref.rel(g["dweight"], t[1].grad) < TOL[F32] * 4
            if res is not None:
                assert ref.rel(g["dresidual"], t[2].grad) < TOL[rt] or (d == 1 and not with_dres)
            if sc is not None:
                assert ref.rel(g["dscale"], t[3].grad) < TOL[F32] * 4 or (d == 1 and not with_dres)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("before", [False, True])
@pytest.mark.parametrize("size", [s + (1,) for s in SIZES] + [(65, 120, 3), (33, 1536, 8), (9, 40, 40), (3, 32768, 2)])
def test_gated_norm(ss, size, before, dtype):
    rows, d, groups = size
    say(f"gated norm {size} before={before} {dtype}")
    normal = make(rows + d)
    y, z, w = normal(rows, d, dt=dtype), normal(rows, d, dt=dtype), normal(d, scale=0.2, mean=1.0)
    dout = normal(rows, d, dt=dtype)
    out = ss.gated_norm_fwd(y, z, w, groups=groups, norm_before_gate=before)
    g = ss.gated_norm_bwd(dout, y, z, w, groups=groups, norm_before_gate=before)
    t = [ref.wide(v, True) for v in (y, z, w)]
    want = ref.gated_norm(*t, groups, before=before)
    want.backward(ref.wide(dout))
    assert ref.rel(out, want) < TOL[dtype]
    one = d // groups == 1   # a single channel's norm is its sign: its gradients are differences of equal terms
    for name, v in (("dy", t[0]), ("dz", t[1])):
        assert torch.isfinite(g[name].float()).all()
        assert one or ref.rel(g[name], v.grad) < TOL[dtype], name
    assert ref.rel(g["dweight"], t[2].grad) < 4 * TOL[F32]


def test_gated_norm_reads_column_ranges(ss):
    """z as columns of a wider projection, rows unaligned for vectors and aligned ones, in three dimensions."""
    say("gated norm views")
    normal = make(3)
    for off, width in ((8, 600), (3, 601)):
        proj = normal(3, 17, width, dt=BF16)
        z, y, w = proj[..., off:off + 512], normal(3, 17, 512, dt=BF16), normal(512, mean=1.0)
        assert not z.is_contiguous()
        out = ss.gated_norm(y, z, w, groups=2)
        assert torch.equal(out, ss.gated_norm_fwd(y, z.contiguous(), w, groups=2))
        g = ss.gated_norm_bwd(y, y, z, w, groups=2)
        k = ss.gated_norm_bwd(y, y, z.contiguous(), w, groups=2)
        for name in g:
            assert torch.equal(g[name], k[name]), name


def test_in_place_residual_and_autograd(ss):
    say("residual norm in place, autograd")
    normal = make(4)
    x, res, w, sc = normal(9, 320, dt=BF16), normal(9, 320), normal(320, mean=1.0), normal(320, mean=0.5)
    out, r = ss.residual_norm_fwd(x, w, residual=res, scale=sc)
    keep = res.clone()
    out2, r2 = ss.residual_norm_fwd(x, w, residual=keep, scale=sc, residual_out=keep)
    assert r2.data_ptr() == keep.data_ptr() and torch.equal(r, keep) and torch.equal(out, out2)
    leaves = [v.clone().requires_grad_(True) for v in (x, w, res, sc)]
    o, s = ss.residual_norm(leaves[0], leaves[1], residual=leaves[2], scale=leaves[3])
    dout, dres = normal(9, 320, dt=BF16), normal(9, 320)
    torch.autograd.backward([o, s], [dout, dres])
    g = ss.residual_norm_bwd(dout, r, w, dresidual_out=dres, x=x, scale=sc)
    for v, name in zip(leaves, ("dx", "dweight", "dresidual", "dscale")):
        assert torch.equal(v.grad, g[name]), name
    y, z = normal(9, 320, dt=BF16), normal(9, 320, dt=BF16)
    leaves = [v.clone().requires_grad_(True) for v in (y, z, w)]
    ss.gated_norm(*leaves, groups=4).backward(dout)
    g = ss.gated_norm_bwd(dout, y, z, w, groups=4)
    for v, name in zip(leaves, ("dy", "dz", "dweight")):
        assert torch.equal(v.grad, g[name]), name


def test_gradients_against_differences(ss):
    """Central differences of the fp32 forward along random directions: at a step of 2^-6 the difference is within
    1e-2 of the derivative's scale (its square times a third derivative of order one, and 2^-24 / 2^-6 of the sum)."""
    say("norm differences")
    normal = make(6)
    e = 2.0 ** -6
    dout, dres = normal(5, 48), normal(5, 48)

    def compare(loss, leaves, got):
        for i, (v, gr) in enumerate(zip(leaves, got)):
            d = normal(*v.shape)
            up, down = (loss(*leaves[:i], v + s * e * d, *leaves[i + 1:]) for s in (1, -1))
            want, have = ((up - down) / (2 * e)).item(), (gr.double() * d.double()).sum().item()
            assert abs(want - have) < 1e-2 * max(abs(want), gr.double().norm().item()), (i, want, have)

    def res_loss(x, w, res, sc):
        o, r = ss.residual_norm_fwd(x, w, residual=res, scale=sc)
        return (o.double() * dout.double()).sum() + (r.double() * dres.double()).sum()

    leaves = [normal(5, 48), normal(48, mean=1.0), normal(5, 48), normal(48, mean=0.5)]
    r = ss.residual_norm_fwd(leaves[0], leaves[1], residual=leaves[2], scale=leaves[3])[1]
    g = ss.residual_norm_bwd(dout, r, leaves[1], dresidual_out=dres, x=leaves[0], scale=leaves[3])
    compare(res_loss, leaves, [g["dx"], g["dweight"], g["dresidual"], g["dscale"]])
    for before in (False, True):
        def gate_loss(y, z, w):
            return (ss.gated_norm_fwd(y, z, w, groups=3, norm_before_gate=before).double() * dout.double()).sum()

        leaves = [normal(5, 48), normal(5, 48), normal(48, mean=1.0)]
        g = ss.gated_norm_bwd(dout, *leaves, groups=3, norm_before_gate=before)
        compare(gate_loss, leaves, [g["dy"], g["dz"], g["dweight"]])


def test_zero_rows_and_zero_values(ss):
    """A row of zeros has out = 0 and finite gradients (eps under the root); no rows give empty outputs."""
    say("norm zeros")
    w = torch.ones(64, device=DEV)
    zero = torch.zeros(3, 64, device=DEV)
    out, r = ss.residual_norm_fwd(zero, w, residual=zero)
    assert not out.any() and not r.any()
    g = ss.residual_norm_bwd(zero + 1, r, w)
    assert torch.isfinite(g["dx"]).all()
    assert not ss.gated_norm_fwd(zero, zero, w).any()
    assert torch.isfinite(ss.gated_norm_bwd(zero + 1, zero, zero, w)["dy"]).all()
    empty = zero[:0]
    assert ss.residual_norm_fwd(empty, w)[0].shape == (0, 64)
    assert not ss.gated_norm_bwd(empty, empty, empty, w)["dweight"].any()


def test_refusals(ss):
    say("norm refusals")
    x, w = torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    for bad in (lambda: ss.residual_norm_fwd(x.half(), w), lambda: ss.residual_norm_fwd(x, w.to(BF16)),
                lambda: ss.residual_norm_fwd(x, w, residual=x.to(BF16)), lambda: ss.gated_norm_fwd(x, x.to(BF16), w)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ss.residual_norm_fwd(x, w[:32]), lambda: ss.residual_norm_fwd(x.t(), torch.ones(4, device=DEV)),
                lambda: ss.gated_norm_fwd(x, x[:2], w), lambda: ss.residual_norm_bwd(x, x, w, scale=w),
                lambda: ss.gated_norm_fwd(x.cpu(), x, w)):
        with pytest.raises(ValueError):
            bad()
    for bad, code in ((lambda: ss.gated_norm_fwd(x, x, w, groups=5), -2), (lambda: ss.gated_norm_fwd(x, x, w, groups=0), -2),
                      (lambda: ss.gated_norm_fwd(x, x, w, eps=-1.0), -2), (lambda: ss.gated_norm_fwd(x, x, w, out=x), -7),
                      (lambda: ss.residual_norm_fwd(torch.zeros(1, 16385, device=DEV), torch.ones(16385, device=DEV)), -4),
                      (lambda: ss.residual_norm_fwd(x, w, out=x), -7)):
        with pytest.raises(ss.SSError) as e:
            bad()
        assert e.value.code == code
