"""Cases and plain forms of the operators around the head-wise selective scan.

Operators (names as in the package):

  head_scan_fwd / head_scan_bwd   the recurrence with one decay per head and a (P, N) state per head
  head_state_update               its single-token form on a persistent state
  residual_norm_fwd / _bwd        r = residual + scale * x, out = rmsnorm(r) * weight
  gated_norm_fwd / _bwd           rmsnorm over groups of channels of y * silu(z) (or rmsnorm(y) * silu(z))

With ``own`` false, run() computes them with elementary torch operations in 32 bits; with ``own`` true it calls the
package.  exact() is a step-by-step form in 64 bits.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DEV = "cuda"


def _ss():
    import selective_state_space_softplus_amd as ss

    return ss


# ----------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # Prefill of the long workload: its 5120 channels as 80 heads of 64, x, B and C views of one projection.
        dict(name="scan-fwd-long", op="scan", train=False, b=4, L=8192, H=80, P=64, N=128, G=1, dtype="bf16",
             packed=True, state=True),
        # One prompt of ordinary, odd length at 24 heads (1536 channels), continuing a cached state.
        dict(name="scan-fwd-prompt", op="scan", train=False, b=1, L=777, H=24, P=64, N=64, G=1, dtype="bf16",
             packed=True, state=True),
        # A training step of the mid workload (b = 8, L = 2048, 1536 channels).
        dict(name="scan-train-mid", op="scan", train=True, b=8, L=2048, H=24, P=64, N=128, G=1, dtype="bf16",
             packed=True, state=False),
        # Training on one long sequence with several B / C groups.
        dict(name="scan-train-long", op="scan", train=True, b=1, L=16384, H=80, P=64, N=128, G=8, dtype="bf16",
             packed=True, state=False),
        # Training in fp32 with odd sizes, an initial state and a gradient of the last state (truncated backward).
        dict(name="scan-train-odd-fp32", op="scan", train=True, b=2, L=1001, H=12, P=33, N=40, G=3, dtype="fp32",
             packed=False, state=True),
        # Decoding one sequence: latency.
        dict(name="step-one", op="step", b=1, H=24, P=64, N=128, G=1, dtype="bf16"),
        # Decoding the decode workload's batch (b = 256, 5120 channels).
        dict(name="step-batch", op="step", b=256, H=80, P=64, N=128, G=1, dtype="bf16"),
        # The norm before a block in training, bf16 activations on an fp32 residual stream, per-channel residual scale.
        dict(name="resnorm-train", op="resnorm", train=True, rows=32768, d=2560, dtype="bf16", res="fp32", scale=True),
        # The same norm while decoding a few sequences.
        dict(name="resnorm-decode", op="resnorm", train=False, rows=7, d=2560, dtype="bf16", res="bf16", scale=False),
        # The norm after the scan in training: the gate and the mean square over all channels.
        dict(name="gatenorm-train", op="gatenorm", train=True, rows=16384, d=5120, groups=1, dtype="bf16", before=False),
        # The same in fp32 with odd sizes and groups, the norm taken before the gate.
        dict(name="gatenorm-odd-fp32", op="gatenorm", train=True, rows=1001, d=1995, groups=3, dtype="fp32",
             before=True),
        # The norm after the scan while decoding a batch, per group.
        dict(name="gatenorm-decode", op="gatenorm", train=False, rows=256, d=5120, groups=8, dtype="bf16",
             before=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One case of the listed ones' ranges (3072, a size that no workload here has, is drawn again)."""
    while True:
        case = _draw(rng)
        if 3072 not in list(case.values()) + [case.get("H", 0) * case.get("P", 0)]:
            return case


def _draw(rng):
    kind = rng.choice(["scan", "scan", "scan-train", "scan-train", "step", "resnorm", "gatenorm"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind == "step":
        G = rng.choice([1, 1, 2, 5])
        H = G * _log_int(rng, 1, 80 // G)
        b = _log_int(rng, 1, 256)
        return dict(op="step", b=b, H=H, P=rng.choice([16, 33, 64, 64, 80 if H <= 40 else 64]),
                    N=rng.choice([16, 31, 64, 128]), G=G, dtype=dtype)
    if kind in ("scan", "scan-train"):
        train = kind == "scan-train"
        # fp32 products run at a sixteenth of the bf16 rate, and a training step costs several forwards.
        most = (4 * 8192 * 5120 if not train else 16384 * 5120) // (1 if dtype == "bf16" else 16)
        G = rng.choice([1, 1, 2, 4])
        H = G * _log_int(rng, 1, 80 // G)
        P = rng.choice([16, 33, 40, 64, 64, 64, 80, 112])
        L = _log_int(rng, 1, 16384)
        while L * H * P > most:
            L = max(1, L // 2) | 1
        b = _log_int(rng, 1, max(1, min(16, most // (L * H * P))))
        return dict(op="scan", train=train, b=b, L=L, H=H, P=P, N=rng.choice([8, 16, 31, 64, 64, 100, 128]), G=G,
                    dtype=dtype, packed=rng.random() < 0.5, state=rng.random() < 0.5)
    d = _log_int(rng, 64, 8192) | rng.choice([0, 1])
    rows = _log_int(rng, 1, min(32768, 16384 * 5120 // d // (1 if dtype == "bf16" else 2)))
    if kind == "resnorm":
        train = rng.random() < 0.6
        res = "fp32" if train or dtype == "fp32" else rng.choice(["bf16", "fp32"])
        return dict(op="resnorm", train=train, rows=rows, d=d, dtype=dtype, res=res, scale=rng.random() < 0.5)
    groups = rng.choice([1, 1, 2, 3, 8])
    d = max(1, d // groups) * groups
    return dict(op="gatenorm", train=rng.random() < 0.6, rows=rows, d=d, groups=groups, dtype=dtype,
                before=rng.random() < 0.3)


# ---------------------------------------------------------------------------------------------------------- the inputs

EPS = 1e-5


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = BF16 if case["dtype"] == "bf16" else F32

    def normal(*shape, dtype=dt, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale + mean).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device=DEV) * (hi - lo) + lo

    s = dict(case=dict(case))
    if case["op"] in ("scan", "step"):
        b, H, P, N, G = (case[k] for k in ("b", "H", "P", "N", "G"))
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))   # the initialisation of the step size
        s["bias"] = step + torch.log(-torch.expm1(-step))              # its inverse softplus
        s["A_log"] = torch.log(uniform(1.0, 16.0, H))
        s["D"] = normal(H, dtype=F32)
    if case["op"] == "scan":
        L = case["L"]
        if case["packed"]:
            # x, B and C lie side by side in each token's row, as one projection leaves them.
            row = normal(b, L, H * P + 2 * G * N)
            s["x"] = row[..., :H * P].unflatten(-1, (H, P))
            s["B"] = row[..., H * P:H * P + G * N].unflatten(-1, (G, N))
            s["C"] = row[..., H * P + G * N:].unflatten(-1, (G, N))
        else:
            s["x"], s["B"], s["C"] = normal(b, L, H, P), normal(b, L, G, N), normal(b, L, G, N)
        s["delta"] = normal(b, L, H)
        s["h0"] = normal(b, H, P, N, dtype=F32, scale=0.3) if case["state"] else None
        if case["train"]:
            s["dy"] = normal(b, L, H, P)
            s["dlast"] = normal(b, H, P, N, dtype=F32, scale=0.3) if case["state"] else None
    elif case["op"] == "step":
        s["x"], s["B"], s["C"] = normal(b, H, P), normal(b, G, N), normal(b, G, N)
        s["delta"] = normal(b, H)
        s["h"] = normal(b, H, P, N, dtype=F32, scale=0.3)
    elif case["op"] == "resnorm":
        rows, d = case["rows"], case["d"]
        rt = BF16 if case["res"] == "bf16" else F32
        s["x"], s["residual"] = normal(rows, d), normal(rows, d, dtype=rt, scale=2.0)
        s["w"] = normal(d, dtype=F32, scale=0.2, mean=1.0)
        s["scale"] = normal(d, dtype=F32, scale=0.1, mean=0.5) if case["scale"] else None
        if case["train"]:
            s["dout"], s["dres"] = normal(rows, d), normal(rows, d, dtype=rt)
    else:
        rows, d = case["rows"], case["d"]
        s["y"], s["z"] = normal(rows, d), normal(rows, d)
        s["w"] = normal(d, dtype=F32, scale=0.2, mean=1.0)
        if case["train"]:
            s["dout"] = normal(rows, d)
    return s


# ------------------------------------------------------------------------------------------------------ the plain forms

CHUNK = 64


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _plain_scan(x, delta, A_log, B, C, D, bias, h0):
    """The recurrence over chunks of the sequence: products inside a chunk, and the chunks' states joined by the decays
    between chunks.  All in fp32."""
    b, L, H, P = x.shape
    G, N = B.shape[2:]
    nc = -(-L // CHUNK)
    pad = nc * CHUNK - L
    step = _softplus(delta + bias)
    logs = -torch.exp(A_log) * step

    def chunks(t):          # (b, L, H, k) -> (b, H, nc, CHUNK, k)
        t = torch.cat([t, t.new_zeros(b, pad, *t.shape[2:])], 1) if pad else t
        return t.reshape(b, nc, CHUNK, t.shape[2], -1).permute(0, 3, 1, 2, 4)

    xc, sc, gc = chunks(x), chunks(step.unsqueeze(-1)), chunks(logs.unsqueeze(-1)).squeeze(-1)
    Bc = chunks(B).repeat_interleave(H // G, 1)
    Cc = chunks(C).repeat_interleave(H // G, 1)
    cum = torch.cumsum(gc, -1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp((cum.unsqueeze(-1) - cum.unsqueeze(-2)).masked_fill(~lower, float("-inf")))
    xs = xc * sc
    y = ((Cc @ Bc.transpose(-1, -2)) * decay) @ xs
    local = xs.transpose(-1, -2) @ (Bc * torch.exp(cum[..., -1:] - cum).unsqueeze(-1))      # (b, H, nc, P, N)
    # Decay from the end of chunk j to the start of chunk i, j < i (column 0: from the initial state): the sums over
    # the chunks between are formed term by term.
    total = torch.cat([torch.zeros_like(cum[..., :1, -1]), cum[..., -1]], -1)               # (b, H, nc + 1)
    k = torch.arange(nc + 1, device=x.device)
    between = torch.cumsum(total.unsqueeze(-1).expand(-1, -1, -1, nc + 1).masked_fill(k[:, None] <= k[None, :], 0.0), -2)
    carry = torch.exp(between.masked_fill(k[:, None] < k[None, :], float("-inf")))
    first = h0.unsqueeze(2) if h0 is not None else local.new_zeros(b, H, 1, P, N)
    states = (carry @ torch.cat([first, local], 2).flatten(-2)).unflatten(-1, (P, N))       # at every chunk's start, and the end
    y = y + (Cc * torch.exp(cum).unsqueeze(-1)) @ states[:, :, :-1].transpose(-1, -2)
    y = y.permute(0, 2, 3, 1, 4).reshape(b, nc * CHUNK, H, P)[:, :L] + D[:, None] * x
    return y, states[:, :, -1]


def _plain_resnorm(x, residual, w, scale, rt):
    r = residual + (x if scale is None else x * scale)
    r = r + (r.detach().to(rt).float() - r.detach())     # the residual stream as it is stored
    return r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * w, r


def _plain_gatenorm(y, z, w, groups, before):
    gate = z / (1 + torch.exp(-z))
    v = (y if before else y * gate).unflatten(-1, (groups, -1))
    v = (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)).flatten(-2) * w
    return v * gate if before else v


def _wide(t, grad):
    return None if t is None else t.detach().float().requires_grad_(grad)


def _grads(outs, weights, wrt):
    """Gradients of the pairs' sum of products, with respect to the tensors of the dict ``wrt`` that are there."""
    keys = [k for k, v in wrt.items() if v is not None]
    pairs = [(o, w.float()) for o, w in zip(outs, weights) if w is not None]
    got = torch.autograd.grad([o for o, _ in pairs], [wrt[k] for k in keys], [w for _, w in pairs])
    return dict(zip(keys, got))


def _run_plain(s):
    c = s["case"]
    if c["op"] == "scan":
        names = ("x", "delta", "A_log", "B", "C", "D", "bias", "h0")
        t = {k: _wide(s[k], c["train"]) for k in names}
        y, last = _plain_scan(*(t[k] for k in names))
        out = dict(y=y.detach().to(s["x"].dtype))
        if c["state"]:
            out["last"] = last.detach()
        if c["train"]:
            g = _grads((y, last), (s["dy"], s["dlast"]), t)
            out.update({"d" + k: v.to(s[k].dtype) for k, v in g.items()})
        return out
    if c["op"] == "step":
        x, B, C, h = s["x"].float(), s["B"].float(), s["C"].float(), s["h"]
        rep = c["H"] // c["G"]
        step = _softplus(s["delta"].float() + s["bias"])
        B, C = (t.repeat_interleave(rep, 1).unsqueeze(2) for t in (B, C))
        h.mul_(torch.exp(-torch.exp(s["A_log"]) * step)[..., None, None]).add_((step.unsqueeze(-1) * x).unsqueeze(-1) * B)
        y = (h * C).sum(-1) + s["D"][:, None] * x
        return dict(y=y.to(s["x"].dtype), h=h)
    if c["op"] == "resnorm":
        rt = s["residual"].dtype
        t = {k: _wide(s[k], c["train"]) for k in ("x", "residual", "w", "scale")}
        out, r = _plain_resnorm(t["x"], t["residual"], t["w"], t["scale"], rt)
        got = dict(out=out.detach().to(s["x"].dtype), r=r.detach().to(rt))
        if c["train"]:
            g = _grads((out, r), (s["dout"], s["dres"]), t)
            got.update({"d" + k: v.to(s[k].dtype) for k, v in g.items()})
        return got
    t = {k: _wide(s[k], c["train"]) for k in ("y", "z", "w")}
    out = _plain_gatenorm(t["y"], t["z"], t["w"], c["groups"], c["before"])
    got = dict(out=out.detach().to(s["y"].dtype))
    if c["train"]:
        g = _grads((out,), (s["dout"],), t)
        got.update({"d" + k: v.to(s[k].dtype) for k, v in g.items()})
    return got


# --------------------------------------------------------------------------------------------------- the package's calls

def _run_own(s):
    ss, c = _ss(), s["case"]
    if c["op"] == "scan":
        args = (s["x"], s["delta"], s["A_log"], s["B"], s["C"], s["D"])
        out = {}
        if c["state"]:
            out["y"], out["last"] = ss.head_scan_fwd(*args, delta_bias=s["bias"], initial_state=s["h0"],
                                                     return_last_state=True)
        else:
            out["y"] = ss.head_scan_fwd(*args, delta_bias=s["bias"])
        if c["train"]:
            g = ss.head_scan_bwd(*args, s["dy"], delta_bias=s["bias"], initial_state=s["h0"], dlast_state=s["dlast"])
            out.update(dx=g["dx"], ddelta=g["ddelta"], dA_log=g["dA_log"], dB=g["dB"], dC=g["dC"], dD=g["dD"],
                       dbias=g["ddelta_bias"])
            if c["state"]:
                out["dh0"] = g["dinitial_state"]
        return out
    if c["op"] == "step":
        y = ss.head_state_update(s["h"], s["x"], s["delta"], s["A_log"], s["B"], s["C"], s["D"], dt_bias=s["bias"])
        return dict(y=y, h=s["h"])
    if c["op"] == "resnorm":
        out, r = ss.residual_norm_fwd(s["x"], s["w"], residual=s["residual"], scale=s["scale"], eps=EPS)
        got = dict(out=out, r=r)
        if c["train"]:
            g = ss.residual_norm_bwd(s["dout"], r, s["w"], dresidual_out=s["dres"], x=s["x"], scale=s["scale"], eps=EPS)
            got.update(dx=g["dx"], dresidual=g["dresidual"], dw=g["dweight"])
            if s["scale"] is not None:
                got["dscale"] = g["dscale"]
        return got
    got = dict(out=ss.gated_norm_fwd(s["y"], s["z"], s["w"], groups=c["groups"], eps=EPS, norm_before_gate=c["before"]))
    if c["train"]:
        g = ss.gated_norm_bwd(s["dout"], s["y"], s["z"], s["w"], groups=c["groups"], eps=EPS,
                              norm_before_gate=c["before"])
        got.update(dy=g["dy"], dz=g["dz"], dw=g["dweight"])
    return got


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("scan", "step"):
        b, H, P, N, G = (case[k] for k in ("b", "H", "P", "N", "G"))
        L = case.get("L", 1)
        rows = b * L
        args = e * rows * (H * P + H + 2 * G * N) + 12 * H           # x, delta, B, C and the heads' parameters
        y = e * rows * H * P
        state = 4 * b * H * P * N
        # A step of one head: the update of its state and the readout, a multiply-add for each state element.
        flops = 4.0 * rows * H * P * N
        if case["op"] == "step":
            return dict(bytes=args + y + 2 * state, flops=flops)
        total = args + y + (2 * state if case["state"] else 0)
        if case["train"]:
            # The backward reads the arguments and dy again and writes a gradient for each argument; it forms the
            # adjoint state and the products for x, B and C.
            total += args + y + args + (3 * state if case["state"] else 0)
            flops += 10.0 * rows * H * P * N
        return dict(bytes=total, flops=flops)
    n, d = case["rows"] * case["d"], case["d"]
    if case["op"] == "resnorm":
        er = 2 if case["res"] == "bf16" else 4
        params = 4 * d * (2 if case["scale"] else 1)
        total = n * (2 * e + 2 * er) + params                        # x, residual, out, r
        if case["train"]:
            # dout, r, its gradient (and x for the scale's) read; dx, dresidual and the parameters' written
            total += n * (2 * e + 3 * er + (e if case["scale"] else 0)) + 2 * params
        return dict(bytes=total, flops=n * (6.0 + (12.0 if case["train"] else 0.0)))
    total = n * 3 * e + 4 * d
    if case["train"]:
        total += n * 5 * e + 8 * d                                   # dout, y, z read; dy, dz written
    return dict(bytes=total, flops=n * (10.0 + (25.0 if case["train"] else 0.0)))


# ----------------------------------------------------------------------------------- step by step, in 64 bits

def _exact_scan(s):
    c = s["case"]
    b, L, H, P, N, G = (c[k] for k in ("b", "L", "H", "P", "N", "G"))
    R = H // G
    x = s["x"].double().reshape(b, L, G, R, P)
    B, C = s["B"].double(), s["C"].double()
    raw = s["delta"].double() + s["bias"].double()
    step = torch.logaddexp(raw, torch.zeros_like(raw)).reshape(b, L, G, R)
    A = -torch.exp(s["A_log"].double()).reshape(G, R)
    D = s["D"].double().reshape(G, R)
    a = torch.exp(step * A)
    xs = x * step.unsqueeze(-1)
    h = x.new_zeros(b, G, R, P, N) if s["h0"] is None else s["h0"].double().reshape(b, G, R, P, N).clone()
    seg = 128
    kept, ys = [], []

    def advance(h, t):
        return h * a[:, t, :, :, None, None] + xs[:, t].unsqueeze(-1) * B[:, t, :, None, None, :]

    for t in range(L):
        if c["train"] and t % seg == 0:
            kept.append(h)
        h = advance(h, t)
        ys.append(torch.matmul(h.reshape(b, G, R * P, N), C[:, t].unsqueeze(-1)).reshape(b, G, R, P))
    y = torch.stack(ys, 1) + D.unsqueeze(-1) * x
    out = dict(y=y.reshape(b, L, H, P))
    if c["state"]:
        out["last"] = h.reshape(b, H, P, N)
    if not c["train"]:
        return out
    dy = s["dy"].double().reshape(b, L, G, R, P)
    q = torch.zeros_like(h) if s["dlast"] is None else s["dlast"].double().reshape(b, G, R, P, N).clone()
    dxs, dB, dC, dlog = torch.empty_like(x), torch.empty_like(B), torch.empty_like(C), torch.empty_like(step)
    for k in reversed(range(len(kept))):
        hs = [kept[k]]
        end = min(L, (k + 1) * seg)
        for t in range(k * seg, end):
            hs.append(advance(hs[-1], t))
        for t in reversed(range(k * seg, end)):
            now, before = hs[t - k * seg + 1], hs[t - k * seg]
            dC[:, t] = torch.matmul(dy[:, t].reshape(b, G, 1, R * P), now.reshape(b, G, R * P, N)).squeeze(2)
            q = q + dy[:, t].unsqueeze(-1) * C[:, t, :, None, None, :]
            dB[:, t] = torch.matmul(xs[:, t].reshape(b, G, 1, R * P), q.reshape(b, G, R * P, N)).squeeze(2)
            dxs[:, t] = torch.matmul(q.reshape(b, G, R * P, N), B[:, t].unsqueeze(-1)).reshape(b, G, R, P)
            q = q * a[:, t, :, :, None, None]
            dlog[:, t] = (q * before).sum((-1, -2))        # d/d(step A): the decay times its own derivative's factor
        del hs
    dx = dxs * step.unsqueeze(-1) + D.unsqueeze(-1) * dy
    dstep = dlog * A + (dxs * x).sum(-1)
    ddelta = dstep.reshape(b, L, H) * torch.sigmoid(raw)
    out.update(dx=dx.reshape(b, L, H, P), ddelta=ddelta, dA_log=(dlog * step * A).sum((0, 1)).reshape(H), dB=dB, dC=dC,
               dD=(dy * x).sum((0, 1, 4)).reshape(H), dbias=ddelta.sum((0, 1)))
    if c["state"]:
        out["dh0"] = q.reshape(b, H, P, N)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "scan":
        return _exact_scan(s)
    if c["op"] == "step":
        b, H, P, N, G = (c[k] for k in ("b", "H", "P", "N", "G"))
        raw = s["delta"].double() + s["bias"].double()
        step = torch.logaddexp(raw, torch.zeros_like(raw))
        head = torch.arange(H, device=DEV) // (H // G)
        a = torch.exp(-torch.exp(s["A_log"].double()) * step)
        x = s["x"].double()
        h = s["h"].double() * a[:, :, None, None]
        h += torch.einsum("bhp,bhn->bhpn", x * step.unsqueeze(-1), s["B"].double()[:, head])
        y = torch.einsum("bhpn,bhn->bhp", h, s["C"].double()[:, head]) + s["D"].double()[:, None] * x
        return dict(y=y, h=h)
    if c["op"] == "resnorm":
        x, w = s["x"].double(), s["w"].double()
        k = torch.ones_like(w) if s["scale"] is None else s["scale"].double()
        r = (s["residual"].double() + k * x)
        r = r.to(s["residual"].dtype).double() if c["res"] == "bf16" else r
        inv = 1 / torch.sqrt((r * r).sum(-1, keepdim=True) / c["d"] + EPS)
        got = dict(out=r * inv * w, r=r)
        if c["train"]:
            dout = s["dout"].double()
            hat = r * inv
            dr = s["dres"].double() + inv * (dout * w - hat * ((dout * w * hat).sum(-1, keepdim=True) / c["d"]))
            got.update(dx=dr * k, dresidual=dr, dw=(dout * hat).sum(0))
            if c["scale"]:
                got["dscale"] = (dr * x).sum(0)
        return got
    shape = (c["rows"], c["groups"], c["d"] // c["groups"])
    y, z = s["y"].double().reshape(shape), s["z"].double().reshape(shape)
    w = s["w"].double().reshape(shape[1:])
    sig = torch.sigmoid(z)
    gate = z * sig
    v = y if c["before"] else y * gate
    inv = 1 / torch.sqrt((v * v).sum(-1, keepdim=True) / shape[2] + EPS)
    hat = v * inv
    o = hat * w * gate if c["before"] else hat * w
    got = dict(out=o.reshape(c["rows"], c["d"]))
    if c["train"]:
        dout = s["dout"].double().reshape(shape)
        dn = dout * gate if c["before"] else dout                    # gradient of hat * w
        dv = inv * (dn * w - hat * ((dn * w * hat).sum(-1, keepdim=True) / shape[2]))
        dgate = dout * hat * w if c["before"] else dv * y
        got.update(dy=(dv if c["before"] else dv * gate).reshape(c["rows"], c["d"]),
                   dz=(dgate * (sig + gate * (1 - sig))).reshape(c["rows"], c["d"]),
                   dw=(dn * hat).sum(0).reshape(c["d"]))
    return got
