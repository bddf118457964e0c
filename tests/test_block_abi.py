"""CPU: the C ABI of ss_block.h -- every declared entry point is exported and bound, sizes of workspaces, and bad
arguments rejected with the documented status before the GPU is touched (the pointers are fake addresses that
validation never dereferences)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ss_block.h")

NULL, SHAPE, DTYPE, UNSUP, WS, ALIAS, ALIGN = -1, -2, -3, -4, -5, -7, -8


@pytest.fixture(scope="module")
def ss():
    import selective_state_space_softplus_amd as ss

    return ss


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return set(re.findall(r"\b(ss_[a-z_]+)\s*\(", text))


def test_declared_exported_and_bound(ss):
    from selective_state_space_softplus_amd import block

    lib = ctypes.CDLL(ss.LIBRARY)
    assert declared() == set(block.EXPORTS)
    for name in declared():
        assert hasattr(lib, name), name
        assert getattr(ss.lib, name).argtypes
    text = open(HEADER).read()
    for name in ("SS_MAX_HEAD_STATE", "SS_MAX_HEAD_DIM", "SS_MAX_NORM_CHANNELS"):
        assert re.search(rf"#define {name} {getattr(block, name)}\b", text), name


BASE = 1 << 40


def addr(i):
    return BASE + i * (1 << 36)


def fwd(ss, **over):
    a = dict(x=addr(1), delta=addr(2), A_log=addr(3), B=addr(4), C=addr(5), D=addr(6), bias=addr(7), sp=1, h0=addr(8),
             y=addr(9), last=addr(10), b=2, L=3000, H=4, P=64, N=64, G=2, dtype=1, strides=None, ws=addr(11),
             bytes=1 << 34, stream=None)
    a.update(over)
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_int64 * 8)(*a["strides"])
    return ss.lib.ss_head_scan_fwd(*a.values())


FWD_CASES = [
    (dict(x=None), NULL), (dict(delta=None), NULL), (dict(A_log=None), NULL), (dict(B=None), NULL),
    (dict(C=None), NULL), (dict(D=None), NULL), (dict(y=None), NULL),
    (dict(b=0), SHAPE), (dict(L=0), SHAPE), (dict(H=-4), SHAPE), (dict(P=0), SHAPE), (dict(N=0), SHAPE),
    (dict(G=0), SHAPE), (dict(G=3), SHAPE), (dict(G=8), SHAPE), (dict(L=1 << 31), SHAPE),
    (dict(b=1 << 20, L=1 << 20, H=1 << 10), SHAPE), (dict(b=1 << 12, L=1 << 18, H=4, P=64), SHAPE),
    (dict(H=1 << 19, G=1, b=1, L=64), SHAPE),
    (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
    (dict(N=129), UNSUP), (dict(P=1025), UNSUP),
    (dict(strides=[0, -1] + [0, 8] * 3), SHAPE), (dict(strides=[0, (1 << 24) + 1] + [0, 8] * 3), SHAPE),
    (dict(ws=None), WS), (dict(bytes=256), WS), (dict(ws=addr(11) + 128), ALIGN),
    (dict(x=addr(1) + 1), ALIGN), (dict(dtype=0, B=addr(4) + 2), ALIGN), (dict(h0=addr(8) + 2), ALIGN),
    (dict(y=addr(1) + 64), ALIAS), (dict(last=addr(5)), ALIAS), (dict(ws=addr(9)), ALIAS), (dict(last=addr(8) + 4), ALIAS),
    (dict(y=addr(8)), ALIAS),
]


@pytest.mark.parametrize("over,code", FWD_CASES)
def test_forward_rejects(ss, over, code):
    assert fwd(ss, **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(dB=None), NULL), (dict(dD=None), NULL), (dict(dA=None), NULL),
    (dict(G=3), SHAPE), (dict(dtype=5), DTYPE), (dict(N=200), UNSUP), (dict(ws=None), WS), (dict(bytes=1000), WS),
    (dict(dx=addr(1)), ALIAS), (dict(dB=addr(16)), ALIAS), (dict(dh0=addr(8)), ALIAS), (dict(ws=addr(2)), ALIAS),
    (dict(dy=addr(9) + 1), ALIGN), (dict(dA=addr(13) + 2), ALIGN), (dict(ws=addr(20) + 64), ALIGN),
])
def test_backward_rejects(ss, over, code):
    a = dict(x=addr(1), delta=addr(2), A_log=addr(3), B=addr(4), C=addr(5), D=addr(6), bias=addr(7), sp=1, h0=addr(8),
             dy=addr(9), dlast=addr(10), dx=addr(11), dd=addr(12), dA=addr(13), dB=addr(15), dC=addr(16), dD=addr(17),
             db=addr(18), dh0=addr(19), b=2, L=300, H=4, P=64, N=64, G=2, dtype=1, strides=None, ws=addr(20),
             bytes=1 << 34, stream=None)
    a.update(over)
    assert ss.lib.ss_head_scan_bwd(*a.values()) == code


@pytest.mark.parametrize("over,code", [
    (dict(state=None), NULL), (dict(y=None), NULL), (dict(H=3), SHAPE), (dict(b=0), SHAPE), (dict(b=1 << 24), SHAPE),
    (dict(dtype=9), DTYPE), (dict(N=130), UNSUP), (dict(P=2000), UNSUP), (dict(state=addr(1) + 2), ALIGN),
    (dict(y=addr(2)), ALIAS), (dict(state=addr(5)), ALIAS), (dict(y=addr(1)), ALIAS),
])
def test_step_rejects(ss, over, code):
    a = dict(state=addr(1), x=addr(2), dt=addr(3), A_log=addr(4), B=addr(5), C=addr(6), D=addr(7), bias=None, sp=1,
             y=addr(8), b=2, H=4, P=64, N=64, G=2, dtype=1, stream=None)
    a.update(over)
    assert ss.lib.ss_head_state_update(*a.values()) == code


def test_norms_reject(ss):
    lib = ss.lib
    good = dict(x=addr(1), res=addr(2), scale=addr(3), w=addr(4), out=addr(5), ro=addr(6), rows=8, d=64, eps=1e-5, dt=1,
                rt=0, xs=64, stream=None)
    for over, code in ((dict(x=None), NULL), (dict(ro=None), NULL), (dict(rows=0), SHAPE), (dict(d=0), SHAPE),
                       (dict(xs=63), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
                       (dict(d=16385, xs=16385), UNSUP), (dict(dt=3), DTYPE), (dict(dt=0, rt=1), DTYPE),
                       (dict(w=addr(4) + 1), ALIGN), (dict(out=addr(1)), ALIAS), (dict(ro=addr(2) + 4), ALIAS),
                       (dict(out=addr(6)), ALIAS)):
        assert lib.ss_residual_norm_fwd(*dict(good, **over).values()) == code, over
    good = dict(dout=addr(1), dro=addr(2), ro=addr(3), x=addr(4), scale=addr(5), w=addr(6), dx=addr(7), dres=addr(8),
                dw=addr(9), ds=addr(10), rows=8, d=64, eps=1e-5, dt=1, rt=0, xs=64, ws=addr(11), bytes=1 << 30, stream=None)
    for over, code in ((dict(dout=None), NULL), (dict(ds=None), NULL), (dict(x=None), NULL), (dict(scale=None), NULL),
                       (dict(ws=None), WS), (dict(bytes=0), WS), (dict(ws=addr(11) + 8), ALIGN), (dict(dx=addr(8)), ALIAS),
                       (dict(dw=addr(11)), ALIAS), (dict(rt=7), DTYPE), (dict(d=20000, xs=20000), UNSUP)):
        assert lib.ss_residual_norm_bwd(*dict(good, **over).values()) == code, over
    good = dict(y=addr(1), z=addr(2), w=addr(3), out=addr(4), rows=8, d=64, groups=4, eps=1e-5, before=0, dt=1, ys=64,
                zs=100, stream=None)
    for over, code in ((dict(z=None), NULL), (dict(groups=5), SHAPE), (dict(groups=0), SHAPE), (dict(zs=10), SHAPE),
                       (dict(dt=2), DTYPE), (dict(out=addr(2) + 64), ALIAS), (dict(y=addr(1) + 1), ALIGN),
                       (dict(d=16385 * 2, groups=2, ys=40000, zs=40000), UNSUP)):
        assert lib.ss_gated_norm_fwd(*dict(good, **over).values()) == code, over


def test_workspace_sizes(ss):
    fwd_ws, bwd_ws = ss.lib.ss_head_scan_fwd_workspace_bytes, ss.lib.ss_head_scan_bwd_workspace_bytes
    assert fwd_ws(4, 64, 80, 64, 128, 1, 1) == 0                     # one chunk: nothing to carry
    assert fwd_ws(1, 8192, 8, 64, 128, 1, 1) >= 8 * 64 * 128 * 4     # segments of one sequence
    # The backward keeps the state and its adjoint at every chunk.
    assert bwd_ws(1, 6400, 8, 64, 128, 1, 1) >= 2 * 100 * 8 * 64 * 128 * 4
    for bad in ((0, 1, 1, 1, 1, 1, 0), (1, 0, 1, 1, 1, 1, 0), (1, 1, 4, 1, 1, 3, 0), (1, 1, 1, 1, 129, 1, 0),
                (1, 1, 1, 1, 1, 1, 4)):
        assert fwd_ws(*bad) == 0 and bwd_ws(*bad) == 0, bad
    assert ss.lib.ss_residual_norm_bwd_workspace_bytes(100, 64) > 0
    assert ss.lib.ss_residual_norm_bwd_workspace_bytes(0, 64) == 0
    assert ss.lib.ss_gated_norm_bwd_workspace_bytes(100, 64, 3) == 0


def test_bindings_need_a_gpu_tensor_set(ss):
    """The checks that come before the library: types and shapes, on CPU tensors."""
    import torch

    x = torch.zeros(1, 4, 4, 8)
    B = torch.zeros(1, 4, 2, 8)
    v = torch.zeros(4)
    with pytest.raises(ValueError):
        ss.head_scan_fwd(x[0], torch.zeros(1, 4, 4), v, B, B, v)
    with pytest.raises(ValueError):
        ss.head_scan_fwd(x, torch.zeros(1, 4, 4), v, B[:, :, :0], B[:, :, :0], v)
    with pytest.raises(TypeError):
        ss.head_scan_fwd(x.double(), torch.zeros(1, 4, 4).double(), v, B.double(), B.double(), v)
    with pytest.raises(ValueError):
        ss.gated_norm_fwd(torch.zeros(()), torch.zeros(()), v)
