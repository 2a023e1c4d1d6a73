"""What the linear attention and block norm entry points refuse, through the C ABI and the
binding, without a GPU: every refusal comes before anything reaches a device.  Pointers
here are fake addresses, never dereferenced; no call with valid arguments is made."""
import ctypes

import pytest
import torch

import selective_state_space_68_amd as ssm
from selective_state_space_68_amd import _lib

F = 0x100000          # fake, 1 MiB-aligned device addresses
MB = 1 << 20
INV, UNS = _lib.SSM_ERR_INVALID_ARG, _lib.SSM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return _lib.load_library()


def at(i):
    return F + i * 64 * MB


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def fwd(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), qs=None, ks=None, vs=None, g=at(3), scale=1.0, n=None, s0=None, o=at(4),
             fin=at(5), B=2, L=64, H=4, Hq=4, Hk=2, Hv=1, K=64, V=32, dt=1, ws=at(8), ws_bytes=32 * MB)
    a.update(kw)
    return lib.ssm_linear_attention_fwd(
        a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["scale"], a["n"], a["s0"], a["o"], a["fin"], a["B"],
        a["L"], a["H"], a["Hq"], a["Hk"], a["Hv"], a["K"], a["V"], a["dt"], a["ws"], a["ws_bytes"], None)


def bwd(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), d=at(3), qs=None, ks=None, vs=None, ds=None, g=at(4), scale=1.0, n=None, s0=None,
             df=None, dq=at(5), dk=at(6), dv=at(7), d0=at(9), B=2, L=64, H=4, Hq=4, Hk=2, Hv=1, K=64, V=32, dt=1,
             ws=at(10), ws_bytes=32 * MB)
    a.update(kw)
    return lib.ssm_linear_attention_bwd(
        a["q"], a["k"], a["v"], a["d"], a["qs"], a["ks"], a["vs"], a["ds"], a["g"], a["scale"], a["n"], a["s0"], a["df"],
        a["dq"], a["dk"], a["dv"], a["d0"], a["B"], a["L"], a["H"], a["Hq"], a["Hk"], a["Hv"], a["K"], a["V"], a["dt"],
        a["ws"], a["ws_bytes"], None)


def step(lib, **kw):
    a = dict(si=at(0), so=at(0), q=at(1), k=at(2), v=at(3), qs=None, ks=None, vs=None, g=at(4), scale=1.0, slots=None,
             o=at(5), B=3, S=3, H=4, Hq=4, Hk=2, Hv=1, K=64, V=32, dt=1)
    a.update(kw)
    return lib.ssm_linear_attention_step(
        a["si"], a["so"], a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["scale"], a["slots"], a["o"],
        a["B"], a["S"], a["H"], a["Hq"], a["Hk"], a["Hv"], a["K"], a["V"], a["dt"], None)


COMMON = [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(g=None), INV),
    (dict(B=-1), INV), (dict(H=-4), INV),
    (dict(Hq=3), INV), (dict(Hk=0), INV), (dict(Hv=8), INV),
    (dict(K=0), UNS), (dict(K=129), UNS), (dict(V=0), UNS), (dict(V=129), UNS), (dict(dt=2), UNS),
    (dict(q=at(0) + 1), INV), (dict(g=at(3) + 2), INV),
    (dict(B=1 << 40), UNS), (dict(H=1 << 17, Hq=1, Hk=1, Hv=1), UNS),
]
PROMPT = COMMON + [
    (dict(L=-1), INV), (dict(L=1 << 30), UNS), (dict(B=1 << 20, H=2, Hq=1, Hk=1, Hv=1), UNS),
    (dict(qs=strides(-1, 256, 64)), INV), (dict(vs=strides(1 << 62, 256, 64)), INV),
    (dict(n=at(3) + 2), INV), (dict(s0=at(12) + 2), INV), (dict(ws=at(8) + 8), INV), (dict(ws=None), INV),
]


@pytest.mark.parametrize("kw,status", PROMPT + [
    (dict(o=None), INV), (dict(o=at(0)), INV), (dict(o=at(0) + 64), INV), (dict(o=at(3)), INV),
    (dict(fin=at(1)), INV), (dict(fin=at(4) + 256), INV), (dict(fin=at(5) + 2), INV),
    (dict(s0=at(4)), INV), (dict(s0=at(5) + 64), INV),               # partly under the final state
    (dict(ws=at(2)), INV), (dict(ws=at(4)), INV), (dict(ws=at(5)), INV), (dict(s0=at(8)), INV),
    (dict(n=at(4)), INV),                                           # lengths inside the output
    (dict(q=at(0), qs=strides(0, 0, 0), o=at(0) + 64, K=64), INV),  # a broadcast view's one row
    (dict(L=8192, B=1, ws_bytes=4096), INV),                        # less than the queried workspace
])
def test_forward_refuses(lib, kw, status):
    assert fwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", PROMPT + [
    (dict(d=None), INV), (dict(dq=None), INV), (dict(dk=None), INV), (dict(dv=None), INV),
    (dict(dq=at(0)), INV), (dict(dk=at(3) + 128), INV), (dict(dv=at(5)), INV), (dict(d0=at(6)), INV),
    (dict(df=at(9), d0=at(9)), INV), (dict(ws=at(5)), INV), (dict(ws=at(3)), INV), (dict(ds=strides(-4, 1, 1)), INV),
    (dict(ws_bytes=1024), INV),                                     # shared heads need room for partial sums
])
def test_gradient_refuses(lib, kw, status):
    assert bwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(si=None), INV), (dict(so=None), INV), (dict(o=None), INV), (dict(S=2), INV), (dict(S=-1, slots=at(8)), INV),
    (dict(so=at(0) + 64), INV), (dict(so=at(1)), INV), (dict(o=at(2)), INV), (dict(o=at(0) + 128), INV),
    (dict(slots=at(8) + 2), INV), (dict(slots=at(5)), INV), (dict(si=at(0) + 2, so=at(0) + 2), INV),
    (dict(ks=strides(-1, 64)), INV),
])
def test_step_refuses(lib, kw, status):
    assert step(lib, **kw) == status


def test_workspace_sizes(lib):
    size, gsize = lib.ssm_linear_attention_workspace_size, lib.ssm_linear_attention_bwd_workspace_size
    assert size(8, 2048, 32, 128, 128, 1) == 0                      # a workgroup for every CU: one segment
    assert gsize(8, 2048, 32, 32, 32, 32, 128, 128, 1) == 0
    n = size(1, 131072, 20, 128, 128, 1)
    assert n > 0 and n % (20 * 128 * 128 * 4) == 0                  # one state a head and segment
    assert gsize(8, 2048, 32, 32, 8, 8, 128, 128, 1) == 2 * 8 * 2048 * 32 * 128 * 4   # partial sums of dk and dv
    for bad in (size(-1, 64, 4, 64, 64, 1), size(1, 64, 4, 129, 64, 1), size(1, 64, 4, 64, 64, 9),
                gsize(1, 64, 4, 3, 4, 4, 64, 64, 1), size(0, 64, 4, 64, 64, 1), size(1, 0, 4, 64, 64, 1)):
        assert bad == 0


def nfwd(lib, **kw):
    a = dict(x=at(0), xs=None, res=at(1), gate=at(2), gs=None, w1=at(3), rs=at(4), w2=at(5), h=at(6), y=at(7), rows=8,
             D=64, groups=2, eps=1e-5, dt=1, rdt=0)
    a.update(kw)
    xs, gs = (a["D"] if a[n] is None else a[n] for n in ("xs", "gs"))
    return lib.ssm_block_norm_fwd(a["x"], xs, a["res"], a["gate"], gs, a["w1"], a["rs"], a["w2"], a["h"], a["y"],
                                  a["rows"], a["D"], a["groups"], a["eps"], a["dt"], a["rdt"], None)


def nbwd(lib, **kw):
    a = dict(x=at(0), xs=None, h=at(1), dy=at(2), dh=at(3), gate=at(4), gs=None, w1=at(5), rs=at(6), w2=at(7), dx=at(8),
             dg=at(9), dr=at(10), dw1=at(11), drs=at(12), dw2=at(13), rows=8, D=64, groups=2, eps=1e-5, dt=1, rdt=0,
             ws=at(14), ws_bytes=MB)
    a.update(kw)
    xs, gs = (a["D"] if a[n] is None else a[n] for n in ("xs", "gs"))
    return lib.ssm_block_norm_bwd(a["x"], xs, a["h"], a["dy"], a["dh"], a["gate"], gs, a["w1"], a["rs"], a["w2"],
                                  a["dx"], a["dg"], a["dr"], a["dw1"], a["drs"], a["dw2"], a["rows"], a["D"], a["groups"],
                                  a["eps"], a["dt"], a["rdt"], a["ws"], a["ws_bytes"], None)


NORM = [
    (dict(x=None), INV), (dict(rows=-1), INV), (dict(D=0), UNS), (dict(D=16385), UNS), (dict(D=-1), INV),
    (dict(rows=(1 << 22) + 1), UNS), (dict(groups=0), INV), (dict(groups=3), INV), (dict(groups=16), UNS),
    (dict(D=96, groups=8), UNS), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(dt=3), UNS),
    (dict(rdt=7), UNS), (dict(dt=0, rdt=1), UNS), (dict(xs=63), INV), (dict(gs=10), INV), (dict(x=at(0) + 1), INV),
    (dict(w1=at(5) + 2), INV),
]


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(y=None), INV), (dict(w2=None), INV), (dict(h=None, y=None, w2=None), INV), (dict(h=at(0)), INV),
    (dict(h=at(1) + 64), INV), (dict(y=at(1)), INV), (dict(y=at(2) + 32), INV), (dict(y=at(6)), INV), (dict(h=at(4)), INV),
    (dict(res=at(1) + 2), INV),
])
def test_norm_refuses(lib, kw, status):
    assert nfwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(dx=None), INV), (dict(dy=None), INV), (dict(h=None), INV), (dict(dg=None), INV), (dict(gate=None), INV),
    (dict(dw1=None), INV), (dict(w1=None), INV), (dict(drs=None), INV), (dict(rs=None), INV), (dict(dw2=None), INV),
    (dict(ws=None), INV), (dict(ws_bytes=64), INV), (dict(ws=at(14) + 8), INV), (dict(dx=at(0)), INV),
    (dict(dr=at(3) + 64), INV), (dict(dr=at(1)), INV), (dict(dx=at(3)), INV), (dict(dw1=at(12)), INV),
    (dict(ws=at(10)), INV), (dict(ws=at(3)), INV),
])
def test_norm_gradient_refuses(lib, kw, status):
    assert nbwd(lib, **kw) == status


# ---- the binding: shapes before devices, for tensors on the CPU

def t(*s, dtype=torch.float32):
    return torch.zeros(*s, dtype=dtype)


def attention(**kw):
    a = dict(q=t(2, 8, 4, 16), k=t(2, 8, 2, 16), v=t(2, 8, 1, 24), log_decay=t(4))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,match", [
    (dict(q=t(2, 8, 64)), "dimensions"), (dict(log_decay=t(4, 1)), "dimensions"), (dict(q=None), "dimensions"),
    (dict(k=t(2, 8, 2, 15)), "must have shape"), (dict(k=t(2, 9, 2, 16)), "must have shape"),
    (dict(v=t(1, 8, 1, 24)), "must have shape"), (dict(q=t(2, 8, 3, 16)), "does not divide"),
    (dict(lengths=t(3, dtype=torch.int32)), "must have shape"), (dict(initial_state=t(2, 4, 24, 16)), "must have shape"),
    (dict(), "must live on the GPU"),
])
def test_binding_refuses_attention(kw, match):
    with pytest.raises(ValueError, match=match):
        ssm.linear_attention_fwd(**attention(**kw))
    with pytest.raises(ValueError, match=match):
        ssm.linear_attention_bwd(**attention(**kw), dout=t(2, 8, 4, 24))


def test_binding_refuses_outputs_and_types():
    with pytest.raises(ValueError, match="must have shape"):
        ssm.linear_attention_fwd(**attention(), out=t(2, 8, 4, 16))
    with pytest.raises(ValueError, match="must have shape"):
        ssm.linear_attention_fwd(**attention(), final_state=t(2, 4, 16, 16))
    with pytest.raises(ValueError, match="must have shape"):
        ssm.linear_attention_bwd(**attention(), dout=t(2, 8, 4, 16))
    with pytest.raises(ValueError, match="must have shape"):
        ssm.linear_attention_bwd(**attention(), dout=t(2, 8, 4, 24), dfinal_state=t(2, 4, 16, 23))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssm.linear_attention_fwd(**attention(q=t(2, 8, 4, 16, dtype=torch.float16)))


@pytest.mark.parametrize("kw,match", [
    (dict(q_t=t(3, 2, 4, 16)), "dimensions"), (dict(state=t(3, 4, 16)), "dimensions"),
    (dict(state=t(3, 4, 24, 16)), "must have shape"), (dict(state=t(2, 4, 16, 24)), "as many states"),
    (dict(slots=t(2, dtype=torch.int32)), "must have shape"), (dict(out_state=t(2, 4, 16, 24)), "must have shape"),
    (dict(out=t(3, 4, 16)), "must have shape"), (dict(k_t=t(3, 3, 16)), "does not divide"),
    (dict(), "must live on the GPU"),
])
def test_binding_refuses_steps(kw, match):
    a = dict(state=t(3, 4, 16, 24), q_t=t(3, 4, 16), k_t=t(3, 2, 16), v_t=t(3, 1, 24), log_decay=t(4))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        ssm.linear_attention_step(**a)


@pytest.mark.parametrize("kw,match", [
    (dict(gate=t(3, 15)), "must have shape"), (dict(residual=t(2, 16)), "must have shape"),
    (dict(post_weight=t(15)), "must have shape"), (dict(pre_weight=t(16, 1)), "must have shape"),
    (dict(res_scale=t(3)), "must have shape"), (dict(h=t(3, 15)), "must have shape"), (dict(groups=3), "must divide"),
    (dict(groups=0), "must divide"), (dict(x=None), "expected x"), (dict(), "must live on the GPU"),
])
def test_binding_refuses_norms(kw, match):
    a = dict(x=t(3, 16))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        ssm.block_norm_fwd(**a)


def test_binding_refuses_norm_gradients():
    x, w = t(3, 16), t(16)
    with pytest.raises(ValueError, match="exactly when"):
        ssm.block_norm_bwd(x, x, None, x, pre_weight=w)
    with pytest.raises(ValueError, match="exactly when"):
        ssm.block_norm_bwd(x, x, x, x)
    with pytest.raises(ValueError, match="is needed"):
        ssm.block_norm_bwd(x, None, x, x, pre_weight=w)
    with pytest.raises(ValueError, match="must have shape"):
        ssm.block_norm_bwd(x, t(3, 15), x, x, pre_weight=w)
    with pytest.raises(ValueError, match="must live on the GPU"):
        ssm.block_norm_bwd(x, x, x, x, pre_weight=w)
