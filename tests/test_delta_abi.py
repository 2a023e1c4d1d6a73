"""What the gated delta rule and the query and key norms refuse, through the C ABI and the binding, without a GPU: every
refusal comes before anything reaches a device.  Pointers here are fake addresses, never dereferenced; no call with
valid arguments is made."""
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
    a = dict(q=at(0), k=at(1), v=at(2), qs=None, ks=None, vs=None, g=at(3), b=at(6), scale=1.0, n=None, s0=None, o=at(4),
             fin=at(5), B=2, L=64, H=4, Hq=4, Hk=2, Hv=1, K=64, V=32, dt=1, ws=at(8), ws_bytes=32 * MB)
    a.update(kw)
    return lib.ssm_gated_delta_fwd(
        a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["b"], a["scale"], a["n"], a["s0"], a["o"], a["fin"],
        a["B"], a["L"], a["H"], a["Hq"], a["Hk"], a["Hv"], a["K"], a["V"], a["dt"], a["ws"], a["ws_bytes"], None)


def bwd(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), d=at(3), qs=None, ks=None, vs=None, ds=None, g=at(4), b=at(5), scale=1.0, n=None,
             s0=None, df=None, dq=at(6), dk=at(7), dv=at(8), dg=at(9), db=at(11), d0=at(10), B=2, L=64, H=4, Hq=4, Hk=2,
             Hv=1, K=64, V=32, dt=1, ws=at(12), ws_bytes=32 * MB)
    a.update(kw)
    return lib.ssm_gated_delta_bwd(
        a["q"], a["k"], a["v"], a["d"], a["qs"], a["ks"], a["vs"], a["ds"], a["g"], a["b"], a["scale"], a["n"], a["s0"],
        a["df"], a["dq"], a["dk"], a["dv"], a["dg"], a["db"], a["d0"], a["B"], a["L"], a["H"], a["Hq"], a["Hk"], a["Hv"],
        a["K"], a["V"], a["dt"], a["ws"], a["ws_bytes"], None)


def step(lib, **kw):
    a = dict(si=at(0), so=at(0), q=at(1), k=at(2), v=at(3), qs=None, ks=None, vs=None, g=at(4), b=at(6), scale=1.0,
             slots=None, o=at(5), B=3, S=3, H=4, Hq=4, Hk=2, Hv=1, K=64, V=32, dt=1)
    a.update(kw)
    return lib.ssm_gated_delta_step(
        a["si"], a["so"], a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["b"], a["scale"], a["slots"], a["o"],
        a["B"], a["S"], a["H"], a["Hq"], a["Hk"], a["Hv"], a["K"], a["V"], a["dt"], None)


COMMON = [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(g=None), INV), (dict(b=None), INV),
    (dict(B=-1), INV), (dict(H=-4), INV),
    (dict(Hq=3), INV), (dict(Hk=0), INV), (dict(Hv=8), INV),
    (dict(K=0), UNS), (dict(K=129), UNS), (dict(V=0), UNS), (dict(V=129), UNS), (dict(dt=2), UNS),
    (dict(q=at(0) + 1), INV), (dict(g=at(3) + 2), INV), (dict(b=at(6) + 2), INV),
    (dict(B=1 << 40), UNS), (dict(H=1 << 17, Hq=1, Hk=1, Hv=1), UNS),
]
PROMPT = COMMON + [
    (dict(L=-1), INV), (dict(L=1 << 30), UNS), (dict(B=1 << 20, H=2, Hq=1, Hk=1, Hv=1), UNS),
    (dict(B=1 << 10, L=1 << 28, H=1, Hq=1, Hk=1, Hv=1), UNS),       # more chunks than are counted
    (dict(qs=strides(-1, 256, 64)), INV), (dict(vs=strides(1 << 62, 256, 64)), INV),
    (dict(n=at(3) + 2), INV), (dict(s0=at(14) + 2), INV), (dict(ws=at(8) + 8), INV), (dict(ws=None), INV),
    (dict(ws_bytes=1024), INV),                                     # every call with tokens needs one
]


@pytest.mark.parametrize("kw,status", PROMPT + [
    (dict(o=None), INV), (dict(o=at(0)), INV), (dict(o=at(0) + 64), INV), (dict(o=at(3)), INV), (dict(o=at(6) + 16), INV),
    (dict(fin=at(1)), INV), (dict(fin=at(4) + 256), INV), (dict(fin=at(5) + 2), INV),
    (dict(s0=at(4)), INV), (dict(s0=at(5) + 64), INV),               # partly under the final state
    (dict(ws=at(2)), INV), (dict(ws=at(4)), INV), (dict(ws=at(5)), INV), (dict(ws=at(6)), INV), (dict(s0=at(8)), INV),
    (dict(n=at(4)), INV),                                           # lengths inside the output
    (dict(q=at(0), qs=strides(0, 0, 0), o=at(0) + 64, K=64), INV),  # a broadcast view's one row
])
def test_forward_refuses(lib, kw, status):
    assert fwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", PROMPT + [
    (dict(d=None), INV), (dict(dq=None), INV), (dict(dk=None), INV), (dict(dv=None), INV), (dict(dg=None), INV),
    (dict(db=None), INV), (dict(dg=at(9) + 2), INV), (dict(dg=at(4)), INV), (dict(db=at(9)), INV), (dict(db=at(5) + 16), INV),
    (dict(dq=at(0)), INV), (dict(dk=at(3) + 128), INV), (dict(dv=at(6)), INV), (dict(d0=at(7)), INV),
    (dict(df=at(10), d0=at(10)), INV), (dict(ws=at(6)), INV), (dict(ws=at(3)), INV), (dict(ds=strides(-4, 1, 1)), INV),
])
def test_gradient_refuses(lib, kw, status):
    assert bwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(si=None), INV), (dict(so=None), INV), (dict(o=None), INV), (dict(S=2), INV), (dict(S=-1, slots=at(8)), INV),
    (dict(so=at(0) + 64), INV), (dict(so=at(1)), INV), (dict(o=at(2)), INV), (dict(o=at(0) + 128), INV),
    (dict(slots=at(8) + 2), INV), (dict(slots=at(5)), INV), (dict(si=at(0) + 2, so=at(0) + 2), INV),
    (dict(ks=strides(-1, 64)), INV), (dict(o=at(6)), INV),
])
def test_step_refuses(lib, kw, status):
    assert step(lib, **kw) == status


def test_workspace_sizes(lib):
    size, gsize = lib.ssm_gated_delta_workspace_size, lib.ssm_gated_delta_bwd_workspace_size
    assert size(8, 2048, 32, 128, 128, 1) == 8 * 32 * 32 * (18 + 2 + 12) * 1024     # the chunks' records alone
    assert size(1, 131072, 20, 128, 128, 1) > 20 * 2048 * 32 * 1024                  # and states of segments
    assert gsize(8, 2048, 32, 32, 8, 8, 128, 128, 1) == gsize(8, 2048, 32, 32, 32, 32, 128, 128, 1) + 2 * 8 * 2048 * 32 * 128 * 4
    for bad in (size(-1, 64, 4, 64, 64, 1), size(1, 64, 4, 129, 64, 1), size(1, 64, 4, 64, 64, 9),
                gsize(1, 64, 4, 3, 4, 4, 64, 64, 1), size(0, 64, 4, 64, 64, 1), size(1, 0, 4, 64, 64, 1)):
        assert bad == 0


def qk(lib, **kw):
    a = dict(q=at(0), k=at(1), qs=None, ks=None, qw=at(2), kw=at(3), f=at(4), p=at(5), qo=at(6), ko=at(7), B=2, L=8, Hq=4,
             Hk=2, K=64, r=32, i=0, norm=0, eps=1e-6, dt=1)
    a.update(kw)
    return lib.ssm_qk_norm_fwd(a["q"], a["k"], a["qs"], a["ks"], a["qw"], a["kw"], a["f"], a["p"], a["qo"], a["ko"], a["B"],
                               a["L"], a["Hq"], a["Hk"], a["K"], a["r"], a["i"], a["norm"], a["eps"], a["dt"], None)


def qkb(lib, **kw):
    a = dict(q=at(0), k=at(1), gq=at(8), gk=at(9), qs=None, ks=None, gqs=None, gks=None, qw=at(2), kw=at(3), f=at(4), p=at(5),
             qo=at(6), ko=at(7), dqw=at(10), dkw=at(11), B=2, L=8, Hq=4, Hk=2, K=64, r=32, i=0, norm=0, eps=1e-6, dt=1,
             ws=at(12), ws_bytes=4 * MB)
    a.update(kw)
    return lib.ssm_qk_norm_bwd(a["q"], a["k"], a["gq"], a["gk"], a["qs"], a["ks"], a["gqs"], a["gks"], a["qw"], a["kw"],
                               a["f"], a["p"], a["qo"], a["ko"], a["dqw"], a["dkw"], a["B"], a["L"], a["Hq"], a["Hk"], a["K"],
                               a["r"], a["i"], a["norm"], a["eps"], a["dt"], a["ws"], a["ws_bytes"], None)


NORM = [
    (dict(q=None), INV), (dict(k=None), INV), (dict(f=None), INV), (dict(qo=None), INV), (dict(ko=None), INV),
    (dict(B=-1), INV), (dict(Hk=-1), INV), (dict(r=-2), INV), (dict(r=31), INV), (dict(r=66), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(K=0, r=0), UNS), (dict(K=257), UNS), (dict(Hq=1 << 16), UNS), (dict(L=1 << 30), UNS),
    (dict(B=1 << 39), UNS), (dict(dt=2), UNS), (dict(norm=2), UNS), (dict(q=at(0) + 1), INV), (dict(qw=at(2) + 2), INV),
    (dict(f=at(4) + 1), INV), (dict(p=at(5) + 2), INV), (dict(qo=at(6) + 1), INV), (dict(qs=strides(-1, 256, 64)), INV),
    (dict(ko=at(2)), INV), (dict(qo=at(4)), INV), (dict(qo=at(5)), INV), (dict(qo=at(7)), INV),
    (dict(qo=at(1)), INV), (dict(ko=at(0) + 128), INV),
]


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(qo=at(0) + 128), INV),                                    # partly under q
    (dict(qo=at(0), qs=strides(2048 + 64, 256, 64)), INV),          # in place, but q is not packed
])
def test_qk_norm_refuses(lib, kw, status):
    assert qk(lib, **kw) == status


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(gq=None), INV), (dict(gk=None), INV), (dict(dqw=None), INV), (dict(kw=None), INV), (dict(ws=None), INV),
    (dict(ws_bytes=64), INV), (dict(ws=at(12) + 8), INV), (dict(dqw=at(10) + 2), INV), (dict(dkw=at(10)), INV),
    (dict(qo=at(0)), INV), (dict(ko=at(9) + 128), INV), (dict(qo=at(9)), INV), (dict(ko=at(8)), INV), (dict(ws=at(6)), INV),
    (dict(ws=at(9)), INV), (dict(qo=at(8), gqs=strides(2048 + 64, 256, 64)), INV), (dict(gqs=strides(1, 1, -1)), INV),
])
def test_qk_norm_gradient_refuses(lib, kw, status):
    assert qkb(lib, **kw) == status


# ---- the binding: shapes before devices, for tensors on the CPU

def t(*s, dtype=torch.float32):
    return torch.zeros(*s, dtype=dtype)


def delta(**kw):
    a = dict(q=t(2, 8, 4, 16), k=t(2, 8, 2, 16), v=t(2, 8, 1, 24), g=t(2, 8, 4), beta=t(2, 8, 4))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,match", [
    (dict(q=t(2, 8, 64)), "dimensions"), (dict(g=t(4)), "dimensions"), (dict(q=None), "dimensions"), (dict(g=None), "dimensions"),
    (dict(k=t(2, 8, 2, 15)), "must have shape"), (dict(k=t(2, 9, 2, 16)), "must have shape"),
    (dict(g=t(2, 9, 4)), "must have shape"), (dict(beta=t(2, 8, 3)), "must have shape"), (dict(beta=None), "must be a tensor"),
    (dict(v=t(1, 8, 1, 24)), "must have shape"), (dict(q=t(2, 8, 3, 16)), "does not divide"),
    (dict(lengths=t(3, dtype=torch.int32)), "must have shape"), (dict(initial_state=t(2, 4, 24, 16)), "must have shape"),
    (dict(), "must live on the GPU"),
])
def test_binding_refuses_delta(kw, match):
    with pytest.raises(ValueError, match=match):
        ssm.gated_delta_fwd(**delta(**kw))
    with pytest.raises(ValueError, match=match):
        ssm.gated_delta_bwd(**delta(**kw), dout=t(2, 8, 4, 24))


def test_binding_refuses_outputs_and_types():
    for kw in (dict(out=t(2, 8, 4, 16)), dict(final_state=t(2, 4, 16, 16))):
        with pytest.raises(ValueError, match="must have shape"):
            ssm.gated_delta_fwd(**delta(), **kw)
    for kw in (dict(dout=t(2, 8, 4, 16)), dict(dout=t(2, 8, 4, 24), dfinal_state=t(2, 4, 16, 23))):
        with pytest.raises(ValueError, match="must have shape"):
            ssm.gated_delta_bwd(**delta(), **kw)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        ssm.gated_delta_bwd(**delta(), dout=None)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssm.gated_delta_fwd(**delta(q=t(2, 8, 4, 16, dtype=torch.float16)))


@pytest.mark.parametrize("kw,match", [
    (dict(q_t=t(3, 2, 4, 16)), "dimensions"), (dict(state=t(3, 4, 16)), "dimensions"), (dict(g_t=t(4)), "dimensions"),
    (dict(state=t(3, 4, 24, 16)), "must have shape"), (dict(state=t(2, 4, 16, 24)), "as many states"),
    (dict(slots=t(2, dtype=torch.int32)), "must have shape"), (dict(out_state=t(2, 4, 16, 24)), "must have shape"),
    (dict(out=t(3, 4, 16)), "must have shape"), (dict(k_t=t(3, 3, 16)), "does not divide"),
    (dict(beta_t=t(2, 4)), "must have shape"), (dict(), "must live on the GPU"),
])
def test_binding_refuses_steps(kw, match):
    a = dict(state=t(3, 4, 16, 24), q_t=t(3, 4, 16), k_t=t(3, 2, 16), v_t=t(3, 1, 24), g_t=t(3, 4), beta_t=t(3, 4))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        ssm.gated_delta_step(**a)


@pytest.mark.parametrize("kw,match", [
    (dict(q=t(2, 64)), r"\[tokens, heads, K\]"), (dict(k=t(2, 8, 16)), "dimensions"), (dict(k=t(2, 8, 3, 15)), "must have shape"),
    (dict(q_weight=t(15)), "must have shape"), (dict(k_weight=t(16, 1)), "must have shape"), (dict(norm="max"), "norm must be"),
    (dict(inv_freq=t(9)), "more than 16 columns"), (dict(inv_freq=t(2, 2)), "dimensions"),
    (dict(positions=t(2, 8, dtype=torch.int32)), "without inv_freq"),
    (dict(inv_freq=t(4), positions=t(8, dtype=torch.int32)), "must have shape"),
    (dict(k=None, k_weight=t(16)), "without k"), (dict(), "must live on the GPU"),
])
def test_binding_refuses_qk_norms(kw, match):
    a = dict(q=t(2, 8, 4, 16), k=t(2, 8, 3, 16))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        ssm.qk_norm_fwd(**a)
    with pytest.raises(ValueError, match=match):
        ssm.qk_norm_bwd(**a, dq_out=t(2, 8, 4, 16), dk_out=None if a["k"] is None else t(2, 8, 3, 16))


def test_binding_refuses_qk_norm_forms():
    q, k = t(5, 4, 16), t(5, 2, 16)
    with pytest.raises(ValueError, match="positions are needed"):
        ssm.qk_norm_fwd(q, k, inv_freq=t(4))
    with pytest.raises(ValueError, match="must have shape"):
        ssm.qk_norm_fwd(q, k, q_out=t(5, 4, 15))
    with pytest.raises(ValueError, match="without k"):
        ssm.qk_norm_fwd(q, k_out=k)
    with pytest.raises(ValueError, match="exactly when"):
        ssm.qk_norm_bwd(q, None, q, k)
    with pytest.raises(ValueError, match="exactly when"):
        ssm.qk_norm_bwd(q, k, q, None)
    with pytest.raises(ValueError, match="must have shape"):
        ssm.qk_norm_bwd(q, k, q, t(5, 2, 15))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssm.qk_norm_fwd(t(5, 4, 16, dtype=torch.float16))
