"""GPU parity of linear attention (prompt form, gradient, single token) with the token
recurrence in float64.

Error of a row (one token's V values of one head; one row of a state): the 2-norm of the
difference over the root mean square 2-norm of that head's rows.  Bounds, from the
roundings on the way:
  float32  a value is a sum of at most 64 + 128 products per chunk in float32, so at most
           192 * 2^-24 = 1.1e-5 of the terms' size, plus the chunks' decays: 5e-5.
  bfloat16 outputs: rounded to 8 bits, as the masked scores were at first (2^-9 of each term;
           they are in two terms now); a row's terms may be a few times its head's mean size: 8 * 2^-9 = 1.6e-2.
  states   float32 from exact products (bfloat16 inputs included): 5e-5.
"""
import pytest
import torch

import lm_reference as ref

pytestmark = pytest.mark.gpu

OUT = {torch.float32: 5e-5, torch.bfloat16: 1.6e-2}
STATE = 5e-5


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ssm():
    import selective_state_space_68_amd as ssm
    return ssm


def _err(got, want):
    """Largest row error; rows are the last axis, heads the one before it (outputs) or two before it (states)."""
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    d, r = (got - want).norm(dim=-1), want.norm(dim=-1)
    axes = (0, 1) if d.dim() == 3 else (0, 2)
    size = r.square().mean(axes, keepdim=True).sqrt()
    if d.numel() == 0:
        return 0.0
    return float((d / size.clamp(min=1e-30)).max()) if float(d.max()) > 0 else 0.0


def _check(got, want, dtype, what):
    tol = STATE if "state" in what else OUT[dtype]
    e = _err(got, want)
    print(f"{what} {tuple(got.shape)} {dtype}: {e:.2e}", flush=True)
    assert e <= tol, (what, e)


def _inputs(B, L, H, K, V, dtype, heads=None, seed=0, decay=(0.8, 0.999)):
    Hq, Hk, Hv = heads or (H, H, H)
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    g = torch.log(torch.linspace(decay[0], decay[1], H))
    t = dict(q=r(B, L, Hq, K), k=r(B, L, Hk, K) * K ** -0.5, v=r(B, L, Hv, V), do=r(B, L, H, V))
    t = {n: x.to(dtype) for n, x in t.items()}
    return t, g, r(B, H, K, V), r(B, H, K, V)


def _cuda(t):
    return {n: x.cuda() for n, x in t.items()}


SHAPES = [   # batch, L, H, K, V, heads of q, k, v
    (1, 1, 1, 64, 64, None),
    (2, 64, 2, 64, 64, None),
    (1, 65, 2, 128, 128, None),
    (2, 200, 4, 64, 128, (4, 2, 2)),
    (1, 130, 6, 128, 64, (2, 6, 3)),
    (2, 77, 3, 72, 40, (1, 1, 3)),       # vectors, tiles partly empty
    (1, 129, 2, 33, 17, None),           # element by element
    (1, 70, 1, 1, 1, None),
    (3, 63, 2, 100, 128, (2, 1, 1)),
    (2, 193, 2, 100, 100, None),         # words
    (1, 140, 3, 34, 98, (3, 1, 1)),
    (2, 300, 2, 128, 50, (1, 2, 2)),
    (1, 1500, 2, 64, 64, None),
    (1, 1100, 2, 100, 36, (1, 2, 2)),    # the others in segments
    (1, 1030, 1, 33, 17, None),
    (1, 1200, 2, 96, 128, None),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,L,H,K,V,heads", SHAPES)
def test_forward(B, L, H, K, V, heads, dtype):
    t, g, s0, _ = _inputs(B, L, H, K, V, dtype, heads, seed=L + K)
    d = _cuda(t)
    out, fin = _ssm().linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), initial_state=s0.cuda())
    want, wfin = ref.attention(t["q"], t["k"], t["v"], g, K ** -0.5, s0)
    _check(out, want, dtype, "out")
    _check(fin, wfin, dtype, "final_state")
    out2, none = _ssm().linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), 0.3, return_final_state=False)
    assert none is None
    _check(out2, ref.attention(t["q"], t["k"], t["v"], g, 0.3)[0], dtype, "out")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,L,H,K,V,heads", SHAPES)
def test_gradient(B, L, H, K, V, heads, dtype):
    t, g, s0, df = _inputs(B, L, H, K, V, dtype, heads, seed=L + V)
    d = _cuda(t)
    got = _ssm().linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], initial_state=s0.cuda(),
                                      dfinal_state=df.cuda())
    want = ref.attention_grad(t["q"], t["k"], t["v"], g, t["do"], K ** -0.5, s0, df)
    assert got.keys() == want.keys()
    for n in want:
        _check(got[n], want[n], dtype, n)
    got = _ssm().linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], 0.3)
    assert got["dinitial_state"] is None
    want = ref.attention_grad(t["q"], t["k"], t["v"], g, t["do"], 0.3)
    for n in ("dq", "dk", "dv"):
        _check(got[n], want[n], dtype, n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_absent_tokens_hold_anything(dtype):
    B, L, H, K, V = 6, 150, 3, 64, 72
    lengths = torch.tensor([150, 0, 1, 64, 65, 149], dtype=torch.int32)
    t, g, s0, df = _inputs(B, L, H, K, V, dtype, (3, 1, 1), seed=3)
    absent = torch.arange(L)[None] >= lengths[:, None]
    bad = {n: x.clone() for n, x in t.items()}
    for i, x in enumerate(bad.values()):
        x[absent] = (float("nan"), float("inf"), float("-inf"), torch.finfo(dtype).min)[i]
    d = _cuda(bad)
    n = lengths.cuda()
    out, fin = _ssm().linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), initial_state=s0.cuda(), lengths=n)
    want, wfin = ref.attention(t["q"], t["k"], t["v"], g, K ** -0.5, s0, lengths.tolist())
    _check(out, want, dtype, "out")
    _check(fin, wfin, dtype, "final_state")
    assert not out.cpu()[absent].any()
    assert torch.equal(fin[1].cpu(), s0[1])                 # no token: the state as it was
    got = _ssm().linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], initial_state=s0.cuda(),
                                      dfinal_state=df.cuda(), lengths=n)
    want = ref.attention_grad(t["q"], t["k"], t["v"], g, t["do"], K ** -0.5, s0, df, lengths.tolist())
    for name in want:
        _check(got[name], want[name], dtype, name)
    for name in ("dq", "dk", "dv"):
        assert not got[name].cpu()[absent].any()
    assert torch.equal(got["dinitial_state"][1].cpu(), df[1])
    # lengths outside [0, L] are clamped
    out2, _ = _ssm().linear_attention_fwd(d["q"][:2], d["k"][:2], d["v"][:2], g.cuda(),
                                          lengths=torch.tensor([1000, -5], dtype=torch.int32, device="cuda"))
    assert torch.isfinite(out2[0]).all() and not out2[1].any()


@pytest.mark.parametrize("log_decay", [0.0, -1e-4, -5.0, -100.0, float("-inf")])
def test_decays_from_none_to_all(log_decay):
    B, L, H, K, V = 1, 200, 2, 64, 64
    t, _, s0, df = _inputs(B, L, H, K, V, torch.float32, seed=4)
    g = torch.full((H,), log_decay)
    d = _cuda(t)
    ref_g = g.clamp(min=-1e5)                               # (exp(-1e5) is 0 in float64 too)
    out, fin = _ssm().linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), initial_state=s0.cuda())
    want, wfin = ref.attention(t["q"], t["k"], t["v"], ref_g, K ** -0.5, s0)
    _check(out, want, torch.float32, "out")
    _check(fin, wfin, torch.float32, "final_state")
    got = _ssm().linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], initial_state=s0.cuda(),
                                      dfinal_state=df.cuda())
    want = ref.attention_grad(t["q"], t["k"], t["v"], ref_g, t["do"], K ** -0.5, s0, df)
    for n in want:
        if float(want[n].abs().max()) < 1e-30:              # (dinitial_state where nothing is carried)
            assert float(got[n].abs().max()) < 1e-30
        else:
            _check(got[n], want[n], torch.float32, n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,V,offset", [(64, 64, 0), (64, 64, 1), (64, 64, 2), (128, 96, 2), (40, 24, 0)])
def test_views_of_one_projection(K, V, offset, dtype):
    # q, k, v and dout as slices of wider rows; with an odd offset rows are not even 4-byte aligned in bfloat16, with 2 not 16-byte
    B, L, H, Hk = 2, 100, 4, 2
    gen = torch.Generator().manual_seed(5)
    wide = torch.randn(B, L, (H + Hk) * K + Hk * V + H * V + 8, generator=gen).to(dtype)
    cut = lambda x, at, n, w: x[..., offset + at:offset + at + n * w].unflatten(-1, (n, w))
    def split(x):
        return (cut(x, 0, H, K), cut(x, H * K, Hk, K), cut(x, (H + Hk) * K, Hk, V),
                cut(x, (H + Hk) * K + Hk * V, H, V))
    q, k, v, do = split(wide.cuda())
    g = torch.log(torch.linspace(0.9, 0.99, H))
    hq, hk, hv, hdo = split(wide)
    out, fin = _ssm().linear_attention_fwd(q, k, v, g.cuda(), 0.1)
    want, wfin = ref.attention(hq, hk, hv, g, 0.1)
    _check(out, want, dtype, "out")
    _check(fin, wfin, dtype, "final_state")
    got = _ssm().linear_attention_bwd(q, k, v, g.cuda(), do, 0.1)
    want = ref.attention_grad(hq, hk, hv, g, hdo, 0.1)
    for n in ("dq", "dk", "dv"):
        _check(got[n], want[n], dtype, n)
    # a transposed order of the axes: [L, batch, heads, width]
    tq = hq.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    out2, _ = _ssm().linear_attention_fwd(tq, k, v, g.cuda(), 0.1)
    assert torch.equal(out, out2) or _err(out2, out.double().cpu()) <= OUT[dtype]
    # one head broadcast over the tokens by a stride of zero
    q0 = hq[:, :1].cuda().expand(B, L, H, K)
    out3, _ = _ssm().linear_attention_fwd(q0, k, v, g.cuda(), 0.1)
    _check(out3, ref.attention(hq[:, :1].expand(B, L, H, K), hk, hv, g, 0.1)[0], dtype, "out")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_sequences_run_in_segments(dtype):
    # one head: cut into segments wherever the workspace is not empty; the recurrence over all of it
    ssm = _ssm()
    B, L, H, K, V = 1, 4133, 2, 32, 32
    t, g, s0, df = _inputs(B, L, H, K, V, dtype, seed=6, decay=(0.99, 0.9999))
    d = _cuda(t)
    n = torch.tensor([4111], dtype=torch.int32)
    for lengths in (None, n):
        dn = None if lengths is None else lengths.cuda()
        hn = None if lengths is None else lengths.tolist()
        out, fin = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), initial_state=s0.cuda(), lengths=dn)
        want, wfin = ref.attention(t["q"], t["k"], t["v"], g, K ** -0.5, s0, hn)
        _check(out, want, dtype, "out")
        _check(fin, wfin, dtype, "final_state")
        got = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], initial_state=s0.cuda(),
                                       dfinal_state=df.cuda(), lengths=dn)
        want = ref.attention_grad(t["q"], t["k"], t["v"], g, t["do"], K ** -0.5, s0, df, hn)
        for name in want:
            _check(got[name], want[name], dtype, name)


def test_pieces_equal_the_whole_and_state_in_place():
    ssm = _ssm()
    t, g, s0, _ = _inputs(2, 300, 2, 64, 64, torch.float32, seed=7)
    d = _cuda(t)
    whole, fin = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), initial_state=s0.cuda())
    state = s0.cuda()
    parts = []
    for a, b in ((0, 100), (100, 101), (101, 300)):
        o, st = ssm.linear_attention_fwd(d["q"][:, a:b], d["k"][:, a:b], d["v"][:, a:b], g.cuda(), initial_state=state,
                                         final_state=state)
        assert st is state
        parts.append(o)
    assert _err(torch.cat(parts, 1), whole.double().cpu()) <= 2 * OUT[torch.float32]
    assert _err(state, fin.double().cpu()) <= 2 * STATE


def test_no_tokens():
    ssm = _ssm()
    t, g, s0, df = _inputs(2, 0, 2, 16, 8, torch.bfloat16)
    d = _cuda(t)
    out, fin = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda(), initial_state=s0.cuda())
    assert out.shape == (2, 0, 2, 8) and torch.equal(fin.cpu(), s0)
    _, fin = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda())
    assert not fin.any()
    got = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], dfinal_state=df.cuda(),
                                   want_dinitial_state=True)
    assert torch.equal(got["dinitial_state"].cpu(), df)


@pytest.mark.parametrize("name", ["q", "k", "v", "initial_state"])
def test_gradient_against_differences(name):
    # each argument enters linearly, so a step of 1 has no truncation; what is left is the
    # float32 rounding of the two losses, 5e-5 of their terms' size
    ssm = _ssm()
    t, g, s0, df = _inputs(1, 150, 2, 64, 64, torch.float32, seed=8)
    args = {"q": t["q"], "k": t["k"], "v": t["v"], "initial_state": s0}
    d = _cuda(args)
    do, dfc = t["do"].cuda(), df.cuda()
    got = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), do, initial_state=d["initial_state"],
                                   dfinal_state=dfc)["d" + name]
    step = torch.randn(args[name].shape, generator=torch.Generator().manual_seed(9)).cuda()

    def loss(sign):
        a = dict(d)
        a[name] = a[name] + sign * step
        o, f = ssm.linear_attention_fwd(a["q"], a["k"], a["v"], g.cuda(), initial_state=a["initial_state"])
        return (o.double() * do).sum() + (f.double() * dfc).sum()

    diff = float(loss(1) - loss(-1)) / 2
    size = float(got.double().norm() * step.double().norm())
    assert abs(diff - float((got.double() * step).sum())) <= 5e-5 * size


def test_results_do_not_change_from_call_to_call():
    ssm = _ssm()
    t, g, s0, df = _inputs(2, 2100, 3, 64, 128, torch.bfloat16, (3, 1, 1), seed=10)
    d = _cuda(t)
    a = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], initial_state=s0.cuda(),
                                 dfinal_state=df.cuda())
    f = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda())
    for _ in range(2):
        b = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], g.cuda(), d["do"], initial_state=s0.cuda(),
                                     dfinal_state=df.cuda())
        assert all(torch.equal(a[n], b[n]) for n in a)
        assert all(torch.equal(x, y) for x, y in zip(f, ssm.linear_attention_fwd(d["q"], d["k"], d["v"], g.cuda())))


def test_runs_on_the_given_stream_and_in_a_graph():
    ssm = _ssm()
    t, g, s0, _ = _inputs(1, 2000, 2, 64, 64, torch.bfloat16, seed=11)
    d = _cuda(t)
    gc, st = g.cuda(), s0.cuda()
    want = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], gc, initial_state=st)
    out, fin = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(max(1, ssm.linear_attention_workspace_size(1, 2000, 2, 64, 64)), dtype=torch.uint8, device="cuda")
    call = lambda: ssm.linear_attention_fwd(d["q"], d["k"], d["v"], gc, initial_state=st, out=out, final_state=fin,
                                            workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(fin, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for i in range(3):
        out.zero_()
        fin.zero_()
        st.copy_(s0.cuda() * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        eager = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], gc, initial_state=st)
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(fin, eager[1])


# ---- one token

STEPS = [(1, 1, 64, 64, None), (5, 6, 64, 64, (6, 2, 3)), (3, 4, 128, 128, (1, 1, 4)), (2, 2, 72, 40, None),
         (3, 2, 33, 17, None), (2, 1, 1, 1, None), (4, 2, 128, 100, None), (2, 3, 16, 4, None)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,H,K,V,heads", STEPS)
def test_step(S, H, K, V, heads, dtype):
    t, g, s0, _ = _inputs(S, 1, H, K, V, dtype, heads, seed=K + V)
    q, k, v = (t[n][:, 0].cuda() for n in "qkv")
    want, wfin = ref.attention(t["q"], t["k"], t["v"], g, K ** -0.5, s0)
    state = s0.cuda()
    out = _ssm().linear_attention_step(state, q, k, v, g.cuda())
    _check(out[:, None], want, dtype, "out")
    _check(state, wfin, dtype, "state")
    other = torch.full_like(state, float("nan"))
    start = s0.cuda()
    out2 = _ssm().linear_attention_step(start, q, k, v, g.cuda(), out_state=other)
    assert torch.equal(out, out2) and torch.equal(other, state) and torch.equal(start.cpu(), s0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step_by_slots_leaves_other_states_alone(dtype):
    S, pool, H, K, V = 7, 11, 3, 64, 72
    t, g, _, _ = _inputs(S, 1, H, K, V, dtype, (3, 1, 1), seed=12)
    s0 = torch.randn(pool, H, K, V, generator=torch.Generator().manual_seed(13))
    slots = torch.tensor([3, -1, 10, 0, 11, 7, -2147483648], dtype=torch.int32)
    live = [i for i, x in enumerate(slots.tolist()) if 0 <= x < pool]
    q, k, v = (t[n][:, 0].cuda() for n in "qkv")
    state = s0.cuda()
    out = _ssm().linear_attention_step(state, q, k, v, g.cuda(), slots=slots.cuda())
    at = slots[live].long()
    want, wfin = ref.attention(*(t[n][live] for n in "qkv"), g, K ** -0.5, s0[at])
    _check(out[live][:, None], want, dtype, "out")
    _check(state[at.cuda()], wfin, dtype, "state")
    idle = [i for i in range(S) if i not in live]
    assert not out[idle].any()
    rest = [i for i in range(pool) if i not in at.tolist()]
    assert torch.equal(state[rest].cpu(), s0[rest])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_continue_a_prompt(dtype):
    # the prompt's final state, then token by token, equals the prompt form over all of it;
    # q, k, v of a token are views of the sequence
    ssm = _ssm()
    t, g, s0, _ = _inputs(2, 70, 4, 64, 64, dtype, (4, 2, 2), seed=14)
    d = _cuda(t)
    want, wfin = ref.attention(t["q"], t["k"], t["v"], g, 64 ** -0.5, s0)
    _, state = ssm.linear_attention_fwd(d["q"][:, :66], d["k"][:, :66], d["v"][:, :66], g.cuda(),
                                        initial_state=s0.cuda())
    outs = [ssm.linear_attention_step(state, d["q"][:, i], d["k"][:, i], d["v"][:, i], g.cuda())
            for i in range(66, 70)]
    _check(torch.stack(outs, 1), want[:, 66:], dtype, "out")
    _check(state, wfin, dtype, "state")


def test_step_states_past_32_bits():
    # the last state of a pool of over 2^32 bytes, and over 2^31 elements of offset in bytes
    ssm = _ssm()
    H, K, V = 40, 128, 128
    pool = (1 << 32) // (H * K * V * 4) + 2
    state = torch.zeros(pool, H, K, V, device="cuda")
    t, g, s0, _ = _inputs(1, 1, H, K, V, torch.bfloat16, seed=15)
    state[-1] = s0[0].cuda()
    q, k, v = (t[n][:, 0].cuda() for n in "qkv")
    out = ssm.linear_attention_step(state, q, k, v, g.cuda(),
                                    slots=torch.tensor([pool - 1], dtype=torch.int32, device="cuda"))
    want, wfin = ref.attention(t["q"], t["k"], t["v"], g, K ** -0.5, s0)
    _check(out[:, None], want, torch.bfloat16, "out")
    _check(state[-1:], wfin, torch.bfloat16, "state")
    assert not state[:-1].any()


@pytest.mark.parametrize("which", ["batch", "token"])
def test_views_past_32_bits_of_elements(which):
    # rows of a batch 2^31 elements apart (vector loads), tokens 2^30 apart (element by element): the same bits
    # as packed copies, forwards and in the gradient
    ssm = _ssm()
    B, L, H, K = (2, 70, 2, 64) if which == "batch" else (1, 4, 2, 64)
    far = (1 << 31) + 64 if which == "batch" else 1 << 30
    span = (B - 1) * far if which == "batch" else (L - 1) * far
    store = torch.zeros(span + 4 * L * H * K, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(21)
    views = {}
    for i, n in enumerate(("q", "k", "v", "do")):
        strides = (far, H * K, K, 1) if which == "batch" else (0, far, K, 1)
        views[n] = store.as_strided((B, L, H, K), strides, i * L * H * K)
        views[n].copy_(torch.randn(B, L, H, K, device="cuda", generator=gen))
    t = {n: x.contiguous() for n, x in views.items()}
    g = torch.tensor([-0.01, -0.2], device="cuda")
    for a, b in zip(ssm.linear_attention_fwd(views["q"], views["k"], views["v"], g),
                    ssm.linear_attention_fwd(t["q"], t["k"], t["v"], g)):
        assert torch.equal(a, b)
    a = ssm.linear_attention_bwd(views["q"], views["k"], views["v"], g, views["do"])
    b = ssm.linear_attention_bwd(t["q"], t["k"], t["v"], g, t["do"])
    for n in ("dq", "dk", "dv"):
        assert torch.equal(a[n], b[n]), n


def test_outputs_past_32_bits_of_elements():
    # 2^31 output elements and more: the last tokens from the state before them
    ssm = _ssm()
    H, K, V, tail = 64, 64, 128, 100
    L = (1 << 31) // (H * V) + tail
    gen = torch.Generator("cuda").manual_seed(22)
    r = lambda heads, d: torch.randn(1, L, heads, d, device="cuda", dtype=torch.bfloat16, generator=gen)
    q, k, v = r(1, K), r(1, K), r(H, V)
    g = torch.log(torch.linspace(0.5, 0.9, H, device="cuda"))     # what is 1000 tokens back is below 0.9^1000
    out, fin = ssm.linear_attention_fwd(q, k, v, g)
    n = L - tail - 1000
    t = [x[:, n:].cpu() for x in (q, k, v)]
    want, wfin = ref.attention(*t, g.cpu(), K ** -0.5, None)
    _check(out[:, -tail:], want[:, -tail:], torch.bfloat16, "out")
    _check(fin, wfin, torch.bfloat16, "state")
