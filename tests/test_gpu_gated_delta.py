"""GPU parity of the gated delta rule (prompt form, single token) with the token recurrence in float64.

Error of a row (one token's V values of one head; one row of a state): the 2-norm of the difference over the row's own
2-norm plus the root mean square 2-norm of that head's rows.  Bounds, from the roundings on the way:
  float32  a chunk's value is a sum of at most 128 + 64 products, as is each of the three before it in the chain (K E, T X,
           the state), in float32: 4 * 192 * 2^-24 = 4.6e-5 of the terms' size if all roundings agreed, and the square
           root of their number, 4 * sqrt(192) * 2^-24 = 3.3e-6, times the few sizes that a term may exceed its head's
           mean by, as they fall: 2e-5.
  states   float32 from operands of 24 bits (bfloat16 inputs included): the same 2e-5.
  the initial state's gradient is what its first chunk leaves of the gradient that enters it, exp(G_Q) F - K^T (beta
           exp(G) Y) + scale (exp(G) Q)^T D: where the keys are alike the terms cancel (with K = 1 a chunk takes the
           product of 64 factors 1 - beta off F), and float32 sums are good to 2^-24 of their terms, not of what is
           left.  The terms' 2-norms are added to that row's size.
  bfloat16 outputs: rounded by up to 2^-8 of each value, operands of 16 bits before that (2^-16 a product, far below):
           2^-8 * 1.02 + 2e-5.
"""
import pytest
import torch

import delta_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
OUT = {F32: 2e-5, BF16: 2.0 ** -8 * 1.02 + 2e-5}
STATE = 2e-5


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ssm():
    import selective_state_space_68_amd as ssm
    return ssm


def _first_chunk_terms(t, s0, df, scale):
    """[B, H, K]: the 2-norms of the terms whose sum is the initial state's gradient, row by row."""
    H = t["g"].shape[-1]
    x = {n: ref.heads(t[n], H) if n in "qkv" else t[n].double() for n in t}
    first, rest = ({n: y[:, i] for n, y in x.items()} for i in (slice(0, 64), slice(64, None)))
    state = ref.delta(*(first[n] for n in ("q", "k", "v", "g", "beta")), scale, s0)[1]
    F = ref.delta_grad(*rest.values(), scale, state, df)["dinitial_state"]
    dv = ref.delta_grad(*first.values(), scale, s0, F)["dv"]
    decay = first["g"].cumsum(1).exp()                          # [B, L, H]
    both = first["k"].abs() * dv.norm(dim=-1, keepdim=True) + scale * first["q"].abs() * first["do"].norm(dim=-1, keepdim=True)
    return decay[:, -1, :, None] * F.norm(dim=-1) + (decay[..., None] * both).sum(1)


def _check(got, want, tol, what, more=0.0):
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape
    assert torch.isfinite(got).all(), what
    d, r = (got - want).norm(dim=-1), want.norm(dim=-1)
    if d.numel() == 0:
        return
    axes = (0, 1) if d.dim() == 3 and "state" not in what else (0, 2)
    size = r + r.square().mean(axes, keepdim=True).sqrt() + more
    e = float((d / size.clamp(min=1e-30)).max()) if float(d.max()) > 0 else 0.0
    print(f"{what} {tuple(got.shape)}: {e:.2e}", flush=True)
    assert e <= tol, (what, e)


def _cuda(t):
    return {n: x.cuda() for n, x in t.items()}


def _forward(t, s0=None, lengths=None, scale=None, **named):
    d = _cuda(t)
    return _ssm().gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], scale,
                                  initial_state=None if s0 is None else s0.cuda(),
                                  lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda(),
                                  **named)


def _want(t, scale, s0=None, lengths=None):
    return ref.delta(t["q"], t["k"], t["v"], t["g"], t["beta"], scale, s0, lengths)


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
    (1, 1500, 2, 128, 128, None),
    (1, 1100, 2, 100, 36, (1, 2, 2)),
    (1, 1030, 1, 33, 17, None),
    (1, 1200, 2, 96, 128, None),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,H,K,V,heads", SHAPES)
def test_forward(B, L, H, K, V, heads, dtype):
    t, s0, _ = ref.inputs(B, L, H, K, V, dtype, heads, seed=L + K)
    out, fin = _forward(t, s0)
    want, wfin = _want(t, K ** -0.5, s0)
    _check(out, want, OUT[dtype], "out")
    _check(fin, wfin, STATE, "final_state")
    out2, none = _forward(t, scale=0.3, return_final_state=False)
    assert none is None
    _check(out2, _want(t, 0.3)[0], OUT[dtype], "out")


def _gradient(t, s0=None, df=None, lengths=None, scale=None, **named):
    d = _cuda(t)
    return _ssm().gated_delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], scale,
                                  initial_state=None if s0 is None else s0.cuda(),
                                  dfinal_state=None if df is None else df.cuda(),
                                  lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda(),
                                  **named)


def _check_grads(got, want, dtype, terms=0.0):
    """g's and beta's gradients are float32 and a row of theirs is a head's tokens."""
    for n, w in want.items():
        if got[n] is None:
            continue
        if n in ("dg", "dbeta"):
            _check(got[n].transpose(1, 2)[:, :, None], w.transpose(1, 2)[:, :, None], OUT[F32], n)
        else:
            _check(got[n], w, STATE if "state" in n else OUT[dtype], n, terms if "state" in n else 0.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,H,K,V,heads", SHAPES)
def test_gradient(B, L, H, K, V, heads, dtype):
    t, s0, df = ref.inputs(B, L, H, K, V, dtype, heads, seed=L + V)
    got = _gradient(t, s0, df)
    want = ref.delta_grad(*t.values(), K ** -0.5, s0, df)
    assert got.keys() == want.keys()
    _check_grads(got, want, dtype, _first_chunk_terms(t, s0, df, K ** -0.5))
    got = _gradient(t, scale=0.3)
    assert got["dinitial_state"] is None
    _check_grads(got, ref.delta_grad(*t.values(), 0.3), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K,V", [(12, 10), (66, 126), (6, 12), (12, 6), (126, 66), (10, 62)])
def test_words(K, V, dtype):
    """Rows that move as words: their last columns are read with those before them."""
    lengths = [70, 130]
    t, s0, df = ref.inputs(2, 130, 2, K, V, dtype, (1, 2, 2), seed=K)
    want, wfin = _want(t, K ** -0.5, s0, lengths)
    wg = ref.delta_grad(*t.values(), K ** -0.5, None, df, lengths)
    for x in ("q", "k", "v", "do"):
        t[x][0, 70:] = float("nan")
    out, fin = _forward(t, s0, lengths)
    _check(out, want, OUT[dtype], "out")
    _check(fin, wfin, STATE, "final_state")
    _check_grads(_gradient(t, None, df, lengths), wg, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_absent_tokens_hold_anything(dtype):
    B, L, H, K, V = 6, 150, 3, 64, 72
    lengths = [150, 0, 1, 64, 65, 149]
    t, s0, _ = ref.inputs(B, L, H, K, V, dtype, (3, 1, 1), seed=3)
    absent = torch.arange(L)[None] >= torch.tensor(lengths)[:, None]
    bad = {n: x.clone() for n, x in t.items()}
    for i, x in enumerate(bad.values()):
        x[absent] = (float("nan"), float("inf"), float("-inf"), float("nan"), float("inf"), torch.finfo(dtype).min)[i]
    out, fin = _forward(bad, s0, lengths)
    want, wfin = _want(t, K ** -0.5, s0, lengths)
    _check(out, want, OUT[dtype], "out")
    _check(fin, wfin, STATE, "final_state")
    assert not out.cpu()[absent].any()
    assert torch.equal(fin[1].cpu(), s0[1])                 # no token: the state as it was
    out2, fin2 = _forward(t, s0, [1000, -5, 1, 64, 65, 149])    # clamped to [0, L]
    assert torch.equal(out2, out) and torch.equal(fin2, fin)
    df = torch.randn(B, H, K, V, generator=torch.Generator().manual_seed(2))
    got = _gradient(bad, s0, df, lengths)
    _check_grads(got, ref.delta_grad(*t.values(), K ** -0.5, s0, df, lengths), dtype)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert not got[n].cpu()[absent].any(), n
    assert torch.equal(got["dinitial_state"][1].cpu(), df[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (72, 33)])
def test_step(K, V, dtype):
    """The step from a pool, and the prompt form continued by it, against the recurrence over all tokens."""
    B, L, H = 4, 70, 6
    t, s0, _ = ref.inputs(B, L, H, K, V, dtype, (3, 2, 6), seed=K + V)
    want, wfin = _want(t, K ** -0.5, s0)
    cut = 60
    _, fin = _forward({n: x[:, :cut] for n, x in t.items()}, s0)
    gen = torch.Generator("cuda").manual_seed(1)
    pool = torch.randn(7, H, K, V, device="cuda", generator=gen)
    before = pool.clone()
    slots = torch.tensor([5, 0, 6, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = fin
    for i in range(cut, L):
        d = {n: x[:, i].cuda() for n, x in t.items()}
        out = _ssm().gated_delta_step(pool, d["q"], d["k"], d["v"], d["g"], d["beta"], slots=slots)
        _check(out[:, None], want[:, i:i + 1], OUT[dtype], f"out {i}")
    _check(pool[slots.long()], wfin, STATE, "final_state")
    for i in (1, 3, 4):
        assert torch.equal(pool[i], before[i])


# ---- decays, strengths and keys of every kind

@pytest.mark.parametrize("gate", [0.0, -1e-4, -5.0, -100.0, float("-inf"), 0.01])
@pytest.mark.parametrize("strength", [0.0, 1.0, 1.9])
def test_constant_gates(gate, strength):
    """From no decay to all of it, and a little growth; from nothing written to more than the whole value replaced.  a = 0
    keeps nothing: compared with a decay of exp(-1e5), which is 0 in float64 too."""
    t, s0, df = ref.inputs(1, 150, 2, 64, 64, F32, seed=4)
    t["g"].fill_(gate)
    t["beta"].fill_(strength)
    host = dict(t, g=t["g"].clamp(min=-1e5))
    out, fin = _forward(t, s0)
    want, wfin = _want(host, 0.125, s0)
    _check(out, want, OUT[F32], "out")
    if float(wfin.abs().max()) < 1e-30:                     # (nothing is carried and nothing written)
        assert float(fin.abs().max()) < 1e-30
    else:
        _check(fin, wfin, STATE, "final_state")
    got, wgrad = _gradient(t, s0, df), ref.delta_grad(*host.values(), 0.125, s0, df)
    terms = _first_chunk_terms(host, s0, df, 0.125)
    for n, w in wgrad.items():
        if n == "dg":                                       # (a difference: against the sizes of what it is taken from)
            size = float(df.norm() * (wfin.norm() + s0.norm()) + t["do"].norm() * want.norm())
            assert float((got[n].double().cpu() - w).abs().max()) <= STATE * size, n
        elif float(w.abs().max()) < 1e-30:
            assert float(got[n].abs().max()) < 1e-30, n
        elif n == "dbeta":
            _check(got[n].transpose(1, 2)[:, :, None], w.transpose(1, 2)[:, :, None], OUT[F32], n)
        else:
            _check(got[n], w, STATE, n, terms if "state" in n else 0.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_alike_keys(dtype):
    """All keys of a head alike, written whole: the chunk's matrix is as far from the identity as it comes."""
    t, s0, _ = ref.inputs(1, 130, 2, 64, 64, dtype, seed=8)
    t["k"] = t["k"][:, :1].expand(1, 130, 2, 64).contiguous()
    t["beta"].fill_(1.0)
    t["g"].fill_(-0.001)
    out, fin = _forward(t, s0)
    want, wfin = _want(t, 0.125, s0)
    _check(out, want, OUT[dtype], "out")
    _check(fin, wfin, STATE, "final_state")


# ---- layouts

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K,V,offset", [(64, 64, 0), (64, 64, 1), (64, 64, 2), (128, 128, 1), (128, 96, 2), (40, 24, 0)])
def test_views_of_one_projection(K, V, offset, dtype):
    """Slices of wider rows, with an odd offset not even 4-byte aligned, with 2 not 16-byte: the bits of packed copies."""
    B, L, H, Hk = 2, 100, 4, 2
    gen = torch.Generator("cuda").manual_seed(5)
    wide = 0.1 * torch.randn(B, L, (H + Hk) * K + Hk * V + H * V + 8, device="cuda", generator=gen).to(dtype)
    cut = lambda at, n, w: wide[..., offset + at:offset + at + n * w].unflatten(-1, (n, w))
    q, k, v, do = (cut(0, H, K), cut(H * K, Hk, K), cut((H + Hk) * K, Hk, V), cut((H + Hk) * K + Hk * V, H, V))
    g = -torch.rand(B, L, H, device="cuda", generator=gen)
    beta = torch.rand(B, L, H, device="cuda", generator=gen)
    ssm = _ssm()
    packed = [x.contiguous() for x in (q, k, v)]
    for a, b in zip(ssm.gated_delta_fwd(q, k, v, g, beta), ssm.gated_delta_fwd(*packed, g, beta)):
        assert torch.equal(a, b)
    a, b = ssm.gated_delta_bwd(q, k, v, g, beta, do), ssm.gated_delta_bwd(*packed, g, beta, do.contiguous())
    for n in a:
        assert a[n] is None or torch.equal(a[n], b[n]), n
    # [L, batch, heads, width] in memory, and one head broadcast over the tokens by a stride of zero
    tq = q.transpose(0, 1).contiguous().transpose(0, 1)
    q0 = q[:, :1].expand(B, L, H, K)
    for x, y in ((tq, packed[0]), (q0, q0.contiguous())):
        for a, b in zip(ssm.gated_delta_fwd(x, k, v, g, beta), ssm.gated_delta_fwd(y, k, v, g, beta)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("which", ["batch", "token"])
def test_views_past_32_bits_of_elements(which):
    """Rows of a batch 2^31 elements apart, tokens 2^30 apart: the bits of packed copies."""
    ssm = _ssm()
    B, L, H, K = (2, 70, 2, 64) if which == "batch" else (1, 4, 2, 64)
    far = (1 << 31) + 64 if which == "batch" else 1 << 30
    span = (B - 1) * far if which == "batch" else (L - 1) * far
    store = torch.zeros(span + 4 * L * H * K, dtype=BF16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(21)
    views = {}
    for i, n in enumerate(("q", "k", "v", "do")):
        strides = (far, H * K, K, 1) if which == "batch" else (0, far, K, 1)
        views[n] = store.as_strided((B, L, H, K), strides, i * L * H * K)
        views[n].copy_(0.1 * torch.randn(B, L, H, K, device="cuda", generator=gen))
    t = {n: x.contiguous() for n, x in views.items()}
    gates = [-torch.rand(B, L, H, device="cuda", generator=gen), torch.rand(B, L, H, device="cuda", generator=gen)]
    for a, b in zip(ssm.gated_delta_fwd(views["q"], views["k"], views["v"], *gates),
                    ssm.gated_delta_fwd(t["q"], t["k"], t["v"], *gates)):
        assert torch.equal(a, b)
    a = ssm.gated_delta_bwd(views["q"], views["k"], views["v"], *gates, views["do"])
    b = ssm.gated_delta_bwd(t["q"], t["k"], t["v"], *gates, t["do"])
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(a[n], b[n]), n


def test_step_states_past_32_bits():
    ssm = _ssm()
    H, K, V = 40, 128, 128
    pool = (1 << 32) // (H * K * V * 4) + 2
    state = torch.zeros(pool, H, K, V, device="cuda")
    t, s0, _ = ref.inputs(1, 1, H, K, V, BF16, seed=15)
    state[-1] = s0[0].cuda()
    d = {n: x[:, 0].cuda() for n, x in t.items()}
    out = ssm.gated_delta_step(state, d["q"], d["k"], d["v"], d["g"], d["beta"],
                               slots=torch.tensor([pool - 1], dtype=torch.int32, device="cuda"))
    want, wfin = _want(t, K ** -0.5, s0)
    _check(out[:, None], want, OUT[BF16], "out")
    _check(state[-1:], wfin, STATE, "final_state")
    assert not state[:-1].any()


# ---- segments, pieces, states

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K,V", [(32, 32), (128, 128), (96, 128), (64, 128)])
def test_long_sequences_run_in_segments(K, V, dtype):
    """Few heads over many chunks, ragged: the last segment half there, and rows that end in an earlier one."""
    B, L, H = 3, 2100, 2
    t, s0, df = ref.inputs(B, L, H, K, V, dtype, (1, 2, 2), seed=6, rate=(0.001, 0.05))
    for lengths in (None, [2099, 700, 0]):
        out, fin = _forward(t, s0, lengths)
        want, wfin = _want(t, K ** -0.5, s0, lengths)
        _check(out, want, OUT[dtype], "out")
        _check(fin, wfin, STATE, "final_state")
        got = _gradient(t, s0, df, lengths)
        _check_grads(got, ref.delta_grad(*t.values(), K ** -0.5, s0, df, lengths), dtype)


def test_many_heads_without_segments():
    """A workgroup for every CU: whole sequences, 128 columns at a time."""
    t, s0, df = ref.inputs(9, 200, 16, 128, 128, BF16, (4, 4, 16), seed=7)
    out, fin = _forward(t, s0)
    want, wfin = _want(t, 128 ** -0.5, s0)
    _check(out, want, OUT[BF16], "out")
    _check(fin, wfin, STATE, "final_state")
    _check_grads(_gradient(t, s0, df), ref.delta_grad(*t.values(), 128 ** -0.5, s0, df), BF16)


def test_stretches_of_several_chunks():
    """Enough chunks for kept states to lie several apart: a head's gradients against those of a call of its own."""
    ssm = _ssm()
    B, L, H = 8, 1900, 16
    t, s0, df = ref.inputs(B, L, H, 64, 64, F32, seed=12)
    got = _gradient(t, s0, df)
    for b, h in ((0, 0), (7, 15)):
        one = {n: x[b:b + 1, :, h:h + 1] for n, x in t.items()}
        want = ref.delta_grad(*one.values(), 0.125, s0[b:b + 1, h:h + 1], df[b:b + 1, h:h + 1])
        part = {n: x[b:b + 1, h:h + 1] if "state" in n else x[b:b + 1, :, h:h + 1] for n, x in got.items()}
        _check_grads(part, want, F32)


def test_pieces_equal_the_whole_and_state_in_place():
    ssm = _ssm()
    t, s0, _ = ref.inputs(2, 300, 2, 64, 64, F32, seed=7)
    d = _cuda(t)
    whole, fin = _forward(t, s0)
    state = s0.cuda()
    parts = []
    for a, b in ((0, 100), (100, 101), (101, 300)):
        o, st = ssm.gated_delta_fwd(*(d[n][:, a:b].contiguous() if n in ("g", "beta") else d[n][:, a:b]
                                      for n in ("q", "k", "v", "g", "beta")), initial_state=state, final_state=state)
        assert st is state
        parts.append(o)
    _check(torch.cat(parts, 1), whole.double().cpu(), 2 * OUT[F32], "out")
    _check(state, fin.double().cpu(), 2 * STATE, "state")


def test_what_is_asked_for_changes_nothing_else():
    """Outputs with and without states, in outputs and workspaces full of NaN, and into given tensors: the same bits."""
    ssm = _ssm()
    for L, H in ((1500, 2), (130, 20)):
        t, s0, df = ref.inputs(2, L, H, 64, 128, BF16, (1, 2, 2), seed=10)
        d = _cuda(t)
        args = [d[n] for n in ("q", "k", "v", "g", "beta")]
        out, fin = ssm.gated_delta_fwd(*args)
        alone, none = ssm.gated_delta_fwd(*args, return_final_state=False)
        zeros, fin0 = ssm.gated_delta_fwd(*args, initial_state=torch.zeros_like(s0).cuda())
        assert none is None and torch.equal(out, alone) and torch.equal(out, zeros) and torch.equal(fin, fin0)
        ws = torch.full((ssm.gated_delta_workspace_size(2, L, H, 64, 128),), 255, dtype=torch.uint8, device="cuda")
        nan = lambda x: torch.full_like(x, float("nan"))
        o, f = ssm.gated_delta_fwd(*args, workspace=ws, out=nan(out), final_state=nan(fin))
        assert torch.equal(o, out) and torch.equal(f, fin)
        a = ssm.gated_delta_bwd(*args, d["do"], initial_state=s0.cuda(), dfinal_state=df.cuda())
        n = ssm.gated_delta_bwd_workspace_size(2, L, H, 64, 128, Hq=1, Hk=2, Hv=2)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        b = ssm.gated_delta_bwd(*args, d["do"], initial_state=s0.cuda(), dfinal_state=df.cuda(), workspace=ws,
                                out={x: nan(y) for x, y in a.items()})
        assert all(torch.equal(a[x], b[x]) for x in a)


def test_no_tokens():
    ssm = _ssm()
    t, s0, df = ref.inputs(2, 0, 2, 16, 8, BF16)
    out, fin = _forward(t, s0)
    assert out.shape == (2, 0, 2, 8) and torch.equal(fin.cpu(), s0)
    assert not _forward(t)[1].any()
    got = _gradient(t, None, df, want_dinitial_state=True)
    assert torch.equal(got["dinitial_state"].cpu(), df)
    none = torch.zeros(3, 0, 16, device="cuda")
    state = torch.ones(3, 0, 16, 8, device="cuda")
    with pytest.raises(ValueError):
        ssm.gated_delta_step(state, none, none, none[..., :8], none[..., 0], none[..., 0])
    # no rows
    d = {n: x[:0] for n, x in _cuda(ref.inputs(1, 5, 2, 16, 8, BF16)[0]).items()}
    out, fin = ssm.gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"])
    assert out.shape == (0, 5, 2, 8) and fin.shape == (0, 2, 16, 8)


def test_one_token_without_a_state_has_no_decay_to_learn():
    t, _, _ = ref.inputs(3, 1, 2, 64, 64, BF16, seed=1)
    got = _gradient(t)
    assert not got["dg"].any() and got["dbeta"].any()


# ---- values that are not finite

BAD = {"nan": float("nan"), "inf": float("inf")}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("token,value", [(0, "nan"), (1, "inf"), (31, "nan"), (63, "inf"), (64, "nan"), (100, "inf"), (149, "nan")])
def test_one_bad_value(token, value, name, dtype):
    """One value of one head: outputs before its token, of other rows, heads and (for v) columns are the others'; where the
    recurrence is not finite, neither is the result."""
    t, s0, _ = ref.inputs(2, 150, 2, 64, 64, dtype, seed=token)
    clean, cfin = _forward(t, s0)
    at = (1, token, 0) if name in ("g", "beta") else (1, token, 0, 37)
    t[name][at] = BAD[value]
    out, fin = _forward(t, s0)
    hit = torch.zeros(2, 150, 2, 64, dtype=torch.bool)
    if name == "q":
        hit[1, token, 0] = True
    elif name == "v":
        hit[1, token:, 0, 37] = True
    else:
        hit[1, token:, 0] = True
    hit = hit.cuda()
    assert torch.equal(out[~hit], clean[~hit])
    assert not torch.isfinite(out[hit]).any()
    keep = torch.ones_like(fin, dtype=torch.bool)
    if name == "v":
        keep[1, 0, :, 37] = False
    elif name != "q":
        keep[1, 0] = False
    assert torch.equal(fin[keep], cfin[keep])
    assert not torch.isfinite(fin[~keep]).any()


def test_masks_of_the_lowest_value():
    """A gate of float32's lowest value is a decay of 0, as -inf is."""
    t, s0, _ = ref.inputs(1, 100, 2, 64, 64, F32, seed=3)
    t["g"][0, 50] = torch.finfo(F32).min
    a = _forward(t, s0)
    t["g"][0, 50] = float("-inf")
    b = _forward(t, s0)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    want, wfin = _want(dict(t, g=t["g"].clamp(min=-1e5)), 0.125, s0)
    _check(a[0], want, OUT[F32], "out")
    _check(a[1], wfin, STATE, "final_state")


# ---- the gradient against differences, streams, graphs

@pytest.mark.parametrize("name", ["q", "v", "initial_state", "k", "g", "beta"])
def test_gradient_against_differences(name):
    """q, v and the state enter linearly, so a step of 1 has no truncation; the others by a step of 2^-7 in central differences,
    whose truncation is a third of 2^-14 of third derivatives, at most some tens of the terms' size: 2^-10 of it.  Either
    way the losses round to 2e-5 of their terms."""
    ssm = _ssm()
    t, s0, df = ref.inputs(1, 150, 2, 64, 64, F32, seed=8)
    d, dfc = _cuda(t), df.cuda()
    do = d.pop("do")
    d["initial_state"] = s0.cuda()
    h = 1.0 if name in ("q", "v", "initial_state") else 2.0 ** -7
    way = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(9)).cuda()

    def call(f, a, **kw):
        return f(a["q"], a["k"], a["v"], a["g"], a["beta"], **kw)

    got = ssm.gated_delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], do, initial_state=d["initial_state"],
                              dfinal_state=dfc)["d" + name]

    def loss(sign):
        a = dict(d)
        a[name] = a[name] + sign * h * way
        o, f = call(ssm.gated_delta_fwd, a, initial_state=a["initial_state"])
        return (o.double() * do).sum() + (f.double() * dfc).sum()

    diff = float(loss(1) - loss(-1)) / (2 * h)
    size = float(got.double().norm() * way.double().norm())
    bound = 2e-5 * size if h == 1.0 else 2.0 ** -10 * size + 2e-5 * float(do.norm() * d["v"].norm()) / h
    assert abs(diff - float((got.double() * way).sum())) <= bound


def test_results_do_not_change_from_call_to_call():
    t, s0, df = ref.inputs(2, 2100, 3, 64, 128, BF16, (3, 1, 1), seed=10)
    a, f = _gradient(t, s0, df), _forward(t, s0)
    for _ in range(2):
        b = _gradient(t, s0, df)
        assert all(torch.equal(a[n], b[n]) for n in a)
        assert all(torch.equal(x, y) for x, y in zip(f, _forward(t, s0)))


def test_runs_on_the_given_stream_and_in_graphs():
    """A forward pass, a gradient and a step captured together and replayed with other inputs and eager work between."""
    ssm = _ssm()
    t, s0, df = ref.inputs(1, 1100, 2, 64, 64, BF16, seed=11)
    d = _cuda(t)
    st, dfc, pool = s0.cuda(), df.cuda(), s0.cuda().repeat(3, 1, 1, 1)
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    last = [x[:, -1].contiguous() for x in args]
    slots = torch.tensor([2], dtype=torch.int32, device="cuda")
    call = lambda ws=None, wb=None: (*ssm.gated_delta_fwd(*args, initial_state=st, workspace=ws),
                                     *ssm.gated_delta_bwd(*args, d["do"], initial_state=st, dfinal_state=dfc,
                                                          workspace=wb).values(),
                                     ssm.gated_delta_step(pool, *last, slots=slots))
    ws = torch.empty(ssm.gated_delta_workspace_size(1, 1100, 2, 64, 64), dtype=torch.uint8, device="cuda")
    wb = torch.empty(ssm.gated_delta_bwd_workspace_size(1, 1100, 2, 64, 64), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    start = pool.clone()
    want = call()
    pool.copy_(start)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(ws, wb)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pool.copy_(start)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call(ws, wb)
    for i in range(3):
        st.copy_(s0.cuda() * (i + 1))
        pool.copy_(start * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        kept, after = [x.clone() for x in got], pool.clone()
        pool.copy_(start * (i + 1))
        eager = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager)) and torch.equal(after, pool)


STEPS = [(1, 1, 64, 64, None), (5, 6, 64, 64, (6, 2, 3)), (3, 4, 128, 128, (1, 1, 4)), (2, 2, 72, 40, None),
         (3, 2, 33, 17, None), (2, 1, 1, 1, None), (4, 2, 128, 100, None), (2, 3, 16, 4, None), (2, 1, 128, 127, None)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S,H,K,V,heads", STEPS)
def test_step_shapes(S, H, K, V, heads, dtype):
    t, s0, _ = ref.inputs(S, 1, H, K, V, dtype, heads, seed=K + V)
    d = {n: x[:, 0].cuda() for n, x in t.items()}
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    want, wfin = _want(t, K ** -0.5, s0)
    state = s0.cuda()
    out = _ssm().gated_delta_step(state, *args)
    _check(out[:, None], want, OUT[dtype], "out")
    _check(state, wfin, STATE, "state")
    other, start = torch.full_like(state, float("nan")), s0.cuda()
    out2 = _ssm().gated_delta_step(start, *args, out_state=other)
    assert torch.equal(out, out2) and torch.equal(other, state) and torch.equal(start.cpu(), s0)


def test_step_by_slots_leaves_other_states_alone():
    S, pool, H, K, V = 7, 11, 3, 64, 72
    t, _, _ = ref.inputs(S, 1, H, K, V, BF16, (3, 1, 1), seed=12)
    s0 = torch.randn(pool, H, K, V, generator=torch.Generator().manual_seed(13))
    slots = torch.tensor([3, -1, 10, 0, 11, 7, -2147483648], dtype=torch.int32)
    live = [i for i, x in enumerate(slots.tolist()) if 0 <= x < pool]
    d = {n: x[:, 0].cuda() for n, x in t.items()}
    state = s0.cuda()
    out = _ssm().gated_delta_step(state, d["q"], d["k"], d["v"], d["g"], d["beta"], slots=slots.cuda())
    at = slots[live].long()
    want, wfin = _want({n: x[live] for n, x in t.items()}, K ** -0.5, s0[at])
    _check(out[live][:, None], want, OUT[BF16], "out")
    _check(state[at.cuda()], wfin, STATE, "state")
    assert not out[[i for i in range(S) if i not in live]].any()
    rest = [i for i in range(pool) if i not in at.tolist()]
    assert torch.equal(state[rest].cpu(), s0[rest])
