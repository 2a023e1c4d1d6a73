"""GPU parity of the block norms (forward and gradient) with the row formulas in float64.

Error: the 2-norm of the difference over the 2-norm of the result (whole tensor), and the
largest difference over max(|value|, root mean square).  Bounds: float32 results come from
row sums of at most 16384 float32 terms added in strands (about 16384 / 64 * 2^-24 = 1.5e-5
at worst, far less in norm) and the hardware exponential (1e-6 of the sigmoid): 2e-5 in
norm, 1e-4 at most.  bfloat16 results add one rounding, 2^-9 = 2e-3: 4e-3 in norm, 8e-3 at
most.  Column sums run over `rows` float32 terms that cancel: 2e-5 of the norm holds with the terms
random, as here.
"""
import pytest
import torch

import lm_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NORM = {F32: 2e-5, BF16: 4e-3}
MOST = {F32: 1e-4, BF16: 8e-3}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ssm():
    import selective_state_space_68_amd as ssm
    return ssm


def _check(got, want, what):
    g, w = got.detach().double().cpu(), want.double()
    assert g.shape == w.shape and torch.isfinite(g).all(), what
    if w.numel() == 0:
        return
    norm = float((g - w).norm() / w.norm().clamp(min=1e-30))
    rms = w.square().mean().sqrt()
    most = float(((g - w).abs() / torch.maximum(w.abs(), rms).clamp(min=1e-30)).max())
    print(f"{what} {tuple(got.shape)} {got.dtype}: norm {norm:.2e}, most {most:.2e}", flush=True)
    assert norm <= NORM[got.dtype] and most <= MOST[got.dtype], (what, norm, most)


FORMS = {   # what is there: residual, gate, post, scale, pre
    "all": "rgpsn", "gated": "gp", "pre": "n", "residual_pre": "rn", "both_norms": "rpn", "scaled": "rps",
    "gate_only": "g", "no_residual": "gpsn", "residual_only": "r",
}


def _inputs(rows, D, dtype, rdtype, form, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    has = FORMS[form]
    return dict(x=r(rows, D).to(dtype), residual=(2 * r(rows, D)).to(rdtype) if "r" in has else None,
                gate=r(rows, D).to(dtype) if "g" in has else None,
                post_weight=1 + 0.2 * r(D) if "p" in has else None,
                res_scale=0.5 + 0.3 * r(D) if "s" in has else None,
                pre_weight=1 + 0.2 * r(D) if "n" in has else None), r(rows, D).to(dtype), r(rows, D).to(rdtype)


def _cuda(a):
    return {k: None if v is None else v.cuda() for k, v in a.items()}


TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]
SIZES = [(1, 1, 1), (3, 7, 1), (5, 33, 1), (2, 64, 1), (9, 512, 4), (3, 513, 1), (4, 1000, 5), (6, 1024, 8),
         (3, 769, 1), (2, 1536, 2), (4, 2048, 32), (2, 2560, 20), (3, 4096, 32), (2, 5120, 80), (2, 6144, 6),
         (1, 8192, 128), (2, 9000, 9), (1, 16384, 1), (1, 16381, 1)]


def _run(a, dy, dh, groups, rdtype, eps=1e-5):
    ssm = _ssm()
    d = _cuda(a)
    h, y = ssm.block_norm_fwd(**d, groups=groups, eps=eps, residual_dtype=rdtype)
    wh, wy = ref.block_norm(**a, groups=groups, eps=eps)
    assert h.dtype == rdtype and (y is None) == (wy is None)
    _check(h, wh, "h")
    if y is not None:
        _check(y, wy, "y")
    rest = {k: d[k] for k in ("gate", "post_weight", "res_scale", "pre_weight")}
    got = ssm.block_norm_bwd(d["x"], h, dy.cuda() if y is not None else None, dh.cuda(), **rest, groups=groups, eps=eps,
                             residual_dtype=rdtype if a["residual"] is not None else None)
    want = ref.block_norm_grad(a["x"], h.cpu(), dy, dh, *(a[k] for k in rest), groups=groups, eps=eps)
    for k, w in want.items():
        if k == "dresidual" and a["residual"] is None:
            assert got[k] is None
        else:
            _check(got[k], w, k)
    assert {k for k, v in got.items() if v is not None} == {k for k in want if k != "dresidual"} | (
        {"dresidual"} if a["residual"] is not None else set())


@pytest.mark.parametrize("dtype,rdtype", TYPES)
@pytest.mark.parametrize("rows,D,groups", SIZES)
def test_sizes(rows, D, groups, dtype, rdtype):
    a, dy, dh = _inputs(rows, D, dtype, rdtype, "all", seed=D)
    _run(a, dy, dh, groups, rdtype)


@pytest.mark.parametrize("dtype,rdtype", TYPES)
@pytest.mark.parametrize("form", FORMS)
def test_forms(form, dtype, rdtype):
    a, dy, dh = _inputs(37, 384, dtype, rdtype, form, seed=1)
    _run(a, dy, dh, 3 if a["post_weight"] is not None else 1, rdtype)


@pytest.mark.parametrize("dtype,rdtype", TYPES)
def test_many_rows(dtype, rdtype):
    a, dy, dh = _inputs(3001, 136, dtype, rdtype, "all", seed=2)
    _run(a, dy, dh, 1, rdtype)


@pytest.mark.parametrize("dtype,rdtype", TYPES)
@pytest.mark.parametrize("rows,D,groups", [(1100, 769, 1), (700, 2560, 20), (600, 5120, 1), (520, 5121, 1), (300, 8192, 64),
                                           (290, 9000, 1), (270, 12296, 1)])
def test_many_wide_rows(rows, D, groups, dtype, rdtype):
    # more rows than workgroups: the column sums run over several rows of one
    a, dy, dh = _inputs(rows, D, dtype, rdtype, "all", seed=D)
    _run(a, dy, dh, groups, rdtype)


def test_zero_rows_and_large_values():
    # eps bounds the norm of a row of zeros; squares of 1e18 stay in float32's range
    a, dy, dh = _inputs(4, 96, F32, F32, "both_norms", seed=3)
    a["x"][0] = 0.0
    a["residual"][0] = 0.0
    a["x"][1] *= 1e18
    _run(a, dy, dh, 2, F32, eps=1e-3)
    # a gate of either infinity's size: silu is 0 or the gate
    b, dy, dh = _inputs(2, 64, F32, F32, "gated", seed=4)
    b["gate"][0], b["gate"][1] = -200.0, 200.0
    _run(b, dy, dh, 1, F32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset,D,groups", [(0, 128, 2), (1, 128, 2), (3, 65, 1)])
def test_strided_rows(offset, D, groups, dtype):
    # x and gate as slices of one projection's rows, aligned and not
    ssm = _ssm()
    gen = torch.Generator().manual_seed(5)
    wide = torch.randn(2, 11, 3 * D + 8, generator=gen).to(dtype)
    cut = lambda t: (t[..., offset:offset + D], t[..., offset + D:offset + 2 * D])
    w = 1 + 0.1 * torch.randn(D, generator=gen)
    x, z = cut(wide.cuda())
    hx, hz = cut(wide)
    h, _ = ssm.block_norm_fwd(x, gate=z, post_weight=w.cuda(), groups=groups)
    _check(h, ref.block_norm(hx, gate=hz, post_weight=w, groups=groups)[0], "h")
    dh = torch.randn(2, 11, D, generator=gen).to(dtype)
    got = ssm.block_norm_bwd(x, dh=dh.cuda(), gate=z, post_weight=w.cuda(), groups=groups)
    want = ref.block_norm_grad(hx, None, None, dh, hz, w, groups=groups)
    for k in ("dx", "dgate", "dpost_weight"):
        _check(got[k], want[k], k)


def test_in_place_residual_and_h_not_stored():
    ssm = _ssm()
    a, dy, dh = _inputs(9, 256, BF16, F32, "all", seed=6)
    d = _cuda(a)
    h, y = ssm.block_norm_fwd(**d)
    keep = d["residual"]
    h2, y2 = ssm.block_norm_fwd(**d, h=keep)
    assert h2 is keep and torch.equal(h, h2) and torch.equal(y, y2)
    none, y3 = ssm.block_norm_fwd(**{**d, "residual": a["residual"].cuda()}, return_h=False)
    assert none is None and torch.equal(y, y3)
    rest = {k: d[k] for k in ("gate", "post_weight", "res_scale", "pre_weight")}
    g1 = ssm.block_norm_bwd(d["x"], h, dy.cuda(), dh.cuda(), **rest, residual_dtype=F32)
    buf = dh.cuda()
    g2 = ssm.block_norm_bwd(d["x"], h, dy.cuda(), buf, **rest, residual_dtype=F32, out={"dresidual": buf})
    assert g2["dresidual"] is buf and all(torch.equal(g1[k], g2[k]) for k in g1)
    # without a gradient from elsewhere
    g3 = ssm.block_norm_bwd(d["x"], h, dy.cuda(), None, **rest, residual_dtype=F32)
    want = ref.block_norm_grad(a["x"], h.cpu(), dy, None, *(a[k] for k in rest))
    for k, w in want.items():
        _check(g3[k], w, k)


def test_no_rows():
    ssm = _ssm()
    a, dy, dh = _inputs(0, 64, BF16, F32, "all")
    d = _cuda(a)
    h, y = ssm.block_norm_fwd(**d)
    assert h.shape == y.shape == (0, 64)
    g = ssm.block_norm_bwd(d["x"], h, dy.cuda(), dh.cuda(), d["gate"], d["post_weight"], d["res_scale"], d["pre_weight"],
                           residual_dtype=F32)
    assert not any(g[k].any() for k in ("dpost_weight", "dres_scale", "dpre_weight"))


@pytest.mark.parametrize("name", ["x", "residual", "gate", "post_weight", "res_scale", "pre_weight"])
def test_gradient_against_differences(name):
    # central differences of the float32 kernel: truncation step^2 = 1e-4 of the third derivative, rounding 1e-6 / step
    ssm = _ssm()
    a, dy, dh = _inputs(6, 200, F32, F32, "all", seed=7)
    d, dyc, dhc = _cuda(a), dy.cuda(), dh.cuda()
    h, _ = ssm.block_norm_fwd(**d, groups=5)
    got = ssm.block_norm_bwd(d["x"], h, dyc, dhc, d["gate"], d["post_weight"], d["res_scale"], d["pre_weight"], groups=5,
                             residual_dtype=F32)["d" + name]
    step = 1e-2
    to = torch.randn(a[name].shape, generator=torch.Generator().manual_seed(8)).cuda()

    def loss(s):
        h, y = ssm.block_norm_fwd(**{**d, name: d[name] + s * to}, groups=5)
        return (h.double() * dhc).sum() + (y.double() * dyc).sum()

    diff = float(loss(step) - loss(-step)) / (2 * step)
    size = float(got.double().norm() * to.double().norm())
    assert abs(diff - float((got.double() * to).sum())) <= 1e-3 * size


def test_runs_on_the_given_stream_and_in_a_graph():
    ssm = _ssm()
    a, dy, dh = _inputs(700, 512, BF16, F32, "all", seed=9)
    d = _cuda(a)
    dyc, dhc = dy.cuda(), dh.cuda()
    rest = [d[k] for k in ("gate", "post_weight", "res_scale", "pre_weight")]
    ws = torch.empty(ssm.block_norm_bwd_workspace_size(700, 512), dtype=torch.uint8, device="cuda")
    h, y = ssm.block_norm_fwd(**d)
    g = ssm.block_norm_bwd(d["x"], h, dyc, dhc, *rest, residual_dtype=F32)
    h2, y2, g2 = torch.empty_like(h), torch.empty_like(y), {k: torch.empty_like(v) for k, v in g.items()}

    def call():
        ssm.block_norm_fwd(**d, h=h2, y=y2)
        ssm.block_norm_bwd(d["x"], h2, dyc, dhc, *rest, residual_dtype=F32, workspace=ws, out=g2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(3):
        for t in (h2, y2, *g2.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g)
        ssm.block_norm_fwd(**d)                             # (eager work between the replays)
        torch.cuda.synchronize()


def test_rows_past_32_bits_of_elements():
    ssm = _ssm()
    rows, D, far = 4, 136, 1 << 30
    store = torch.zeros((rows - 1) * far + 2 * D, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(23)
    views = [store.as_strided((rows, D), (far, 1), i * D) for i in range(2)]
    for x in views:
        x.copy_(torch.randn(rows, D, device="cuda", generator=gen))
    x, gate = (a.contiguous() for a in views)
    w = torch.randn(D, device="cuda", generator=gen)
    for a, b in zip(ssm.block_norm_fwd(views[0], None, views[1], w, pre_weight=w),
                    ssm.block_norm_fwd(x, None, gate, w, pre_weight=w)):
        assert torch.equal(a, b)
    dh = torch.randn(rows, D, device="cuda", generator=gen).bfloat16()
    a = ssm.block_norm_bwd(views[0], None, None, dh, views[1], w)
    b = ssm.block_norm_bwd(x, None, None, dh, gate, w)
    for n in ("dx", "dgate", "dpost_weight"):
        assert torch.equal(a[n], b[n]), n
