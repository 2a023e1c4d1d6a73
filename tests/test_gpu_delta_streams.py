"""The gated delta rule and the query and key norms on a stream of their own (`stream=`), with everything allocated by the
call: what the current stream allocates, fills and frees around the call reaches neither scratch memory nor outputs."""
import pytest
import torch

import delta_reference as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ssm():
    import selective_state_space_68_amd as ssm
    return ssm


def _delta(L, grad):
    t, _, _ = ref.inputs(1, L, 4, 64, 64, BF16, (2, 2, 4), seed=L)
    return [t[n].cuda() for n in ("q", "k", "v", "g", "beta") + (("do",) if grad else ())]


def _step():
    t, s0, _ = ref.inputs(3, 1, 4, 64, 64, BF16, seed=1)
    return [s0.cuda()] + [t[n][:, 0].cuda() for n in ("q", "k", "v", "g", "beta")]


def _heads(n, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(2, 300, h, 64, device="cuda", generator=gen).to(BF16) for h in (4, 2)] * n


CALLS = {   # name: (inputs, named)
    "gated_delta_fwd": (lambda: _delta(1500, False), {}),
    "gated_delta_bwd": (lambda: _delta(1500, True), {}),
    "gated_delta_step": (_step, {}),
    "qk_norm_fwd": (lambda: _heads(1, 2), {"q_weight": lambda: torch.ones(64, device="cuda"),
                                          "inv_freq": lambda: torch.full((16,), 0.5, device="cuda")}),
    "qk_norm_bwd": (lambda: _heads(2, 3), {"k_weight": lambda: torch.ones(64, device="cuda")}),
}


def _tensors(got):
    got = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
    return [t for t in got if t is not None]


def _scribble():
    """Blocks of every size of the calls on the current stream, filled and freed."""
    for n in range(9, 25):
        for _ in range(4):
            torch.empty(1 << n, dtype=torch.uint8, device="cuda").fill_(0xff)


@pytest.mark.parametrize("late", ["current", "side"])
@pytest.mark.parametrize("name", CALLS)
def test_call_on_a_stream_of_its_own(name, late):
    inputs, named = CALLS[name]
    fn = getattr(_ssm(), name)
    want = [t.clone() for t in _tensors(fn(*inputs(), **{n: f() for n, f in named.items()}))]
    args, kw = inputs(), {n: f() for n, f in named.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side if late == "side" else torch.cuda.current_stream()):
        torch.cuda._sleep(20_000_000)                       # the call's kernels wait behind this, or the scribbles
    _scribble()
    got = fn(*args, **kw, stream=side if late == "side" else side.cuda_stream)
    del args, kw
    _scribble()
    side.synchronize()
    got = [t.cpu() for t in _tensors(got)]
    torch.cuda.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b.cpu()) for a, b in zip(got, want))


def test_two_calls_at_once():
    """The same call on two streams, each with its own scratch memory."""
    ssm = _ssm()
    args = _delta(1500, True)
    want = ssm.gated_delta_bwd(*args)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [ssm.gated_delta_bwd(*args, stream=s) for s in sides for _ in range(2)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(g[n], want[n]) for n in want if want[n] is not None)


def test_a_workspace_on_another_kind_of_memory_is_refused():
    ssm = _ssm()
    args = _delta(100, False)
    with pytest.raises(ValueError):
        ssm.gated_delta_fwd(*args, workspace=torch.empty(1 << 24, dtype=torch.uint8))
    with pytest.raises(ValueError):
        ssm.gated_delta_fwd(*args, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_qk_norm_in_a_graph():
    ssm = _ssm()
    q, k, dq, dk = _heads(2, 5)
    w, f = torch.rand(64, device="cuda") + 0.5, torch.rand(32, device="cuda")
    at = torch.zeros(2, 300, dtype=torch.int32, device="cuda")
    ws = torch.empty(ssm.qk_norm_bwd_workspace_size(64), dtype=torch.uint8, device="cuda")
    call = lambda ws=None: (*ssm.qk_norm_fwd(q, k, w, w, inv_freq=f, positions=at),
                            *ssm.qk_norm_bwd(q, k, dq, dk, w, w, inv_freq=f, positions=at, workspace=ws).values())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call(ws)
    for i in range(3):
        at.fill_(1000 * i)
        w.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in got]
        eager = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager))
