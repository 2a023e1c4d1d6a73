"""Calls on a stream of their own (`stream=`) with everything allocated by the call: what the current stream
allocates, fills and frees around the call reaches neither the scratch memory nor the outputs, and the inputs may
be dropped at once.  Results equal the same call's on the current stream bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ssm():
    import selective_state_space_68_amd as ssm
    return ssm


def _rand(*shape, dtype=torch.float32):
    gen = torch.Generator("cuda").manual_seed(sum(shape))
    return torch.randn(*shape, device="cuda", generator=gen).to(dtype)


def _attention(L, heads):
    return [_rand(1, L, 4, 64, dtype=BF16), _rand(1, L, heads, 64, dtype=BF16), _rand(1, L, heads, 64, dtype=BF16),
            torch.tensor([-0.01, -0.1, -0.5, -1.0], device="cuda")]


def _scan(L):
    return [_rand(1, 8, L), _rand(1, 8, L), -_rand(8, 16).exp(), _rand(1, L, 16), _rand(1, L, 16)]


CALLS = {   # name: (inputs, call)
    "linear_attention_fwd": (lambda: _attention(1500, 4), "linear_attention_fwd", {}),
    "linear_attention_bwd": (lambda: _attention(1500, 2) + [_rand(1, 1500, 4, 64, dtype=BF16)], "linear_attention_bwd", {}),
    "linear_attention_step": (lambda: [_rand(3, 4, 64, 64), _rand(3, 4, 64), _rand(3, 4, 64), _rand(3, 4, 64),
                                       torch.full((4,), -0.1, device="cuda")], "linear_attention_step", {}),
    "block_norm_fwd": (lambda: [_rand(300, 256), _rand(300, 256)], "block_norm_fwd", {"pre_weight": lambda: _rand(256)}),
    "block_norm_bwd": (lambda: [_rand(300, 256), _rand(300, 256), _rand(300, 256)], "block_norm_bwd",
                       {"pre_weight": lambda: _rand(256)}),
    "selective_scan_fwd": (lambda: _scan(700), "selective_scan_fwd", {}),
    "selective_scan_bwd": (lambda: _scan(700) + [_rand(1, 8, 700)], "selective_scan_bwd", {}),
    "ssd_scan_fwd": (lambda: [_rand(1, 4096, 2, 64, dtype=BF16), _rand(1, 4096, 2, dtype=BF16), -_rand(2).exp(),
                              _rand(1, 4096, 64, dtype=BF16), _rand(1, 4096, 64, dtype=BF16)], "ssd_scan_fwd", {}),
}


def _tensors(got):
    got = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
    return [t for t in got if t is not None]


def _make(name):
    inputs, fn, named = CALLS[name]
    return getattr(_ssm(), fn)(*inputs(), **{n: f() for n, f in named.items()})


def _scribble():
    """Blocks of every size of the calls on the current stream, filled and freed."""
    for n in range(9, 25):
        for _ in range(4):
            torch.empty(1 << n, dtype=torch.uint8, device="cuda").fill_(0xff)


@pytest.mark.parametrize("late", ["current", "side"])
@pytest.mark.parametrize("name", CALLS)
def test_call_on_a_stream_of_its_own(name, late):
    want = [t.clone() for t in _tensors(_make(name))]
    inputs, fn, named = CALLS[name]
    args, kw = inputs(), {n: f() for n, f in named.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side if late == "side" else torch.cuda.current_stream()):
        torch.cuda._sleep(20_000_000)                       # the call's kernels wait behind this, or the scribbles
    _scribble()
    got = getattr(_ssm(), fn)(*args, **kw, stream=side if late == "side" else side.cuda_stream)
    del args, kw
    _scribble()
    side.synchronize()
    got = [t.cpu() for t in _tensors(got)]
    torch.cuda.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b.cpu()) for a, b in zip(got, want))


def test_results_are_the_streams_memory():
    # what the call allocated goes back to the stream's own blocks: none of them is handed out on the current stream
    ssm = _ssm()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = _attention(1500, 2)
    do = _rand(1, 1500, 4, 64, dtype=BF16)
    side.wait_stream(torch.cuda.current_stream())
    got = ssm.linear_attention_bwd(*a, do, stream=side)
    mine = {t.data_ptr() for t in _tensors(got)}
    del got
    torch.cuda.synchronize()
    assert not mine & {torch.empty(t, device="cuda").data_ptr() for t in [(1, 1500, 2, 64)] * 4}


def test_stream_of_no_tensor_is_refused():
    ssm = _ssm()
    with pytest.raises(ValueError, match="must live on the GPU"):
        x = torch.zeros(3, 16)
        ssm.block_norm_fwd(x, stream=torch.cuda.Stream())
