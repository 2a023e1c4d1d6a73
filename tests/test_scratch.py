"""The scratch memory that a call allocates for itself lives until its kernels are launched, on the CPU: the
tensors say that they live on GPU 0, the library's launches are replaced by a look at which allocations are
still held (the foreign call lets other threads run, so a block that is free by then may be another call's)."""
import weakref

import pytest
import torch

import selective_state_space_68_amd as ssm
from selective_state_space_68_amd import _lib, lm_ops, ops

BF16 = torch.bfloat16


class OnGpu(torch.Tensor):
    """A CPU tensor that passes for one of GPU 0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


class Host:
    """Stands for the library: sizes are its own, a launch looks at the allocations."""

    def __init__(self, library):
        self.library, self.allocated, self.launches = library, [], 0

    def empty(self, make):
        def empty(shape, *args, **kw):
            t = make(shape, *args, **kw).as_subclass(OnGpu)
            if kw.get("dtype") is torch.uint8:
                self.allocated.append(weakref.ref(t))
            return t
        return empty

    def launch(self, *args):
        self.launches += 1
        assert self.allocated, "the call was to need scratch memory"
        assert all(t() is not None for t in self.allocated), "scratch memory is free before the launch"
        return 0

    def __getattr__(self, name):
        return getattr(self.library, name) if name.endswith("_size") else self.launch


@pytest.fixture
def host(monkeypatch):
    h = Host(_lib.load_library())
    monkeypatch.setattr(torch, "empty", h.empty(torch.empty))
    monkeypatch.setattr(_lib, "load_library", lambda: h)
    monkeypatch.setattr(ops, "_stream", lambda: 0)
    monkeypatch.setattr(lm_ops, "_entry", lambda name: getattr(h, name))
    monkeypatch.setattr(lm_ops, "_run", lambda fn, index, *args: fn(*args))
    return h


def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def attention(heads=2, L=1500):
    return [t(1, L, heads, 64, dtype=BF16) for _ in range(3)] + [t(2)]


def scan(L):
    u = [t(1, 8, L) for _ in range(2)]
    return u + [t(8, 16), t(1, L, 16), t(1, L, 16)]


CALLS = {
    "linear_attention_fwd": lambda: ssm.linear_attention_fwd(*attention()),
    "linear_attention_bwd": lambda: ssm.linear_attention_bwd(*attention(), dout=t(1, 1500, 2, 64, dtype=BF16)),
    "linear_attention_bwd, shared heads": lambda: ssm.linear_attention_bwd(
        *attention(1, 30), dout=t(1, 30, 2, 64, dtype=BF16)),
    "block_norm_bwd": lambda: ssm.block_norm_bwd(t(4, 64), t(4, 64), t(4, 64), None, pre_weight=t(64)),
    "selective_scan_bwd": lambda: ssm.selective_scan_bwd(*scan(2048), t(1, 8, 2048)),
    "ssd_scan_fwd": lambda: ssm.ssd_scan_fwd(t(1, 4096, 2, 64, dtype=BF16), t(1, 4096, 2, dtype=BF16), t(2),
                                             t(1, 4096, 64, dtype=BF16), t(1, 4096, 64, dtype=BF16)),
}


@pytest.mark.parametrize("name", CALLS)
def test_scratch_lives_until_the_launch(host, name):
    CALLS[name]()
    assert host.launches == 1


def test_workspace_of_another_gpu_is_refused(host):
    class Elsewhere(OnGpu):
        device = property(lambda self: torch.device("cuda", 1))

    workspace = torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        ssm.linear_attention_fwd(*attention(), workspace=workspace)
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        ssm.ssd_scan_fwd(t(1, 4096, 2, 64, dtype=BF16), t(1, 4096, 2, dtype=BF16), t(2), t(1, 4096, 64, dtype=BF16),
                         t(1, 4096, 64, dtype=BF16), workspace=workspace)
    assert host.launches == 0
