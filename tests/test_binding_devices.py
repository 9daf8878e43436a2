"""Which device the binding's calls run on, with stand-ins for tensors of two
devices (no GPU): the library is replaced by a record of what it is given."""
import pytest
import torch

from masked_attention_backward_gb300 import binding as mab


class Tensor:
    """What the binding asks of a tensor."""

    is_cuda = True

    def __init__(self, shape, device=1, dtype=torch.float16):
        self.shape, self.index, self.dtype = torch.Size(shape), device, dtype
        self.device = torch.device("cuda", device)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 0x7F0000000000


@pytest.fixture
def calls(monkeypatch):
    """Current device and stream of each call that reaches the library."""
    seen, current = [], [0]

    class Guard:
        def __init__(self, dev):
            self.dev = dev if isinstance(dev, int) else dev.index

        def __enter__(self):
            self.before, current[0] = current[0], self.dev

        def __exit__(self, *_):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(mab, "_raw_stream", lambda dev: 1000 + dev)
    for n in ("attn_fwd", "attn_bwd", "attn_get_device_status"):
        monkeypatch.setattr(mab, n, lambda *a: seen.append((current[0], a[-1])) or mab.ATTN_OK)
    return seen


@pytest.mark.parametrize("dev", [0, 1])
def test_the_status_is_read_on_the_workspace_s_device(calls, dev):
    # the stream that is waited for first has to be that device's
    assert mab.device_status(Tensor([4096], dev, torch.uint8)) == mab.ATTN_OK
    assert calls == [(dev, 1000 + dev)]
