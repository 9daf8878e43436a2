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


S, HQ, HKV = 64, 4, 2
MASK = mab.Mask(kind=mab.ATTN_MASK_CAUSAL)


def _run(monkeypatch, which, dev, mask=MASK, **other):
    q, k = Tensor([1, HQ, S, 128], dev), Tensor([1, HKV, S, 128], dev)
    t = dict(q=q, k=k, v=k, sink=Tensor([HQ], dev, torch.float32),
             ws=Tensor([1 << 20], dev, torch.uint8))
    if which == "fwd":
        monkeypatch.setattr(torch, "empty_like", lambda x: x)
        monkeypatch.setattr(torch, "empty", lambda s, **kw: Tensor(s, dev))
        t.update(other)
        return mab.fwd(t["q"], t["k"], t["v"], t["sink"], mask, 0.1, ws=t["ws"])
    t.update(o=q, dO=q, lse=Tensor([1, HQ, S], dev, torch.float32), dq=q, dk=k, dv=k,
             dsink=t["sink"])
    t.update(other)
    return mab.bwd(t["q"], t["k"], t["v"], t["o"], t["dO"], t["lse"], t["sink"], mask, 0.1,
                   ws=t["ws"], out=(t["dq"], t["dk"], t["dv"], t["dsink"]))


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("dev", [0, 1])
def test_a_call_runs_on_its_tensors_device(monkeypatch, calls, which, dev):
    _run(monkeypatch, which, dev)
    assert calls == [(dev, 1000 + dev)]


KV = Tensor([1, HKV, S, 128], 1)
LENS = torch.ones(1, dtype=torch.int32)


@pytest.mark.parametrize("which,other", [
    ("fwd", dict(k=KV)), ("fwd", dict(v=KV)), ("fwd", dict(sink=torch.zeros(HQ))),
    ("fwd", dict(sink=Tensor([HQ], 1, torch.float32))),
    ("fwd", dict(ws=Tensor([1 << 20], 1, torch.uint8))),
    ("fwd", dict(mask=mab.Mask(kind=mab.ATTN_MASK_CAUSAL, seqlen_q=LENS, seqlen_k=LENS))),
    ("fwd", dict(mask=mab.Mask(kind=mab.ATTN_MASK_BLOCK, bx=64, by=64,
                               block_mask=torch.ones(1, HQ, 1, 1, dtype=torch.uint8)))),
    ("bwd", dict(v=KV)), ("bwd", dict(sink=torch.zeros(HQ))), ("bwd", dict(dk=KV)),
    ("bwd", dict(dsink=torch.zeros(HQ))), ("bwd", dict(lse=Tensor([1, HQ, S], 1, torch.float32))),
    ("bwd", dict(mask=mab.Mask(kind=mab.ATTN_MASK_CAUSAL, seqlen_q=LENS, seqlen_k=LENS)))])
def test_tensors_of_the_host_or_of_several_devices_are_refused(monkeypatch, calls, which, other):
    with pytest.raises(ValueError):
        _run(monkeypatch, which, 0, **other)
    assert calls == []


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("sink", [Tensor([HQ], 0, torch.bfloat16), Tensor([HQ - 1], 0, torch.float32),
                                  Tensor([HQ], 0, torch.float64)])
def test_sinks_of_another_type_or_size_are_refused(monkeypatch, calls, which, sink):
    with pytest.raises(ValueError):
        _run(monkeypatch, which, 0, sink=sink)
    assert calls == []
