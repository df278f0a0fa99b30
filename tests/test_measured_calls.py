"""The handles that the measured calls keep (perf/operators.py), without a GPU."""
from types import SimpleNamespace

import torch

from perf import operators as O
from speculative_decoding_verification_pipeline_amd import sampler as SM


class Handle:
    def __init__(self, device, **limits):
        self.device, self.limits = device, limits


def test_handles_belong_to_a_device_and_a_stream(monkeypatch):
    at = SimpleNamespace(device=0, stream=11)
    monkeypatch.setattr(SM, "Sampler", Handle)
    monkeypatch.setattr(O, "_samplers", {})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at.device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=at.stream))
    a = O._sampler(max_batch=2, vocab_size=5)
    assert O._sampler(vocab_size=5, max_batch=2) is a and a.device == 0
    at.stream = 12
    b = O._sampler(max_batch=2, vocab_size=5)
    at.device = 1
    c = O._sampler(max_batch=2, vocab_size=5)
    assert len({id(x) for x in (a, b, c)}) == 3 and c.device == 1
    for V in range(6, 12):  # many sizes: what nobody uses any more is let go
        O._sampler(max_batch=2, vocab_size=V)
        assert len(O._samplers) <= 4
