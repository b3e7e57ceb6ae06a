"""RGDR_VALIDATE checks the lengths of the calls that take no slots."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_rgdr_amd as m
    m.library()
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("op", ["rope", "norm"])
@pytest.mark.parametrize("own_stream", [False, True])
def test_lengths_are_validated(rg, monkeypatch, op, own_stream):
    x = torch.randn(2, 3, 4, 64, device="cuda")
    freq, w = torch.ones(32, device="cuda"), torch.ones(64, device="cuda")
    stream = torch.cuda.Stream() if own_stream else None
    torch.cuda.synchronize()

    def call(lens, x=x):
        if op == "rope":
            return rg.la_rope(x, None, freq, actual_seq_lengths=lens, stream=stream)[0]
        return rg.la_norm_gate(x, w, actual_seq_lengths=lens, stream=stream)
    want = call(ints([4, 2]))
    clamped = call(ints([9, -1]))
    monkeypatch.setattr(rg, "VALIDATE", True)
    assert torch.equal(call(ints([4, 2])), want)
    torch.cuda.synchronize()
    for bad in ([5, 2], [4, -1]):
        with pytest.raises(RuntimeError, match="index arrays"):
            call(ints(bad))
    call(None)
    call(ints([]), x[:0])
    for wrong in (ints([1]), ints([1, 2]).long(), torch.tensor([1, 2], dtype=torch.int32)):
        with pytest.raises(RuntimeError, match="actual_seq_lengths"):
            call(wrong)
    monkeypatch.setattr(rg, "VALIDATE", False)
    assert torch.equal(call(ints([9, -1])), clamped)
    torch.cuda.synchronize()
