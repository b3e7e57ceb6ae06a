"""The state space scan at the ends of what it accepts (bounds: ssm_util)."""
import pytest
import torch

from ssm_form import prefill_form
from ssm_util import U, HALF, TINY
from test_gpu_ssm import Case, rg  # noqa: F401  (rg is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("operand", ["x", "dt", "z", "Bm", "Cm"])
@pytest.mark.parametrize("dtype,N", [("bf16", 16), ("f32", 32)])
def test_far_tokens_over_several_chunks(rg, operand, dtype, N):  # noqa: F811
    """Tokens as far apart as is allowed, 2^25 bytes, in a call of 16 lanes for each channel, whose chunks have
    128 tokens: the second one starts 2^32 bytes behind the first."""
    T, C = 140, 64
    assert prefill_form(1, T, C, N, 1)[0] == 16
    c = Case(1, T, C, N, 1, dtype, "f32", 31, lens=[T], acc=[T], layout="whole", slow=0.1)
    ref = c.reference()
    near = getattr(c, operand)
    step = 2 ** 25 // near.element_size()
    far = torch.empty((T - 1) * step + 64, dtype=near.dtype, device="cuda")
    view = far.as_strided(near.shape, (8, step, *near.stride()[2:]))
    view.copy_(near)
    setattr(c, operand, view)
    out, after = c.call(rg, "ssm_prefill")
    c.check(out, after, ref, f"{operand} {dtype}")


@pytest.mark.parametrize("fn", ["ssm_decode", "ssm_prefill"])
def test_softplus_over_its_range(rg, fn):  # noqa: F811
    """With x = 1, B = 1, C picking one state and a pool of zeros the output is the step itself: softplus is
    good to (3 |s| + 16) u of its value (ssm_util) at every s, also where 1 + e^s is the next number to 1."""
    T, C = 8, 4096
    dt = torch.linspace(-110, 40, T * C).reshape(1, T, C)
    x = torch.ones(1, T, C)
    Bm, Cm = torch.ones(1, T, 1, 8), torch.zeros(1, T, 1, 8)
    Cm[..., 0] = 1
    A = torch.full((C, 8), -float("inf"))  # nothing is left of the state before
    pool = torch.zeros(1, C, 8)
    out, _ = getattr(rg, fn)(*(t.cuda() for t in (x, dt, A, Bm, Cm, pool)))
    want = torch.logaddexp(dt.double(), torch.zeros((), dtype=torch.float64))
    # a step below 2^-126 may be zero
    err = (out.double().cpu() - want).abs() - (3 * dt.double().abs() + 16) * U * want - TINY[torch.float32] - HALF[torch.float32] * want
    assert err.max() <= 0, f"off by {float(err.max()):.3g} more than the bound at dt = {float(dt.flatten()[err.argmax()])}"


def test_more_workgroups_than_the_wider_form_may_have(rg):  # noqa: F811
    """300000 entries of 2048 channels: 19 million workgroups with 8 lanes for each channel, 9.6 with four. All
    entries but three have no slot; their rows are zeros."""
    B, C, N = 300000, 2048, 8
    assert prefill_form(B, 1, C, N, 1)[0] == 4
    c = Case(3, 1, C, N, 1, "bf16", "f32", 32, slots=3, lens=[1] * 3, acc=[1] * 3, idx=[2, 0, 1], layout="whole")
    ref = c.reference()
    at = [0, 123457, B - 1]

    def rows(t):
        wide = torch.zeros(B, *t.shape[1:], dtype=t.dtype, device="cuda")
        wide[at] = t
        return wide
    idx = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    idx[at] = c.idx.cuda()
    out, after = rg.ssm_prefill(rows(c.x), rows(c.dt), c.A, rows(c.Bm), rows(c.Cm), c.pool, None, idx, D=c.D,
                                z=rows(c.z), dt_bias=c.bias)
    c.check(out[at], after, ref, "300000 entries")
    out[at] = 0
    assert not out.any()
