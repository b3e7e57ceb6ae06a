"""Linear attention where large terms cancel: what fp32 arithmetic gives, and operands of the matrix
products that hold fewer bits than fp32 do not."""
import pytest
import torch

from la_util import BF16_HALF

pytestmark = pytest.mark.gpu
CALLS = [("la_decode", 3), ("la_decode", 8), ("la_prefill", 3), ("la_prefill", 65), ("la_prefill", 700)]  # the last in segments


@pytest.fixture(scope="module")
def rg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_rgdr_amd as m
    m.library()
    return m


def zeros(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def call(rg, fn, q, k, v, g, pool):
    out, pool = getattr(rg, fn)(q.cuda(), k.cuda(), v.cuda(), g.cuda(), pool.cuda())
    torch.cuda.synchronize()
    return out.double().cpu(), pool.double().cpu()


@pytest.mark.parametrize("Dk", [64, 128, 256])
@pytest.mark.parametrize("fn,T", CALLS)
def test_difference_of_two_rows(rg, fn, T, Dk):
    """q picks one row of the state and takes another away. Both are 1 + 2^-9 + a 2^-22 (24 bits), every
    product, partial sum and the difference a fp32 number, the last one a bf16 number: exact."""
    r = torch.Generator().manual_seed(Dk)
    a = torch.randint(-60, 61, (2, 2, 64), generator=r).double()
    pool = torch.zeros(1, 2, Dk, 64)
    pool[0, :, 3], pool[0, :, Dk - 5] = ((1 + 2.0 ** -9 + a * 2.0 ** -22).float())
    q = zeros(1, 1, T, Dk)
    q[..., 3], q[..., Dk - 5] = 1, -1
    out, after = call(rg, fn, q, zeros(1, 1, T, Dk), zeros(1, 2, T, 64), torch.zeros(1, 2, T), pool)
    want = (a[0] - a[1])[None, :, None] * 2.0 ** -22
    assert torch.equal(out, want.expand(1, 2, T, 64))
    assert torch.equal(after, pool.double())


@pytest.mark.parametrize("Dk", [64, 128, 256])
@pytest.mark.parametrize("fn,T", CALLS)
def test_difference_of_two_scores(rg, fn, T, Dk):
    """Scores of the first two tokens, 1 + 2^-9 and 1 + 2^-9 + 2^-22, on values 1 and -1: exactly -2^-22
    at every token behind them, by way of the scores or of the state (whose row is then -2^-11)."""
    q, k, v = zeros(1, 1, T, Dk), zeros(1, 1, T, Dk), zeros(1, 1, T, 96)
    q[..., 0], q[..., Dk - 1], q[..., 7] = 1, 2.0 ** -11, 1
    k[:, :, :2, 0], k[:, :, 1, Dk - 1], k[:, :, :2, 7] = 1, 2.0 ** -11, 2.0 ** -9
    v[:, :, 0], v[:, :, 1] = 1, -1
    out, _ = call(rg, fn, q, k, v, torch.zeros(1, 1, T), torch.zeros(1, 1, Dk, 96))
    assert torch.equal(out[:, :, 1:], torch.full((1, 1, T - 1, 96), -2.0 ** -22, dtype=torch.float64))


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("fn,T", CALLS)
def test_state_of_two_tokens_that_cancel(rg, fn, T, state):
    """One row of the state: exp(d) (exp(c) v0 - v1), the first decay at token 1, the other at the
    last one, v1 the bf16 number next to exp(c) v0. Of the magnitudes' sum A, each of the two decays is
    off by 2^-26 for its exponent's rounding (it is below 0.5 in magnitude), 2^-23 for the exponential and
    2^-24 for its product, a value in three bf16 parts by 2^-27, and each of the up to four sums into
    which the terms go by 2^-24 (2^-23 where it truncates): below 2^-20 A. A bf16 state rounds by half
    a step more."""
    H, Dk, Dv = 32, 64, 128
    r = torch.Generator().manual_seed(T)
    g = torch.zeros(1, H, T)
    g[0, :, 1] = -0.25 * torch.rand(H, generator=r) - 0.05
    g[0, :, T - 1] = -0.25 * torch.rand(H, generator=r) - 0.05
    k, v = zeros(1, 1, T, Dk), zeros(1, H, T, Dv)
    k[:, :, :2, 5] = 1
    v[0, :, 0] = (1 + torch.arange(Dv) / 128).bfloat16()
    kept = torch.exp(g[0, :, 1].double())[:, None] * v[0, :, 0].double()
    v[0, :, 1] = (-kept).bfloat16()
    last = torch.exp(g[0, :, T - 1].double())[:, None]
    want = last * (kept + v[0, :, 1].double())
    size = last * (kept + v[0, :, 1].double().abs())
    _, pool = call(rg, fn, zeros(1, 1, T, Dk), k, v, g, torch.zeros(1, H, Dk, Dv, dtype=state))
    bound = 2.0 ** -20 * size + (BF16_HALF * (want.abs() + 2.0 ** -20 * size) if state == torch.bfloat16 else 0)
    over = (pool[0, :, 5] - want).abs() - bound
    assert over.max() <= 0, f"{(over > 0).sum()} of {over.numel()} off, by {over.max():.3g} more than the bound"
    pool[0, :, 5] = 0
    assert torch.all(pool == 0)
