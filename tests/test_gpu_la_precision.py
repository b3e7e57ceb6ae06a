"""Linear attention where large terms cancel (what fp32 arithmetic gives, and operands of the matrix
products that hold fewer bits than fp32 do not), and over many steps on rounded states."""
import pytest
import torch

from la_util import BF16_HALF, c_out, c_state, mx_step
from test_gpu_la import Case, rg  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
CALLS = [("la_decode", 3), ("la_decode", 8), ("la_prefill", 3), ("la_prefill", 65), ("la_prefill", 700)]  # the last in segments


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


@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
def test_many_steps_against_unrounded_states(rg, state):
    """A prompt and sixty steps of one to three tokens, against states that are never rounded. Per element
    the error after a step is what was there, decayed, the step's own arithmetic, and the commit's rounding
    of what it then holds; an output is off by the state's errors at its token, weighted by |q|, and its
    own rounding."""
    B, Hv, D = 2, 2, 64
    steps = [40] + [1, 1, 3] * 20
    T = sum(steps)
    c = Case(B, 1, Hv, T, D, D, state, seed=33, N=B, lens=[T] * B, acc=[T] * B, idx=[1, 0], decay=0.2)
    S = c.S0[c.idx.long()].double().cpu()
    off = torch.zeros_like(S)
    pool, scales = c.pool, c.scales
    at = 0
    for n in steps:
        d = Case.__new__(Case)
        d.__dict__.update(c.__dict__)
        d.q, d.k, d.v, d.g = (x[:, :, at:at + n] for x in (c.q, c.k, c.v, c.g))
        d.lens = d.acc = torch.tensor([n] * B, dtype=torch.int32)
        out = d.call(rg, "la_prefill" if n > 8 else "la_decode", pool=pool, scales=scales)[0].double().cpu()
        q, k, v, g = (x.double().cpu() for x in (d.q, d.k, d.v, d.g))
        A = S.abs() + off
        for t in range(n):
            keep = torch.exp(g[:, :, t])[..., None, None]
            term = k[:, :, t, :, None] * v[:, :, t, None, :]
            S, A, off = keep * S + term, keep * A + term.abs(), keep * off
            qt = (q[:, :, t] * c.scale).expand(B, Hv, D)[..., None]
            ref, bound = (qt * S).sum(2), (qt.abs() * (off + c_out(n, D) * A)).sum(2)
            over = (out[:, :, t] - ref).abs() - bound - BF16_HALF * (ref.abs() + bound)
            assert over.max() <= 0, f"{state} token {at + t}: out off by {over.max():.3g} more than its bound"
        off = off + c_state(n) * A
        if state == "bf16":
            off = off + BF16_HALF * (S.abs() + off)
        elif state == "i8":
            off = off + mx_step(S.abs() + off) / 2
        got = c.values(pool, scales)[c.idx.long()].double().cpu()
        over = (got - S).abs() - off
        assert over.max() <= 0, f"{state} after token {at + n}: state off by {over.max():.3g} more than its bound"
        at += n
    assert at == T
