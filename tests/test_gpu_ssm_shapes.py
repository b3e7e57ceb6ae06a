"""Sizes of the state space scan that choose variants of their own (lanes for each channel, segments, tokens by
way of LDS), and far offsets; bounds: ssm_util."""
import pytest
import torch

from test_gpu_ssm import Case, rg  # noqa: F401  (rg is a fixture)

pytestmark = pytest.mark.gpu

MANY = [  # B, T, C, N, G: enough channels for four lanes for each
    (64, 37, 512, 16, 1), (96, 20, 264, 16, 3), (64, 33, 512, 8, 8), (70, 31, 448, 32, 7), (40, 66, 1024, 16, 16),
]


@pytest.mark.parametrize("types", [("bf16", "f32"), ("f16", "bf16"), ("f32", "f32")], ids="-".join)
@pytest.mark.parametrize("shape", MANY, ids=str)
def test_many_channels(rg, shape, types):  # noqa: F811
    c = Case(*shape, *types, seed=sum(shape), slow=0.1)
    assert rg.ssm_prefill_workspace_size(*shape) == 0
    before = c.rest(c.pool).clone()
    ref = c.reference()
    out, after = c.call(rg, "ssm_prefill")
    c.check(out, after, ref, str(shape))
    assert torch.equal(c.rest(c.pool), before)


SEGMENTS = [(1, 900, 64, 8, 1), (2, 1100, 24, 32, 1), (1, 1300, 80, 16, 10), (3, 2100, 8, 16, 1)]


@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SEGMENTS, ids=str)
def test_segments(rg, shape, dtype, state):  # noqa: F811
    """In segments, and (without a workspace) in one pass; counts that end within a segment, at its end and
    before the first token; a pool apart."""
    B, T = shape[:2]
    assert rg.ssm_prefill_workspace_size(*shape) > 0
    for lens, acc in (([T, T - 1, 70][:B], [T - 77, 64, 0][:B]), ([T - 65, 1, 0][:B], [128, 1, 0][:B]), ([T] * B, [T] * B)):
        c = Case(*shape, dtype, state, seed=sum(shape), lens=lens, acc=acc, slow=0.02)
        ref = c.reference()
        new = torch.zeros_like(c.pool)
        for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):
            out, after = c.call(rg, "ssm_prefill", state_out=new, workspace=ws)
            c.check(out, after, ref, f"{shape} {lens} {acc} {ws}")
        out, after = c.call(rg, "ssm_prefill")
        c.check(out, after, ref, f"{shape} {lens} {acc} in place")


TOKENS = [  # by way of LDS from 5 tokens, or 3 in large calls, where a group fills a workgroup
    (2, 5, 128, 16, 1), (3, 8, 264, 16, 1), (2, 6, 1024, 8, 2), (5, 7, 96, 32, 1), (2, 8, 520, 16, 1),
    (160, 3, 1024, 16, 1), (160, 4, 1032, 16, 1), (300, 2, 64, 16, 1), (33, 1, 72, 32, 1),
]


@pytest.mark.parametrize("types", [("bf16", "f32"), ("f16", "bf16"), ("f32", "bf16")], ids="-".join)
@pytest.mark.parametrize("shape", TOKENS, ids=str)
def test_few_tokens(rg, shape, types):  # noqa: F811
    c = Case(*shape, *types, seed=sum(shape))
    before = c.rest(c.pool).clone()
    ref = c.reference()
    new = torch.zeros_like(c.pool)
    out, after = c.call(rg, "ssm_decode", state_out=new)
    c.check(out, after, ref, f"{shape} apart")
    out, after = c.call(rg, "ssm_decode")
    c.check(out, after, ref, str(shape))
    assert torch.equal(c.rest(c.pool), before)


@pytest.mark.parametrize("fn,T", [("ssm_decode", 1), ("ssm_decode", 8), ("ssm_prefill", 40), ("ssm_prefill", 500)])
def test_far_slots(rg, fn, T):  # noqa: F811
    """A slot past 2^32 bytes of the pool."""
    c = Case(2, T, 64, 16, 1, "bf16", "f32", 20, slots=4, lens=[T] * 2, acc=[T] * 2, idx=[0, 3], slow=0.1)
    ref = c.reference()
    slots = 2 ** 30 // (64 * 16) + 5
    pool = torch.empty(slots, 64, 16, device="cuda")
    c.idx, c.slots = torch.tensor([0, slots - 1], dtype=torch.int32), slots
    pool[0], pool[-1] = c.pool[0], c.pool[3]
    out, after = c.call(rg, fn, pool=pool)
    c.check(out, after, ref, fn)


def test_token_strides(rg):  # noqa: F811
    """Tokens as far apart as is allowed (2^25 bytes), and one element further: refused."""
    c = Case(1, 70, 64, 16, 1, "bf16", "f32", 21, lens=[70], acc=[70], layout="whole", slow=0.1)
    ref = c.reference()
    step = 2 ** 24
    far = torch.empty(70 * step, dtype=torch.bfloat16, device="cuda")
    view = far.as_strided((1, 70, 64), (8, step, 1))
    view.copy_(c.x)
    c.x = view
    out, after = c.call(rg, "ssm_prefill")
    c.check(out, after, ref, "far tokens")
    c.x = far.as_strided((1, 2, 64), (8, step + 8, 1))
    c.dt, c.z, c.Bm, c.Cm = c.dt[:, :2], c.z[:, :2], c.Bm[:, :2], c.Cm[:, :2]
    for fn in ("ssm_decode", "ssm_prefill"):
        with pytest.raises(RuntimeError, match="SHAPE"):
            c.call(rg, fn)
    c.x, c.dt, c.z, c.Bm, c.Cm = (t[:, :1] for t in (c.x, c.dt, c.z, c.Bm, c.Cm))
    c.lens, c.acc, c.T = c.lens * 0 + 1, c.acc * 0 + 1, 1
    ref = c.reference()
    c.check(*c.call(rg, "ssm_prefill"), ref, "one token at any stride")


def test_groups_of_channels(rg):  # noqa: F811
    """Groups that do not fill a wave or a workgroup, against one group each."""
    c = Case(2, 50, 136, 16, 17, "bf16", "f32", 22, lens=[50] * 2, acc=[50] * 2, layout="whole")
    pool = c.pool.clone()
    out, after = c.call(rg, "ssm_prefill")
    for g in range(17):
        s = slice(8 * g, 8 * g + 8)
        x, dt, z, Bm, Cm = (t.contiguous() for t in (c.x[..., s], c.dt[..., s], c.z[..., s], c.Bm[:, :, g:g + 1], c.Cm[:, :, g:g + 1]))
        one = pool[:, s].contiguous()
        o, _ = rg.ssm_prefill(x, dt, c.A[s].contiguous(), Bm, Cm, one, ssm_state_indices=c.idx.cuda(), D=c.D[s].contiguous(),
                              z=z, dt_bias=c.bias[s].contiguous())
        assert torch.equal(o, out[..., s])
        named = c.idx.long()
        assert torch.equal(one[named], after[named][:, s])


def test_longest_prompt(rg):  # noqa: F811
    c = Case(1, 65536, 8, 8, 1, "bf16", "f32", 23, lens=[65536], acc=[65536], slow=0.02)
    ref = c.reference()
    for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):
        out, after = c.call(rg, "ssm_prefill", pool=c.pool.clone(), workspace=ws)
        c.check(out, after, ref, "65536 tokens")


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("shape", [(1, 1000, 64, 16, 1), (2, 200, 128, 16, 2), (64, 37, 512, 16, 1), (1, 900, 64, 8, 1)], ids=str)
def test_rejected_values_that_are_not_finite(rg, shape, value):  # noqa: F811
    """In segments, with roles, with four lanes: the values of a rejected token stay out of the state, of the
    outputs before it and, but for B, out of other channels."""
    B, T, C, N, G = shape
    t0 = T // 3 * 2
    c = Case(*shape, "bf16", "f32", 24, lens=[T] * B, acc=[t0] * B, slow=0.05)
    want, after = c.call(rg, "ssm_prefill", pool=c.pool.clone())
    c.x[:, t0, 3] = value
    c.dt[:, t0 + 1, 5] = value
    c.z[:, t0 + 2, 6] = value
    keep = c.pool.clone()
    out, got = c.call(rg, "ssm_prefill")
    assert torch.equal(got, after)
    others = [i for i in range(C) if i not in (3, 5, 6)]
    assert torch.equal(out[..., others], want[..., others])
    assert torch.equal(out[:, :t0], want[:, :t0]) and not torch.isfinite(out[:, t0, 3]).any()
    assert torch.equal(out[:, t0 + 3:, 6], want[:, t0 + 3:, 6])
    c.Bm[:, t0] = value
    out, got = c.call(rg, "ssm_prefill", pool=keep)
    assert torch.equal(got, after) and torch.equal(out[:, :t0], want[:, :t0])
