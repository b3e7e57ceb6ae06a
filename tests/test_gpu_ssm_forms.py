"""Each form of ssm_prefill with workgroups that are not full and prompts of several chunks; the form that a shape
takes is asked for, so that a change of the plan cannot drop one unnoticed. Bounds: ssm_util."""
import pytest
import torch

from ssm_form import prefill_form
from test_gpu_ssm import Case, rg  # noqa: F401  (rg is a fixture)

pytestmark = pytest.mark.gpu

FORMS = [  # B, T, C, N, G; lanes for each channel, roles
    ((24, 70, 2376, 16, 3), 4, False),   # groups of 792: 12 workgroups of 64 channels and one of 24
    ((30, 75, 2056, 32, 1), 4, False),
    ((13, 300, 1000, 16, 1), 16, False),  # chunks of 128 tokens, workgroups of 16 channels, the last of 8
    ((6, 290, 1000, 32, 1), 16, False),
    ((10, 200, 1000, 8, 1), 8, False),    # of 64 tokens and 32 channels
    ((3, 300, 536, 16, 1), 16, True),
    ((2, 270, 520, 32, 1), 16, True),
    ((4, 210, 200, 8, 5), 8, True),
    ((20, 75, 2056, 8, 1), 4, False),     # (in fp32 eight lanes)
]


@pytest.mark.parametrize("types", [("bf16", "f32"), ("f32", "bf16")], ids="-".join)
@pytest.mark.parametrize("shape,ways,roles", FORMS, ids=str)
def test_forms(rg, shape, ways, roles, types):  # noqa: F811
    """Full lengths (no count shortens a chunk), then ragged ones with counts within chunks."""
    B, T, C, N, G = shape
    if types[0] == "f32" and (N, ways) == (8, 4):
        ways = 8
    assert prefill_form(*shape, one_pass=True, f32=types[0] == "f32") == (ways, roles, 1, T)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    for lens, acc in (([T] * B, [T] * B), ("ragged", "ragged")):
        c = Case(*shape, *types, seed=sum(shape), lens=lens, acc=acc, slow=0.05)
        before = c.rest(c.pool).clone()
        ref = c.reference()
        out, after = c.call(rg, "ssm_prefill", workspace=none)
        c.check(out, after, ref, f"{shape} {types} {lens}")
        assert torch.equal(c.rest(c.pool), before)


def test_four_lanes_for_few_states(rg):  # noqa: F811
    """N = 8 in four lanes for each channel, several chunks, with more workgroups than the grid could have with
    eight. All entries but four have no slot; inputs are one row for all of them."""
    B, T, G, N = 65536, 45, 129, 8
    C = 40 * G
    assert prefill_form(B, T, C, N, G) == (4, False, 1, T)
    c = Case(4, T, C, N, G, "bf16", "f32", 41, slots=4, lens=[T, T, 33, 7], acc=[T, 40, 33, 0], idx=[2, 0, 1, 3],
             layout="whole", slow=0.1)
    for name in ("x", "dt", "z", "Bm", "Cm"):
        t = getattr(c, name)
        setattr(c, name, t[:1].expand_as(t))
    ref = c.reference()
    at = [0, 4097, 40000, B - 1]
    lens, idx, acc = (torch.full((B,), v, dtype=torch.int32, device="cuda") for v in (T, -1, T))
    lens[at], idx[at], acc[at] = c.lens.cuda(), c.idx.cuda(), c.acc.cuda()
    x, dt, z, Bm, Cm = (t[:1].expand(B, *t.shape[1:]) for t in (c.x, c.dt, c.z, c.Bm, c.Cm))
    out, after = rg.ssm_prefill(x, dt, c.A, Bm, Cm, c.pool, lens, idx, acc, D=c.D, z=z, dt_bias=c.bias)
    c.check(out[at], after, ref, "four lanes, 8 states")
    for b in (1, 4096, 4098, 39999, 65534):
        assert not out[b].any()
