"""Linear attention, state moves and the norm at sizes that choose kernel variants of their own, and at
the sizes' limits (references and bounds: la_util)."""
import pytest
import torch

from test_gpu_la import Case, rg  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_heads_past_whole_rounds_of_the_launch(rg):
    """One query/key head with 2^21 value heads: within the sizes that the header allows, and more
    workgroups than a launch takes if heads are kept together in whole rounds over the XCDs. From
    zero states out is bf16(scale (q.k) v) and the state k v^T."""
    Hv, Dk, Dv = 1 << 21, 64, 32
    r = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.randn(1, 1, 1, Dk, generator=r, device="cuda").sign().bfloat16() for _ in range(2))
    v = torch.randn(1, Hv, 1, Dv, generator=r, device="cuda").bfloat16()
    pool = torch.zeros(1, Hv, Dk, Dv, dtype=torch.bfloat16, device="cuda")
    out, _ = rg.la_prefill(q, k, v, torch.zeros(Hv, device="cuda"), pool, scale=0.25)
    # signs: q.k is a whole number below 64, its product with v and 1/4 is exact in fp32
    want = (0.25 * (q.float() * k.float()).sum() * v.float()).bfloat16()
    assert torch.equal(out, want)
    for h in range(0, Hv, 1 << 18):
        part = slice(h, h + (1 << 18))
        assert torch.equal(pool[0, part], k[0, 0, 0, :, None] * v[0, part, 0, None, :])
