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


def reference_part(c, out, pool, scales, entries, tag):
    """The call's result against the reference at some of its entries (all of them would keep the CPU
    busy for long)."""
    d = Case.__new__(Case)
    d.__dict__.update(c.__dict__)
    d.B = len(entries)
    d.q, d.k, d.v, d.g = (x[entries] for x in (c.q, c.k, c.v, c.g))
    d.lens, d.acc, d.idx = c.lens[entries], c.acc[entries], c.idx[entries]
    d.check(out[entries], pool, scales, tag)


def untouched(c, out, before, sbefore, tag):
    """Rows behind each length are zero and slots that no entry names as they were."""
    late = torch.arange(c.T)[None] >= c.lens.clamp(0, c.T)[:, None]
    assert torch.all(out.transpose(1, 2)[late.cuda()].contiguous().view(torch.int16) == 0), tag
    named = torch.zeros(c.N, dtype=torch.bool)
    named[c.idx.long()] = True
    assert torch.equal(c.pool[~named], before[~named]), tag
    assert sbefore is None or torch.equal(c.scales[~named], sbefore[~named]), tag


def run_large(rg, fn, c, entries, tag):
    before, sbefore = c.pool.clone(), None if c.scales is None else c.scales.clone()
    out = c.call(rg, fn)[0]
    untouched(c, out, before, sbefore, tag)
    reference_part(c, out, c.pool, c.scales, entries, tag)


# la_decode's variants for full batches: one token in tiles of 128 columns from B H_v D_v / 128 = 512 on
# (the first two: just below and at it); 2 to 8 tokens with two blocks of 32 columns for each wave from
# B H_v D_v / 64 = 2048 on, for 16-bit and 8-bit states.
@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("shape", [(15, 16, 32, 1, 64, 128), (16, 16, 32, 1, 64, 128), (16, 8, 32, 1, 128, 128),
                                   (4, 1, 64, 1, 256, 256), (32, 16, 32, 5, 64, 128), (31, 16, 32, 8, 64, 128),
                                   (32, 8, 32, 8, 128, 128), (64, 8, 32, 2, 64, 64), (16, 4, 32, 3, 256, 320)],
                         ids=str)
def test_full_batches(rg, shape, state):
    c = Case(*shape, state, seed=sum(shape))
    run_large(rg, "la_decode", c, [0, 1, 2, shape[0] - 2, shape[0] - 1], f"decode {shape} {state}")


@pytest.mark.parametrize("state", ["bf16", "i8"])
@pytest.mark.parametrize("T", [1, 4])
def test_full_batches_into_another_pool(rg, T, state):
    """The full-batch variants (as above) with a separate output pool: entries of no token, and none
    accepted, are copied."""
    c = Case(32, 16, 32, T, 64, 128, state, seed=T, lens=[T, 0, T, 1] * 8, acc=[T, 0, 0, 1] * 8)
    keep = c.pool.clone()
    kw = {"state_out": torch.zeros_like(c.pool)}
    if state == "i8":
        kw["state_scales_out"] = torch.zeros_like(c.scales)
    out, *new = c.call(rg, "la_decode", **kw)
    assert torch.equal(c.pool, keep)
    reference_part(c, out, new[0], new[1] if state == "i8" else None, [0, 1, 2, 3, 30], f"apart {T} {state}")


# la_prefill in one pass: more than 64 entries (not sorted by length), units of heads on one XCD (8 heads
# and more) and one by one (the second), each with several columns tiles, whole and not, and D_k = 256.
@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("shape", [(70, 1, 2, 70, 64, 64), (3, 1, 4, 90, 128, 256), (4, 2, 4, 90, 128, 256),
                                   (4, 2, 4, 90, 64, 160), (8, 1, 2, 130, 256, 256), (9, 1, 2, 70, 256, 96)],
                         ids=str)
def test_prompts_in_one_pass(rg, shape, state):
    B, _, Hv, T, Dk, Dv = shape
    assert rg.la_prefill_workspace_size(B, Hv, T, Dk, Dv) == 0
    c = Case(*shape, state, seed=sum(shape))
    entries = list(range(B)) if B < 16 else [0, 1, 2, 33, 63, 64, 65, 68, 69]
    run_large(rg, "la_prefill", c, entries, f"prompts {shape} {state}")


# ... and in segments (the workspace says so), the accepted count off and on a segment's border (1024 is
# one of segments of two chunks of 64 tokens, 960 of segments of three).
SEGMENTED = [(1, 1, 2, 1500, 64, 64), (2, 1, 1, 1300, 128, 128), (1, 1, 2, 1500, 256, 64), (1, 1, 1, 1100, 256, 256),
             (1, 2, 2, 1300, 128, 160), (1, 2, 2, 1300, 64, 256)]


@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("accepted", [1037, 1024, 960])
@pytest.mark.parametrize("shape", SEGMENTED, ids=str)
def test_prompts_in_segments(rg, shape, accepted, state):
    B, _, Hv, T, Dk, Dv = shape
    assert rg.la_prefill_workspace_size(B, Hv, T, Dk, Dv) > 0
    c = Case(*shape, state, seed=sum(shape), lens=[T - 13, 1060][:B], acc=[accepted] * B, decay=0.05)
    run_large(rg, "la_prefill", c, list(range(B)), f"segments {shape} {accepted} {state}")


@pytest.mark.parametrize("state", ["bf16", "i8"])
@pytest.mark.parametrize("D", [128, 256])
def test_segments_into_another_pool(rg, D, state):
    """... with a separate output pool, entries without tokens and with none accepted among them."""
    T = 1200
    assert rg.la_prefill_workspace_size(3, 1, T, D, 64) > 0
    c = Case(3, 1, 1, T, D, 64, state, seed=D, lens=[T, 0, T - 1], acc=[700, 0, 0], decay=0.05)
    keep = c.pool.clone()
    kw = {"state_out": torch.zeros_like(c.pool)}
    if state == "i8":
        kw["state_scales_out"] = torch.zeros_like(c.scales)
    out, *new = c.call(rg, "la_prefill", **kw)
    assert torch.equal(c.pool, keep)
    c.check(out, new[0], new[1] if state == "i8" else None, f"segments apart {D} {state}")


# State moves with four units for each thread: from 1024 workgroups of them on, which 32 states of these
# sizes are past (fp32 4096, bf16 2048), and an odd size whose last workgroup is not full.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("n,H,Dk,Dv", [(32, 32, 128, 128), (33, 31, 64, 160)])
def test_many_states_move(rg, n, H, Dk, Dv, dtype):
    from la_util import mx_values
    from test_gpu_la import mx_reference
    r = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n + 3, H, Dk, Dv, generator=r, device="cuda")
    x = (x * torch.exp2(torch.randint(-9, 9, (n + 3, H, Dk, 1), generator=r, device="cuda").float())).to(dtype)
    src = torch.randperm(n + 3, generator=r, device="cuda")[:n].to(torch.int32)
    dst = torch.randperm(n + 1, generator=r, device="cuda")[:n].to(torch.int32)
    codes = torch.full((n + 1, H, Dk, Dv), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((n + 1, H, Dk, Dv // 32), 44, dtype=torch.uint8, device="cuda")
    rg.la_state_quantize(x, codes, scales, src_slots=src, dst_slots=dst)
    left = sorted(set(range(n + 1)) - set(dst.tolist()))[0]
    assert torch.all(codes[left] == 99) and torch.all(scales[left] == 44)
    for i in (0, 1, n - 1):
        want, e = mx_reference(x[src[i]])
        assert torch.equal(codes[dst[i]].cpu().double(), want)
        assert torch.equal(scales[dst[i]].cpu().double(), e)
    back = torch.full_like(x, 7.0)
    rg.la_state_dequantize(codes, scales, back, src_slots=dst, dst_slots=src)
    named = torch.zeros(n + 3, dtype=torch.bool)
    named[src.long().cpu()] = True
    assert torch.all(back[~named.cuda()] == 7)
    for i in range(n):
        assert torch.equal(back[src[i]].double().cpu(), mx_values(codes[dst[i]], scales[dst[i]]))


# The norm with two rows for each group of lanes, from 2048 workgroups' rows on: a workgroup has 256 / 8 rows up
# to 128 bytes each, 256 / 16 up to 256, 256 / 32 up to 512 and 256 / 64 up to 1024 (the last shape's
# fp32 rows are longer).
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("shape", [(2, 32, 513, 128), (3, 7, 3130, 64), (2, 5, 1641, 256), (4, 9, 461, 200),
                                   (1, 3, 2731, 504)], ids=str)
def test_norm_of_many_rows(rg, shape, dtype):
    from test_gpu_la import norm_bound, norm_reference
    B, H, T, D = shape
    r = torch.Generator().manual_seed(D)
    x = torch.randn(B, H, T, D, generator=r).to(dtype).cuda()
    gate = (3 * torch.randn(B, T, H, D, generator=r)).to(dtype).cuda()
    lens = torch.tensor([T, T // 2, 0, T - 1][:B], dtype=torch.int32)
    w = torch.randn(H, D, generator=r)
    y = rg.la_norm_gate(x, w.cuda(), gate, actual_seq_lengths=lens.cuda())
    ref = norm_reference(x, w, gate, 1e-6, False, lens)
    over = (y.double().cpu() - ref).abs() - norm_bound(ref, D, dtype)
    assert over.max() <= 0, f"{shape} {dtype}: off by {over.max():.3g} more than the bound"
