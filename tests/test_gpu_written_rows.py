"""Every row of an output is written, whatever the buffer held before: entries without a slot that have lengths and
counts, empty ones, short ones; each form of the convolution, rotary positions, the state space scan, linear attention
and the gated delta rule."""
import pytest
import torch

from ssm_form import prefill_form

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def rg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_rgdr_amd as m
    m.library()
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def entries(B, T):
    """Lengths, slots and counts: full, without a slot, empty, short, without a slot again, over-long."""
    lens = [T, T, 0, (T + 1) // 2, T, T + 3]
    idx = [0, -1, 2, 3, B + 9, 5]
    acc = [T, T, T, T // 3, T, 1]
    return [[v[b % 6] if v is not idx else (b if 0 <= v[b % 6] < 6 else v[b % 6]) for b in range(B)] for v in (lens, idx, acc)]


def both(make, shape, dtype, valid):
    """The call's output into buffers of NaN and of ones: the same bits, and +0.0 where `valid` [B, T] is not."""
    outs = []
    for value in (float("nan"), 1.0):
        outs.append(make(torch.full(shape, value, dtype=dtype, device="cuda")))
    bits = [o.view(torch.int16 if dtype != torch.float32 else torch.int32) for o in outs]
    assert torch.equal(*bits)
    assert torch.isfinite(outs[0]).all()
    assert not bits[0][~valid].any()
    return outs[0]


def valid_rows(lens, idx, T, slots):
    ok = torch.zeros(len(lens), T, dtype=torch.bool, device="cuda")
    for b, (n, s) in enumerate(zip(lens, idx)):
        if 0 <= s < slots:
            ok[b, :max(0, min(n, T))] = True
    return ok


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C", [(6, 1, 72), (6, 8, 264), (6, 77, 72), (12, 200, 4104)])
def test_conv(rg, B, T, C, dtype):
    lens, idx, acc = entries(B, T)
    x = torch.randn(B, T, C, device="cuda").to(TYPES[dtype])
    w, pool = torch.randn(C, 4, device="cuda"), torch.randn(B + 2, 3, C, device="cuda").to(TYPES[dtype])
    both(lambda out: rg.la_conv(x, w, pool.clone(), ints(lens), ints(idx), ints(acc), out=out)[0], (B, T, C), TYPES[dtype],
         valid_rows(lens, idx, T, B + 2))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,R", [(1, 64, 64), (7, 128, 64), (30, 72, 18), (9, 1024, 2), (5, 96, 24), (6, 24, 0)])
def test_rope(rg, T, D, R, dtype, interleaved):
    B = 6
    lens, _, _ = entries(B, T)
    q = torch.randn(B, 3, T, D, device="cuda").to(TYPES[dtype])
    freq = torch.rand(R // 2, device="cuda")
    ok = valid_rows(lens, [0] * B, T, 1)[:, None].expand(B, 3, T)
    for which in (0, 1):
        def make(out):
            return rg.la_rope(q, q, freq, ints([5] * B), interleaved=interleaved, actual_seq_lengths=ints(lens),
                              **{("query_out", "key_out")[which]: out})[which]
        both(make, q.shape, TYPES[dtype], ok)


SCANS = [("ssm_decode", 12, 1, 72, 16, 1), ("ssm_decode", 6, 3, 72, 8, 1), ("ssm_decode", 6, 8, 264, 32, 1),
         ("ssm_prefill", 6, 5, 72, 16, 3), ("ssm_prefill", 6, 300, 264, 16, 1), ("ssm_prefill", 6, 300, 1032, 16, 1),
         ("ssm_prefill", 60, 70, 1032, 16, 1), ("ssm_prefill", 6, 130, 72, 8, 1), ("ssm_prefill", 6, 3000, 72, 16, 1),
         ("ssm_prefill", 6, 3000, 40, 8, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fn,B,T,C,N,G", SCANS)
def test_scan(rg, fn, B, T, C, N, G, dtype):
    lens, idx, acc = entries(B, T)
    r = torch.Generator(device="cuda").manual_seed(T)
    x, dt, z = (torch.randn(B, T, C, generator=r, device="cuda").to(TYPES[dtype]) for _ in range(3))
    Bm, Cm = (torch.randn(B, T, G, N, generator=r, device="cuda").to(TYPES[dtype]) for _ in range(2))
    A = -torch.rand(C, N, generator=r, device="cuda")
    pool = torch.randn(B + 2, C, N, generator=r, device="cuda")
    pools = []

    def make(out):
        pools.append(pool.clone())
        return getattr(rg, fn)(x, dt, A, Bm, Cm, pools[-1], ints(lens), ints(idx), ints(acc), z=z, out=out)[0]
    both(make, (B, T, C), TYPES[dtype], valid_rows(lens, idx, T, B + 2))
    assert torch.equal(*pools)
    rest = [s for s in range(B + 2) if s not in idx]
    assert torch.equal(pools[0][rest], pool[rest])


def test_the_scan_s_forms():
    """The prompts above are of every form."""
    seen = {prefill_form(B, T, C, N, G)[:2] + (prefill_form(B, T, C, N, G)[2] > 1,)
            for fn, B, T, C, N, G in SCANS if fn == "ssm_prefill"}
    assert seen >= {(4, False, False), (4, False, True), (16, False, False), (16, True, False), (8, True, False)}, seen


@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("fn,T,D", [("la_decode", 1, 64), ("la_decode", 5, 128), ("la_prefill", 70, 64),
                                    ("la_prefill", 900, 128)])
def test_linear_attention(rg, fn, T, D, state):
    B = 6
    lens, idx, acc = entries(B, T)
    r = torch.Generator(device="cuda").manual_seed(T)
    q, k = (torch.nn.functional.normalize(torch.randn(B, 2, T, D, generator=r, device="cuda"), dim=-1).bfloat16()
            for _ in range(2))
    v, g = torch.randn(B, 4, T, 96, generator=r, device="cuda").bfloat16(), -torch.rand(B, 4, T, generator=r, device="cuda")
    pool, scales = torch.randn(B + 2, 4, D, 96, generator=r, device="cuda"), None
    if state == "bf16":
        pool = pool.bfloat16()
    if state == "i8":
        pool, scales = rg.la_state_quantize(pool)

    def make(out):
        return getattr(rg, fn)(q, k, v, g, pool.clone(), ints(lens), ints(idx), ints(acc), out=out,
                               state_scales=None if scales is None else scales.clone())[0]
    both(make, v.shape, torch.bfloat16, valid_rows(lens, idx, T, B + 2)[:, None].expand(B, 4, T))


@pytest.mark.parametrize("fn,T,Dk,Dv", [
    ("rgdr_decode", 1, 128, 128), ("rgdr_decode", 1, 64, 512), ("rgdr_decode", 2, 64, 64), ("rgdr_decode", 8, 128, 128),
    ("rgdr_decode", 8, 64, 512), ("rgdr_prefill", 40, 128, 128), ("rgdr_prefill", 40, 64, 256),
    ("rgdr_prefill_ws", 900, 128, 128), ("rgdr_prefill_ws", 900, 64, 256), ("rgdr_prefill_noalloc", 900, 128, 64)])
def test_gated_delta_rule(rg, fn, T, Dk, Dv):
    B = 6
    lens, idx, acc = entries(B, T)
    r = torch.Generator(device="cuda").manual_seed(T)
    q, k = (torch.nn.functional.normalize(torch.randn(B, 2, T, Dk, generator=r, device="cuda"), dim=-1).bfloat16()
            for _ in range(2))
    v = torch.randn(B, 4, T, Dv, generator=r, device="cuda").bfloat16()
    beta = torch.rand(B, 4, T, generator=r, device="cuda").bfloat16()
    g, gk = -torch.rand(B, 4, T, generator=r, device="cuda"), -0.1 * torch.rand(B, 4, T, Dk, generator=r, device="cuda")
    pool = torch.randn(B + 2, 4, Dk, Dv, generator=r, device="cuda").bfloat16()
    if fn in ("rgdr_prefill_ws", "rgdr_prefill_noalloc"):
        assert rg.rgdr_prefill_workspace_size(B, 4, T, Dk, Dv) > 0

    def make(out):
        return getattr(rg, fn)(q, k, v, beta, pool.clone(), ints(lens), ints(idx), g, gk, ints(acc), out=out)[0]
    both(make, v.shape, torch.bfloat16, valid_rows(lens, idx, T, B + 2)[:, None].expand(B, 4, T))
