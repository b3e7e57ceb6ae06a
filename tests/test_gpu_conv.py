"""la_conv against a plain reference in 64 bits (bounds: ssm_util)."""
import pytest
import torch

from ssm_util import TYPES, check, clamp, conv, zero_bits

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def rg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_rgdr_amd as m
    m.library()
    return m


class Case:
    def __init__(self, B, T, C, W, dtype, seed, *, N=None, lens="ragged", acc="ragged", idx=None,
                 act=True, bias=True, pad=0):
        r = torch.Generator().manual_seed(seed)
        self.B, self.T, self.C, self.W, self.act = B, T, C, W, act
        self.N, self.dtype = N or B + 2, TYPES[dtype]
        x = torch.randn(B, T, C + pad, generator=r).to(self.dtype).cuda()
        self.x = x[..., pad:]
        self.w = torch.randn(C, W, generator=r).cuda()
        self.bias = torch.randn(C, generator=r).cuda() if bias else None
        self.pool = torch.randn(self.N, W - 1, C, generator=r).to(self.dtype).cuda()
        if lens == "ragged":
            lens = [T - (b * T) // max(B, 1) if b % 3 else T for b in range(B)]
            lens[-1] = lens[-1] if B < 3 else 0
        if acc == "ragged":
            acc = [max(0, n - b % 4) for b, n in enumerate(lens)]
        self.lens, self.acc = (torch.tensor(v, dtype=torch.int32) for v in (lens, acc))
        self.idx = torch.tensor(idx, dtype=torch.int32) if idx is not None else \
            torch.randperm(self.N, generator=r)[:B].to(torch.int32)

    def call(self, rg, pool=None, **kw):
        out, after = rg.la_conv(self.x, self.w, self.pool if pool is None else pool, self.lens.cuda(),
                                self.idx.cuda(), self.acc.cuda(), bias=self.bias, silu=self.act, **kw)
        torch.cuda.synchronize()
        return out, after

    def reference(self, pool=None):
        return conv(self.x, self.w, self.bias, self.pool if pool is None else pool, self.lens,
                    self.idx, self.acc, self.act)

    def check(self, out, after, ref, tag):
        """Also that every slot which no entry names is as in ref, the reference's pool."""
        check(out, ref[0], ref[1], tag)
        assert torch.equal(after.double().cpu(), ref[2]), f"{tag}: state"
        for b in range(self.B):
            e = clamp(self.lens, self.idx, self.acc, b, self.T, self.N)
            assert zero_bits(out[b, e[0] if e else 0:]), f"{tag}: padded row"


SHAPES = [  # B, T, C, W, pad
    (1, 1, 8, 4, 0), (3, 1, 264, 3, 8), (5, 1, 4104, 2, 0), (2, 2, 16, 4, 16), (4, 3, 72, 3, 0),
    (3, 7, 136, 2, 8), (2, 8, 2056, 4, 0), (3, 9, 40, 4, 0), (2, 15, 8, 3, 8), (1, 16, 64, 2, 0),
    (2, 17, 1032, 4, 8), (3, 77, 24, 4, 0), (2, 130, 520, 3, 0), (1, 1025, 8, 4, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_conv(rg, shape, dtype):
    B, T, C, W, pad = shape
    c = Case(B, T, C, W, dtype, sum(shape), pad=pad, act=T % 2 == 1, bias=B % 2 == 1)
    ref = c.reference()
    c.check(*c.call(rg), ref, f"{shape} {dtype}")


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 5, 8, 40])
def test_lengths_slots_and_counts(rg, T, W):
    """Empty and over-long lengths, counts past the length, slots out of range, every count up to past
    the taps; in place, and into another pool that is left as it was elsewhere."""
    lens = [T, 0, T + 5, -2, 1, T, T, (T + 1) // 2, T, T]
    acc = [T + 9, 0, 1, 3, 1, -1, T, 0, 2, 3]
    idx = [4, 8, 0, 2, 7, 1, -1, 12, 3, 6]
    c = Case(10, T, 48, W, "bf16", 5, N=12, lens=lens, acc=acc, idx=idx)
    ref = c.reference()
    new = torch.full_like(c.pool, 7.0)
    keep = c.pool.clone()
    out, after = c.call(rg, state_out=new)
    assert after is new and torch.equal(c.pool, keep)
    want = torch.full_like(ref[2], 7.0)
    for b in range(c.B):
        if clamp(c.lens, c.idx, c.acc, b, T, c.N):
            want[idx[b]] = ref[2][idx[b]]
    c.check(out, after, (ref[0], ref[1], want), "apart")
    c.check(*c.call(rg), ref, "in place")


@pytest.mark.parametrize("T", [1, 6, 30])
def test_what_is_not_read(rg, T):
    """NaN in padding, in slots that are not named and behind an entry without a slot does not show; a
    rejected token's stays out of the slot."""
    c = Case(4, T, 64, 4, "bf16", 9, N=6, lens=[T, T // 2, 0, T], acc=[T - 1, T // 2, 0, T],
             idx=[1, 3, 0, 9])
    for b, n in enumerate([T, T // 2, 0, 0]):
        c.x[b, n:] = NAN
    c.pool[[2, 4, 5]] = NAN
    ref = c.reference(torch.nan_to_num(c.pool))
    c.x[0, T - 1] = NAN
    out, after = c.call(rg)
    assert torch.isnan(out[0, T - 1]).all()
    out[0, T - 1] = ref[0][0, T - 1].to(out.dtype)
    check(out, ref[0], ref[1], "out")
    for s in (0, 1, 3):
        assert torch.equal(after[s].double().cpu(), ref[2][s])


def test_no_accepted_token_leaves_the_slot(rg):
    c = Case(2, 4, 64, 4, "f32", 10, lens=[4, 0], acc=[0, 0])
    keep = c.pool.clone()
    c.call(rg)
    assert torch.equal(c.pool, keep)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_parts_equal_the_whole(rg, dtype):
    """A prompt in one call, and as parts of 1 to 40 tokens on the slot."""
    c = Case(2, 100, 72, 4, dtype, 11, lens=[100, 100], acc=[100, 100])
    pool = c.pool.clone()
    whole, after = c.call(rg)
    got, t = [], 0
    for n in (1, 1, 2, 3, 8, 40, 45):
        got.append(rg.la_conv(c.x[:, t:t + n], c.w, pool, ssm_state_indices=c.idx.cuda(),
                              bias=c.bias)[0])
        t += n
    assert torch.equal(torch.cat(got, 1), whole) and torch.equal(pool, after)


def test_strides_and_given_out(rg):
    c = Case(3, 20, 64, 4, "bf16", 12)
    ref = c.reference()
    wide = torch.full((20, 3, 200), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide[..., 64:128].transpose(0, 1)
    x = torch.empty(20, 3, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    x.copy_(c.x)
    c.x = x
    got, after = c.call(rg, out=out)
    assert got.data_ptr() == out.data_ptr()
    c.check(out, after, ref, "strided")
    assert torch.all(wide[..., :64] == 5) and torch.all(wide[..., 128:] == 5)
    # one input for all entries
    x = torch.randn(1, 20, 64, device="cuda").bfloat16()
    a = rg.la_conv(x.expand(3, 20, 64), c.w, c.pool.clone())[0]
    b = rg.la_conv(x.repeat(3, 1, 1), c.w, c.pool.clone())[0]
    assert torch.equal(a, b)


def test_defaults(rg):
    """Without index arrays: all tokens, slot b, all accepted."""
    c = Case(2, 6, 64, 3, "f16", 13, N=3, lens=[6, 6], acc=[6, 6], idx=[0, 1], bias=False)
    ref = c.reference()
    out, after = rg.la_conv(c.x, c.w, c.pool)
    c.check(out, after, ref, "defaults")


@pytest.mark.parametrize("T", [1, 5, 33])
def test_captured_equals_eager(rg, T):
    c = Case(3, T, 136, 4, "bf16", 14)
    first = c.pool.clone()
    lens, idx, acc = c.lens.cuda(), c.idx.cuda(), c.acc.cuda()
    stream = torch.cuda.Stream()
    out = torch.empty_like(c.x)
    rg.la_conv(c.x, c.w, c.pool, lens, idx, acc, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        rg.la_conv(c.x, c.w, c.pool, lens, idx, acc, out=out)
    for k in range(4):
        c.x.copy_(torch.randn(c.x.shape).to(c.x.dtype))
        c.pool.copy_(first)
        want, pool = rg.la_conv(c.x, c.w, first.clone(), lens, idx, acc)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c.pool, pool), k


def test_other_stream(rg):
    c = Case(2, 50, 512, 4, "bf16", 15)
    want = rg.la_conv(c.x, c.w, c.pool.clone(), bias=c.bias)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = rg.la_conv(c.x, c.w, c.pool, bias=c.bias, stream=s)[0]
    s.synchronize()
    assert torch.equal(out, want)


def test_large_offsets(rg):
    """Rows past 2^31 elements from the first."""
    x = torch.zeros(2, 5, 64, dtype=torch.bfloat16, device="cuda")
    far = torch.empty(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    view = far.as_strided((2, 5, 64), (2 ** 31, 64, 1))
    x.copy_(torch.randn(2, 5, 64))
    view.copy_(x)
    w = torch.randn(64, 4, device="cuda")
    pool = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    out = far.as_strided((2, 5, 64), (2 ** 31, 64, 1), 4096)
    want = rg.la_conv(x, w, pool.clone())[0]
    rg.la_conv(view, w, pool, out=out)
    assert torch.equal(out, want)


def test_index_arrays_are_validated(rg, monkeypatch):
    c = Case(2, 4, 64, 4, "bf16", 16, N=4)
    monkeypatch.setattr(rg, "VALIDATE", True)
    rg.la_conv(c.x, c.w, c.pool)
    with pytest.raises(RuntimeError, match="index arrays"):
        rg.la_conv(c.x, c.w, c.pool, ssm_state_indices=torch.tensor([1, 1], dtype=torch.int32).cuda())


def test_refusals_on_the_device(rg):
    c = Case(2, 4, 64, 4, "bf16", 17)
    x, w, pool = c.x, c.w, c.pool
    for call in (lambda: rg.la_conv(x.double(), w, pool), lambda: rg.la_conv(x, w.bfloat16(), pool),
                 lambda: rg.la_conv(x, w[:, :1].contiguous(), pool[:, :0]),
                 lambda: rg.la_conv(x, w, pool.float()), lambda: rg.la_conv(x, w, pool[:, :2]),
                 lambda: rg.la_conv(x.transpose(1, 2), w, pool), lambda: rg.la_conv(x[..., 1:33], w[:32].contiguous(), pool[..., :32].contiguous()),
                 lambda: rg.la_conv(x, w, pool, bias=w[0]), lambda: rg.la_conv(x, w, pool[:1]),
                 lambda: rg.la_conv(x, w, pool, out=x), lambda: rg.la_conv(x, w, pool, out=x[:1]),
                 lambda: rg.la_conv(x, w, pool, torch.tensor([1, 2]).cuda()),
                 lambda: rg.la_conv(x, w, pool, torch.tensor([1], dtype=torch.int32).cuda()),
                 lambda: rg.la_conv(x, w, pool, state_out=pool[:2]),
                 lambda: rg.la_conv(x[..., :20], w[:20].contiguous(), pool[..., :20].contiguous()),
                 lambda: rg.la_conv(x[0], w, pool), lambda: rg.la_conv(x, w.cpu(), pool)):
        with pytest.raises((RuntimeError, TypeError)):
            call()


def test_empty_batch(rg):
    c = Case(2, 4, 64, 4, "bf16", 18)
    out, _ = rg.la_conv(c.x[:0], c.w, c.pool)
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("dtype,W", [("bf16", 4), ("f16", 3), ("f32", 2)])
def test_many_rows(rg, dtype, W):
    """Enough rows for 16 tokens to each thread; ragged, counts of all sorts, columns of a wider buffer."""
    c = Case(16, 130, 4104, W, dtype, 19, pad=8)
    ref = c.reference()
    new = torch.zeros_like(c.pool)
    out, after = c.call(rg, state_out=new)
    check(out, ref[0], ref[1], "apart")
    for b in range(c.B):
        assert torch.equal(new[int(c.idx[b])].double().cpu(), ref[2][int(c.idx[b])])
    c.check(*c.call(rg), ref, "in place")


def test_longest_prompt(rg):
    x = torch.randn(1, 65536, 16, generator=torch.Generator().manual_seed(20))
    w, pool = torch.randn(16, 4), torch.randn(1, 3, 16)
    want = torch.cat([pool, x], 1).double().unfold(1, 4, 1)
    # five roundings of the terms' magnitudes
    err = 5 * 2.0 ** -24 * (want * w.double()).abs().sum(-1)
    out, after = rg.la_conv(x.cuda(), w.cuda(), pool.cuda(), silu=False)
    check(out, (want * w.double()).sum(-1), err, "65536 tokens")
    assert torch.equal(after.cpu(), x[:, -3:])
