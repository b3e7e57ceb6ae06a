"""la_rope against a plain reference in 64 bits (bounds: ssm_util)."""
import pytest
import torch

from ssm_util import TYPES, check, rope, zero_bits

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def rg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_rgdr_amd as m
    m.library()
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(r, B, H, T, D, dtype, layout):
    if layout == "bhtd":
        return torch.randn(B, H, T, D, generator=r).to(TYPES[dtype]).cuda()
    return torch.randn(B, T, H, D, generator=r).to(TYPES[dtype]).cuda().transpose(1, 2)


SHAPES = [  # B, Hq, Hk, T, D, R
    (1, 1, 1, 1, 8, 8), (1, 16, 16, 1, 128, 128), (2, 3, 1, 1, 64, 32), (3, 2, 2, 5, 72, 18),
    (2, 5, 5, 3, 80, 80), (1, 8, 2, 33, 96, 24), (2, 1, 3, 7, 256, 64), (1, 4, 4, 130, 64, 64),
    (2, 2, 0, 9, 128, 128), (1, 70, 3, 2, 40, 2), (1, 2, 1, 6, 1024, 1024), (2, 2, 1, 4, 24, 0),
    (1, 3, 1, 5, 48, 20),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rope(rg, shape, interleaved, dtype):
    B, Hq, Hk, T, D, R = shape
    r = torch.Generator().manual_seed(sum(shape))
    layout = "bthd" if T % 2 else "bhtd"
    q = rows(r, B, Hq, T, D, dtype, layout)
    k = rows(r, B, Hk, T, D, dtype, layout) if Hk else None
    freq = torch.exp(-8 * torch.rand(R // 2, generator=r)).cuda()
    pos = torch.randint(0, 100000, (B,), generator=r).to(torch.int32).cuda()
    lens = ints([T - b % 2 * (T // 2) for b in range(B)])
    qo, ko = rg.la_rope(q, k, freq, pos, interleaved=interleaved, factor=1.25, actual_seq_lengths=lens)
    assert (ko is None) == (k is None)
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            assert y.is_contiguous() and y.dtype == x.dtype
            check(y, *rope(x, freq, pos, 1.25, interleaved, lens), f"{shape} {dtype}")
            for b in range(B):
                assert zero_bits(y[b, :, int(lens[b]):])
            # what is not turned is copied, to the bit
            n = int(lens[0])
            assert torch.equal(y[0, :, :n, R:], x[0, :, :n, R:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(rg, interleaved):
    """Positions at which a 32-bit angle is off by radians, and negative ones; a position for each
    token, in any order."""
    r = torch.Generator().manual_seed(3)
    q, k = rows(r, 2, 2, 6, 64, "f32", "bthd"), rows(r, 2, 1, 6, 64, "f32", "bthd")
    freq, _ = rg.la_rope_frequencies(64)
    each = ints([[0, 1, 2 ** 31 - 1, 16777217, 999983, -5], [-2 ** 31, 7, 7, 123456789, 3, 2 ** 30 + 1]])
    for pos in (each, ints([2 ** 31 - 1, -2 ** 31]), ints([1234567, 0]), None):
        got = rg.la_rope(q, k, freq, pos, interleaved=interleaved)
        for x, y in zip((q, k), got):
            check(y, *rope(x, freq, pos, 1.0, interleaved, [6, 6]), str(pos))


@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (72, 18)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(rg, D, R, interleaved):
    r = torch.Generator().manual_seed(4)
    both = torch.randn(2, 9, 5 * D, generator=r).bfloat16().cuda()
    q = both[..., :3 * D].unflatten(-1, (3, D)).transpose(1, 2)
    k = both[..., 3 * D:].unflatten(-1, (2, D)).transpose(1, 2)
    freq, _ = rg.la_rope_frequencies(R)
    pos = ints([5, 77])
    want = rg.la_rope(q, k, freq, pos, interleaved=interleaved)
    got = rg.la_rope(q, k, freq, pos, interleaved=interleaved, query_out=q, key_out=k)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    # turned back by the same angles with their signs changed
    q32 = torch.randn(1, 2, 9, D, generator=r).cuda()
    there, _ = rg.la_rope(q32, None, freq, ints([40]), interleaved=interleaved)
    back, _ = rg.la_rope(there, None, -freq, ints([40]), interleaved=interleaved)
    # |u| + |v| < 8, and at most sqrt(2) times that after a turn: (1 + 2 sqrt(2)) bounds of one turn,
    # the first one's also turned
    assert (back - q32).abs().max() <= 4 * 8 * (2.0 ** -21 + 2.0 ** -24)


def test_scores_go_by_distance(rg):
    """q . k after the turn is that of the distance alone, in both layouts of the pairs."""
    r = torch.Generator().manual_seed(5)
    q, k = rows(r, 1, 1, 1, 64, "f32", "bhtd"), rows(r, 1, 1, 1, 64, "f32", "bhtd")
    freq, _ = rg.la_rope_frequencies(64)
    for interleaved in (False, True):
        s = []
        for at in (0, 11, 5000, 1000003):
            a, _ = rg.la_rope(q, None, freq, ints([at + 9]), interleaved=interleaved)
            b, _ = rg.la_rope(k, None, freq, ints([at]), interleaved=interleaved)
            s.append((a.double() * b.double()).sum())
        # each of 64 columns off by (|u| + |v|) 2^-21, against the other's magnitude
        bound = 4 * 2.0 ** -21 * (q.abs().sum() * k.abs().max() + k.abs().sum() * q.abs().max())
        assert max(abs(x - s[0]) for x in s) <= bound


def test_padding_is_not_read(rg):
    r = torch.Generator().manual_seed(6)
    for interleaved in (False, True):
        for R in (64, 32, 18):
            q, k = rows(r, 3, 2, 8, 64, "bf16", "bthd"), rows(r, 3, 1, 8, 64, "bf16", "bthd")
            lens = [8, 3, 0]
            for b, n in enumerate(lens):
                q[b, :, n:], k[b, :, n:] = NAN, float("inf")
            freq, _ = rg.la_rope_frequencies(R)
            for lens in (ints([8, 3, 0]), ints([99, 3, -4])):
                for y in rg.la_rope(q, k, freq, ints([1, 2, 3]), interleaved=interleaved,
                                    actual_seq_lengths=lens):
                    assert torch.isfinite(y).all()
                    assert zero_bits(y[1, :, 3:]) and zero_bits(y[2])


def test_values_that_are_not_finite(rg):
    """They show in their own pair and nowhere else, and pass where columns are copied."""
    x = torch.ones(1, 1, 1, 32, device="cuda")
    x[..., 3], x[..., 20], x[..., 31] = NAN, float("inf"), -float("inf")
    freq, _ = rg.la_rope_frequencies(16)
    for interleaved in (False, True):
        y, _ = rg.la_rope(x, None, freq, ints([3]), interleaved=interleaved)
        bad = {2, 3} if interleaved else {3, 11}
        assert {int(i) for i in torch.isnan(y[0, 0, 0]).nonzero()} == bad
        assert y[0, 0, 0, 20] == float("inf") and y[0, 0, 0, 31] == -float("inf")


def test_frequencies(rg):
    freq, factor = rg.la_rope_frequencies(64, 10000.0, device="cpu")
    i = torch.arange(32, dtype=torch.float64)
    plain = 10000.0 ** (-i / 32)
    assert factor == 1.0 and torch.equal(freq, plain.float())
    assert torch.equal(rg.la_rope_frequencies(64, scaling="linear", scale=4.0, device="cpu")[0], (plain / 4).float())
    based = rg.la_rope_frequencies(64, scaling="base", scale=4.0, device="cpu")[0]
    assert based[0] == 1.0 and abs(float(based[-1]) / float(plain[-1]) - 0.25) < 1e-6
    blend, factor = rg.la_rope_frequencies(64, scaling="blend", scale=4.0, original_length=4096, device="cpu")
    assert blend[0] == 1.0 and abs(float(blend[-1]) / float(plain[-1]) - 0.25) < 1e-6
    ratio = blend.double() / plain
    assert torch.all(ratio[1:] <= ratio[:-1] + 1e-6) and 1.1 < factor < 1.2
    for kw in (dict(scaling="yes"), dict(scaling="blend"), dict(scale=0.5), dict(base=1.0)):
        with pytest.raises(RuntimeError):
            rg.la_rope_frequencies(64, **{"device": "cpu", **kw})
    for odd in (0, 7, -2):
        with pytest.raises(RuntimeError):
            rg.la_rope_frequencies(odd, device="cpu")


@pytest.mark.parametrize("T", [1, 40])
def test_captured_equals_eager(rg, T):
    r = torch.Generator().manual_seed(8)
    q, k = rows(r, 2, 4, T, 64, "bf16", "bthd"), rows(r, 2, 2, T, 64, "bf16", "bthd")
    freq, _ = rg.la_rope_frequencies(64)
    pos = ints([3, 9])
    qo, ko = rg.la_rope(q, k, freq, pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        rg.la_rope(q, k, freq, pos, query_out=qo, key_out=ko)
    for n in range(4):
        pos.copy_(ints([n * 1000, 5]))
        q.copy_(torch.randn(q.shape).bfloat16())
        want = rg.la_rope(q, k, freq, pos)
        qo.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]), n


def test_other_stream(rg):
    q = torch.randn(2, 4, 300, 64, device="cuda").bfloat16()
    freq, _ = rg.la_rope_frequencies(64)
    want = rg.la_rope(q, q, freq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = rg.la_rope(q, q, freq, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals_on_the_device(rg):
    q = torch.randn(2, 2, 4, 64, device="cuda").bfloat16()
    freq, _ = rg.la_rope_frequencies(64)
    pos = ints([0, 0])
    for call in (lambda: rg.la_rope(q.double(), None, freq), lambda: rg.la_rope(q, q.float(), freq),
                 lambda: rg.la_rope(q, q[:, :, :3], freq), lambda: rg.la_rope(q, q[..., :32], freq),
                 lambda: rg.la_rope(q, None, freq.double()), lambda: rg.la_rope(q, None, torch.ones(33, device="cuda")),
                 lambda: rg.la_rope(q, None, freq, pos.long()), lambda: rg.la_rope(q, None, freq, pos[:1]),
                 lambda: rg.la_rope(q, None, freq, pos, key_out=q), lambda: rg.la_rope(q, None, freq.cpu()),
                 lambda: rg.la_rope(q, None, freq, pos, query_out=q[:, :1]),
                 lambda: rg.la_rope(q, None, freq, pos, query_out=q.as_strided(q.shape, (512, 0, 64, 1))),
                 lambda: rg.la_rope(q, None, freq, pos, query_out=q.as_strided(q.shape, (512, 64, 128, 1))),
                 lambda: rg.la_rope(q[..., 1:33], None, freq[:16].contiguous()), lambda: rg.la_rope(q.transpose(2, 3), None, freq[:1]),
                 lambda: rg.la_rope(q[0], None, freq), lambda: rg.la_rope(q, None, freq, pos, actual_seq_lengths=pos[:1])):
        with pytest.raises((RuntimeError, TypeError)):
            call()


@pytest.mark.parametrize("shape", [(0, 2, 4, 64), (2, 0, 4, 64), (2, 2, 0, 64)])
def test_empty_calls(rg, shape):
    q = torch.empty(shape, device="cuda")
    freq, _ = rg.la_rope_frequencies(64)
    out, none = rg.la_rope(q, None, freq)
    assert out.shape == q.shape and none is None
