"""Linear attention with a decay for each head (la_decode, la_prefill), 8-bit state pools and the
gated norm, against token-by-token references in 64 bits (bounds: la_util)."""
import numpy as np
import pytest
import torch

from la_util import attention, check_out, check_state, mx_step, mx_values

pytestmark = pytest.mark.gpu
NAN = float("nan")
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8}


@pytest.fixture(scope="module")
def rg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_rgdr_amd as m
    m.library()
    return m


class Case:
    """Inputs of one call, made on the CPU from a seed."""

    def __init__(self, B, Hq, Hv, T, Dk, Dv, state, seed, *, N=None, lens="ragged", acc="ragged",
                 decay=0.3, layout="bthd", idx=None, size=0.3):
        r = torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.Hv, self.T, self.Dk, self.Dv = B, Hq, Hv, T, Dk, Dv
        self.N, self.state = N or B + 2, state

        def rows(H, D, unit):
            x = torch.randn(B, T, H, D, generator=r)
            if unit:
                x = x / x.norm(dim=-1, keepdim=True)
            x = x.to(torch.bfloat16).cuda()
            return x.transpose(1, 2) if layout == "bthd" else x.transpose(1, 2).contiguous()

        self.q, self.k, self.v = rows(Hq, Dk, True), rows(Hq, Dk, True), rows(Hv, Dv, False)
        g = -decay * torch.rand(B, T, Hv, generator=r) ** 2
        self.g = g.cuda().transpose(1, 2)
        self.scale = Dk ** -0.5
        if lens == "ragged":
            lens = [T - (b * T) // max(B, 1) if b % 3 else T for b in range(B)]
            lens[-1] = lens[-1] if B < 3 else 0
        if acc == "ragged":
            acc = [max(0, n - b % 4) for b, n in enumerate(lens)]
        self.lens, self.acc = (torch.tensor(x, dtype=torch.int32) for x in (lens, acc))
        self.idx = torch.tensor(idx, dtype=torch.int32) if idx is not None else \
            torch.randperm(self.N, generator=r)[:B].to(torch.int32)
        S = torch.randn(self.N, Hv, Dk, Dv, generator=r) * size
        self.scales = None
        if state == "i8":
            self.scales = torch.randint(116, 124, (self.N, Hv, Dk, Dv // 32), generator=r,
                                        dtype=torch.uint8).cuda()
            self.pool = torch.randint(-127, 128, S.shape, generator=r, dtype=torch.int8).cuda()
            self.S0 = mx_values(self.pool, self.scales)
        else:
            self.pool = S.to(DT[state]).cuda()
            self.S0 = self.pool.double().cpu()

    def call(self, rg, fn, pool=None, scales=None, **kw):
        if self.scales is not None:
            kw["state_scales"] = self.scales if scales is None else scales
        r = getattr(rg, fn)(self.q, self.k, self.v, self.g, self.pool if pool is None else pool,
                            self.lens.cuda(), self.idx.cuda(), self.acc.cuda(), self.scale, **kw)
        torch.cuda.synchronize()
        return r

    def values(self, pool, scales):
        return pool if scales is None else mx_values(pool, scales)

    def check(self, out, pool, scales, tag):
        """out and the pool after a call in place (or into a copy of the pool)."""
        ref, states, mag, smags = attention(self.q, self.k, self.v, self.g, self.S0, self.lens,
                                            self.idx, self.acc, self.scale)
        check_out(out, ref, mag, self.T, self.Dk, tag)
        for b in range(self.B):
            ok = states[b] is not None
            for t in range(min(max(int(self.lens[b]), 0), self.T) if ok else 0, self.T):
                assert torch.all(out[b, :, t].contiguous().view(torch.int16) == 0), f"{tag}: padded row"
            if ok:
                s = int(self.idx[b])
                got = self.values(pool[s:s + 1], None if scales is None else scales[s:s + 1])[0]
                check_state(got, states[b], smags[b], self.T, DT[self.state], f"{tag} entry {b}")


def rest(case, pool):
    """Slots that no entry names."""
    named = set(int(i) for i in case.idx)
    keep = [s for s in range(case.N) if s not in named]
    return pool[keep]


SHAPES = [  # B, Hq, Hv, T, Dk, Dv
    (1, 1, 1, 1, 64, 32), (1, 2, 4, 1, 128, 128), (3, 1, 2, 2, 64, 96), (4, 2, 2, 3, 128, 64),
    (5, 3, 6, 5, 64, 256), (2, 1, 3, 7, 256, 160), (3, 2, 4, 8, 128, 128), (2, 2, 2, 8, 256, 32),
    (9, 4, 8, 1, 64, 512), (3, 5, 5, 4, 128, 544),
]
PROMPTS = [
    (1, 1, 1, 1, 64, 32), (2, 1, 2, 15, 64, 64), (2, 2, 2, 16, 128, 128), (1, 1, 1, 31, 64, 96),
    (1, 1, 1, 32, 256, 32), (3, 1, 3, 33, 128, 160), (2, 2, 4, 63, 64, 128), (2, 1, 1, 64, 128, 64),
    (3, 1, 2, 65, 128, 128), (4, 2, 4, 127, 64, 32), (2, 1, 2, 129, 256, 192), (1, 2, 2, 300, 128, 128),
    (1, 1, 1, 577, 64, 544),
]


@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("fn,shape", [("la_decode", s) for s in SHAPES] +
                         [("la_prefill", s) for s in PROMPTS], ids=str)
def test_attention(rg, fn, shape, state):
    c = Case(*shape, state, seed=sum(shape), layout="bthd" if shape[0] % 2 else "bhtd")
    before = rest(c, c.pool).clone()
    sbefore = None if c.scales is None else rest(c, c.scales).clone()
    out = c.call(rg, fn)[0]
    c.check(out, c.pool, c.scales, f"{fn} {shape} {state}")
    assert torch.equal(rest(c, c.pool), before)
    if sbefore is not None:
        assert torch.equal(rest(c, c.scales), sbefore)


@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("fn,T", [("la_decode", 1), ("la_decode", 6), ("la_prefill", 70), ("la_prefill", 400)])
def test_lengths_slots_and_counts(rg, fn, T, state):
    """Empty and over-long lengths, counts past the length, slots out of range, and a pool that
    stays as it was beside a separate output pool."""
    c = Case(8, 2, 4, T, 128, 128, state, seed=77, N=9,
             lens=[T, 0, T + 5, -2, 1, T, T, (T + 1) // 2], acc=[T + 9, 0, 1, 3, 1, -1, T, 0],
             idx=[4, 8, 0, 2, 7, 1, -1, 9])
    keep, skeep = c.pool.clone(), None if c.scales is None else c.scales.clone()
    new = torch.zeros_like(c.pool)
    if c.scales is None:
        out, got = c.call(rg, fn, state_out=new)
        snew = None
    else:
        out, got, snew = c.call(rg, fn, state_out=new, state_scales_out=torch.zeros_like(c.scales))
    assert got is new and torch.equal(c.pool, keep)
    assert skeep is None or torch.equal(c.scales, skeep)
    c.check(out, new, snew, f"{fn} T={T} {state}")
    assert torch.all(rest(c, new) == 0)
    assert torch.all(out[6:].contiguous().view(torch.int16) == 0)


@pytest.mark.parametrize("fn,T", [("la_decode", 1), ("la_decode", 4), ("la_prefill", 40)])
def test_codes_in_place_scales_apart(rg, fn, T):
    """Scales into an array of their own while the codes stay: entries without tokens, and with
    none accepted, get theirs too."""
    c = Case(4, 1, 2, T, 64, 64, "i8", seed=15, lens=[T, 0, T, T], acc=[T, 0, 0, T])
    out, pool, scales = c.call(rg, fn, state_out=c.pool, state_scales_out=torch.zeros_like(c.scales))
    c.check(out, pool, scales, f"{fn} scales apart")


@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("fn,T", [("la_decode", 1), ("la_decode", 4), ("la_prefill", 40)])
def test_no_token_on_a_state_that_is_not_finite(rg, fn, T, state):
    """Outputs of an entry without tokens are zero whatever its state holds, and that state is
    copied."""
    c = Case(2, 1, 2, T, 64, 64, state, seed=16, lens=[0, T], acc=[0, T], idx=[1, 0], N=2)
    kw = {"state_out": torch.zeros_like(c.pool)}
    if state == "i8":
        c.scales[1] = 255
        kw["state_scales_out"] = torch.zeros_like(c.scales)
    else:
        c.pool[1, 0], c.pool[1, 1] = NAN, float("inf")
    out, *new = c.call(rg, fn, **kw)
    assert torch.all(out[0].contiguous().view(torch.int16) == 0)
    got = c.values(new[0], new[1] if state == "i8" else None)[1]
    want = c.values(c.pool, c.scales)[1]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(want))


@pytest.mark.parametrize("state", ["bf16", "i8"])
@pytest.mark.parametrize("fn,T", [("la_decode", 1), ("la_decode", 4), ("la_prefill", 40), ("la_prefill", 700)])
def test_no_accepted_token_leaves_the_slot(rg, fn, T, state):
    """In place, an entry whose tokens are all rejected keeps its slot's bytes (codes that a new
    rounding would choose otherwise too), and a padding entry of length 0 that names a slot in
    use does not disturb it."""
    c = Case(3, 1, 2, T, 64, 64, state, seed=17, lens=[T, T, 0], acc=[T, 0, 0], idx=[1, 3, 2], N=4)
    if state == "i8":
        c.pool //= 8
    before, sbefore = c.pool.clone(), None if c.scales is None else c.scales.clone()
    clean = c.call(rg, fn, pool=before.clone(), scales=None if sbefore is None else sbefore.clone())
    for s in (0, 2, 3):
        assert torch.equal(clean[1][s], before[s])
        assert sbefore is None or torch.equal(clean[2][s], sbefore[s])
    c.idx[2] = 1
    got = c.call(rg, fn)
    for x, y in zip(got, clean):
        assert torch.equal(x, y)


@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("fn,T", [("la_decode", 1), ("la_decode", 2), ("la_decode", 7), ("la_prefill", 90),
                                  ("la_prefill", 700)])
def test_rejected_tokens_do_not_reach_the_state(rg, fn, T, state):
    """NaN and infinity in tokens behind the accepted ones."""
    acc = [T // 2, T - 1, 0, T]
    c = Case(4, 1, 2, T, 64, 64, state, seed=18, lens=[T] * 4, acc=acc)
    clean = c.call(rg, fn, pool=c.pool.clone(), scales=None if c.scales is None else c.scales.clone())
    c.q, c.k, c.v, c.g = (x.clone() for x in (c.q, c.k, c.v, c.g))
    for b, n in enumerate(acc):
        c.q[b, :, n:], c.k[b, :, n:], c.v[b, :, n:], c.g[b, :, n:] = NAN, float("inf"), NAN, NAN
    got = c.call(rg, fn)
    for x, y in zip(got[1:], clean[1:]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("state", ["f32", "i8"])
@pytest.mark.parametrize("fn,T", [("la_decode", 5), ("la_prefill", 90), ("la_prefill", 600)])
def test_padding_is_not_read(rg, fn, T, state):
    """NaN and infinity in padded tokens, in the slots of skipped entries and of nobody."""
    c = Case(4, 1, 2, T, 64, 64, state, seed=3, N=6, lens=[T, T - 2, 1, T], acc=[T, T - 3, 1, T],
             idx=[3, 1, 5, 6])
    clean = c.call(rg, fn, pool=c.pool.clone(), scales=None if c.scales is None else c.scales.clone())
    c.q, c.k, c.v, c.g = (x.clone() for x in (c.q, c.k, c.v, c.g))
    for b, n in enumerate([T, T - 2, 1, 0]):
        c.q[b, :, n:], c.k[b, :, n:], c.v[b, :, n:] = NAN, float("inf"), NAN
        c.g[b, :, n:] = NAN
    for s in (0, 2, 4):
        if state == "i8":
            c.scales[s] = 255
        else:
            c.pool[s] = NAN
    got = c.call(rg, fn)
    assert torch.equal(got[0].contiguous().view(torch.int16), clean[0].contiguous().view(torch.int16))
    for s in (1, 3, 5):
        for x, y in zip(got[1:], clean[1:]):
            assert torch.equal(x[s], y[s])


@pytest.mark.parametrize("fn,T", [("la_decode", 6), ("la_prefill", 130), ("la_prefill", 500)])
def test_extreme_decays(rg, fn, T):
    """Decays that forget everything at a token (-infinity and finite), none at all, and growth."""
    c = Case(3, 1, 3, T, 64, 64, "f32", seed=11)
    c.lens[:] = T
    c.acc[:] = T
    c.g = c.g.contiguous()
    c.g[0] = 0.0
    c.g[1, 0, ::3] = -float("inf")
    c.g[1, 1, 1::4] = -500.0
    c.g[1, 2] = -1e30
    c.g[2] = 0.01
    out = c.call(rg, fn)[0]
    c.check(out, c.pool, None, f"{fn} extreme decays")


@pytest.mark.parametrize("fn,T", [("la_decode", 4), ("la_prefill", 100)])
def test_decay_for_each_head(rg, fn, T):
    """A [H_v] decay equals the same decay at every token."""
    c = Case(2, 2, 4, T, 128, 64, "bf16", seed=21)
    per_head = -torch.rand(4).cuda()
    c.g = per_head[None, :, None].expand(2, 4, T).contiguous()
    one = c.call(rg, fn, pool=c.pool.clone())
    c.g = per_head
    two = c.call(rg, fn, pool=c.pool.clone())
    for x, y in zip(one, two):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fn,T", [("la_decode", 4), ("la_prefill", 100), ("la_prefill", 700)])
def test_strides(rg, fn, T):
    """Slices of one projection's output, an out that lies in the projection's layout, and the
    contiguous call give the same bits."""
    B, Hq, Hv, D = 2, 2, 4, 64
    r = torch.Generator().manual_seed(4)
    x = torch.randn(B, T, (2 * Hq + Hv) * D, generator=r).to(torch.bfloat16).cuda()
    q, k, v = (y.reshape(B, T, -1, D).transpose(1, 2) for y in
               (x[..., :Hq * D], x[..., Hq * D:2 * Hq * D], x[..., 2 * Hq * D:]))
    g = -torch.rand(B, T, Hv, generator=r).cuda()
    pool = torch.randn(B, Hv, D, D, generator=r).cuda()
    out = torch.empty(B, T, Hv, D, dtype=torch.bfloat16, device="cuda")
    p1, p2 = pool.clone(), pool.clone()
    f = getattr(rg, fn)
    f(q, k, v, g.transpose(1, 2), p1, scale=0.125, out=out.transpose(1, 2))
    o2, _ = f(q.contiguous(), k.contiguous(), v.contiguous(), g.transpose(1, 2).contiguous(), p2,
              scale=0.125)
    torch.cuda.synchronize()
    assert torch.equal(out.transpose(1, 2).contiguous(), o2) and torch.equal(p1, p2)


@pytest.mark.parametrize("fn", ["la_decode", "la_prefill"])
def test_codes_are_those_of_the_state(rg, fn):
    """An 8-bit commit rounds a state that is good to fp32, so a code differs from the exact state's
    only where that is within fp32's error of a step's middle. Two tokens, every one accepted, so
    S = d S0 + w k1 v1 + k2 v2: of the sum's magnitudes, d and w are off by 2^-24 for their
    exponent's rounding (it is below 1), 2^-23 for the exponential and 2^-24 for the product, what is
    left of a value in three bf16 parts is 2^-27, and each of the up to four sums into which the terms
    go rounds by 2^-24 (2^-23 where it truncates): 2^-20 for all."""
    c = Case(4, 8, 16, 2, 128, 128, "i8", seed=21, lens=[2] * 4, acc=[2] * 4)
    _, pool, scales = c.call(rg, fn)
    _, states, _, smags = attention(c.q, c.k, c.v, c.g, c.S0, c.lens, c.idx, c.acc, c.scale)
    for b in range(c.B):
        got = mx_values(pool[c.idx[b]], scales[c.idx[b]])
        slack = 2.0 ** -20 * smags[b]
        over = (got - states[b]).abs() - mx_step(states[b].abs() + slack) / 2 - slack
        assert over.max() <= 0, f"{(over > 0).sum()} codes, off by {over.max():.3g} more than half a step"


def test_shared_entries(rg):
    """One prompt for every entry (stride 0 along the batch)."""
    c = Case(3, 1, 2, 40, 64, 64, "f32", seed=9, lens=[40, 17, 40], acc=[40, 17, 3])
    c.q, c.k, c.v = (x[:1].expand(3, -1, -1, -1) for x in (c.q, c.k, c.v))
    out = c.call(rg, "la_prefill")[0]
    c.check(out, c.pool, None, "shared entries")


@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
def test_prompt_then_tokens(rg, state):
    """A prompt in two halves and then single tokens, against one reference over all of them. The
    stored state is rounded between the calls, so the reference is rounded there too."""
    c = Case(2, 1, 2, 150, 128, 128, state, seed=31, N=2, lens=[150, 150], acc=[150, 150], idx=[1, 0])
    cut = [0, 64, 147, 148, 149, 150]
    for a, b in zip(cut, cut[1:]):
        fn = "la_decode" if b - a <= 8 else "la_prefill"
        d = Case.__new__(Case)
        d.__dict__.update(c.__dict__)
        d.q, d.k, d.v, d.g = (x[:, :, a:b] for x in (c.q, c.k, c.v, c.g))
        d.T = b - a
        d.lens = d.acc = torch.tensor([b - a] * 2, dtype=torch.int32)
        d.S0 = d.values(c.pool, c.scales).double().cpu()
        out = d.call(rg, fn)[0]
        d.check(out, c.pool, c.scales, f"{fn} tokens {a}..{b} {state}")


def test_long_prompt_same_as_parts(rg):
    """A prompt over many segments, ragged, against the reference; the accepted count lies inside
    one of them."""
    c = Case(2, 1, 2, 2100, 64, 64, "f32", seed=41, lens=[2100, 1333], acc=[1025, 1333], decay=0.05)
    out = c.call(rg, "la_prefill")[0]
    c.check(out, c.pool, None, "long prompt")


@pytest.mark.parametrize("D", [64, 128])
def test_with_and_without_workspace(rg, D):
    """Both forms of la_prefill, through the C entry, hold the reference."""
    c = Case(1, 1, 2, 1500, D, D, "f32", seed=43, lens=[1490], acc=[1490], decay=0.1)
    lib = rg.library()
    size = rg.la_prefill_workspace_size(1, 2, 1500, D, D)
    for ws in (0, size):
        pool = c.pool.clone()
        out = torch.empty(1, 2, 1500, D, dtype=torch.bfloat16, device="cuda")
        buf = torch.full((max(ws, 1),), 255, dtype=torch.uint8, device="cuda")
        lens, idx, acc = c.lens.cuda(), c.idx.cuda(), c.acc.cuda()
        args = []
        for t in (c.q, c.k, c.v, c.g):
            args += [t.data_ptr(), rg._Strides(*t.stride()[:3])]
        rc = lib.la_prefill(*args, pool.data_ptr(), None, 0, lens.data_ptr(), idx.data_ptr(),
                            acc.data_ptr(), c.scale, 1, 1, 2, 1500, D, D, c.N, out.data_ptr(), None,
                            pool.data_ptr(), None, buf.data_ptr() if ws else None, ws,
                            torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == 0
        c.check(out, pool, None, f"workspace {ws}")


@pytest.mark.parametrize("fn,T", [("la_decode", 1), ("la_decode", 8), ("la_prefill", 200), ("la_prefill", 1100)])
def test_captured_equals_eager(rg, fn, T):
    """A captured call, replayed with eager work between the replays: each step continues from the
    state that the last one left."""
    c = Case(2, 1, 2, T, 64, 64, "f32", seed=51, lens=[T, T - T // 3], acc=[T, T - T // 3])
    eager = c.pool.clone()
    lens, idx, acc = c.lens.cuda(), c.idx.cuda(), c.acc.cuda()
    f = getattr(rg, fn)
    pool = c.pool.clone()
    warm = pool.clone()
    f(c.q, c.k, c.v, c.g, warm, lens, idx, acc, c.scale)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = f(c.q, c.k, c.v, c.g, pool, lens, idx, acc, c.scale)
    for step in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want, _ = f(c.q, c.k, c.v, c.g, eager, lens, idx, acc, c.scale)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool, eager), f"replay {step}"


def test_other_stream(rg):
    """Calls on a stream of their own, back to back, leave what the default stream's calls do."""
    c = Case(1, 1, 2, 900, 64, 64, "f32", seed=61, lens=[900], acc=[900])
    lens, idx, acc = c.lens.cuda(), c.idx.cuda(), c.acc.cuda()
    a, b = c.pool.clone(), c.pool.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [rg.la_prefill(c.q, c.k, c.v, c.g, a, lens, idx, acc, c.scale, stream=s)[0] for _ in range(3)]
    s.synchronize()
    want = [rg.la_prefill(c.q, c.k, c.v, c.g, b, lens, idx, acc, c.scale)[0] for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(outs, want))


def test_two_calls_at_once(rg):
    """Two prompts on two streams, each cut into segments with a workspace of its own, and decode
    steps under a stream context: what the calls leave one after the other."""
    cs = [Case(1, 2, 4, 1300, 128, 128, "f32", seed=62 + i, lens=[1300 - 77 * i], acc=[900]) for i in range(2)]
    want = [c.call(rg, "la_prefill", pool=c.pool.clone()) for c in cs]
    pools = [c.pool.clone() for c in cs]
    args = [(c.lens.cuda(), c.idx.cuda(), c.acc.cuda(), c.scale) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [None, None]
    for i, (c, st) in enumerate(zip(cs, streams)):
        with torch.cuda.stream(st):
            outs[i] = rg.la_prefill(c.q, c.k, c.v, c.g, pools[i], *args[i])[0]
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want[i][0]) and torch.equal(pools[i], want[i][1])


def test_index_arrays_are_validated(rg, monkeypatch):
    monkeypatch.setattr(rg, "VALIDATE", True)
    c = Case(2, 1, 2, 4, 64, 64, "f32", seed=63, lens=[4, 3], acc=[4, 1], idx=[2, 0])
    out = c.call(rg, "la_decode")[0]
    c.check(out, c.pool, None, "validated")
    rg.la_decode(c.q, c.k, c.v, c.g, c.pool)  # every array left out
    for name, bad in (("idx", [0, 0]), ("idx", [0, 4]), ("lens", [5, 1]), ("acc", [4, 2])):
        d = Case(2, 1, 2, 4, 64, 64, "f32", seed=63, lens=[4, 1], acc=[4, 1], idx=[2, 0])
        setattr(d, name, torch.tensor(bad, dtype=torch.int32))
        with pytest.raises(RuntimeError, match="RGDR_ERR"):
            d.call(rg, "la_prefill")


def test_same_call_same_bits(rg):
    for fn, T in (("la_decode", 1), ("la_decode", 7), ("la_prefill", 333), ("la_prefill", 1500)):
        c = Case(2, 1, 2, T, 128, 128, "f32", seed=71)
        first = c.call(rg, fn, pool=c.pool.clone())
        for _ in range(3):
            again = c.call(rg, fn, pool=c.pool.clone())
            assert all(torch.equal(x, y) for x, y in zip(first, again)), fn


# ---- 8-bit pools ------------------------------------------------------------------------------

def mx_reference(x):
    """Codes and scale bytes by the definition, in 64 bits."""
    x = x.double().cpu()
    step = mx_step(x)
    codes = torch.round(x / step)
    return codes, (torch.log2(step) + 127).reshape(-1, 32)[:, 0].reshape(*x.shape[:-1], -1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shape", [(1, 1, 1, 32), (3, 2, 5, 96), (4, 5, 64, 64), (2, 3, 128, 544)], ids=str)
def test_quantize_and_back(rg, shape, dtype):
    """Codes and scales are those of the definition, bit for bit, and come back exactly."""
    r = torch.Generator().manual_seed(shape[2])
    x = torch.randn(shape, generator=r) * torch.exp2(torch.randint(-30, 30, shape[:-1] + (1,), generator=r).float())
    flat = x.view(-1, 32)
    flat[0] = 0
    flat[-1, 5] = 127.0
    flat[-1, 6:] = 0
    if flat.shape[0] > 2:
        flat[1] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -127.0] + [63.5] * 25)  # ties to even
        flat[2] = torch.tensor([127.5] + [1.0] * 31)                                      # one step up
    x = x.to(dtype).cuda()
    codes, scales = rg.la_state_quantize(x)
    torch.cuda.synchronize()
    want, e = mx_reference(x)
    assert torch.equal(codes.cpu().double(), want) and torch.equal(scales.cpu().double(), e)
    for back in (torch.float32, torch.bfloat16):
        y = rg.la_state_dequantize(codes, scales, dtype=back)
        assert y.dtype == back and torch.equal(y.double().cpu(), mx_values(codes, scales))


def test_quantize_special_values(rg):
    x = torch.zeros(1, 1, 8, 32)
    x[0, 0, 0, 3] = NAN
    x[0, 0, 1, 4] = float("inf")
    x[0, 0, 2, 0] = -float("inf")
    x[0, 0, 3] = 3e38
    x[0, 0, 4] = 2.0 ** -127         # subnormal: one step of the smallest scale
    x[0, 0, 5] = 2.0 ** -130         # rounds to zero
    x[0, 0, 6] = torch.finfo(torch.float32).max
    x[0, 0, 6, 1:] = -1e38
    x[0, 0, 7, 9] = -2.5
    codes, scales = rg.la_state_quantize(x.cuda())
    y = rg.la_state_dequantize(codes, scales, dtype=torch.float32).cpu()[0, 0]
    # Row 6 too: fp32's largest value lies above 127 * 2^121, so its step would be 2^122 and its
    # nearest code 64; 64 * 2^122 = 2^128 is no fp32 number.
    bad, fine = [0, 1, 2, 6], [3, 4, 5, 7]
    assert torch.isnan(y[bad]).all() and scales.cpu()[0, 0, bad].eq(255).all()
    assert torch.isfinite(y[fine]).all()
    want, e = mx_reference(x[:, :, fine])
    assert torch.equal(codes.cpu()[:, :, fine].double(), want)
    assert torch.equal(scales.cpu()[:, :, fine].double(), e)
    assert torch.equal(y[4], torch.full((32,), 2.0 ** -127)) and torch.all(y[5] == 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_slots(rg, dtype):
    """Gather and scatter between pools of different sizes; repeated sources, slots out of range,
    untouched destinations."""
    r = torch.Generator().manual_seed(8)
    x = torch.randn(5, 2, 64, 64, generator=r).to(dtype).cuda()
    codes = torch.full((7, 2, 64, 64), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((7, 2, 64, 2), 44, dtype=torch.uint8, device="cuda")
    src = torch.tensor([4, 4, 5, -1, 0, 1], dtype=torch.int32, device="cuda")
    dst = torch.tensor([6, 0, 2, 3, 7, -5], dtype=torch.int32, device="cuda")
    rg.la_state_quantize(x, codes, scales, src_slots=src, dst_slots=dst)
    want, e = mx_reference(x[4])
    for s in (6, 0):
        assert torch.equal(codes[s].cpu().double(), want) and torch.equal(scales[s].cpu().double(), e)
    for s in (2, 3):  # sources out of range: zero states
        assert torch.all(codes[s] == 0) and torch.all(scales[s] == 0)
    for s in (1, 4, 5):
        assert torch.all(codes[s] == 99) and torch.all(scales[s] == 44)
    y = torch.full((4, 2, 64, 64), 7.0, dtype=dtype, device="cuda")
    back_src = torch.tensor([6, 9, 0], dtype=torch.int32, device="cuda")
    back_dst = torch.tensor([3, 1, 4], dtype=torch.int32, device="cuda")
    rg.la_state_dequantize(codes, scales, y, src_slots=back_src, dst_slots=back_dst)
    torch.cuda.synchronize()
    assert torch.equal(y[3].double().cpu(), mx_values(codes[6:7], scales[6:7])[0])
    assert torch.all(y[1] == 0) and torch.all(y[0] == 7) and torch.all(y[2] == 7)


def test_state_moves_captured(rg):
    x = torch.randn(3, 2, 64, 64, device="cuda")
    codes = torch.zeros(3, 2, 64, 64, dtype=torch.int8, device="cuda")
    scales = torch.zeros(3, 2, 64, 2, dtype=torch.uint8, device="cuda")
    y = torch.zeros_like(x)
    rg.la_state_quantize(x, codes, scales)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rg.la_state_quantize(x, codes, scales)
        rg.la_state_dequantize(codes, scales, y)
    for step in range(3):
        x.mul_(1.7)
        graph.replay()
        torch.cuda.synchronize()
        a, b = rg.la_state_quantize(x)
        assert torch.equal(a, codes) and torch.equal(b, scales)
        assert torch.equal(rg.la_state_dequantize(a, b, dtype=torch.float32), y)


def test_commit_rounds_as_quantize(rg):
    """What a decode step commits to an 8-bit pool is what quantizing its fp32 state gives."""
    c = Case(3, 1, 2, 1, 128, 128, "i8", seed=91, lens=[1, 1, 1], acc=[1, 1, 1])
    wide = rg.la_state_dequantize(c.pool, c.scales, dtype=torch.float32)
    lens, idx = c.lens.cuda(), c.idx.cuda()
    rg.la_decode(c.q, c.k, c.v, c.g, wide, lens, idx, None, c.scale)
    c.call(rg, "la_decode")
    codes, scales = rg.la_state_quantize(wide)
    for b in range(3):
        s = int(c.idx[b])
        assert torch.equal(codes[s], c.pool[s]) and torch.equal(scales[s], c.scales[s])


# ---- the norm and gate ------------------------------------------------------------------------

def norm_reference(x, w, gate, eps, sigmoid, lens):
    x, w = x.double().cpu().transpose(1, 2), w.double().cpu()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w
    if gate is not None:
        z = gate.double().cpu()
        y = y * (torch.sigmoid(z) if sigmoid else z * torch.sigmoid(z))
    if lens is not None:
        for b, n in enumerate(lens):
            y[b, max(0, int(n)):] = 0
    return y


# fp32: the sum of D squares (D/2 units of 2^-24 of the result after the root, at most), root,
# division, three products, exponential and reciprocal of the gate: under D + 40 units in all.
def norm_bound(ref, D, dtype):
    unit = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dtype]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133  # half of the smallest step, or below
    return ref.abs() * ((D + 40) * 2.0 ** -24 + unit * (1 + 2.0 ** -10)) + tiny


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("shape", [(1, 1, 1, 8), (2, 3, 5, 24), (3, 4, 1, 64), (2, 5, 9, 128), (1, 2, 17, 200),
                                   (2, 1, 3, 256), (5, 7, 2, 520), (1, 3, 2, 1000), (1, 2, 3, 4096),
                                   (2, 1, 2, 8192)], ids=str)
def test_norm_gate(rg, shape, dtype):
    B, H, T, D = shape
    r = torch.Generator().manual_seed(D)
    x = (torch.randn(B, H, T, D, generator=r) * torch.exp2(torch.randint(-6, 5, (B, H, T, 1), generator=r).float())).to(dtype).cuda()
    gate = (3 * torch.randn(B, T, H, D, generator=r)).to(dtype).cuda()
    lens = torch.randint(0, T + 2, (B,), generator=r).to(torch.int32)
    for w, z, sig, ln in ((torch.randn(D, generator=r), gate, False, None),
                          (torch.randn(H, D, generator=r), gate, True, lens),
                          (torch.randn(D, generator=r), None, False, lens)):
        y = rg.la_norm_gate(x, w.cuda(), z, sigmoid=sig, eps=1e-5,
                            actual_seq_lengths=None if ln is None else ln.cuda())
        ref = norm_reference(x, w, z, float(np.float32(1e-5)), sig, ln)
        over = (y.double().cpu() - ref).abs() - norm_bound(ref, D, dtype)
        assert over.max() <= 0, f"{shape} {dtype}: off by {over.max():.3g} more than the bound"


def test_norm_gate_special_rows(rg):
    """Zero rows, large gates of both signs, NaN only in padded rows."""
    x = torch.zeros(2, 2, 3, 64, device="cuda")
    x[:, :, 1] = torch.randn(64, device="cuda")
    gate = torch.full((2, 3, 2, 64), 200.0, device="cuda")
    gate[0, :, :, ::2] = -200.0
    x[1, :, 2], gate[1, 2] = NAN, NAN
    w = torch.ones(64, device="cuda")
    lens = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    y = rg.la_norm_gate(x, w, gate, actual_seq_lengths=lens)
    ref = norm_reference(x, w, gate, 1e-6, False, lens.cpu())
    assert torch.all(y[:, 0] == 0) and torch.all(y[1, 2] == 0)
    assert ((y.double().cpu() - ref).abs() <= norm_bound(ref, 64, torch.float32)).all()


def test_norm_gate_layouts(rg):
    """Strided inputs and outputs, and a result in the gate's place, give the plain call's bits."""
    B, H, T, D = 2, 4, 5, 128
    x = torch.randn(B, T, H, D, device="cuda").to(torch.bfloat16).transpose(1, 2)
    both = torch.randn(B, T, 2 * H, D, device="cuda").to(torch.bfloat16)
    gate = both[:, :, H:]
    w = torch.randn(D, device="cuda")
    want = rg.la_norm_gate(x.contiguous(), w, gate.contiguous())
    assert torch.equal(rg.la_norm_gate(x, w, gate), want)
    left = both[:, :, :H].clone()
    assert torch.equal(rg.la_norm_gate(x, w, gate, out=gate), want)
    assert torch.equal(both[:, :, H:], want) and torch.equal(both[:, :, :H], left)


# ---- together ---------------------------------------------------------------------------------

@pytest.mark.parametrize("state", ["f32", "i8"])
def test_layer(rg, state):
    """One layer over a prompt and three more tokens, with the sequences parked in between: gate,
    attention, norm. Each step against its reference on that step's inputs."""
    B, Hq, Hv, D, T = 2, 2, 4, 64, 37
    r = torch.Generator().manual_seed(13)
    a_log = torch.randn(Hv, generator=r).cuda()
    dt_bias = torch.randn(Hv, generator=r).cuda()
    w = torch.randn(D, generator=r).cuda()
    pool = torch.zeros(3, Hv, D, D, dtype=DT[state], device="cuda")
    scales = torch.zeros(3, Hv, D, D // 32, dtype=torch.uint8, device="cuda") if state == "i8" else None
    idx = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    lens = torch.tensor([T, T - 9], dtype=torch.int32, device="cuda")
    for step, n in enumerate((T, 1, 1, 1)):
        x = torch.randn(B, n, (2 * Hq + 2 * Hv) * D, generator=r).to(torch.bfloat16).cuda()
        q, k, v, z = (y.reshape(B, n, -1, D) for y in x.split([Hq * D, Hq * D, Hv * D, Hv * D], -1))
        g, _ = rg.la_gate(torch.randn(B, n, Hv, generator=r).cuda(), dt_bias, -torch.exp(a_log))
        ln = lens if step == 0 else torch.ones_like(lens)
        c = Case.__new__(Case)
        c.B, c.Hq, c.Hv, c.T, c.Dk, c.Dv, c.N, c.state, c.scale = B, Hq, Hv, n, D, D, 3, state, D ** -0.5
        c.q, c.k, c.v, c.g = q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), g.transpose(1, 2)
        c.pool, c.scales, c.idx, c.lens, c.acc = pool, scales, idx.cpu(), ln.cpu(), ln.cpu()
        c.S0 = c.values(pool, scales).double().cpu()
        out = c.call(rg, "la_prefill" if n > 8 else "la_decode")[0]
        c.check(out, pool, scales, f"layer step {step}")
        y = rg.la_norm_gate(out, w, z, actual_seq_lengths=ln)
        ref = norm_reference(out, w, z, float(np.float32(1e-6)), False, ln.cpu())
        assert ((y.double().cpu() - ref).abs() <= norm_bound(ref, D, torch.bfloat16)).all()
        if state == "f32" and step == 1:  # park, and resume into other slots
            codes, sc = rg.la_state_quantize(pool, src_slots=idx)
            pool.zero_()
            idx = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
            rg.la_state_dequantize(codes, sc, pool, dst_slots=idx)
            torch.cuda.synchronize()
            assert torch.equal(pool[idx.long()].double().cpu(), mx_values(codes, sc))


def test_delta_rule_states_park(rg):
    """A pool of the gated delta rule parks too, and decodes on from what came back."""
    import workloads
    from gpu_util import check_decode, oracle_decode, upload
    inp = workloads.make_case(2, 1, 2, 3, 64, 64, 3, seed=88, indices="choice", lengths="uniform")
    d = upload(inp)
    codes, scales = rg.la_state_quantize(d["state"])
    pool = rg.la_state_dequantize(codes, scales)
    torch.cuda.synchronize()
    from gpu_util import dev_to_bits
    inp.state = dev_to_bits(pool)
    out, st = rg.rgdr_decode(d["query"], d["key"], d["value"], d["beta"], pool, d["actual_seq_lengths"],
                             d["ssm_state_indices"], d["g"], d["gk"], d["num_accepted_tokens"], inp.scale)
    torch.cuda.synchronize()
    check_decode(inp, out, st, oracle_decode(inp), "resumed states")


def test_refusals_on_the_device(rg):
    """Shapes, types and places that do not fit raise before anything is launched."""
    c = Case(2, 1, 2, 3, 64, 64, "i8", seed=5)
    good = (c.q, c.k, c.v, c.g, c.pool)
    with pytest.raises(RuntimeError, match="needs state_scales"):
        rg.la_decode(*good)
    with pytest.raises(RuntimeError, match="state_scales must be"):
        rg.la_decode(*good, state_scales=c.scales[:, :, :, :1])
    with pytest.raises(RuntimeError, match="only an int8 pool"):
        rg.la_decode(*good[:4], c.pool.float(), state_scales=c.scales)
    with pytest.raises(RuntimeError, match="last axis"):
        rg.la_decode(c.q.transpose(2, 3).contiguous().transpose(2, 3), *good[1:], state_scales=c.scales)
    with pytest.raises(RuntimeError, match="inconsistent"):
        rg.la_decode(c.q, c.k[:, :, :2], *good[2:], state_scales=c.scales)
    with pytest.raises(RuntimeError, match="RGDR_ERR_ALIGN"):
        wide = torch.zeros(2, 2, 3, 65, dtype=torch.bfloat16, device="cuda")
        rg.la_decode(c.q, c.k, wide[..., :64], *good[3:], state_scales=c.scales)
    with pytest.raises(RuntimeError, match="RGDR_ERR_SHAPE"):
        rg.la_decode(*good, state_scales=c.scales, out=torch.zeros(2, 1, 3, 64, dtype=torch.bfloat16,
                                                                   device="cuda").expand(2, 2, 3, 64))
    with pytest.raises(RuntimeError, match="expected cuda"):
        rg._same_device(c.q, other=torch.zeros(1))
    with pytest.raises(RuntimeError, match="workspace must be"):
        rg.la_prefill(*good, state_scales=c.scales, workspace=torch.zeros(4, device="cuda"))
    with pytest.raises(RuntimeError, match="RGDR_ERR_ALIGN"):
        rg.la_prefill(*good, state_scales=c.scales,
                      workspace=torch.zeros(1024, dtype=torch.uint8, device="cuda")[8:])
    with pytest.raises(RuntimeError, match="actual_seq_lengths must have shape"):
        rg.la_decode(*good, c.lens.cuda()[:1], state_scales=c.scales)
    with pytest.raises(RuntimeError, match="go together"):
        rg.la_state_quantize(c.pool.float(), torch.zeros_like(c.pool))
    with pytest.raises(RuntimeError, match="names slots"):
        rg.la_state_dequantize(c.pool, c.scales, dst_slots=c.idx.cuda())
    with pytest.raises(RuntimeError, match="weight"):
        rg.la_norm_gate(c.v, torch.ones(32, device="cuda"))
    with pytest.raises(RuntimeError, match="gate must be"):
        rg.la_norm_gate(c.v, torch.ones(64, device="cuda"), c.v)


def test_refuses_odd_tensors(rg):
    """Slot arrays that are no arrays, and a decay that torch holds as its negative."""
    x = torch.zeros(2, 2, 64, 64, device="cuda")
    codes, scales = rg.la_state_quantize(x)
    with pytest.raises(TypeError, match="src_slots"):
        rg.la_state_quantize(x, src_slots=[0, 1])
    with pytest.raises(TypeError, match="dst_slots"):
        rg.la_state_dequantize(codes, scales, x, dst_slots=torch.tensor(0, device="cuda"))
    with pytest.raises(RuntimeError, match="state must be"):
        rg.la_state_dequantize(codes, scales, [x])
    c = Case(1, 1, 2, 4, 64, 64, "f32", seed=19)
    c.g = torch.randn(1, 2, 4, dtype=torch.complex64, device="cuda").conj().imag
    assert c.g.is_neg()
    with pytest.raises(RuntimeError, match="unsupported arguments"):
        c.call(rg, "la_decode")


def test_empty_calls(rg):
    q = torch.zeros(0, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(0, 2, 3, device="cuda")
    pool = torch.ones(1, 2, 64, 64, device="cuda")
    for f in (rg.la_decode, rg.la_prefill):
        out, st = f(q, q, q, g, pool)
        assert out.shape == (0, 2, 3, 64) and torch.all(st == 1)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    codes, scales = rg.la_state_quantize(pool, src_slots=none)
    assert codes.shape == (0, 2, 64, 64)
    assert rg.la_state_dequantize(codes, scales).shape == (0, 2, 64, 64)
    assert rg.la_norm_gate(q, torch.ones(64, device="cuda")).shape == (0, 3, 2, 64)


@pytest.mark.parametrize("state", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("Dv,B", [(96, 2), (64, 70)])
@pytest.mark.parametrize("T", [2, 5, 8])
def test_tokens_do_not_reach_earlier_outputs(rg, T, Dv, B, state):
    """NaN and infinities in a drafted token, accepted or not, leave the outputs of the tokens before it
    as they are without them, and show in its own and in the later ones'. (B = 70: two blocks of columns for
    each wave.)"""
    c = Case(B, 16, 32, T, 64, Dv, state, seed=19, lens=[T] * B, acc=[T - 1 - b % 2 for b in range(B)])
    clean = c.call(rg, "la_decode", pool=c.pool.clone(), scales=None if c.scales is None else c.scales.clone())
    c.q, c.k, c.v, c.g = (x.clone() for x in (c.q, c.k, c.v, c.g))
    c.v[0, :, T - 1, 5:40], c.k[0, :, T - 1, 3], c.q[0, :, T - 1, 9], c.g[0, :, T - 1] = NAN, float("inf"), NAN, NAN
    c.v[1, :, T // 2, 7], c.v[1, :, T // 2, 41] = float("inf"), -float("inf")
    out = c.call(rg, "la_decode")[0]
    for b, s in ((0, T - 1), (1, T // 2)):
        assert torch.equal(out[b, :, :s], clean[0][b, :, :s])
        assert not torch.isfinite(out[b, :, s:, 7]).any()
    assert not torch.isfinite(out[1, :, T // 2:, 41]).any()
    rest = [x for x in range(Dv) if x not in (7, 41)]
    assert torch.equal(out[1][..., rest], clean[0][1][..., rest])
    assert torch.equal(out[2:], clean[0][2:])
