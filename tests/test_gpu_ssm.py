"""ssm_decode and ssm_prefill against a token-by-token reference in 64 bits (bounds: ssm_util), and the
operators in front of the recurrences as a layer runs them."""
import pytest
import torch

from ssm_util import TYPES, check, clamp, conv, rope, scan, zero_bits

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def rg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_rgdr_amd as m
    m.library()
    return m


class Case:
    """Inputs of one call, made on the CPU from a seed."""

    def __init__(self, B, T, C, N, G, dtype, state, seed, *, slots=None, lens="ragged", acc="ragged",
                 idx=None, gated=True, layout="sliced", slow=1.0):
        r = torch.Generator().manual_seed(seed)
        self.B, self.T, self.C, self.N, self.G = B, T, C, N, G
        self.slots, self.dtype = slots or B + 2, TYPES[dtype]

        def rows(*shape, size=1.0):
            x = (torch.randn(B, T, *shape, generator=r) * size).to(self.dtype).cuda()
            if layout == "sliced" and len(shape) == 1:  # columns of a wider projection
                wide = torch.full((B, T, shape[0] + 24), NAN, dtype=self.dtype, device="cuda")
                wide[..., 8:8 + shape[0]] = x
                return wide[..., 8:8 + shape[0]]
            return x

        self.x, self.dt, z = rows(C), rows(C), rows(C)
        self.z = z if gated else None
        bc = rows(2 * G * N)
        self.Bm, self.Cm = (bc[..., i * G * N:(i + 1) * G * N].unflatten(-1, (G, N)) for i in (0, 1))
        self.A = (-torch.arange(1, N + 1) * torch.exp(torch.randn(C, N, generator=r)) * slow).cuda()
        self.D = torch.randn(C, generator=r).cuda() if gated else None
        self.bias = (torch.randn(C, generator=r) * 2 - 3).cuda() if gated else None
        self.pool = torch.randn(self.slots, C, N, generator=r).to(TYPES[state]).cuda()
        if lens == "ragged":
            lens = [T - (b * T) // max(B, 1) if b % 3 else T for b in range(B)]
            lens[-1] = lens[-1] if B < 3 else 0
        if acc == "ragged":
            acc = [max(0, n - b % 4) for b, n in enumerate(lens)]
        self.lens, self.acc = (torch.tensor(v, dtype=torch.int32) for v in (lens, acc))
        self.idx = torch.tensor(idx, dtype=torch.int32) if idx is not None else \
            torch.randperm(self.slots, generator=r)[:B].to(torch.int32)

    def call(self, rg, fn, pool=None, **kw):
        r = getattr(rg, fn)(self.x, self.dt, self.A, self.Bm, self.Cm, self.pool if pool is None else pool,
                            self.lens.cuda(), self.idx.cuda(), self.acc.cuda(), D=self.D, z=self.z,
                            dt_bias=self.bias, **kw)
        torch.cuda.synchronize()
        return r

    def reference(self, **kw):
        return scan(self.x, self.dt, self.A, self.Bm, self.Cm, self.pool.clone(), self.lens, self.idx,
                    self.acc, self.D, self.z, self.bias, **kw)

    def check(self, out, after, ref, tag):
        check(out, ref[0], ref[1], tag)
        for b in range(self.B):
            e = clamp(self.lens, self.idx, self.acc, b, self.T, self.slots)
            assert zero_bits(out[b, e[0] if e else 0:]), f"{tag}: padded row"
            if e:
                check(after[int(self.idx[b])], ref[2][b], ref[3][b], f"{tag} state {b}")

    def rest(self, pool):
        """Slots that no entry names."""
        named = {int(i) for i in self.idx}
        return pool[[s for s in range(self.slots) if s not in named]]


SHAPES = [  # B, T, C, N, G
    (1, 1, 8, 8, 1), (3, 1, 72, 16, 1), (2, 1, 512, 32, 2), (2, 2, 136, 16, 17), (5, 3, 64, 8, 8),
    (3, 5, 264, 16, 3), (2, 8, 40, 32, 5), (4, 8, 1032, 16, 1), (9, 1, 128, 16, 16), (3, 4, 24, 8, 1),
]
PROMPTS = [
    (1, 1, 8, 16, 1), (2, 9, 72, 8, 1), (2, 15, 64, 16, 4), (1, 16, 128, 16, 1), (3, 17, 264, 32, 3),
    (2, 31, 200, 16, 25), (2, 32, 64, 8, 1), (2, 33, 136, 16, 1), (1, 63, 64, 16, 8), (3, 64, 72, 16, 1),
    (2, 65, 80, 32, 2), (3, 129, 48, 8, 6), (2, 300, 64, 16, 1), (1, 577, 24, 16, 3), (1, 1030, 16, 16, 1),
]


@pytest.mark.parametrize("types", [("bf16", "f32"), ("f16", "bf16"), ("f32", "f32"), ("bf16", "bf16")], ids="-".join)
@pytest.mark.parametrize("fn,shape", [("ssm_decode", s) for s in SHAPES] + [("ssm_prefill", s) for s in PROMPTS], ids=str)
def test_scan(rg, fn, shape, types):
    c = Case(*shape, *types, seed=sum(shape), gated=shape[0] % 2 == 1 or shape[1] % 2 == 0,
             layout="sliced" if shape[1] % 2 else "whole", slow=1.0 if shape[0] % 2 else 0.05)
    before = c.rest(c.pool).clone()
    ref = c.reference()
    out, after = c.call(rg, fn)
    assert after is c.pool
    c.check(out, after, ref, f"{fn} {shape} {types}")
    assert torch.equal(c.rest(c.pool), before)


FORMS = [("ssm_decode", 1), ("ssm_decode", 6), ("ssm_prefill", 5), ("ssm_prefill", 70), ("ssm_prefill", 300)]


@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("fn,T", FORMS)
def test_lengths_slots_and_counts(rg, fn, T, state):
    """Empty and over-long lengths, counts past the length, slots out of range, and a pool that stays
    as it was beside a separate output pool."""
    c = Case(9, T, 72, 16, 1, "bf16", state, 7, slots=10,
             lens=[T, 0, T + 5, -2, 1, T, T, (T + 1) // 2, T],
             acc=[T + 9, 0, 1, 3, 1, -1, T, 0, T // 2], idx=[4, 8, 0, 2, 7, 1, -1, 10, 3])
    ref = c.reference()
    new = torch.full_like(c.pool, 7.0)
    keep = c.pool.clone()
    out, after = c.call(rg, fn, state_out=new)
    assert after is new and torch.equal(c.pool, keep)
    c.check(out, new, ref, "apart")
    assert torch.all(c.rest(new) == 7.0)
    out, after = c.call(rg, fn)
    c.check(out, after, ref, "in place")
    assert torch.equal(c.rest(c.pool), c.rest(keep))


@pytest.mark.parametrize("fn,T", FORMS)
def test_what_is_not_read(rg, fn, T):
    """NaN in padding, in slots that are not named and in an entry without a slot does not show."""
    c = Case(4, T, 72, 16, 1, "bf16", "f32", 8, slots=6, lens=[T, T // 2, 0, T], acc=[T, T // 2, 0, T],
             idx=[1, 3, 0, 9])
    ref = c.reference()
    for b, n in enumerate([T, T // 2, 0, 0]):
        for t in (c.x, c.dt, c.z, c.Bm, c.Cm):
            t[b, n:] = NAN
    c.pool[[2, 4, 5]] = NAN
    out, after = c.call(rg, fn)
    c.check(out, after, ref, "padding")


@pytest.mark.parametrize("fn,T", FORMS)
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_values_that_are_not_finite(rg, fn, T, value):
    """A token's stay out of the outputs before it and out of other channels, and, where the token is
    rejected, out of the state."""
    t0 = T // 2
    c = Case(2, T, 72, 16, 1, "bf16", "f32", 9, lens=[T, T], acc=[t0, t0])
    want, after = c.call(rg, fn, pool=c.pool.clone())
    c.x[0, t0, 3] = value
    c.dt[1, t0, 5] = value
    c.Bm[1, t0, 0, 2] = value
    out, got = c.call(rg, fn)
    assert torch.equal(got, after)
    assert torch.equal(out[:, :t0], want[:, :t0])
    others = [i for i in range(72) if i != 3]
    assert torch.equal(out[0][:, others], want[0][:, others])
    assert not torch.isfinite(out[0, t0, 3]) and not torch.isfinite(out[1, t0]).any()


@pytest.mark.parametrize("fn,T", FORMS)
def test_no_accepted_token_leaves_the_slot(rg, fn, T):
    c = Case(3, T, 64, 16, 1, "bf16", "f32", 10, lens=[T, 0, T], acc=[0, 0, 0])
    c.pool[int(c.idx[1])] = NAN
    keep = c.pool.clone()
    out, _ = c.call(rg, fn)
    assert torch.equal(torch.nan_to_num(c.pool, 9.0), torch.nan_to_num(keep, 9.0))
    assert zero_bits(out[1])


@pytest.mark.parametrize("fn,T", FORMS)
def test_extreme_steps(rg, fn, T):
    """Steps that forget everything at once, and steps of nothing; as they are, without softplus."""
    c = Case(2, T, 64, 16, 1, "f32", "f32", 11, lens=[T, T], acc=[T, T], gated=False)
    c.dt[0] = torch.where(torch.rand(c.dt[0].shape, device="cuda") < 0.3, 1e4, 0.0)
    c.dt[1] = 0.0
    ref = c.reference(softplus=False)
    out, after = c.call(rg, fn, dt_softplus=False)
    c.check(out, after, ref, "steps")
    assert torch.isfinite(out).all()
    c.dt[0], c.dt[1] = 60.0, -60.0  # softplus: 60, and e^-60
    ref = c.reference()
    c.check(*c.call(rg, fn), ref, "softplus")


@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_prompt_then_tokens(rg, state):
    """A prompt and then tokens one and several at a time, on the slots, against one reference over all
    tokens (a bf16 state is rounded at every commit: only fp32 ones are held to one reference)."""
    T, parts = 150, (97, 1, 1, 8, 3, 40)
    c = Case(2, T, 72, 16, 3, "bf16", state, 12, lens=[T, T], acc=[T, T])
    idx = c.idx.cuda()
    t = 0
    whole = c.reference()
    pool = c.pool.clone()
    for n in parts:
        fn = rg.ssm_decode if n <= 8 else rg.ssm_prefill
        s = slice(t, t + n)
        lens = torch.full((2,), n, dtype=torch.int32)
        step = scan(c.x[:, s], c.dt[:, s], c.A, c.Bm[:, s], c.Cm[:, s], pool.clone(), lens, c.idx, lens,
                    c.D, c.z[:, s], c.bias)
        out, _ = fn(c.x[:, s], c.dt[:, s], c.A, c.Bm[:, s], c.Cm[:, s], pool, ssm_state_indices=idx,
                    D=c.D, z=c.z[:, s], dt_bias=c.bias)
        check(out, step[0], step[1], f"{n} tokens at {t}")
        if state == "f32":
            check(out, whole[0][:, s], whole[1][:, s], f"whole, {n} tokens at {t}")
        t += n
    if state == "f32":
        for b in range(2):
            check(pool[int(c.idx[b])], whole[2][b], whole[3][b], "state")


@pytest.mark.parametrize("C,T", [(64, 1000), (24, 700), (512, 2100)])
def test_with_and_without_workspace(rg, C, T):
    c = Case(1, T, C, 16, 1, "bf16", "f32", 13, lens=[T - 3], acc=[T - 77], slow=0.02)
    size = rg.ssm_prefill_workspace_size(1, T, C, 16)
    ref = c.reference()
    tiny = torch.empty(0, dtype=torch.uint8, device="cuda")
    for ws in (None, tiny, torch.full((max(size, 1),), 255, dtype=torch.uint8, device="cuda")):
        out, after = c.call(rg, "ssm_prefill", pool=c.pool.clone(), workspace=ws)
        c.check(out, after, ref, f"workspace {None if ws is None else ws.numel()} of {size}")


@pytest.mark.parametrize("fn,T", FORMS + [("ssm_prefill", 1500)])
def test_captured_equals_eager(rg, fn, T):
    c = Case(3, T, 72, 16, 1, "bf16", "f32", 14)
    first = c.pool.clone()
    lens, idx, acc = c.lens.cuda(), c.idx.cuda(), c.acc.cuda()
    out = torch.empty(3, T, 72, dtype=torch.bfloat16, device="cuda")

    def call(pool, out=None):
        return getattr(rg, fn)(c.x, c.dt, c.A, c.Bm, c.Cm, pool, lens, idx, acc, D=c.D, z=c.z, dt_bias=c.bias, out=out)
    call(c.pool, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call(c.pool, out)
    for k in range(4):
        c.x.copy_(torch.randn(c.x.shape).bfloat16())
        want, pool = call(first.clone())
        c.pool.copy_(first)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c.pool, pool), k


def test_two_calls_at_once(rg):
    """Two streams, each with its own slots and workspace, both against the calls one by one."""
    c = [Case(1, 1200, 64, 16, 1, "bf16", "f32", s, lens=[1200], acc=[1200]) for s in (15, 16)]
    want = [x.call(rg, "ssm_prefill", pool=x.pool.clone()) for x in c]
    streams = [torch.cuda.Stream() for _ in c]
    torch.cuda.synchronize()
    got = []
    for x, s in zip(c, streams):
        got.append(rg.ssm_prefill(x.x, x.dt, x.A, x.Bm, x.Cm, x.pool, ssm_state_indices=x.idx.cuda(), D=x.D,
                                  z=x.z, dt_bias=x.bias, stream=s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


@pytest.mark.parametrize("fn,T", FORMS + [("ssm_prefill", 1500)])
def test_same_call_same_bits(rg, fn, T):
    c = Case(2, T, 264, 16, 1, "bf16", "f32", 17)
    first = c.call(rg, fn, pool=c.pool.clone())
    for _ in range(3):
        again = c.call(rg, fn, pool=c.pool.clone())
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("fn,T", FORMS)
def test_strides(rg, fn, T):
    """Operands of other orders and repeated ones; an out inside a wider buffer."""
    c = Case(2, T, 64, 16, 2, "bf16", "f32", 18, lens=[T, T], acc=[T, T], layout="whole")
    ref = c.reference()
    for name in ("x", "dt", "z", "Bm", "Cm"):
        t = getattr(c, name)
        setattr(c, name, t.transpose(0, 1).contiguous().transpose(0, 1))
    wide = torch.full((2, T, 200), 5.0, dtype=torch.bfloat16, device="cuda")
    keep = c.pool.clone()
    out, after = c.call(rg, fn, out=wide[..., 64:128])
    c.check(out, after, ref, "other order")
    assert torch.all(wide[..., :64] == 5) and torch.all(wide[..., 128:] == 5)
    # one row of B and C for all tokens, groups and entries
    c.pool = keep
    c.Bm, c.Cm = (t[:1, :1, :1].expand(2, T, 2, 16) for t in (c.Bm, c.Cm))
    ref = c.reference()
    c.check(*c.call(rg, fn), ref, "repeated")


def test_defaults(rg):
    c = Case(3, 20, 64, 16, 1, "bf16", "f32", 19, slots=4, lens=[20] * 3, acc=[20] * 3, idx=[0, 1, 2], gated=False)
    ref = c.reference()
    out, after = rg.ssm_prefill(c.x, c.dt, c.A, c.Bm, c.Cm, c.pool)
    c.check(out, after, ref, "defaults")


def test_large_offsets(rg):
    """A slot past 2^32 bytes of the pool, and rows past 2^31 elements."""
    c = Case(2, 12, 64, 16, 1, "bf16", "f32", 20, slots=4, lens=[12] * 2, acc=[12] * 2, idx=[0, 3], layout="whole")
    ref = c.reference()
    slots = 2 ** 30 // (64 * 16) + 5
    pool = torch.empty(slots, 64, 16, device="cuda")
    c.idx = torch.tensor([0, slots - 1], dtype=torch.int32)
    pool[0], pool[-1] = c.pool[0], c.pool[3]
    far = torch.empty(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    view = far.as_strided((2, 12, 64), (2 ** 31, 64, 1))
    view.copy_(c.x)
    c.x, c.slots = view, slots
    for fn, T in (("ssm_prefill", 12),):
        out, after = c.call(rg, fn, pool=pool)
        c.check(out, after, ref, fn)


def test_index_arrays_are_validated(rg, monkeypatch):
    c = Case(2, 4, 64, 16, 1, "bf16", "f32", 21, slots=4)
    monkeypatch.setattr(rg, "VALIDATE", True)
    rg.ssm_decode(c.x, c.dt, c.A, c.Bm, c.Cm, c.pool)
    for fn in (rg.ssm_decode, rg.ssm_prefill):
        with pytest.raises(RuntimeError, match="index arrays"):
            fn(c.x, c.dt, c.A, c.Bm, c.Cm, c.pool, ssm_state_indices=torch.tensor([1, 1], dtype=torch.int32).cuda())


def test_refusals_on_the_device(rg):
    c = Case(2, 4, 64, 16, 2, "bf16", "f32", 22, layout="whole")
    good = dict(x=c.x, dt=c.dt, A=c.A, B=c.Bm, C=c.Cm, state_pool=c.pool)
    i32 = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = [dict(x=c.x.double()), dict(x=c.x.float()), dict(x=c.x[0]), dict(dt=c.dt[:, :3]), dict(dt=None),
           dict(A=c.A.bfloat16()), dict(A=c.A[:, :15]), dict(A=c.A[:, 0]), dict(B=c.Bm[:, :, :1]), dict(B=c.Bm[..., :8]),
           dict(C=c.Cm.float()), dict(C=None), dict(state_pool=c.pool.half()), dict(state_pool=c.pool[:, :8]),
           dict(state_pool=c.pool[:1]), dict(state_out=c.pool.bfloat16()), dict(D=c.D[:8]), dict(D=c.D.double()),
           dict(z=c.z.float()), dict(z=c.z[:1]), dict(dt_bias=c.bias[None]), dict(out=c.x[:, :1]),
           dict(out=c.x.as_strided(c.x.shape, (256, 0, 1))), dict(actual_seq_lengths=i32), dict(ssm_state_indices=i32.long()),
           dict(x=c.x.cpu()), dict(A=c.A.cpu()), dict(x=c.x.transpose(0, 1)), dict(x=1.0)]
    for fn in (rg.ssm_decode, rg.ssm_prefill):
        for kw in bad:
            with pytest.raises((RuntimeError, TypeError)):
                fn(**{**good, **kw})
    with pytest.raises(RuntimeError):
        rg.ssm_prefill(**good, workspace=i32)
    long = Case(1, 9, 64, 16, 1, "bf16", "f32", 23)
    with pytest.raises(RuntimeError, match="SHAPE"):
        long.call(rg, "ssm_decode")


def test_empty_batch(rg):
    c = Case(2, 4, 64, 16, 1, "bf16", "f32", 24)
    for fn in (rg.ssm_decode, rg.ssm_prefill):
        out, _ = fn(c.x[:0], c.dt[:0], c.A, c.Bm[:0], c.Cm[:0], c.pool)
        assert out.shape == (0, 4, 64)


def test_state_space_layer(rg):
    """Convolution, the projections of its output, and the scan: a prompt in two parts and then single
    tokens, as a server runs them, each call against the references on what the call before left."""
    r = torch.Generator().manual_seed(25)
    B, T, C, N, low = 2, 60, 64, 16, 8
    xz = torch.randn(B, T, 2 * C, generator=r).bfloat16().cuda()
    w, bias = torch.randn(C, 4, generator=r).cuda(), torch.randn(C, generator=r).cuda()
    to_low = (torch.randn(C, low + 2 * N, generator=r) * C ** -0.5).bfloat16().cuda()
    to_dt = (torch.randn(low, C, generator=r) * 0.3).bfloat16().cuda()
    A = -torch.arange(1, N + 1).float().repeat(C, 1).cuda()
    D, dt_bias = torch.ones(C, device="cuda"), (torch.randn(C, generator=r) - 4).cuda()
    last = torch.zeros(B + 1, 3, C, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(B + 1, C, N, device="cuda")
    idx = torch.tensor([2, 0], dtype=torch.int32)
    t = 0
    for n in (37, 20, 1, 1, 1):
        x, z = xz[:, t:t + n, :C], xz[:, t:t + n, C:]
        lens = torch.full((B,), n, dtype=torch.int32)
        want = conv(x, w, bias, last, lens, idx, lens, True)
        y, _ = rg.la_conv(x, w, last, ssm_state_indices=idx.cuda(), bias=bias)
        check(y, want[0], want[1], f"convolution at {t}")
        low_rows = y @ to_low
        dt = low_rows[..., :low] @ to_dt
        Bm, Cm = (low_rows[..., low + i * N:low + (i + 1) * N].unflatten(-1, (1, N)) for i in (0, 1))
        want = scan(y, dt, A, Bm, Cm, pool.clone(), lens, idx, lens, D, z, dt_bias)
        fn = rg.ssm_decode if n <= 8 else rg.ssm_prefill
        o, _ = fn(y, dt, A, Bm, Cm, pool, ssm_state_indices=idx.cuda(), D=D, z=z, dt_bias=dt_bias)
        check(o, want[0], want[1], f"scan at {t}")
        t += n


def test_linear_attention_layer(rg):
    """Convolution of a projection's queries, keys and values, rotary positions, linear attention, norm and
    gate, for a prompt and then a token: rotated rows equal the reference on the convolution's output, and
    the token's output equals the one of a prompt that is a token longer."""
    r = torch.Generator().manual_seed(26)
    B, T, H, D = 2, 40, 2, 64
    qkv = (0.3 * torch.randn(B, T + 1, 3 * H * D, generator=r)).bfloat16().cuda()
    w = (0.5 * torch.randn(3 * H * D, 4, generator=r)).cuda()
    g = (-0.2 * torch.rand(B, H, T + 1, generator=r)).cuda()
    gate = torch.randn(B, T + 1, H, D, generator=r).bfloat16().cuda()
    freq, _ = rg.la_rope_frequencies(D // 2)

    def run(x, g, gate, last, pool, at, fn):
        y, _ = rg.la_conv(x, w, last)
        q, k, v = (y[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)).transpose(1, 2) for i in range(3))
        pos = torch.full((B,), at, dtype=torch.int32, device="cuda")
        q2, k2 = rg.la_rope(q, k, freq, pos)
        for a, b in ((q, q2), (k, k2)):
            check(b, *rope(a, freq, pos, 1.0, False, [x.shape[1]] * B), "rotated")
        o, _ = fn(q2, k2, v, g, pool, scale=D ** -0.5)
        return rg.la_norm_gate(o, torch.ones(D, device="cuda"), gate)

    def fresh():
        return (torch.zeros(B, 3, 3 * H * D, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(B, H, D, D, device="cuda"))
    whole = run(qkv, g, gate, *fresh(), 0, rg.la_prefill)
    last, pool = fresh()
    first = run(qkv[:, :T], g[..., :T], gate[:, :T], last, pool, 0, rg.la_prefill)
    token = run(qkv[:, T:], g[..., T:], gate[:, T:], last, pool, T, rg.la_decode)
    # convolution and turn are the same bits either way; the attention's outputs round once to bf16 (half
    # a step each way), as the norm's do, and their fp32 sums differ by far less
    got = torch.cat([first, token], 1).double()
    bound = 2.0 ** -8 * 4 * whole.double().abs() + 2.0 ** -8 * 0.01
    assert torch.all((got - whole.double()).abs() <= bound)
