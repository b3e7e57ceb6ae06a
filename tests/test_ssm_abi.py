"""la_conv, la_rope, ssm_decode and ssm_prefill without a GPU: every refusal happens on the host, before
anything is launched, so the made-up addresses are never used."""
import ctypes as C

import pytest
import torch

import gated_delta_rule_rgdr_amd as rg

OK, NULL, SHAPE, UNSUP, RANGE, DUP, DTYPE, HIP, ALIGN = range(9)
F32, F16, BF16, MXI8 = range(4)
P, Q = 0x100000, 0x900000


@pytest.fixture(scope="module")
def lib():
    return rg.library()


def with_strides(a, names):
    return {k: rg._Strides(*v) if k in names and v is not None else v for k, v in a.items()}


def conv(lib, **kw):
    a = dict(x=P, xs=None, w=P, bias=P, dt=BF16, pool=P, lens=P, idx=P, acc=P, fl=1, B=2, T=4, C=64, W=4, N=5,
             out=Q, os=None, so=P)
    a = with_strides({**a, **kw}, ("xs", "os"))
    return lib.la_conv(a["x"], a["xs"], a["w"], a["bias"], a["dt"], a["pool"], a["lens"], a["idx"], a["acc"], a["fl"],
                       a["B"], a["T"], a["C"], a["W"], a["N"], a["out"], a["os"], a["so"], None)


BAD_CONV = [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(pool=None), NULL), (dict(out=None), NULL), (dict(so=None), NULL),
    (dict(B=-1), SHAPE), (dict(T=0), SHAPE), (dict(T=65537), SHAPE), (dict(C=0), SHAPE), (dict(N=0), SHAPE),
    (dict(W=0), SHAPE), (dict(idx=None, N=1), SHAPE), (dict(out=P), SHAPE),
    (dict(xs=(-256, 0, 64)), SHAPE), (dict(os=(256, 0, 32)), SHAPE), (dict(os=(64, 0, 64)), SHAPE),
    (dict(xs=(1 << 61, 0, 64)), SHAPE), (dict(B=1 << 24, T=1000), SHAPE),
    (dict(C=12), UNSUP), (dict(W=1), UNSUP), (dict(W=5), UNSUP), (dict(fl=2), UNSUP),
    (dict(dt=MXI8), DTYPE), (dict(dt=-1), DTYPE),
    (dict(x=P + 8), ALIGN), (dict(w=P + 4), ALIGN), (dict(bias=P + 4), ALIGN), (dict(pool=P + 2), ALIGN),
    (dict(out=Q + 8), ALIGN), (dict(so=P + 8), ALIGN), (dict(lens=P + 2), ALIGN), (dict(idx=P + 1), ALIGN),
    (dict(acc=P + 2), ALIGN), (dict(xs=(1024, 0, 68)), ALIGN), (dict(os=(1028, 0, 64)), ALIGN),
]


@pytest.mark.parametrize("kw,want", BAD_CONV, ids=[str(k) for k, _ in BAD_CONV])
def test_conv_refuses(lib, kw, want):
    assert conv(lib, **kw) == want


def test_conv_of_nothing(lib):
    assert conv(lib, B=0, x=None, w=None, pool=None, out=None, so=None) == OK


def rope(lib, **kw):
    a = dict(q=P, qs=None, k=P, ks=None, f=P, pos=P, dt=BF16, lens=P, factor=1.0, fl=0, B=2, Hq=4, Hk=2, T=3, D=128,
             R=64, qo=Q, qos=None, ko=Q, kos=None)
    a = with_strides({**a, **kw}, ("qs", "ks", "qos", "kos"))
    return lib.la_rope(a["q"], a["qs"], a["k"], a["ks"], a["f"], a["pos"], a["dt"], a["lens"], a["factor"], a["fl"],
                       a["B"], a["Hq"], a["Hk"], a["T"], a["D"], a["R"], a["qo"], a["qos"], a["ko"], a["kos"], None)


BAD_ROPE = [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(f=None), NULL), (dict(qo=None), NULL), (dict(ko=None), NULL),
    (dict(B=-1), SHAPE), (dict(Hq=-1), SHAPE), (dict(Hk=-1), SHAPE), (dict(T=-1), SHAPE), (dict(D=-8), SHAPE),
    (dict(R=-2), SHAPE), (dict(Hq=1 << 30, Hk=0x7FFFFFFF), SHAPE), (dict(B=1 << 23, T=100), SHAPE),
    (dict(qs=(-1, 128, 512)), SHAPE), (dict(qos=(1536, 64, 512)), SHAPE), (dict(kos=(0, 128, 256)), SHAPE),
    (dict(qo=P, qos=(1536, 128, 512)), SHAPE),  # in place with other strides
    (dict(ks=(1 << 61, 128, 256)), SHAPE),
    (dict(D=100), UNSUP), (dict(D=1032), UNSUP), (dict(R=63), UNSUP), (dict(R=130), UNSUP), (dict(fl=4), UNSUP),
    (dict(dt=MXI8), DTYPE), (dict(dt=9), DTYPE),
    (dict(q=P + 8), ALIGN), (dict(k=P + 2), ALIGN), (dict(qo=Q + 4), ALIGN), (dict(ko=Q + 8), ALIGN),
    (dict(f=P + 2), ALIGN), (dict(pos=P + 2), ALIGN), (dict(lens=P + 1), ALIGN), (dict(qs=(1536, 132, 512)), ALIGN),
]


@pytest.mark.parametrize("kw,want", BAD_ROPE, ids=[str(k) for k, _ in BAD_ROPE])
def test_rope_refuses(lib, kw, want):
    assert rope(lib, **kw) == want


@pytest.mark.parametrize("size", [dict(B=0), dict(T=0), dict(Hq=0, Hk=0), dict(D=0, R=0)], ids=str)
def test_rope_of_nothing(lib, size):
    assert rope(lib, **size, q=None, k=None, f=None, qo=None, ko=None) == OK


def scan(lib, fn="ssm_decode", **kw):
    a = dict(x=P, xs=None, dt=P, dts=None, A=P, Bm=P, Bs=None, Cm=P, Cs=None, D=P, z=P, zs=None, bias=P, ty=BF16,
             pool=P, st=F32, lens=P, idx=P, acc=P, fl=1, B=2, T=4, C=64, N=16, G=2, slots=5, out=Q, os=None, so=P,
             ws=None, wb=0)
    a = with_strides({**a, **kw}, ("xs", "dts", "Bs", "Cs", "zs", "os"))
    more = (a["ws"], a["wb"]) if fn == "ssm_prefill" else ()
    return getattr(lib, fn)(a["x"], a["xs"], a["dt"], a["dts"], a["A"], a["Bm"], a["Bs"], a["Cm"], a["Cs"], a["D"],
                            a["z"], a["zs"], a["bias"], a["ty"], a["pool"], a["st"], a["lens"], a["idx"], a["acc"],
                            a["fl"], a["B"], a["T"], a["C"], a["N"], a["G"], a["slots"], a["out"], a["os"], a["so"],
                            *more, None)


BAD_SCAN = [
    (dict(x=None), NULL), (dict(dt=None), NULL), (dict(A=None), NULL), (dict(Bm=None), NULL), (dict(Cm=None), NULL),
    (dict(pool=None), NULL), (dict(out=None), NULL), (dict(so=None), NULL),
    (dict(B=-1), SHAPE), (dict(T=0), SHAPE), (dict(C=0), SHAPE), (dict(N=0), SHAPE), (dict(G=0), SHAPE),
    (dict(G=3), SHAPE), (dict(slots=0), SHAPE), (dict(idx=None, slots=1), SHAPE),
    (dict(xs=(-256, 0, 64)), SHAPE), (dict(dts=(1 << 61, 0, 64)), SHAPE), (dict(Bs=(-8, 16, 32)), SHAPE),
    (dict(Cs=(1 << 61, 16, 32)), SHAPE), (dict(os=(256, 0, 32)), SHAPE), (dict(os=(0, 0, 64)), SHAPE),
    (dict(xs=(1 << 30, 0, (1 << 24) + 8)), SHAPE), (dict(Bs=(1 << 30, 16, (1 << 24) + 8)), SHAPE),
    (dict(B=1 << 24, C=1024, G=1), SHAPE),
    (dict(C=60), UNSUP), (dict(G=16), UNSUP), (dict(N=12), UNSUP), (dict(N=64), UNSUP), (dict(fl=2), UNSUP),
    (dict(ty=MXI8), DTYPE), (dict(ty=7), DTYPE), (dict(st=F16), DTYPE), (dict(st=MXI8), DTYPE),
    (dict(x=P + 8), ALIGN), (dict(dt=P + 2), ALIGN), (dict(A=P + 4), ALIGN), (dict(Bm=P + 8), ALIGN),
    (dict(Cm=P + 2), ALIGN), (dict(D=P + 4), ALIGN), (dict(z=P + 8), ALIGN), (dict(bias=P + 8), ALIGN),
    (dict(pool=P + 8), ALIGN), (dict(out=Q + 8), ALIGN), (dict(so=P + 4), ALIGN), (dict(lens=P + 2), ALIGN),
    (dict(acc=P + 2), ALIGN), (dict(xs=(256, 0, 68)), ALIGN), (dict(zs=(260, 0, 64)), ALIGN),
    (dict(Bs=(128, 20, 32)), ALIGN), (dict(Cs=(128, 16, 36)), ALIGN), (dict(os=(260, 0, 64)), ALIGN),
]


@pytest.mark.parametrize("fn", ["ssm_decode", "ssm_prefill"])
@pytest.mark.parametrize("kw,want", BAD_SCAN, ids=[str(k) for k, _ in BAD_SCAN])
def test_scan_refuses(lib, fn, kw, want):
    assert scan(lib, fn, **kw) == want


def test_scan_limits(lib):
    assert scan(lib, "ssm_decode", T=9) == SHAPE
    assert scan(lib, "ssm_prefill", T=65537) == SHAPE
    assert scan(lib, "ssm_prefill", ws=P + 128, wb=1 << 20) == ALIGN
    none = dict.fromkeys(("x", "dt", "A", "Bm", "Cm", "D", "z", "bias", "pool", "out", "so", "lens", "idx", "acc"))
    for fn in ("ssm_decode", "ssm_prefill"):
        assert scan(lib, fn, B=0, **none) == OK


def test_workspace_size_refuses(lib):
    n = C.c_size_t(7)
    size = lib.ssm_prefill_workspace_size
    assert size(1, 64, 64, 16, 1, None) == NULL
    for bad in ((1, 0, 64, 16, 1), (1, 65537, 64, 16, 1), (1, 64, 0, 16, 1), (1, 64, 64, 16, 3), (-1, 64, 64, 16, 1)):
        assert size(*bad, C.byref(n)) == SHAPE
    assert size(1, 64, 60, 16, 1, C.byref(n)) == UNSUP and size(1, 64, 64, 24, 1, C.byref(n)) == UNSUP
    assert size(0, 64, 64, 16, 1, C.byref(n)) == OK and n.value == 0


def test_quick_calls_leave_what_does_not_fit():
    """The CPython module takes no call whose tensors are not on a GPU, or are no tensors, and raises
    where it is called wrongly itself."""
    from gated_delta_rule_rgdr_amd import _la_binding as quick
    x, w, s = torch.zeros(1, 2, 64), torch.zeros(64, 4), torch.zeros(1, 3, 64)
    q, f = torch.zeros(1, 2, 3, 64), torch.zeros(32)
    b, h = torch.zeros(1, 2, 1, 16), torch.zeros(1, 64, 16)
    n3 = [None] * 3
    assert quick.conv(x, w, None, s, *n3, 0, None, s, 0) is None
    assert quick.conv(1, "w", None, s, *n3, 0, None, s, 0) is None
    assert quick.rope(q, q, f, None, None, 1.0, 0, None, None, 0) is None
    assert quick.rope(q, None, 3, None, None, 1.0, 0, None, None, 0) is None
    for prefill in (False, True):
        assert quick.scan(prefill, x, x, h[0], b, b, h, *n3, *n3, 1, None, h, None, 0) is None
        assert quick.scan(prefill, x, x, [], b, b, h, *n3, *n3, 1, None, h, None, 0) is None
    for bad in (lambda: quick.conv(x), lambda: quick.rope(), lambda: quick.scan(x),
                lambda: quick.conv(x, w, None, s, *n3, "0", None, s, 0),
                lambda: quick.rope(q, q, f, None, None, "1", 0, None, None, 0),
                lambda: quick.scan(True, x, x, h[0], b, b, h, *n3, *n3, 1, None, h, None, "0")):
        with pytest.raises(TypeError):
            bad()


def test_python_refuses_host_tensors():
    x, w, s = torch.zeros(1, 2, 64), torch.zeros(64, 4), torch.zeros(1, 3, 64)
    b, h = torch.zeros(1, 2, 1, 16), torch.zeros(1, 64, 16)
    for call in (lambda: rg.la_conv(x, w, s), lambda: rg.la_rope(torch.zeros(1, 2, 3, 64), None, torch.zeros(32)),
                 lambda: rg.ssm_decode(x, x, h[0], b, b, h), lambda: rg.ssm_prefill(x, x, h[0], b, b, h)):
        with pytest.raises(RuntimeError, match="on the GPU"):
            call()
    for call in (lambda: rg.la_conv([1.0], w, s), lambda: rg.la_rope(3, None, w), lambda: rg.ssm_decode(None, x, w, b, b, h)):
        with pytest.raises(TypeError):
            call()


def test_rope_frequencies_of_long_contexts():
    """Where every pair turns often enough, none is divided; where none does, all are; and the ends of the
    range between."""
    i = torch.arange(16, dtype=torch.float64)
    plain = 10000.0 ** (-i / 16)

    def ratio(length):
        freq, factor = rg.la_rope_frequencies(32, scaling="blend", scale=8.0, original_length=length, device="cpu")
        assert abs(factor - 1.2079441541679836) < 1e-12  # 0.1 ln 8 + 1
        return freq.double() / plain
    few = ratio(4)        # pair 0 turns 4 / (2 pi) times
    assert torch.allclose(few, torch.full_like(few, 0.125), rtol=1e-6)
    many = ratio(10 ** 9)
    assert torch.allclose(many, torch.ones_like(many), rtol=1e-6)
    some = ratio(4096)
    turns = 4096 * plain / (2 * torch.pi)
    # the range between is widened to whole pairs, neighbours of which turn 1.78 times as often
    assert torch.all(some[turns > 32 * 1.8] > 0.999) and torch.all(some[turns < 1 / 1.8] < 0.1251)
    assert torch.all(some[1:] <= some[:-1] + 1e-6)
