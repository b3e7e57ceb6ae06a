"""The linear-attention entry points without a GPU: every refusal happens on the host, before
anything is launched, so the made-up addresses are never used."""
import ctypes as C

import pytest
import torch

import gated_delta_rule_rgdr_amd as rg

OK, NULL, SHAPE, UNSUP, RANGE, DUP, DTYPE, HIP, ALIGN = range(9)
F32, F16, BF16, MXI8 = range(4)
P = 0x100000


@pytest.fixture(scope="module")
def lib():
    return rg.library()


def strides(*x):
    return None if x == (None,) else rg._Strides(*x)


def attention(lib, fn="la_decode", **kw):
    a = dict(q=P, qs=None, k=P, ks=None, v=P, vs=None, g=P, gs=None, pool=P, sc=P, dt=BF16,
             lens=P, idx=P, acc=P, B=2, Hq=2, Hv=4, T=4, Dk=128, Dv=128, N=5, out=P, os=None,
             so=P, sco=P, ws=None, wb=0)
    a.update(kw)
    for s in ("qs", "ks", "vs", "gs", "os"):
        if a[s] is not None:
            a[s] = strides(*a[s])
    more = (a["ws"], a["wb"]) if fn == "la_prefill" else ()
    return getattr(lib, fn)(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["g"], a["gs"],
                            a["pool"], a["sc"], a["dt"], a["lens"], a["idx"], a["acc"], 1.0,
                            a["B"], a["Hq"], a["Hv"], a["T"], a["Dk"], a["Dv"], a["N"], a["out"],
                            a["os"], a["so"], a["sco"], *more, None)


BAD_ATTENTION = [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(g=None), NULL),
    (dict(pool=None), NULL), (dict(out=None), NULL), (dict(so=None), NULL),
    (dict(dt=MXI8, sc=None), NULL), (dict(dt=MXI8, sco=None), NULL),
    (dict(B=-1), SHAPE), (dict(T=0), SHAPE), (dict(T=-3), SHAPE), (dict(Hq=0), SHAPE),
    (dict(Hq=3), SHAPE), (dict(Hq=8), SHAPE), (dict(Hv=0), SHAPE), (dict(N=0), SHAPE),
    (dict(idx=None, N=1), SHAPE),              # entry b in slot b needs B slots
    (dict(Dk=96), UNSUP), (dict(Dk=32), UNSUP), (dict(Dv=48), UNSUP), (dict(Dv=4128), UNSUP),
    (dict(dt=F16), DTYPE), (dict(dt=7), DTYPE),
    (dict(q=P + 8), ALIGN), (dict(k=P + 2), ALIGN), (dict(v=P + 4), ALIGN), (dict(g=P + 2), ALIGN),
    (dict(pool=P + 8), ALIGN), (dict(so=P + 8), ALIGN), (dict(out=P + 2), ALIGN),
    (dict(dt=MXI8, sc=P + 4), ALIGN), (dict(lens=P + 1), ALIGN), (dict(acc=P + 2), ALIGN),
    (dict(qs=(1 << 20, 1 << 10, 132)), ALIGN),  # rows not at multiples of 8 elements
    (dict(vs=(1 << 20, 4, 128)), ALIGN),
    (dict(qs=(1 << 20, 1 << 10, -128)), SHAPE),
    (dict(gs=(-4, 4, 1)), SHAPE),
    (dict(ks=(1 << 30, 128, (1 << 24) + 8)), SHAPE),
    (dict(os=(1 << 20, 1 << 10, 64)), SHAPE),   # out rows on top of each other
    (dict(os=(0, 1 << 10, 128)), SHAPE),
    (dict(os=(2048, 128, 256)), SHAPE),         # head 2 of token 0 is head 0 of token 1
    (dict(qs=(1 << 61, 1 << 10, 128)), SHAPE),  # past any address
    (dict(B=1 << 20, Hv=1 << 12, Hq=1 << 12), SHAPE),
    (dict(B=1 << 17, Hv=1 << 7, Hq=1, Dv=128, idx=P, N=4), SHAPE),  # 2^24 workgroups of 256
]


@pytest.mark.parametrize("fn", ["la_decode", "la_prefill"])
@pytest.mark.parametrize("kw,want", BAD_ATTENTION, ids=[str(k) for k, _ in BAD_ATTENTION])
def test_attention_refuses(lib, fn, kw, want):
    assert attention(lib, fn, **kw) == want


def test_attention_limits(lib):
    assert attention(lib, "la_decode", T=9) == SHAPE
    assert attention(lib, "la_prefill", T=65537) == SHAPE
    assert attention(lib, "la_prefill", ws=P + 128, wb=1 << 20) == ALIGN
    # an empty batch: no pointer is looked at
    none = dict.fromkeys(("q", "k", "v", "g", "pool", "sc", "out", "so", "sco", "lens", "idx", "acc"))
    for fn in ("la_decode", "la_prefill"):
        assert attention(lib, fn, B=0, **none) == OK


def test_workspace_size_refuses(lib):
    n = C.c_size_t(7)
    assert lib.la_prefill_workspace_size(1, 4, 64, 128, 128, None) == NULL
    assert lib.la_prefill_workspace_size(1, 0, 64, 128, 128, C.byref(n)) == SHAPE
    assert lib.la_prefill_workspace_size(1, 4, 65537, 128, 128, C.byref(n)) == SHAPE
    assert lib.la_prefill_workspace_size(1, 4, 64, 100, 128, C.byref(n)) == UNSUP
    assert lib.la_prefill_workspace_size(0, 4, 64, 128, 128, C.byref(n)) == OK and n.value == 0


def quantize(lib, back=False, **kw):
    a = dict(x=P, dt=F32, Ns=4, src=P, codes=P, sc=P, Nd=4, dst=P, n=3, H=2, Dk=64, Dv=64)
    a.update(kw)
    if back:
        return lib.la_state_dequantize(a["codes"], a["sc"], a["Ns"], a["src"], a["x"], a["dt"],
                                       a["Nd"], a["dst"], a["n"], a["H"], a["Dk"], a["Dv"], None)
    return lib.la_state_quantize(a["x"], a["dt"], a["Ns"], a["src"], a["codes"], a["sc"], a["Nd"],
                                 a["dst"], a["n"], a["H"], a["Dk"], a["Dv"], None)


BAD_MOVE = [
    (dict(x=None), NULL), (dict(codes=None), NULL), (dict(sc=None), NULL),
    (dict(n=-1), SHAPE), (dict(H=0), SHAPE), (dict(Dk=0), SHAPE), (dict(Dv=0), SHAPE),
    (dict(Ns=0), SHAPE), (dict(Nd=0), SHAPE), (dict(src=None, Ns=2), SHAPE),
    (dict(dst=None, Nd=2), SHAPE), (dict(H=1 << 30, Dk=1 << 30, Dv=32), SHAPE),
    (dict(n=1 << 24), SHAPE),
    (dict(Dv=40), UNSUP), (dict(dt=F16), DTYPE), (dict(dt=MXI8), DTYPE),
    (dict(x=P + 8), ALIGN), (dict(codes=P + 4), ALIGN), (dict(sc=P + 1), ALIGN),
    (dict(src=P + 2), ALIGN), (dict(dst=P + 2), ALIGN),
]


@pytest.mark.parametrize("back", [False, True], ids=["quantize", "dequantize"])
@pytest.mark.parametrize("kw,want", BAD_MOVE, ids=[str(k) for k, _ in BAD_MOVE])
def test_state_moves_refuse(lib, back, kw, want):
    assert quantize(lib, back, **kw) == want


def test_state_moves_of_nothing(lib):
    for back in (False, True):
        assert quantize(lib, back, n=0, x=None, codes=None, sc=None, src=None, dst=None) == OK


def norm(lib, **kw):
    a = dict(x=P, xs=None, gate=P, gs=None, w=P, ws=0, dt=BF16, lens=P, eps=1e-6, fl=0, B=2, H=4,
             T=3, D=128, out=P, os=None)
    a.update(kw)
    for s in ("xs", "gs", "os"):
        if a[s] is not None:
            a[s] = strides(*a[s])
    return lib.la_norm_gate(a["x"], a["xs"], a["gate"], a["gs"], a["w"], a["ws"], a["dt"],
                            a["lens"], a["eps"], a["fl"], a["B"], a["H"], a["T"], a["D"], a["out"],
                            a["os"], None)


BAD_NORM = [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL),
    (dict(B=-1), SHAPE), (dict(H=-1), SHAPE), (dict(T=-1), SHAPE), (dict(D=-8), SHAPE),
    (dict(eps=-1e-6), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(B=1 << 24, H=32, lens=None), SHAPE),
    (dict(xs=(-1, 1, 1)), SHAPE), (dict(ws=-4), SHAPE), (dict(os=(1536, 128, 128)), SHAPE),
    (dict(D=100), UNSUP), (dict(D=8200), UNSUP), (dict(fl=2), UNSUP),
    (dict(dt=MXI8), DTYPE), (dict(dt=9), DTYPE),
    (dict(x=P + 8), ALIGN), (dict(gate=P + 2), ALIGN), (dict(w=P + 4), ALIGN),
    (dict(out=P + 4), ALIGN), (dict(xs=(4096, 1024, 132)), ALIGN), (dict(ws=130), ALIGN),
    (dict(lens=P + 2), ALIGN),
]


@pytest.mark.parametrize("kw,want", BAD_NORM, ids=[str(k) for k, _ in BAD_NORM])
def test_norm_gate_refuses(lib, kw, want):
    assert norm(lib, **kw) == want


@pytest.mark.parametrize("size", ["B", "H", "T", "D"])
def test_norm_gate_of_nothing(lib, size):
    assert norm(lib, **{size: 0}, x=None, w=None, out=None, gate=None, lens=None) == OK


def test_quick_calls_leave_what_does_not_fit():
    """The CPython module takes no call whose tensors are not on a GPU, or are no tensors, and
    raises where it is called wrongly itself."""
    from gated_delta_rule_rgdr_amd import _la_binding as quick
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    g, s = torch.zeros(1, 2, 3), torch.zeros(1, 2, 64, 64)
    none = [None] * 4
    assert quick.attention(False, x, x, x, g, s, *none, 1.0, None, s, None, None, 0) is None
    assert quick.attention(True, 1, "q", x, g, s, *none, 1.0, None, s, None, None, 0) is None
    assert quick.move(False, s, s.to(torch.int8), s, None, None, 1, 0) is None
    assert quick.norm_gate(x, torch.ones(64), None, 1e-6, 0, None, None, 0) is None
    for bad in (lambda: quick.attention(1), lambda: quick.move(), lambda: quick.norm_gate(x),
                lambda: quick.attention(False, x, x, x, g, s, *none, "1", None, s, None, None, 0),
                lambda: quick.norm_gate(x, x, None, "eps", 0, None, None, 0)):
        with pytest.raises(TypeError):
            bad()


def test_python_refuses_host_tensors():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    s = torch.zeros(1, 2, 64, 64)
    with pytest.raises(RuntimeError, match="on the GPU"):
        rg.la_decode(x, x, x, torch.zeros(1, 2, 3), s)
    with pytest.raises(RuntimeError, match="on the GPU"):
        rg.la_prefill(x, x, x, torch.zeros(1, 2, 3), s)
    with pytest.raises(RuntimeError, match="on the GPU"):
        rg.la_state_quantize(s)
    with pytest.raises(RuntimeError, match="on the GPU"):
        rg.la_state_dequantize(s.to(torch.int8), s)
    with pytest.raises(RuntimeError, match="on the GPU"):
        rg.la_norm_gate(x, torch.ones(64))
    with pytest.raises(TypeError):
        rg.la_decode([1.0], x, x, s, s)
    with pytest.raises(RuntimeError, match="float32 or bfloat16"):
        rg.la_state_quantize(s.to(torch.int8))
