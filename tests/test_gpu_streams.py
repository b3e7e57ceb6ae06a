"""Calls on a stream of their own, behind a long piece of work on it: every tensor that was made for the call is
dropped when it returns, and new ones of the same sizes are made and filled on the current stream while it waits."""
import numpy as np
import pytest
import torch

import workloads
from gpu_util import gate_tensors, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_rgdr_amd as m
    m.library()
    return m


def scan_inputs(fn):
    B, T, C, N = 3, 6 if fn == "ssm_decode" else 700, 64, 16
    r = torch.Generator().manual_seed(1)
    x, dt, z = (torch.randn(B, T, C, generator=r) for _ in range(3))
    Bm, Cm = (torch.randn(B, T, 1, N, generator=r) for _ in range(2))
    A, D, bias = -torch.rand(C, N, generator=r), torch.randn(C, generator=r), torch.randn(C, generator=r) - 3
    lens, idx, acc = (torch.tensor(v, dtype=torch.int32) for v in ([T, T - 2, 1], [4, 0, 2], [T, 1, 1]))
    return (x, dt, A, Bm, Cm, torch.randn(5, C, N, generator=r), lens, idx, acc), dict(D=D, z=z, dt_bias=bias)


def attention_inputs(fn):
    B, T = 2, 4 if fn == "la_decode" else 900
    r = torch.Generator().manual_seed(2)
    q, k = (torch.nn.functional.normalize(torch.randn(B, 2, T, 64, generator=r), dim=-1).bfloat16() for _ in range(2))
    v, g = torch.randn(B, 4, T, 64, generator=r).bfloat16(), -torch.rand(B, 4, T, generator=r)
    lens, idx, acc = (torch.tensor(v, dtype=torch.int32) for v in ([T, T - 1], [2, 0], [T, 2]))
    return (q, k, v, g, torch.randn(3, 4, 64, 64, generator=r), lens, idx, acc), {}


def rgdr_inputs(fn):
    T = 900 if "prefill" in fn else 3
    inp = workloads.make_case(2, 2, 4, T, 128, 128, 4, seed=9, indices="choice", lengths="uniform", gate="gated" in fn)
    inp.num_accepted_tokens = np.maximum(1, inp.actual_seq_lengths // 2).astype(np.int32)
    d = {k: v.cpu() for k, v in upload(inp).items()}
    if "gated" in fn:
        gate = [t.cpu() for t in gate_tensors(inp)]
        names = ("state", "actual_seq_lengths", "ssm_state_indices", "gk", "num_accepted_tokens")
        return (d["query"], d["key"], d["value"], *gate, *(d[n] for n in names)), {}
    names = ("query", "key", "value", "beta", "state", "actual_seq_lengths", "ssm_state_indices", "g", "gk",
             "num_accepted_tokens")
    return tuple(d[n] for n in names), {}


def inputs(fn):
    r = torch.Generator().manual_seed(3)
    if fn.startswith("ssm"):
        return scan_inputs(fn)
    if fn.startswith("rgdr"):
        return rgdr_inputs(fn)
    if fn in ("la_decode", "la_prefill"):
        return attention_inputs(fn)
    if fn == "la_conv":
        idx = torch.tensor([3, 1], dtype=torch.int32)
        return (torch.randn(2, 50, 64, generator=r), torch.randn(64, 4, generator=r), torch.randn(4, 3, 64, generator=r),
                None, idx), dict(bias=torch.randn(64, generator=r))
    if fn == "la_rope":
        x = torch.randn(2, 3, 40, 64, generator=r)
        return (x, x.flip(1), torch.rand(32, generator=r), torch.tensor([7, 1000], dtype=torch.int32)), {}
    if fn == "la_norm_gate":
        return (torch.randn(2, 3, 40, 64, generator=r), torch.rand(64, generator=r),
                torch.randn(2, 40, 3, 64, generator=r)), {}
    if fn == "la_gate":
        return (torch.randn(2, 30, 8, generator=r), torch.randn(8, generator=r), torch.randn(8, generator=r),
                torch.randn(2, 30, 8, generator=r)), {}
    assert fn == "la_state_quantize"
    return (torch.randn(4, 2, 64, 64, generator=r),), dict(src_slots=torch.tensor([3, 1], dtype=torch.int32))


FUNCTIONS = ["ssm_decode", "ssm_prefill", "la_conv", "la_rope", "la_norm_gate", "la_gate", "la_state_quantize",
             "la_decode", "la_prefill", "rgdr_decode", "rgdr_decode_snapshots", "rgdr_decode_gated", "rgdr_prefill",
             "rgdr_prefill_ws", "rgdr_prefill_gated_ws"]


def keep_busy(stream, work, times):
    with torch.cuda.stream(stream):
        for _ in range(times):  # 0.4 ms each
            work.mul_(1.0)


@pytest.fixture(scope="module")
def beside():
    """A stream whose work the current one's does not wait for (streams share a few hardware queues)."""
    work = torch.ones(1 << 28, device="cuda")
    for _ in range(16):
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        keep_busy(s, work, 20)
        for _ in range(4):
            torch.ones(1000).cuda().add_(1).cpu()
        if not s.query():
            torch.cuda.synchronize()
            return s
    raise AssertionError("no stream runs beside the current one")


@pytest.mark.parametrize("fn", FUNCTIONS)
@pytest.mark.parametrize("foreign", [False, True], ids=["torch", "handle"])
def test_dropped_tensors(rg, beside, fn, foreign):
    args, kw = inputs(fn)

    def gpu(t):
        return t.cuda() if isinstance(t, torch.Tensor) else t

    def call(stream=None):
        out = getattr(rg, fn)(*map(gpu, args), **{k: gpu(v) for k, v in kw.items()}, stream=stream)
        return out if isinstance(out, tuple) else (out,)
    slots = [t for t in args if isinstance(t, torch.Tensor) and t.dtype == torch.int32]
    assert all(int(t.min()) >= 0 for t in slots)
    want = [t.clone() for t in call() if t is not None]
    torch.cuda.synchronize()
    work, s = torch.ones(1 << 28, device="cuda"), beside  # 1 GiB
    handle = type("Handle", (), {"cuda_stream": s.cuda_stream})() if foreign else s
    for times in (100, 400, 1600):
        keep_busy(s, work, times)
        got = [t for t in call(handle) if t is not None]
        again = [torch.zeros_like(gpu(t)) for t in (*args, *kw.values()) if isinstance(t, torch.Tensor) for _ in range(3)]
        again += [torch.zeros(t.numel(), dtype=torch.uint8, device="cuda") for t in got]
        waited = not s.query()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            if fn == "rgdr_decode_snapshots" and a.dim() == 5:
                continue  # entries past a sequence's length keep what the buffer held
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), fn
        del again, got
        if waited:
            return
    pytest.skip("the work before the call was over too soon")


POOL = {"ssm_prefill": 5, "la_conv": 2, "la_rope": None, "la_prefill": 4, "rgdr_prefill_ws": 4}  # the states' argument


@pytest.mark.parametrize("fn", POOL)
def test_captured_on_its_own_stream(rg, fn):
    """The stream given is the one that captures: tensors made and dropped within the capture, four replays with
    eager work between them."""
    args, kw = inputs(fn)

    def gpu(t):
        return t.cuda() if isinstance(t, torch.Tensor) else t
    fixed, kw = [gpu(t) for t in args], {k: gpu(v) for k, v in kw.items()}
    pool_at = POOL[fn]

    def call(stream, pool):
        now = list(fixed)
        if pool_at is not None:
            now[pool_at] = pool
        now[0] = now[0] + 0  # a tensor of the capture's own
        out = getattr(rg, fn)(*now, **kw, stream=stream)
        return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    first = fixed[pool_at].clone() if pool_at is not None else None
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pool = first.clone() if first is not None else None
    with torch.cuda.stream(s):
        want = [t.clone() for t in call(s, pool)]
    torch.cuda.synchronize()
    if pool is not None:
        pool.copy_(first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = call(s, pool)
    for k in range(4):
        if pool is not None:
            pool.copy_(first)
        for t in got:
            if pool is None or t.data_ptr() != pool.data_ptr():
                t.zero_()
        torch.ones(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k
