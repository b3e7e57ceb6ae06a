"""Plain 64-bit references, on the CPU, of the short convolution, rotary positions and the state space
scan, each with the bound on what fp32 arithmetic may differ from it.

u = 2^-24 is half a step of fp32 (relative). Bounds count roundings to first order, each term doubled
where a step's own slope could matter:

* exp(x) as exp2(x log2 e): the product's rounding moves the argument by |x| u twice (the constant's and
  its own), exp2 itself is good to 2 u: (2 |x| + 4) u relative.
* sigmoid(z) = 1 / (1 + exp(-z)): the exponential's error above weighed by at most 1, the sum's and the
  reciprocal's roundings: (2 |z| + 8) u relative. silu(z) = z sigmoid(z): (2 |z| + 9) u; its slope is
  below 1.1.
* softplus(s) = max(s, 0) + log1p(exp(-|s|)), s = dt + dt_bias: the sum's rounding moves s by |s| u,
  which moves exp(s) by as much relative; with the exponential's own error and a few more roundings:
  (3 |s| + 16) u relative.
* the state: see scan().

A stored value is off by at most half a step of its type more.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def clamp(lens, idx, acc, b, T, N):
    """Valid and accepted tokens of an entry; None for a slot out of range."""
    if not 0 <= int(idx[b]) < N:
        return None
    L = min(max(int(lens[b]), 0), T)
    return L, min(max(int(acc[b]), 0), L)


def silu(y, err):
    """silu(y) and the bound on its value in fp32 for an argument that is off by err."""
    s = y * torch.sigmoid(y)
    return s, 1.1 * err + (2 * y.abs() + 9) * U * s.abs()


def conv(x, w, bias, pool, lens, idx, acc, act):
    """out, its bound before the store, and the pool after the call."""
    B, T, C = x.shape
    W = w.shape[1]
    x, w = x.double().cpu(), w.double().cpu()
    bias = torch.zeros(C, dtype=torch.float64) if bias is None else bias.double().cpu()
    after = pool.double().cpu().clone()
    out = torch.zeros(B, T, C, dtype=torch.float64)
    err = torch.zeros_like(out)
    for b in range(B):
        e = clamp(lens, idx, acc, b, T, pool.shape[0])
        if e is None:
            continue
        L, n = e
        slot = int(idx[b])
        line = torch.cat([pool[slot].double().cpu(), x[b]])
        for t in range(L):
            terms = line[t:t + W] * w.T
            y = bias + terms.sum(0)
            # W products and sums, each rounded once at most to a share of the terms' magnitudes
            r = (W + 1) * U * (bias.abs() + terms.abs().sum(0))
            out[b, t], err[b, t] = silu(y, r) if act else (y, r)
        after[slot] = line[n:n + W - 1]
    return out, err, after


def rope(x, freq, pos, factor, interleaved, lens):
    """One operand's output and its bound before the store. An angle's turns are off by 2^-26 (32 bits
    of at most half a turn) and sine and cosine by 2 u, together 2^-22; two products, a sum and the
    factor's rounding add 4 u of the terms: 2^-21. The 64-bit product and this reference's own add the
    angle's 2^-51."""
    B, H, T, D = x.shape
    half = freq.shape[0]
    x = x.double().cpu()
    pos = torch.zeros(B) if pos is None else pos.cpu()
    pos = pos.double()[:, None] + torch.arange(T) if pos.dim() == 1 else pos.double()
    angle = (pos[..., None] * freq.double().cpu())[:, None]
    cos, sin = torch.cos(angle) * factor, torch.sin(angle) * factor
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    out, err = x.clone(), torch.zeros_like(x)
    p, q = x[..., first], x[..., second]
    out[..., first], out[..., second] = p * cos - q * sin, p * sin + q * cos
    err[..., first] = err[..., second] = (p.abs() + q.abs()) * abs(factor) * (2.0 ** -21 + angle.abs() * 2.0 ** -51)
    for b in range(B):
        n = min(max(int(lens[b]), 0), T)
        out[b, :, n:] = err[b, :, n:] = 0
    return out, err


def scan(x, dt, A, Bm, Cm, pool, lens, idx, acc, D, z, dt_bias, softplus=True):
    """out and its bound before the store, each entry's state (None: slot out of range) and its bound
    before the store.

    M is the recurrence on magnitudes. A step's decay a = exp(d A) is off by (|d A| r + 4 u) relative,
    r the relative error of d and of its products; where tokens are taken together, the decay over
    several is that of a sum of d, off by at most (4 + T / 16) u relative (sums of at most 64 terms
    and of the sums), which adds |d A| (4 + T / 16) u for each step. The new term is off by r + 4 u
    of it, and storing the sum in fp32, also where a state is taken from one part of the tokens to the
    next, by 3 u of M."""
    B, T, C = x.shape
    N = A.shape[1]
    G = Bm.shape[2]
    group = torch.arange(C) // (C // G)
    x, dt, A, Bm, Cm = (v.double().cpu() for v in (x, dt, A, Bm, Cm))
    s = dt if dt_bias is None else dt + dt_bias.double().cpu()
    d_all = torch.logaddexp(s, torch.zeros_like(s)) if softplus else s
    out = torch.zeros(B, T, C, dtype=torch.float64)
    err = torch.zeros_like(out)
    states, serrs = [], []
    for b in range(B):
        e = clamp(lens, idx, acc, b, T, pool.shape[0])
        if e is None:
            states.append(None)
            serrs.append(None)
            continue
        L, n = e
        h = pool[int(idx[b])].double().cpu()
        M, E = h.abs(), torch.zeros_like(h)
        kept, kerr = h, E
        for t in range(L):
            d = d_all[b, t][:, None]
            r = (3 * s[b, t].abs()[:, None] + 16) * U
            da = (d * A).abs()
            a = torch.exp(d * A)
            new = d * x[b, t][:, None] * Bm[b, t, group]
            h = a * h + new
            E = a * E + a * M * (da * (r + (8 + T / 16) * U) + 4 * U) + new.abs() * (r + 4 * U)
            M = a * M + new.abs()
            E = E + 3 * U * M
            c = Cm[b, t, group]
            y = (c * h).sum(1)
            r = (c.abs() * E).sum(1) + (N + 4) * U * (c.abs() * M).sum(1)
            if D is not None:
                skip = D.double().cpu() * x[b, t]
                y, r = y + skip, r + 2 * U * (skip.abs() + y.abs())
            if z is not None:
                zz = z[b, t].double().cpu()
                gate, gerr = silu(zz, 0.0)
                y, r = y * gate, r * gate.abs() + y.abs() * gerr + 2 * U * (y * gate).abs()
            out[b, t], err[b, t] = y, r
            if t + 1 == n:
                kept, kerr = h, E
        states.append(kept)
        serrs.append(kerr)
    return out, err, states, serrs


def check(got, ref, err, tag):
    dtype = got.dtype
    got = got.double().cpu()
    assert not torch.isnan(got).any(), f"{tag}: NaN"
    bound = HALF[dtype] * ref.abs() + err * (1 + 2 * HALF[dtype]) + TINY[dtype]
    over = (got - ref).abs() - bound
    assert over.max() <= 0, f"{tag}: off by {over.max():.3g} more than its bound"


def zero_bits(t):
    return bool(np.all(t.contiguous().cpu().view(torch.uint8).numpy() == 0))
