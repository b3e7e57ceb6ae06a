"""Plain 64-bit references, on the CPU, of the linear-attention operators, and the bounds that
their tests use.

Bounds. A is the same sum with every term's magnitude (abs recurrence on |q|, |k|, |v|, |S|).
fp32 arithmetic over T tokens and D_k rows costs at most about one unit of 2^-24 of A for each of
the T decays (twice: the exponential and the product) and each addition: (3 T + D_k + 64) 2^-24 A.
Where a kernel's matrix products take an operand as the sum of two bf16 numbers, that sum is off
by at most 2^-8 * 2^-8 of the operand; at most two operands of a product are split: 2^-15 A.
A stored bf16 value is off by at most 2^-8 of it more (half a step), an 8-bit code by half the
block's step.
"""
import numpy as np
import torch

BF16_HALF = 2.0 ** -8  # torch.finfo(torch.bfloat16).eps / 2
F16_HALF = 2.0 ** -11


def c_out(T, Dk):
    return 2.0 ** -15 + (3 * T + Dk + 64) * 2.0 ** -24


def c_state(T):
    return (3 * T + 64) * 2.0 ** -24


def attention(q, k, v, g, S0, lens, idx, acc, scale):
    """Token by token. Returns out, state after the accepted tokens for each entry (None where
    the slot is out of range), and the same two with every term's magnitude."""
    q, k, v, g = (x.double().cpu() for x in (q, k, v, g))
    B, Hq, T, Dk = q.shape
    Hv, Dv = v.shape[1], v.shape[3]
    N = S0.shape[0]
    head = torch.arange(Hv) // (Hv // Hq)
    out = torch.zeros(B, Hv, T, Dv, dtype=torch.float64)
    mag = torch.zeros_like(out)
    states, smags = [], []
    scale = float(np.float32(scale))
    for b in range(B):
        slot = int(idx[b])
        if not 0 <= slot < N:
            states.append(None)
            smags.append(None)
            continue
        L = min(max(int(lens[b]), 0), T)
        n = min(max(int(acc[b]), 0), L)
        S = S0[slot].double().cpu().clone()
        A = S.abs()
        kept, kmag = S.clone(), A.clone()
        for t in range(L):
            d = torch.exp(g[b, :, t])[:, None, None]
            kt, qt, vt = k[b, head, t], q[b, head, t] * scale, v[b, :, t]
            S = d * S + kt[:, :, None] * vt[:, None, :]
            A = d * A + (kt[:, :, None] * vt[:, None, :]).abs()
            out[b, :, t] = (qt[:, :, None] * S).sum(1)
            mag[b, :, t] = (qt.abs()[:, :, None] * A).sum(1)
            if t + 1 == n:
                kept, kmag = S.clone(), A.clone()
        states.append(kept)
        smags.append(kmag)
    return out, states, mag, smags


def mx_values(codes, scales):
    """What the codes and scale bytes stand for, in 64 bits."""
    e = scales.cpu().double() - 127
    s = torch.exp2(e)
    s = torch.where(scales.cpu() == 255, torch.full_like(s, float("nan")), s)
    return codes.cpu().double() * s.repeat_interleave(32, -1)


def mx_step(x):
    """The step 2^e of each value's block of 32, by trying the exponents in turn."""
    blocks = x.double().cpu().reshape(-1, 32)
    top = blocks.abs().amax(1)
    e = torch.full_like(top, -127.0)
    for n in range(-127, 123):
        e = torch.where(top > 127 * torch.exp2(e), torch.full_like(e, n + 1.0), e)
    return torch.exp2(e)[:, None].expand(-1, 32).reshape(x.shape)


def check_out(got, ref, mag, T, Dk, tag):
    got = got.double().cpu()
    bound = BF16_HALF * ref.abs() + c_out(T, Dk) * mag * (1 + BF16_HALF)
    over = (got - ref).abs() - bound
    assert not torch.isnan(got).any(), f"{tag}: NaN in out"
    assert over.max() <= 0, f"{tag}: out off by {over.max():.3g} more than its bound"


def check_state(got, ref, mag, T, dtype, tag):
    """One entry's committed state against its reference."""
    got = got.double().cpu()
    slack = c_state(T) * mag
    if dtype == torch.float32:
        bound = slack
    elif dtype == torch.bfloat16:
        bound = BF16_HALF * ref.abs() + slack * (1 + BF16_HALF)
    else:
        bound = mx_step(ref.abs() + slack) / 2 + slack
    over = (got - ref).abs() - bound
    assert over.max() <= 0, f"{tag}: state off by {over.max():.3g} more than its bound"
