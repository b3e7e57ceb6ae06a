"""Measured cases of the operators in front of the recurrences, and of the selective state space scan.

* ``la_conv``: the short causal convolution behind an input projection. For channel c and token t,
  with W taps, the last one on the token itself, and the tokens before the call from a pool:

      y[t,c] = silu(bias[c] + sum_j weight[c,j] x[t - W + 1 + j, c])

* ``la_rope``: rotary positions of queries and keys. Pair i of the head's first R columns (columns
  i and i + R/2, or 2i and 2i + 1 when interleaved) is turned by position * inv_freq[i]; cosine and
  sine are multiplied by a factor.
* ``ssm_decode`` (T <= 8) and ``ssm_prefill``: the selective state space scan, on a pool of states of N
  values for each channel; B and C are shared by the channels of a group:

      d = softplus(dt[t,c] + dt_bias[c])
      h[c,n] = exp(d A[c,n]) h[c,n] + d B[t,n] x[t,c]
      y[t,c] = (sum_n C[t,n] h[c,n] + D[c] x[t,c]) silu(z[t,c])

Lengths, slots and accepted tokens are int32 [B]: a sequence's tokens past its length give zeros, and
what is kept in its slot is what it is after its accepted tokens.

Where ``own`` is false, ``run`` computes the plain forms: elementary torch operations in fp32 (angles
in fp64), rounded once at the end.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
PLAIN_CHUNK = 64  # tokens whose decays the plain form of the scan computes at once


# ---- cases -----------------------------------------------------------------------------------

def _conv(name, B, T, C, W, dtype, ragged=False, silu=True, bias=True, sliced=False):
    case = {"op": "conv", "B": B, "T": T, "C": C, "W": W, "dtype": dtype, "ragged": ragged,
            "silu": silu, "bias": bias, "sliced": sliced}
    return {"name": name, **case} if name else case


def _rope(name, B, T, Hq, Hk, D, R, dtype, interleaved=False, first=0, factor=1.0, ragged=False,
          layout="bthd"):
    case = {"op": "rope", "B": B, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "dtype": dtype,
            "interleaved": interleaved, "first": first, "factor": factor, "ragged": ragged,
            "layout": layout}
    return {"name": name, **case} if name else case


def _ssm(name, op, B, T, C, N, G, dtype, state, ragged=False, gated=True):
    case = {"op": op, "B": B, "T": T, "C": C, "N": N, "G": G, "dtype": dtype, "state": state,
            "ragged": ragged, "gated": gated}
    return {"name": name, **case} if name else case


def listed():
    return [
        # One user's next token, queries, keys and values of a layer side by side: latency alone.
        _conv("conv_one_token", 1, 1, 8192, 4, "bf16"),
        # Speculative decoding: up to 8 drafted tokens of each sequence, some rejected.
        _conv("conv_drafted_tokens", 64, 8, 8192, 4, "bf16", True, sliced=True),
        # A batch of prompts of different lengths.
        _conv("conv_prompts", 16, 1024, 8192, 4, "bf16", True),
        # One user's next token, far into its text.
        _rope("rope_one_token", 1, 1, 16, 16, 128, 128, "bf16", first=30000),
        # A batch of prompts, queries and keys as slices of one projection.
        _rope("rope_prompts", 16, 1024, 16, 16, 128, 128, "bf16", ragged=True),
        # A piece of a very long text: part of the head, interleaved, scaled frequencies.
        _rope("rope_long_context", 1, 8192, 32, 8, 128, 64, "f16", True, 1000000, 1.2, layout="bhtd"),
        # One user's next token.
        _ssm("ssm_one_token", "ssm_decode", 1, 1, 4096, 16, 1, "bf16", "f32"),
        # A full serving batch.
        _ssm("ssm_decode_batch", "ssm_decode", 256, 1, 4096, 16, 1, "bf16", "f32"),
        # Speculative decoding on states held in 16 bits, eight groups of channels.
        _ssm("ssm_drafted_tokens", "ssm_decode", 32, 8, 4096, 16, 8, "f16", "bf16", True),
        # A few short, odd prompts in 32 bits.
        _ssm("ssm_short_odd", "ssm_prefill", 3, 77, 1048, 16, 1, "f32", "f32", True),
        # A batch of prompts of different lengths.
        _ssm("ssm_prompts", "ssm_prefill", 16, 1024, 4096, 16, 1, "bf16", "f32", True),
        # One long prompt: few channels to spread over the card.
        _ssm("ssm_long_prompt", "ssm_prefill", 1, 8192, 4096, 16, 1, "bf16", "f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv", "rope", "rope", "ssm_decode", "ssm_decode", "ssm_prefill", "ssm_prefill"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    ragged = rng.random() < 0.5
    if op == "conv":
        C = 8 * _log_int(rng, 1, 2048)
        T = rng.choice([1, rng.randrange(2, 9), _log_int(rng, 9, 8192)])
        B = min(_log_int(rng, 1, 256), max(1, 2 ** 25 // (T * C)))
        return _conv(None, B, T, C, rng.choice([2, 3, 4, 4, 4]), dtype, ragged, rng.random() < 0.8,
                     rng.random() < 0.7, rng.random() < 0.5)
    if op == "rope":
        D = 8 * rng.choice([4, 8, 9, 10, 12, 16, 16, 16, 24, 32])
        R = min(D, 2 * rng.choice([D // 2, D // 2, D // 4, D // 8, 8 * rng.randrange(1, 5)]))
        Hk = rng.choice([1, 2, 5, 8, 16])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        T = rng.choice([1, _log_int(rng, 2, 8192)])
        B = min(_log_int(rng, 1, 256), max(1, 2 ** 26 // (T * (Hq + Hk) * D)))
        return _rope(None, B, T, Hq, Hk, D, R, dtype, rng.random() < 0.4,
                     _log_int(rng, 1, 2000000), rng.choice([1.0, 1.0, 1.25]), ragged,
                     rng.choice(["bthd", "bhtd"]))
    N = rng.choice([8, 16, 16, 16, 32])
    G = rng.choice([1, 1, 1, 2, 8])
    C = G * 8 * _log_int(rng, 1, 1024 // G)
    state = rng.choice(["f32", "f32", "bf16"])
    if op == "ssm_decode":
        T = rng.choice([1, 1, rng.randrange(2, 9)])
        B = min(_log_int(rng, 1, 256), max(1, 2 ** 24 // (C * N)))
    else:
        T = min(_log_int(rng, 9, 8192), 2 ** 29 // (C * N))
        B = min(_log_int(rng, 1, 32), max(1, 2 ** 29 // (T * C * N)))
    return _ssm(None, op, B, T, C, N, G, dtype, state, ragged, rng.random() < 0.8)


def _lengths(case):
    """Valid tokens and accepted tokens of each entry (the ragged ones: an empty entry, entries of
    one token, full ones, and what lies between)."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B, [T] * B
    full = [T, 1, (2 * T + 2) // 3, T - 1, (T + 1) // 2, T, 0, (7 * T + 7) // 8]
    lens = [full[b % len(full)] for b in range(B)]
    drafted = T <= 8  # drafted tokens are rejected; a prompt's are not
    return lens, [max(0, n - b % 3) if drafted else n for b, n in enumerate(lens)]


# ---- inputs ----------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    st = dict(case)
    B, T, dt = case["B"], case["T"], DTYPES[case["dtype"]]
    lens, acc = _lengths(case)
    st["lens"], st["acc"] = ints(lens), ints(acc)
    slots = B + 3
    st["idx"] = torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32)
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        x = randn(B, T, C + 64 if case["sliced"] else C).to(dt)  # the projection's other columns
        st["x"] = x[..., 64:] if case["sliced"] else x
        st["weight"] = randn(C, W) * W ** -0.5
        st["bias_"] = 0.1 * randn(C) if case["bias"] else None
        st["pool"] = randn(slots, W - 1, C).to(dt)
        return st
    if case["op"] == "rope":
        Hq, Hk, D, R = case["Hq"], case["Hk"], case["D"], case["R"]
        if case["layout"] == "bthd":
            both = randn(B, T, (Hq + Hk) * D).to(dt)
            st["q"] = both[..., :Hq * D].unflatten(-1, (Hq, D)).transpose(1, 2)
            st["k"] = both[..., Hq * D:].unflatten(-1, (Hk, D)).transpose(1, 2)
        else:
            st["q"], st["k"] = randn(B, Hq, T, D).to(dt), randn(B, Hk, T, D).to(dt)
        freq = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64, device="cuda") * 2 / R)
        if case["factor"] != 1.0:  # long contexts: slow turns slower still, fast ones as they were
            slow = (1.0 - freq * 500.0).clamp(0.0, 1.0)
            freq = freq * (1 - slow) + freq / 8.0 * slow
        st["freq"] = freq.float()
        # the sequences are at different places in their texts
        st["pos"] = (case["first"] * (1 + 0.25 * rand(B))).to(torch.int32)
        return st
    C, N, G = case["C"], case["N"], case["G"]
    x = randn(B, T, C)
    st["x"] = (x * torch.sigmoid(x)).to(dt)                    # as the convolution leaves it
    st["dt"] = (0.5 * randn(B, T, C)).to(dt)
    step = torch.exp(rand(C) * math.log(100.0) + math.log(0.001))  # 0.001 to 0.1
    st["dt_bias"] = step + torch.log(-torch.expm1(-step))
    st["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.3 * randn(C, N))
    low = 16                                                   # the same projection's columns for dt
    proj = randn(B, T, low + 2 * G * N).to(dt)
    st["Bm"] = proj[..., low:low + G * N].unflatten(-1, (G, N))
    st["Cm"] = proj[..., low + G * N:].unflatten(-1, (G, N))
    st["D"] = 1 + 0.1 * randn(C) if case["gated"] else None
    st["z"] = randn(B, T, 2 * C).to(dt)[..., C:] if case["gated"] else None
    st["pool"] = (randn(slots, C, N) * 0.3).to(DTYPES[case["state"]])
    return st


# ---- plain forms -----------------------------------------------------------------------------

def _plain_conv(st):
    x, T, W = st["x"].float(), st["T"], st["W"]
    t = torch.arange(T, device=x.device)
    idx = st["idx"].long()
    line = torch.cat([st["pool"][idx].float(), x], 1)
    y = sum(line[:, j:j + T] * st["weight"][:, j] for j in range(W))
    if st["bias_"] is not None:
        y = y + st["bias_"]
    if st["silu"]:
        y = y / (1 + torch.exp(-y))
    valid = t < st["lens"][:, None]
    y = torch.where(valid[..., None], y, torch.zeros((), device=x.device))
    at = st["acc"].long()[:, None] + torch.arange(W - 1, device=x.device)
    kept = line[torch.arange(st["B"], device=x.device)[:, None], at]
    st["pool"][idx] = kept.to(st["pool"].dtype)
    return y.to(st["x"].dtype), st["pool"]


def _plain_rope(st):
    t = torch.arange(st["T"], device=st["pos"].device)
    valid = (t < st["lens"][:, None])[:, None, :, None]
    angle = (st["pos"].double()[:, None] + t)[..., None] * st["freq"].double()
    cos = (torch.cos(angle) * st["factor"]).float()[:, None]
    sin = (torch.sin(angle) * st["factor"]).float()[:, None]
    R = st["R"]
    out = []
    for x in (st["q"], st["k"]):
        y = x.float()
        part = y[..., :R]
        a, b = (part[..., 0::2], part[..., 1::2]) if st["interleaved"] else (part[..., :R // 2], part[..., R // 2:])
        a, b = a * cos - b * sin, a * sin + b * cos
        part = torch.stack([a, b], -1).flatten(-2) if st["interleaved"] else torch.cat([a, b], -1)
        y = torch.cat([part, y[..., R:]], -1)
        out.append(torch.where(valid, y, torch.zeros((), device=y.device)).to(x.dtype))
    return out


def _plain_ssm(st):
    B, T, C, N, G = (st[k] for k in ("B", "T", "C", "N", "G"))
    x, Bm, Cm = st["x"].float(), st["Bm"].float(), st["Cm"].float()
    d = st["dt"].float() + st["dt_bias"]
    d = torch.clamp(d, min=0.0) + torch.log1p(torch.exp(-d.abs()))
    t = torch.arange(T, device=x.device)
    zero = torch.zeros((), device=x.device)
    valid = (t < st["lens"][:, None])[..., None]
    idx, acc = st["idx"].long(), st["acc"][:, None, None]
    h = st["pool"][idx].float()
    kept = h.clone()
    rejects = st["op"] == "ssm_decode"  # else a sequence's accepted tokens are its valid ones
    if not rejects:
        d = torch.where(valid, d, zero)  # a token past the end leaves the state as it is
    y = torch.empty_like(x)
    for t0 in range(0, T, PLAIN_CHUNK):
        s = slice(t0, min(T, t0 + PLAIN_CHUNK))
        decay = torch.exp(d[:, s, :, None] * st["A"])
        new = ((d[:, s] * x[:, s]).unflatten(-1, (G, C // G))[..., None] * Bm[:, s, :, None, :]).flatten(2, 3)
        for i in range(new.shape[1]):
            h = decay[:, i] * h + new[:, i]
            new[:, i] = h
            if rejects:
                kept = torch.where(acc > t0 + i, h, kept)
        y[:, s] = (new.unflatten(2, (G, C // G)) * Cm[:, s, :, None, :]).sum(-1).flatten(-2)
    if st["D"] is not None:
        y = y + st["D"] * x
    if st["z"] is not None:
        z = st["z"].float()
        y = y * z / (1 + torch.exp(-z))
    st["pool"][idx] = (kept if rejects else h).to(st["pool"].dtype)
    return torch.where(valid, y, zero).to(st["x"].dtype), st["pool"]


def _run_plain(st):
    return {"conv": _plain_conv, "rope": _plain_rope}.get(st["op"], _plain_ssm)(st)


# ---- the framework's calls -------------------------------------------------------------------

def _run_own(st):
    import gated_delta_rule_rgdr_amd as rgdr
    if st["op"] == "conv":
        return rgdr.la_conv(st["x"], st["weight"], st["pool"], st["lens"], st["idx"], st["acc"],
                            bias=st["bias_"], silu=st["silu"])
    if st["op"] == "rope":
        return rgdr.la_rope(st["q"], st["k"], st["freq"], st["pos"], interleaved=st["interleaved"],
                            factor=st["factor"], actual_seq_lengths=st["lens"])
    call = rgdr.ssm_decode if st["op"] == "ssm_decode" else rgdr.ssm_prefill
    return call(st["x"], st["dt"], st["A"], st["Bm"], st["Cm"], st["pool"], st["lens"], st["idx"],
                st["acc"], D=st["D"], z=st["z"], dt_bias=st["dt_bias"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    B, T = case["B"], case["T"]
    size = 4 if case["dtype"] == "f32" else 2
    tokens = sum(_lengths(case)[0])
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        return {"bytes": size * C * (tokens + B * T + 2 * B * (W - 1)) + 4 * C * W,
                "flops": (2.0 * W + 4) * tokens * C}
    if case["op"] == "rope":
        heads = case["Hq"] + case["Hk"]
        return {"bytes": size * heads * case["D"] * (tokens + B * T), "flops": 3.0 * tokens * heads * case["R"]}
    C, N, G = case["C"], case["N"], case["G"]
    state = 4 if case["state"] == "f32" else 2
    rows = 3 if case["gated"] else 2
    return {"bytes": size * (tokens * (rows * C + 2 * G * N) + B * T * C) + 2 * B * C * N * state + 4 * C * N,
            "flops": 7.0 * tokens * C * N}


# ---- from the definitions, in 64 bits --------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    lens, acc = _lengths(case)
    B, T = case["B"], case["T"]
    idx = st["idx"].long().tolist()
    if case["op"] == "conv":
        W = case["W"]
        out = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")
        pool = st["pool"].double()
        w = st["weight"].double()
        for b in range(B):
            line = torch.cat([pool[idx[b]], st["x"][b].double()])
            n = lens[b]
            if n:
                y = (line[:n + W - 1].unfold(0, W, 1) * w).sum(-1)
                if case["bias"]:
                    y = y + st["bias_"].double()
                out[b, :n] = y * torch.sigmoid(y) if case["silu"] else y
            pool[idx[b]] = line[acc[b]:acc[b] + W - 1].clone()
        return out, pool
    if case["op"] == "rope":
        R = case["R"]
        pos = st["pos"].double()[:, None, None] + torch.arange(T, device="cuda")[:, None]
        turn = torch.polar(torch.full((), case["factor"], dtype=torch.float64, device="cuda"),
                           pos * st["freq"].double())[:, None]
        out = []
        for x in (st["q"], st["k"]):
            y = x.double().clone(memory_format=torch.contiguous_format)
            first = slice(0, R, 2) if case["interleaved"] else slice(0, R // 2)
            second = slice(1, R, 2) if case["interleaved"] else slice(R // 2, R)
            pair = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
            y[..., first], y[..., second] = pair.real, pair.imag
            for b, n in enumerate(lens):
                y[b, :, n:] = 0
            out.append(y)
        return out
    C, N, G = case["C"], case["N"], case["G"]
    group = torch.arange(C, device="cuda") // (C // G)
    step = torch.nn.functional.softplus(st["dt"].double() + st["dt_bias"].double(), threshold=60.0)
    A, x = st["A"].double(), st["x"].double()
    h = st["pool"].double()[idx]
    pool = st["pool"].double()
    out = torch.zeros_like(x)
    for t in range(T + 1):
        for b in range(B):
            if acc[b] == t:
                pool[idx[b]] = h[b]
        if t == T:
            break
        d = step[:, t, :, None]
        h = torch.exp(d * A) * h + d * x[:, t, :, None] * st["Bm"][:, t].double()[:, group]
        out[:, t] = (h * st["Cm"][:, t].double()[:, group]).sum(-1)
    if st["D"] is not None:
        out = out + st["D"].double() * x
    if st["z"] is not None:
        z = st["z"].double()
        out = out * z * torch.sigmoid(z)
    for b, n in enumerate(lens):
        out[b, n:] = 0
    return out, pool
