"""What is measured of the 4-bit KV cache and of windowed decode attention.

Four operators of a decode loop's serving side, each in its plain form (elementary torch
operations, fp32 or wider) and, with `own` set, through the library's entry points:

  append   new K and V rows are quantised into a 4-bit cache (santa.kv4_append), and the
           rows just written are read back, as a prompt's own attention uses them
  read     rows of a 4-bit cache are read back as bf16 (santa.kv4_read), for example into
           the bf16 cache that the sampled decode modes take
  kv4      one decode step of exact attention over a 4-bit cache (santa.decode_kv4), with
           or without a sliding window and sink tokens
  window   one decode step of exact attention over a bf16 cache under a sliding window with
           sink tokens (santa.decode_window)

The 4-bit format: a row of d values is d/16 groups of 16.  A group has one unsigned 8-bit
scale s with 5 exponent bits (bias 15) and 3 mantissa bits, the number of that form nearest
to max|x| / 6 (ties to even, at most 10240; 255, a NaN, where the group holds a NaN or an
infinity), and 16 codes: sign bit and index into {0, .5, 1, 1.5, 2, 3, 4, 6}, the grid
value nearest to x / s (ties to the even index).  Byte i of a row holds values 2i (low
half) and 2i + 1.  A code stands for sign * grid * s, which bf16 holds exactly.
"""
import math

import torch

own = False
DEV = "cuda"
GROUP = 16
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def _append(name, B, T, H_kv, d, n_max, ragged=False, fused=False):
    return {"name": name, "op": "append", "B": B, "T": T, "H_kv": H_kv, "d": d, "n_max": n_max, "ragged": ragged,
            "fused": fused}


def _read(name, B, T, H_kv, d, n_max, ragged=False):
    return {"name": name, "op": "read", "B": B, "T": T, "H_kv": H_kv, "d": d, "n_max": n_max, "ragged": ragged}


def _decode(name, op, B, H_q, H_kv, d, n_max, n_lo, window, sinks, bf16_out=False):
    """n_lo: sequence lengths are uniform in [n_lo, n_max] (n_lo = n_max: all full)."""
    return {"name": name, "op": op, "B": B, "H_q": H_q, "H_kv": H_kv, "d": d, "n_max": n_max, "n_lo": n_lo,
            "window": window, "sinks": sinks, "bf16_out": bf16_out}


def listed():
    return [
        # a decode step of the Llama-shaped batch: one token per sequence (latency)
        _append("append step b16", 16, 1, 8, 128, 32768),
        # a ragged batch of short prompts, d = 64, K and V slices of one projection's output
        _append("append ragged b7 t333 d64", 7, 333, 4, 64, 1008, ragged=True, fused=True),
        # prompts of 8192 tokens
        _append("append prompt b4 8k", 4, 8192, 8, 128, 8192),
        # a short prefix of odd length, read back for a few sequences
        _read("read b5 t1023 d64", 5, 1023, 4, 64, 2512, ragged=True),
        # a whole 32k context moved into the bf16 cache of the sampled modes
        _read("read b4 32k", 4, 32768, 8, 128, 32768),
        # the smallest step: one short sequence (latency)
        _decode("kv4 b1 777 d64", "kv4", 1, 8, 4, 64, 1008, 777, 0, 0),
        # the single long sequence
        _decode("kv4 b1 32k", "kv4", 1, 32, 8, 128, 32768, 32768, 0, 0),
        # the headline batch
        _decode("kv4 b16 32k", "kv4", 16, 32, 8, 128, 32768, 32768, 0, 0),
        # the ragged long batch under a window, bf16 output for the next layer
        _decode("kv4 b32 ragged w4096", "kv4", 32, 32, 8, 128, 65536, 4096, 4096, 4, True),
        # a window on one long sequence (latency)
        _decode("window b1 32k w4096", "window", 1, 32, 8, 128, 32768, 32768, 4096, 4),
        # a wide window on the headline batch
        _decode("window b16 32k w8192", "window", 16, 32, 8, 128, 32768, 32768, 8192, 16),
        # the ragged batch, an odd window, eight heads to a KV head, bf16 output
        _decode("window b32 ragged w1001 g8", "window", 32, 64, 8, 128, 16384, 1, 1001, 5, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "kv4", "kv4", "window", "window"])
    d = rng.choice([64, 128, 128])
    H_kv = rng.choice([1, 2, 4, 8])
    if op in ("append", "read"):
        B = _log(rng, 1, 32)
        T = max(1, _log(rng, 1, min(32768, (4 << 23) // (B * H_kv * 32))))
        n_max = -(-(T + rng.randrange(0, 500)) // 16) * 16
        ragged = rng.random() < 0.5
        c = _append("", B, T, H_kv, d, n_max, ragged, rng.random() < 0.5) if op == "append" else \
            _read("", B, T, H_kv, d, n_max, ragged)
    else:
        B = _log(rng, 1, 32)
        n_max = _log(rng, 64, min(131072, (1 << 22) // (B * H_kv)))
        if op == "kv4":
            n_max = -(-n_max // 16) * 16
        n_lo = n_max if rng.random() < 0.4 else rng.randrange(1, n_max + 1)
        window = rng.randrange(1, n_max + 1) if op == "window" or rng.random() < 0.4 else 0
        sinks = rng.choice([0, 1, 4, 16, 100]) if window else 0
        c = _decode("", op, B, H_kv * rng.choice([1, 2, 4, 8]), H_kv, d, n_max, n_lo, window, sinks, rng.random() < 0.4)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _rows(gen, *shape):
    """bf16 rows ~ N(0, 1)."""
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _ints(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen, device=DEV).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    B, H_kv, d, n_max, op = case["B"], case["H_kv"], case["d"], case["n_max"], case["op"]
    st = {"case": case}

    def full_cache():  # K and V ~ N(0, 1) rows, quantised one batch row at a time
        parts = [torch.empty(B, H_kv, n_max, w, dtype=torch.uint8, device=DEV) for w in (d // 2, d // GROUP) * 2]
        for b in range(B):
            for i in (0, 2):
                parts[i][b], parts[i + 1][b] = _quantise(_rows(gen, H_kv, n_max, d))
        return tuple(parts)

    if op in ("append", "read"):
        T = case["T"]
        st["pos"] = _ints(gen, 0, n_max - T, B)
        st["counts"] = None
        if case["ragged"]:
            st["counts"] = _ints(gen, 0, T, B)
            st["counts"][0] = T
        st["k_out"], st["v_out"] = (torch.zeros(B, T, H_kv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    if op == "append":
        # channels of unequal size, as keys have them
        size = torch.exp(0.5 * torch.randn(H_kv, d, generator=gen, device=DEV)).to(torch.bfloat16)
        if case["fused"]:  # K and V as slices of the projection's output, heads in the order q, k, v
            qkv = _rows(gen, B, T, 6 * H_kv, d)
            st["k_new"], st["v_new"] = qkv[:, :, 4 * H_kv:5 * H_kv], qkv[:, :, 5 * H_kv:]
            st["k_new"].mul_(size)
        else:
            st["k_new"], st["v_new"] = _rows(gen, B, T, H_kv, d) * size, _rows(gen, B, T, H_kv, d)
        st["cache"] = tuple(torch.zeros(B, H_kv, n_max, w, dtype=torch.uint8, device=DEV)
                            for w in (d // 2, d // GROUP) * 2)
    elif op == "read":
        st["cache"] = full_cache()
    else:
        H_q = case["H_q"]
        g = torch.randn(B, H_q, d, generator=gen, device=DEV, dtype=torch.float32)
        # scores of standard deviation 3 against keys ~ N(0, 1)
        st["q"] = (3.0 * math.sqrt(d) * g / g.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
        st["seq_lens"] = _ints(gen, case["n_lo"], n_max, B)
        if case["n_lo"] < n_max and B >= 4:  # a ragged batch also has a new and an empty row
            st["seq_lens"][0] = 1
            st["seq_lens"][B // 2] = 0
        if op == "kv4":
            st["cache"] = full_cache()
        else:
            st["k"], st["v"] = _rows(gen, B, H_kv, n_max, d), _rows(gen, B, H_kv, n_max, d)
    return st


# ------------------------------------------------------------------ plain forms

def _quantise(x):
    """bf16 [..., d] -> packed codes uint8 [..., d/2], scales uint8 [..., d/16]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    s = torch.where(bad, torch.zeros_like(amax), amax).double() / 6
    m = torch.frexp(s)[0]                              # s = m 2^k with m in [1/2, 1)
    step = torch.where(s > 0, s / torch.where(s > 0, m, torch.ones_like(m)) / 16, torch.zeros_like(s)).clamp(min=2.0 ** -17)
    s = (torch.round(s / step) * step).clamp(max=10240.0)
    y = g.double().abs() / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(-1)
    # ties to the even index
    idx = (y > 0.25).byte() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    idx = idx * (~bad).unsqueeze(-1)
    code = (idx | (torch.signbit(g).byte() << 3)).flatten(-2)
    bits = s.to(torch.float16).view(torch.int16) >> 7  # s is exact in fp16: 5 exponent and 3 mantissa bits
    scale = torch.where(bad, torch.full_like(bits, 255), bits).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _values(codes, scales):
    """fp32 [..., d] of packed codes and scales."""
    table = torch.tensor([v for s in (1.0, -1.0) for v in (s * x for x in GRID)], device=codes.device)
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, GROUP))
    s = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (table[code.int()] * s.unsqueeze(-1)).flatten(-2)


def _token_rows(st):
    """Batch and token index and cache position of the rows that `pos` and `counts` name."""
    B, T = st["case"]["B"], st["case"]["T"]
    t = torch.arange(T, device=DEV).expand(B, T)
    live = t < (st["counts"] if st["counts"] is not None else torch.full_like(st["pos"], T)).unsqueeze(1)
    b, t = live.nonzero(as_tuple=True)
    return b, t, st["pos"].long()[b] + t


def _plain_append(st):
    b, t, at = _token_rows(st)
    kc, ks, vc, vs = st["cache"]
    kc[b, :, at], ks[b, :, at] = _quantise(st["k_new"][b, t])
    vc[b, :, at], vs[b, :, at] = _quantise(st["v_new"][b, t])


def _plain_read(st):
    b, t, at = _token_rows(st)
    kc, ks, vc, vs = st["cache"]
    k, v = st["k_out"].clone(), st["v_out"].clone()
    k[b, t] = _values(kc[b, :, at], ks[b, :, at]).to(torch.bfloat16)
    v[b, t] = _values(vc[b, :, at], vs[b, :, at]).to(torch.bfloat16)
    return k, v


def _visible(case, seq_lens):
    """Key index [B, slots] and whether the slot is seen: the sinks, then the window."""
    n = seq_lens.long().unsqueeze(1)
    if case["window"] == 0:
        at = torch.arange(case["n_max"], device=DEV).unsqueeze(0)
        return at.expand(n.shape[0], -1), at < n
    slot = torch.arange(min(case["sinks"] + case["window"], case["sinks"] + case["n_max"]), device=DEV).unsqueeze(0)
    first = (n - case["window"]).clamp(min=0)
    at = torch.where(slot < case["sinks"], slot, first + slot - case["sinks"])
    seen = torch.where(slot < case["sinks"], slot < first, at < n)
    return at.clamp(max=case["n_max"] - 1), seen


def _plain_decode(st):
    case = st["case"]
    B, H_kv, d = case["B"], case["H_kv"], case["d"]
    at, seen = _visible(case, st["seq_lens"])
    if case["window"] == 0:
        rows = lambda x: x                                             # noqa: E731
    else:
        rows = lambda x: x[torch.arange(B, device=DEV).unsqueeze(1), :, at].transpose(1, 2)  # noqa: E731
    if case["op"] == "kv4":
        kc, ks, vc, vs = st["cache"]
        k, v = _values(rows(kc), rows(ks)), _values(rows(vc), rows(vs))
    else:
        k, v = rows(st["k"]).float(), rows(st["v"]).float()
    q = st["q"].float().view(B, H_kv, -1, d)
    s = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    seen = seen.view(B, 1, 1, -1)
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    w = torch.where(seen, torch.exp(s - torch.where(torch.isfinite(m), m, torch.zeros_like(m))), torch.zeros_like(s))
    o = w @ torch.where(seen.transpose(-1, -2), v, torch.zeros_like(v))
    z = w.sum(-1, keepdim=True)
    o = torch.where(z > 0, o / z, torch.zeros_like(o)).view(B, -1, d)
    return o.to(torch.bfloat16) if case["bf16_out"] else o


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op in ("append", "read"):
            if op == "append":
                _plain_append(state)
            return _plain_read(state)
        return _plain_decode(state)
    from stochastic_sparse_kv_gb300 import santa
    if op == "window":
        return santa.decode_window(state["q"], state["k"], state["v"], state["seq_lens"], case["window"], case["sinks"],
                                   out_dtype=torch.bfloat16 if case["bf16_out"] else torch.float32)
    cache = santa.KV4Cache(*state["cache"])
    if op == "kv4":
        return santa.decode_kv4(state["q"], cache, state["seq_lens"], case["window"], case["sinks"],
                                out_dtype=torch.bfloat16 if case["bf16_out"] else torch.float32)
    if op == "append":
        santa.kv4_append(cache, state["k_new"], state["v_new"], state["pos"], state["counts"])
    return santa.kv4_read(cache, state["pos"], state["k_out"], state["v_out"], state["counts"])


# ------------------------------------------------------------------ work and the 64-bit values

def _mean_visible(case):
    """Visible keys of a sequence, averaged over lengths uniform in [n_lo, n_max]."""
    lo, hi, most = case["n_lo"], case["n_max"], case["window"] + case["sinks"]
    if case["window"] == 0 or most >= hi:
        return (lo + hi) / 2
    if most <= lo:
        return most
    below = most - lo  # lengths lo .. most - 1 are seen whole
    return (below * (lo + most - 1) / 2 + (hi - most + 1) * most) / (hi - lo + 1)


def work(case):
    B, H_kv, d = case["B"], case["H_kv"], case["d"]
    wide, narrow = 2 * d, d // 2 + d // GROUP   # bytes of a bf16 and of a 4-bit row
    if case["op"] in ("append", "read"):
        rows = 2 * B * H_kv * case["T"] * (0.5 if case["ragged"] else 1.0)
        passes = 2 if case["op"] == "append" else 1
        # about 12 operations a value to quantise, 2 to read back
        return {"bytes": passes * rows * (wide + narrow) + 8 * B, "flops": rows * d * (14 if passes == 2 else 2)}
    keys = B * H_kv * _mean_visible(case)
    G = case["H_q"] // H_kv
    moved = 2 * keys * (narrow if case["op"] == "kv4" else wide) + B * case["H_q"] * d * (4 if case["bf16_out"] else 6)
    return {"bytes": moved + 4 * B, "flops": 4.0 * keys * G * d}


# every scale that the cache can hold, in order: code i stands for SCALES[i]
SCALES = [(i & 7) * 2.0 ** -17 if i < 8 else (8 + (i & 7)) * 2.0 ** ((i >> 3) - 18) for i in range(0xE2 + 1)]


def _nearest(x):
    """The value that the cache holds for each x, in 64 bits: the scale by its own bits, the
    code by the smallest distance to the sixteen signed values, ties to the even index."""
    x = x.double().unflatten(-1, (-1, GROUP))
    want = x.abs().amax(-1, keepdim=True) / 6
    numbers = torch.tensor(SCALES, dtype=torch.float64, device=x.device)
    up = torch.searchsorted(numbers, want).clamp(max=0xE2)
    down = (up - 1).clamp(min=0)
    a, b = want - numbers[down], numbers[up] - want
    s = numbers[torch.where((b < a) | ((b == a) & (up % 2 == 0)), up, down)]
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    off = (x.abs().unsqueeze(-1) - grid * s.unsqueeze(-1)).abs()
    best = off.amin(-1, keepdim=True)
    order = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=x.device)  # even indexes first
    pick = torch.where(off == best, order, torch.full_like(order, 8)).amin(-1)
    index = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=x.device)[pick]
    return (torch.sign(x) * grid[index] * s).flatten(-2)


def _held(codes, scales):
    """float64 values of one batch row of a 4-bit cache, from the bits."""
    lo, hi = (codes & 15).long(), (codes >> 4).long()
    c = torch.stack((lo, hi), -1).flatten(-2)
    f = torch.tensor(GRID, dtype=torch.float64, device=c.device)[c & 7]
    s = torch.tensor(SCALES, dtype=torch.float64, device=c.device)[scales.long()]
    return torch.where(c >= 8, -f, f) * s.repeat_interleave(GROUP, -1)


def exact(case, seed):
    st = prepare(case, seed)
    B, H_kv, d = case["B"], case["H_kv"], case["d"]
    if case["op"] in ("append", "read"):
        T = case["T"]
        k, v = (torch.zeros(B, T, H_kv, d, dtype=torch.float64, device=DEV) for _ in range(2))
        for b in range(B):
            n = T if st["counts"] is None else int(st["counts"][b])
            p = int(st["pos"][b])
            for t in range(0, n, 1024):
                u = min(n, t + 1024)
                if case["op"] == "append":
                    k[b, t:u], v[b, t:u] = _nearest(st["k_new"][b, t:u]), _nearest(st["v_new"][b, t:u])
                else:
                    kc, ks, vc, vs = (x[b, :, p + t:p + u] for x in st["cache"])
                    k[b, t:u], v[b, t:u] = _held(kc, ks).transpose(0, 1), _held(vc, vs).transpose(0, 1)
        return k, v
    out = torch.zeros(B, case["H_q"], d, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(st["seq_lens"][b])
        if n == 0:
            continue
        keys = torch.arange(n, device=DEV)
        if case["window"]:
            keys = keys[(keys >= n - case["window"]) | (keys < case["sinks"])]
        if case["op"] == "kv4":
            kc, ks, vc, vs = (x[b][:, keys] for x in st["cache"])
            k, v = _held(kc, ks), _held(vc, vs)
        else:
            k, v = st["k"][b][:, keys].double(), st["v"][b][:, keys].double()
        s = torch.einsum("hgd,hnd->hgn", st["q"][b].double().view(H_kv, -1, d), k) / math.sqrt(d)
        out[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(s, -1), v).reshape(case["H_q"], d)
    return out
