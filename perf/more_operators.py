"""What is measured of rotary positions and of attention over a paged cache.

Three operators of a serving loop, each in its plain form (elementary torch operations, fp32
or wider) and, with `own` set, through the library's entry points:

  rope     rows of a projection's output are rotated to their positions (santa.rope)
  append   new K and V rows go into the pages of a paged cache, K and the queries rotated on
           the way (santa.paged_append)
  attend   causal attention of a chunk of new tokens, one to thousands a sequence, over a
           paged cache that holds them already (santa.attend_paged), with or without a
           sliding window and sink tokens

Rotation: pair i of a head at position p turns by the angle p * f_i; a pair is the features
(i, i + rot/2) ("halves") or (2i, 2i + 1) ("pairs") of the first `rot` ones, the others stay.
f_i = base^(-2i/rot), scaled for long contexts: "linear" f / factor; "bands" f where the
wavelength is below original/high, f / factor where it is above original/low, a blend in
between; "ramp" a blend over the index of the pair, and cos and sin times 0.1 ln(factor) + 1.

Paged cache: K and V are [n_pages, H_kv, page, d]; key j of sequence b is row j % page of page
table[b, j // page].  Token t of sequence b has position pos[b] + t, t < counts[b] are live.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases

def _rope(name, B, T, H, d, rot, layout, scaling, p_max, ragged=False, fused=False):
    return {"name": name, "op": "rope", "B": B, "T": T, "H_q": H, "d": d, "rot": rot, "layout": layout,
            "scaling": scaling, "p_max": p_max, "ragged": ragged, "fused": fused}


def _append(name, B, T, H_q, H_kv, d, page, rot, layout, scaling, n_max, ragged=False):
    return {"name": name, "op": "append", "B": B, "T": T, "H_q": H_q, "H_kv": H_kv, "d": d, "page": page, "rot": rot,
            "layout": layout, "scaling": scaling, "n_max": n_max, "ragged": ragged}


def _attend(name, B, T, H_q, H_kv, d, page, n_lo, n_max, window=0, sinks=0, ragged=False, fused=False):
    """Lengths with the chunk from n_lo to n_max; ragged: live tokens from 0 to T."""
    return {"name": name, "op": "attend", "B": B, "T": T, "H_q": H_q, "H_kv": H_kv, "d": d, "page": page, "n_lo": n_lo,
            "n_max": n_max, "window": window, "sinks": sinks, "ragged": ragged, "fused": fused}


def listed():
    return [
        # the queries of a decode step of the Llama-shaped batch (latency)
        _rope("rope step b16", 16, 1, 32, 128, 128, "halves", "bands", 32768),
        # the queries of prompts of 8192 tokens
        _rope("rope prompt b4 8k", 4, 8192, 32, 128, 128, "halves", "ramp", 8192),
        # a ragged batch of short prompts, half of a small head, slices of one projection's output
        _rope("rope ragged b7 t333 d64", 7, 333, 8, 64, 32, "pairs", "linear", 1008, ragged=True, fused=True),
        # a decode step of the Llama-shaped batch: one token a sequence (latency)
        _append("append step b16", 16, 1, 32, 8, 128, 64, 128, "halves", "bands", 8192),
        # a chunk of 2048 tokens of four prompts, small pages
        _append("append chunk b4 2k", 4, 2048, 32, 8, 128, 16, 128, "halves", "bands", 8192),
        # the smallest step: one short sequence (latency)
        _attend("attend b1 777 d64", 1, 1, 8, 4, 64, 16, 777, 777),
        # the single long sequence, one token
        _attend("attend b1 32k", 1, 1, 32, 8, 128, 64, 32768, 32768),
        # the headline batch, one token
        _attend("attend b16 32k", 16, 1, 32, 8, 128, 64, 32768, 32768),
        # a ragged long batch, five drafted tokens to be verified, a window
        _attend("attend b32 ragged t5 w4096", 32, 5, 32, 8, 128, 64, 4096, 65536, 4096, 4),
        # a chunk of a long prompt on what came before
        _attend("attend chunk b1 2k on 30k", 1, 2048, 32, 8, 128, 128, 32768, 32768),
        # whole prompts of 8192 tokens
        _attend("attend prompt b2 8k", 2, 8192, 32, 8, 128, 64, 8192, 8192),
        # a mixed ragged batch (new, finished and long rows), odd window, eight heads a KV head
        _attend("attend mixed b32 t255 w1001 g8", 32, 255, 64, 8, 128, 16, 256, 16384, 1001, 5, ragged=True, fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    H_kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, 32)
    rot = rng.choice([d, d, d // 2, rng.randrange(1, d // 16 + 1) * 16])
    layout, scaling = rng.choice(["halves", "halves", "pairs"]), rng.choice(["none", "linear", "bands", "ramp"])
    ragged = rng.random() < 0.5
    if op == "rope":
        T = _log(rng, 1, min(8192, max(2, (1 << 27) // (B * H_kv * G * d))))
        c = _rope("", B, T, H_kv * G, d, rot, layout, scaling, T + _log(rng, 1, 100000), ragged, rng.random() < 0.5)
    elif op == "append":
        T = _log(rng, 1, min(4096, max(2, (1 << 25) // (B * H_kv * G * d))))
        page = rng.choice([16, 32, 64, 128, 256])
        n_max = -(-(T + rng.randrange(0, 1000)) // page) * page
        c = _append("", B, T, H_kv * G, H_kv, d, page, rot, layout, scaling, n_max, ragged)
    else:
        T = rng.choice([1, 1, rng.randrange(1, 17), _log(rng, 1, 4096), _log(rng, 1, 4096)])
        most = (1 << 32) // (B * H_kv * G * T * 2)                # the plain form's scores
        n_max = max(T, _log(rng, 64, max(65, min(131072, most, (1 << 22) // (B * H_kv)))))
        n_lo = n_max if rng.random() < 0.4 else rng.randrange(T, n_max + 1)
        window = rng.randrange(1, n_max + 1) if rng.random() < 0.4 else 0
        c = _attend("", B, T, H_kv * G, H_kv, d, rng.choice([16, 32, 64, 128, 256]), n_lo, n_max, window,
                    rng.choice([0, 1, 4, 16, 100]) if window else 0, ragged, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

BASE, ORIGINAL, FACTOR, LOW, HIGH = 500000.0, 8192, 8.0, 1.0, 4.0   # (ramp: LOW..8 HIGH turns)


def _frequencies(case):
    """Radians a position of each pair, and the factor of cos and sin."""
    rot, scaling = case["rot"], case["scaling"]
    f = [BASE ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / FACTOR for x in f], 1.0
    if scaling == "bands":
        def blend(x):
            turns = ORIGINAL * x / (2 * math.pi)              # over the original context
            s = min(max((turns - LOW) / (HIGH - LOW), 0.0), 1.0)
            return (1 - s) * x / FACTOR + s * x
        return [blend(x) for x in f], 1.0
    if scaling == "ramp":
        def index(turns):
            return rot * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(BASE))
        lo, hi = max(math.floor(index(8 * HIGH)), 0), min(math.ceil(index(LOW)), rot - 1)
        hi = max(hi, lo + 0.001)
        ramp = [min(max((i - lo) / (hi - lo), 0.0), 1.0) for i in range(rot // 2)]
        return [x / FACTOR * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(FACTOR) + 1
    return f, 1.0


def _spread(lo, hi, B):
    """B numbers from lo to hi, far ones next to each other."""
    return [hi - (hi - lo) * ((b * 7) % B if B % 7 else b) // max(B - 1, 1) for b in range(B)]


def _lengths(case):
    """Live tokens and positions of the first one, a sequence."""
    B, T = case["B"], case["T"]
    counts = _spread(0, T, B) if case["ragged"] and B > 1 else [T] * B
    if case["op"] == "attend":
        return counts, [n - c for n, c in zip(_spread(max(case["n_lo"], T), max(case["n_max"], T), B), counts)]
    last = (case["p_max"] if case["op"] == "rope" else case["n_max"]) - T
    return counts, _spread(last // 2, last, B)


def _rows(gen, *shape):
    """bf16 rows ~ N(0, 1)."""
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    B, T, H_q, d, op = case["B"], case["T"], case["H_q"], case["d"], case["op"]
    counts, pos = _lengths(case)
    st = {"case": case, "pos": torch.tensor(pos, dtype=torch.int32, device=DEV),
          "counts": torch.tensor(counts, dtype=torch.int32, device=DEV) if case["ragged"] else None,
          "out": torch.zeros(B, T, H_q, d, dtype=torch.bfloat16, device=DEV)}
    if op != "attend":
        f, st["amplitude"] = _frequencies(case)
        st["f"] = torch.tensor(f, dtype=torch.float64, device=DEV)
        # in units of 2^-64 of a full turn
        st["turns"] = torch.tensor([int(x / (2 * math.pi) * 2.0 ** 64) for x in f], dtype=torch.int64, device=DEV)
    if op == "rope":
        # queries as slices of the projection's output, or rows of their own
        x = _rows(gen, B, T, H_q + 4, d)[:, :, :H_q] if case["fused"] else _rows(gen, B, T, H_q, d)
        return {**st, "x": x}
    H_kv, page = case["H_kv"], case["page"]
    cols = -(-max(case["n_max"], T) // page)
    n_pages = B * cols + 3
    # pages in no order; entries that no token needs name no page
    table = torch.randperm(n_pages, generator=gen, device=DEV)[:B * cols].view(B, cols).to(torch.int32)
    need = torch.tensor([-(-(p + c) // page) for p, c in zip(pos, counts)], device=DEV)
    st["table"] = torch.where(torch.arange(cols, device=DEV) < need.unsqueeze(1), table, torch.full_like(table, -1))
    if op == "append":
        qkv = _rows(gen, B, T, H_q + 2 * H_kv, d)         # heads in the order q, k, v
        st["q"], st["k_new"], st["v_new"] = qkv.split((H_q, H_kv, H_kv), 2)
        st["k"], st["v"] = (torch.zeros(n_pages, H_kv, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        return st
    g = torch.randn(B, T, H_q, d, generator=gen, device=DEV, dtype=torch.float32)
    # scores of standard deviation 3 against keys ~ N(0, 1)
    q = (3.0 * math.sqrt(d) * g / g.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    st["q"] = torch.cat((q, q[:, :, :1].expand(-1, -1, 2 * H_kv, -1)), 2)[:, :, :H_q] if case["fused"] else q
    st["k"], st["v"] = _rows(gen, n_pages, H_kv, page, d), _rows(gen, n_pages, H_kv, page, d)
    return st


# ------------------------------------------------------------------ plain forms

def _live(st):
    """[B, T]: whether token t is live."""
    t = torch.arange(st["case"]["T"], device=DEV).unsqueeze(0)
    n = st["counts"] if st["counts"] is not None else torch.full_like(st["pos"], st["case"]["T"])
    return t < n.unsqueeze(1)


def _rotate(st, x):
    """bf16 rows [B, T, H, d] at their positions; angles in 64 bits, products in 32, one rounding."""
    case = st["case"]
    rot = case["rot"]
    p = st["pos"].double().unsqueeze(1) + torch.arange(case["T"], device=DEV, dtype=torch.float64)
    a = (p.unsqueeze(-1) * st["f"]).unsqueeze(2)                  # [B, T, 1, rot/2]
    c, s = (torch.cos(a) * st["amplitude"]).float(), (torch.sin(a) * st["amplitude"]).float()
    y = x.float()
    u, v = (y[..., :rot // 2], y[..., rot // 2:rot]) if case["layout"] == "halves" else (y[..., 0:rot:2], y[..., 1:rot:2])
    u, v = u * c - v * s, u * s + v * c
    turned = torch.cat((u, v), -1) if case["layout"] == "halves" else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((turned, y[..., rot:]), -1).to(torch.bfloat16)


def _plain_rope(st, x):
    return torch.where(_live(st).unsqueeze(-1).unsqueeze(-1), _rotate(st, x), st["out"])


def _plain_append(st):
    page = st["case"]["page"]
    b, t = _live(st).nonzero(as_tuple=True)
    at = st["pos"].long()[b] + t
    where, row = st["table"].long()[b, at // page], at % page
    st["k"][where, :, row] = _rotate(st, st["k_new"])[b, t]
    st["v"][where, :, row] = st["v_new"][b, t]
    return st["k"], st["v"], _plain_rope(st, st["q"])


def _plain_attend(st):
    case = st["case"]
    B, T, H_kv, d, page = (case[x] for x in ("B", "T", "H_kv", "d", "page"))
    # keys in order: a page that no token needs is read as page 0 and masked
    pages = st["table"].long().clamp(min=0)
    k, v = (x[pages].transpose(2, 3).flatten(1, 2).transpose(1, 2).float() for x in (st["k"], st["v"]))  # [B, H_kv, n, d]
    j = torch.arange(k.shape[2], device=DEV)
    p = (st["pos"].long().unsqueeze(1) + torch.arange(T, device=DEV)).unsqueeze(-1)                      # [B, T, 1]
    seen = j <= p
    if case["window"]:
        seen = seen & ((j > p - case["window"]) | (j < case["sinks"]))
    q = st["q"].float().unflatten(2, (H_kv, -1)).permute(0, 2, 3, 1, 4)                                 # [B, H_kv, G, T, d]
    s = q.flatten(2, 3) @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    s = s.unflatten(2, (-1, T)).masked_fill_(~seen.unsqueeze(1).unsqueeze(1), -math.inf)
    w = s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = (w.flatten(2, 3) @ v).unflatten(2, (-1, T)) / w.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(torch.bfloat16)
    return torch.where(_live(st).unsqueeze(-1).unsqueeze(-1), o, st["out"])


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return _plain_rope(state, state["x"]) if op == "rope" else _plain_append(state) if op == "append" else _plain_attend(state)
    from stochastic_sparse_kv_gb300 import santa
    pos, counts = state["pos"], state["counts"]
    if op == "attend":
        cache = santa.PagedCache(state["k"], state["v"], state["table"])
        return santa.attend_paged(state["q"], cache, pos, counts, case["window"], case["sinks"], out=state["out"])
    table = santa.RopeTable(state["turns"], case["rot"], case["layout"], state["amplitude"])
    if op == "rope":
        return santa.rope(state["x"], table, pos, counts, out=state["out"])
    cache = santa.PagedCache(state["k"], state["v"], state["table"])
    q = santa.paged_append(cache, state["k_new"], state["v_new"], pos, counts, rope=table, q=state["q"], q_out=state["out"])
    return state["k"], state["v"], q


# ------------------------------------------------------------------ work and the 64-bit values

def _seen(case, p0, n):
    """(pairs of tokens p0 .. p0 + n - 1 and visible keys, keys that any of them sees)."""
    w, s = case["window"], case["sinks"]

    def upto(p):       # pairs of the tokens 0 .. p - 1, each with p + 1 keys
        return p * (p + 1) // 2
    pairs = upto(p0 + n) - upto(p0)
    keys = p0 + n
    if w:
        # of a token's p + 1 keys, p + 1 - w - s at most are hidden
        a, b = max(p0, w + s), max(p0 + n, w + s)
        pairs -= (upto(b) - upto(a)) - (b - a) * (w + s)
        keys -= max(0, p0 + 1 - w - s)
    return pairs, keys


def work(case):
    counts, pos = _lengths(case)
    rows, d = sum(counts), case["d"]
    if case["op"] != "attend":
        turned = rows * (case["H_q"] + case.get("H_kv", 0))
        return {"bytes": 4 * d * (turned + rows * case.get("H_kv", 0)) + 8 * case["B"], "flops": 3 * turned * case["rot"]}
    seen = [_seen(case, p, n) for p, n in zip(pos, counts) if n]
    return {"bytes": 4 * d * (case["H_kv"] * sum(k for _, k in seen) + rows * case["H_q"]) + 8 * case["B"],
            "flops": 4.0 * d * case["H_q"] * sum(x for x, _ in seen)}


def _turned(st, b, t, x):
    """Row x [H, d] of token t: its pairs as complex numbers, times A e^(i angle), in 64 bits."""
    case = st["case"]
    rot, y = case["rot"], x.double()
    a = (int(st["pos"][b]) + t).double().unsqueeze(-1) * st["f"]
    z = torch.polar(torch.full_like(a, st["amplitude"]), a).unsqueeze(1)
    if case["layout"] == "halves":
        r = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * z
        first = torch.cat((r.real, r.imag), -1)
    else:
        r = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z
        first = torch.view_as_real(r).flatten(-2)
    return torch.cat((first, y[..., rot:]), -1)


def exact(case, seed):
    st = prepare(case, seed)
    B, T, d = case["B"], case["T"], case["d"]
    counts, pos = _lengths(case)
    out = st["out"].double()
    if case["op"] != "attend":
        x = st["x"] if case["op"] == "rope" else st["q"]
        k, v = (st[n].double() if n in st else None for n in ("k", "v"))
        for b in range(B):
            t = torch.arange(counts[b], device=DEV)
            out[b, :counts[b]] = _turned(st, b, t, x[b, :counts[b]])
            if case["op"] == "append":
                rows = _turned(st, b, t, st["k_new"][b, :counts[b]])
                for lo in range(pos[b] - pos[b] % case["page"], pos[b] + counts[b], case["page"]):   # page by page
                    first, last = max(lo, pos[b]), min(lo + case["page"], pos[b] + counts[b])
                    where = int(st["table"][b, lo // case["page"]])
                    k[where, :, first - lo:last - lo] = rows[first - pos[b]:last - pos[b]].transpose(0, 1)
                    v[where, :, first - lo:last - lo] = st["v_new"][b, first - pos[b]:last - pos[b]].double().transpose(0, 1)
        return out if case["op"] == "rope" else (k, v, out)
    G = case["H_q"] // case["H_kv"]
    for b in range(B):
        n, p0 = counts[b], pos[b]
        if n == 0:
            continue
        pages = st["table"][b, :-(-(p0 + n) // case["page"])].long()
        for h in range(case["H_kv"]):
            k, v = (st[x][pages, h].flatten(0, 1)[:p0 + n].double() for x in ("k", "v"))
            q = st["q"][b, :n, h * G:(h + 1) * G].double()
            for t in range(0, n, 1024):
                at = torch.arange(p0 + t, p0 + min(t + 1024, n), device=DEV).unsqueeze(-1)
                hidden = torch.arange(p0 + n, device=DEV) > at
                if case["window"]:
                    far = torch.arange(p0 + n, device=DEV)
                    hidden |= (far <= at - case["window"]) & (far >= case["sinks"])
                s = torch.einsum("tgd,nd->gtn", q[t:t + 1024], k) / math.sqrt(d)
                p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
                out[b, t:t + 1024][:n - t, h * G:(h + 1) * G] = torch.einsum("gtn,nd->tgd", p, v)
    return out
