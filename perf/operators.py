"""The 4-bit KV cache's operators, each in a plain form and as the library's calls.

Two operators over a cache whose K and V rows are held in 4 bits:

* ``store``: rows are quantised as they are appended, and read back.
* ``attend``: grouped-query attention over such a cache (bottom-right causal,
  ragged rows, optional sliding window, contiguous, paged or ring storage);
  ``step`` is the same with the chunk's append in front, as a decode loop
  calls it.

Format of one row x[0 .. d-1] (one token of one KV head), each operation
rounded to float32 unless said otherwise:
  lo = min(0, min x), hi = max(0, max x)
  s  = bfloat16((hi - lo) / 15)                        the row's step
  z  = rint(-lo * (1 / s))                             its zero point, 0 .. 15
  c  = min(15, max(0, rint(x * (1 / s)) + z))          the codes (ties to even)
  value = s * (c - z)
A row whose range hi - lo is not finite has s = NaN, and a row with
s < 2^-126 has s = 0 and z = 0 and codes 0.
Eight values share a little-endian 32-bit word: value 2i at bits 4i, value
2i + 1 at bits 16 + 4i.  The row's scale word holds s (bfloat16) in its high
16 bits and z in its low 16.
"""

import math

import numpy as np
import torch

own = False

PAGE = 128
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)  # of values 0 .. 7 in their word


# --------------------------------------------------------------------- cases
def _case(name, op, B, Hkv, G, d, T, lens, ragged=False, cap=0, window=0, layout="flat"):
    """lens: longest prior length; ragged rows have less (0 among them).  cap: max_len (0: as needed)."""
    return {"name": name, "op": op, "B": B, "Hkv": Hkv, "G": G, "d": d, "T": T, "lens": lens, "ragged": ragged,
            "cap": cap, "window": window, "layout": layout}


def listed():
    return [
        # one decode step's rows of a batch of 32 (8 KV heads): latency
        _case("store_decode_b32", "store", 32, 8, 4, 128, 1, 8191, cap=8192),
        # ragged last chunks of prompts, 64-wide heads, pages
        _case("store_ragged_paged_d64", "store", 7, 2, 4, 64, 77, 1000, ragged=True, layout="paged"),
        # a prefill chunk of 512 tokens
        _case("store_chunk512_b4", "store", 4, 8, 4, 128, 512, 15872, cap=16384),
        # whole prompts written at once
        _case("store_prompt8192_b4", "store", 4, 8, 4, 128, 8192, 0, cap=8192),
        # one short sequence: launch and latency
        _case("attend_one_row_short", "attend", 1, 2, 4, 128, 1, 44),
        # the decode step of an 8-KV-head model, batch 32, ragged lengths up to 8192
        _case("step_decode_b32_len8192", "step", 32, 8, 4, 128, 1, 8191, ragged=True, cap=8192),
        # the same with 64-wide heads, rows of no tokens among them, pages
        _case("attend_decode_paged_d64", "attend", 32, 8, 4, 64, 1, 8191, ragged=True, layout="paged"),
        # seven query heads a KV head, a sliding window, odd sizes
        _case("attend_decode_window_g7", "attend", 13, 2, 7, 128, 1, 9001, ragged=True, window=1000),
        # speculative verify, 5 tokens a row
        _case("step_verify_b64_t5", "step", 64, 8, 4, 128, 5, 4091, cap=4096),
        # long-context decode
        _case("attend_decode_len131072_b4", "attend", 4, 8, 4, 128, 1, 131071, cap=131072),
        # chunked prefill, every chunk behind a prior context
        _case("attend_prefill_chunk512_b4", "attend", 4, 8, 4, 128, 512, 15872, ragged=True, cap=16384),
        # a ragged last chunk over pages
        _case("attend_prefill_ragged_paged", "attend", 3, 4, 3, 128, 333, 4000, ragged=True, layout="paged"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "step"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    layout = rng.choice(["flat", "flat", "paged", "ring"])
    kind = "rows" if op == "store" else rng.choice(["decode", "decode", "verify", "prefill"])
    B = _log(rng, 1, 64)
    window = 0
    if kind == "rows":
        T = _log(rng, 1, 8192)
        B = max(1, min(B, 32768 // T))
        L = _log(rng, 1, 8000)
    elif kind == "decode":
        T = 1
        L = _log(rng, 1, max(2, min(131000, 4 * 131000 // B)))
        window = rng.choice([0, 0, 0, _log(rng, 1, 4000)])
    elif kind == "verify":
        T = rng.randint(2, 8)
        L = _log(rng, 1, 16000 if B <= 16 else 4000)
        window = rng.choice([0, 0, 0, _log(rng, 1, 4000)])
    else:
        d = 128
        T = _log(rng, 16, 512)
        B = min(B, 4)
        L = _log(rng, 1, 15000)
        window = rng.choice([0, 0, _log(rng, 1, 4000)])
    if layout == "ring":
        # a ring keeps what a window needs beside the chunk
        window = window or _log(rng, 1, 4000)
    return {"op": op, "B": B, "Hkv": Hkv, "G": G, "d": d, "T": T, "lens": L, "ragged": rng.random() < 0.7, "cap": 0,
            "window": window, "layout": layout}


# -------------------------------------------------------------------- inputs
def _plan(case, seed):
    """Lengths and chunk sizes, from the seed alone: (prior, n_new, capacity)."""
    rng = np.random.default_rng([seed, 77])
    B, T, L = case["B"], case["T"], case["lens"]
    if case["ragged"]:
        prior = rng.integers(min(L, L // 2), L + 1, size=B)
        prior[rng.random(B) < 0.05] = 0
        prior[0] = L
        n_new = rng.integers(max(0, T - T // 3 - (1 if B > 8 else 0)), T + 1, size=B)
        n_new[0] = T
    else:
        prior = np.full(B, L)
        n_new = np.full(B, T)
    if case["layout"] == "ring":
        cap = -(-(case["window"] + T) // PAGE) * PAGE
    elif case["layout"] == "paged":
        cap = -(-(L + T) // PAGE) * PAGE
    else:
        cap = max(case["cap"], L + T)
    return prior.astype(np.int64), n_new.astype(np.int64), int(cap)


def _slots(case, cap):
    """Rows of a layer's buffers: (leading entries, tokens in each)."""
    if case["layout"] == "paged":
        return case["B"] * (cap // PAGE), PAGE
    return case["B"], cap


def _rows(gen, shape, bias, dev):
    """bf16 rows with a spread of sizes and a few large channels, as keys have them."""
    x = torch.randn(shape, generator=gen, device=dev)
    return (x + bias).bfloat16()


def _fill(gen, shape, bias, dev):
    """Codes and scale words of a filled buffer [N, Hkv, tokens]."""
    N, H, S, d = shape
    words = torch.empty(N, H, S, d // 8, dtype=torch.int32, device=dev)
    scale = torch.zeros(N, H, -(-S // 4) * 4, dtype=torch.int32, device=dev)
    step = max(1, (1 << 26) // max(1, H * S * d))
    for i in range(0, N, step):
        x = _rows(gen, (min(step, N - i), H, S, d), bias, dev)
        c, s, z = _quantise(x)
        words[i:i + step] = _pack(c)
        scale[i:i + step, :, :S] = _word(s, z)
    return words, scale


def _inputs(case, seed):
    B, Hkv, G, d, T = (case[k] for k in ("B", "Hkv", "G", "d", "T"))
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 11)
    prior, n_new, cap = _plan(case, seed)
    kb = torch.randn((Hkv, 1, d), generator=gen, device=dev) * 0.5
    big = torch.rand((Hkv, 1, d), generator=gen, device=dev) < 0.03
    kb = torch.where(big, kb * 6.0, kb)
    vb = torch.zeros((Hkv, 1, d), device=dev)
    N, S = _slots(case, cap)
    k, ks = _fill(gen, (N, Hkv, S, d), kb, dev)
    v, vs = _fill(gen, (N, Hkv, S, d), vb, dev)
    st = {"case": dict(case), "prior": prior, "n_new": n_new, "cap": cap, "k": k, "ks": ks, "v": v, "vs": vs}
    if case["layout"] == "paged":
        st["table"] = torch.randperm(N, generator=gen, device=dev).to(torch.int32).view(B, cap // PAGE)
    st["k_new"] = _rows(gen, (B, Hkv, T, d), kb, dev)
    st["v_new"] = _rows(gen, (B, Hkv, T, d), vb, dev)
    st["q"] = torch.randn((B, Hkv * G, T, d), generator=gen, device=dev).bfloat16()
    st["k_out"] = torch.zeros((B, Hkv, T, d), dtype=torch.bfloat16, device=dev)
    st["v_out"] = torch.zeros((B, Hkv, T, d), dtype=torch.bfloat16, device=dev)
    # device copies of the lengths, for the plain form's masks
    st["d_prior"] = torch.as_tensor(prior, device=dev)
    st["d_n_new"] = torch.as_tensor(n_new, device=dev)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from gqa_attention_preallocated_gb300 import KVCache, PagedKVCache

        B, Hkv, d, cap = case["B"], case["Hkv"], case["d"], st["cap"]
        if case["layout"] == "paged":
            mpr = cap // PAGE
            cache = PagedKVCache(1, B, Hkv, PAGE, B * mpr, mpr, d, dtype="q4")
            cache.block_table.copy_(st["table"])
        else:
            cache = KVCache(1, B, Hkv, cap, d, dtype="q4")
        if case["window"]:
            cache.set_window(case["window"], ring=case["layout"] == "ring")
        cache.k[0].copy_(st["k"].view(torch.uint8).view(cache.k[0].shape))
        cache.v[0].copy_(st["v"].view(torch.uint8).view(cache.v[0].shape))
        cache.k_scale[0].copy_(st["ks"])
        cache.v_scale[0].copy_(st["vs"])
        del st["k"], st["v"], st["ks"], st["vs"]
        st["cache"] = cache
        if case["op"] == "attend":
            cache.set_lens(0, st["prior"] + st["n_new"])
        else:
            cache.set_lens(0, st["prior"])
    return st


# ---------------------------------------------------------------- plain form
def _quantise(x):
    """Codes [..., d], step and zero point [...] of rows x [..., d]."""
    x = x.float()
    lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
    span = hi - lo
    s = (span / torch.full_like(span, 15.0)).bfloat16().float()  # (a scalar divisor would be a product)
    none = s < 2.0 ** -126
    r = 1.0 / s
    z = torch.where(none, torch.zeros_like(s), torch.round(-lo * r))
    c = torch.round(x * r[..., None]) + z[..., None]
    c = torch.where(none[..., None], torch.zeros_like(c), c).clamp(0.0, 15.0)
    s = torch.where(none, torch.zeros_like(s), s)
    bad = ~torch.isfinite(span)
    s = torch.where(bad, torch.full_like(s, math.nan), s)
    z = torch.where(bad, torch.zeros_like(z), z)
    c = torch.where(bad[..., None], torch.zeros_like(c), c)
    return c.to(torch.int32), s, z.to(torch.int32)


def _pack(c):
    c = c.view(*c.shape[:-1], c.shape[-1] // 8, 8)
    w = c[..., 0]
    for i in range(1, 8):
        w = w | (c[..., i] << SHIFTS[i])
    return w


def _word(s, z):
    return (s.bfloat16().view(torch.int16).to(torch.int32) << 16) | z


def _values(words, scale):
    """float32 values [..., d] of code words [..., d / 8] and scale words [...]."""
    sh = torch.tensor(SHIFTS, dtype=torch.int32, device=words.device)
    c = (words[..., None] >> sh) & 15
    s = (scale & -65536).view(torch.float32)
    z = scale & 65535
    c = c.flatten(-2) - z[..., None]
    return c.float() * s[..., None]


def _where(st, pos):
    """Buffer entry and token offset of positions pos [B, n]."""
    case, B = st["case"], st["case"]["B"]
    rows = torch.arange(B, device=pos.device)[:, None].expand_as(pos)
    if case["layout"] == "paged":
        return st["table"].long()[rows, pos // PAGE], pos % PAGE
    return rows, pos % st["cap"] if case["layout"] == "ring" else pos


def _plain_store(st):
    """Quantise the chunk's rows into the buffers, then read them back."""
    T = st["case"]["T"]
    t = torch.arange(T, device=st["q"].device)
    live = t[None, :] < st["d_n_new"][:, None]
    bi, ti = live.nonzero(as_tuple=True)
    n, at = _where(st, st["d_prior"][:, None] + t[None, :])
    n, at = n[bi, ti], at[bi, ti]
    for new, codes, scale, out in (("k_new", "k", "ks", "k_out"), ("v_new", "v", "vs", "v_out")):
        c, s, z = _quantise(st[new][bi, :, ti])
        st[codes][n, :, at] = _pack(c)
        st[scale][n, :, at] = _word(s, z)
        st[out][bi, :, ti] = _values(st[codes][n, :, at], st[scale][n, :, at]).bfloat16()
    return st["k_out"], st["v_out"]


def _plain_attend(st):
    case = st["case"]
    B, Hkv, G, d, T, W = (case[k] for k in ("B", "Hkv", "G", "d", "T", "window"))
    last = st["d_prior"] + st["d_n_new"]
    # the key positions that any query of a row may see
    S = int((st["prior"] + st["n_new"]).max())
    first = torch.zeros_like(last)
    if W:
        first = (st["d_prior"] - W + 1).clamp(min=0)
        S = min(S, W + T)
    pos = first[:, None] + torch.arange(S, device=last.device)[None, :]
    held = pos < last[:, None]
    n, at = _where(st, torch.where(held, pos, torch.zeros_like(pos)))
    q = st["q"].float().view(B, Hkv, G * T, d)
    k = _values(st["k"][n, :, at], st["ks"][n, :, at])  # [B, S, Hkv, d]
    k = torch.where(held[:, :, None, None], k, torch.zeros_like(k)).transpose(1, 2)
    sc = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)  # [B, Hkv, G*T, S]
    del k
    t = torch.arange(T, device=last.device)
    p = st["d_prior"][:, None] + t[None, :]  # the queries' positions [B, T]
    see = (pos[:, None, :] <= p[:, :, None]) & held[:, None, :] & (t[None, :] < st["d_n_new"][:, None])[:, :, None]
    if W:
        see = see & (pos[:, None, :] > p[:, :, None] - W)
    see = see[:, None, None].expand(B, 1, G, T, S).reshape(B, 1, G * T, S)
    sc = torch.where(see, sc, torch.full_like(sc, -math.inf))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(sc - top)
    del sc
    total = e.sum(-1, keepdim=True)
    v = _values(st["v"][n, :, at], st["vs"][n, :, at])
    v = torch.where(held[:, :, None, None], v, torch.zeros_like(v)).transpose(1, 2)
    o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.bfloat16().view(B, Hkv * G, T, d)


# ----------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        cache, n_new = st["cache"], st["n_new"]
        if op == "attend":
            return cache.gqa_attention(0, st["q"], n_new)
        cache.set_lens(0, st["prior"])
        if op == "store":
            cache.append(0, st["k_new"], st["v_new"], n_new)
            return cache.read(0, st["prior"], n_new, k_out=st["k_out"], v_out=st["v_out"])
        out = cache.append_attention(0, st["q"], st["k_new"], st["v_new"], n_new)
        k, v = cache.read(0, st["prior"], n_new, k_out=st["k_out"], v_out=st["v_out"])
        return out, k, v
    if op == "attend":
        return _plain_attend(st)
    k, v = _plain_store(st)
    if op == "store":
        return k, v
    return _plain_attend(st), k, v


# --------------------------------------------------------------------- work
def work(case):
    B, Hkv, G, d, T, W = (case[k] for k in ("B", "Hkv", "G", "d", "T", "window"))
    # as the seed leaves it: ragged rows are three quarters as long on the mean
    prior = case["lens"] * (0.75 if case["ragged"] and B > 1 else 1.0)
    new = T * (5 / 6 if case["ragged"] and B > 1 and T > 1 else 1.0)
    row = d // 2 + 4  # codes and scale word of one K or V row
    rows = B * Hkv * new
    moved = rows * 2 * (2 * d + row + 2 * d)  # bf16 in, codes out, bf16 back
    if case["op"] == "store":
        return {"bytes": int(moved), "flops": int(rows * 2 * 4 * d)}
    keys = min(prior + new, W + new) if W else prior + new
    seen = min(W, prior + (new + 1) / 2) if W else prior + (new + 1) / 2
    byts = B * Hkv * keys * 2 * row + 2 * B * Hkv * G * new * d * 2
    flops = 4 * B * Hkv * G * new * seen * d
    if case["op"] == "step":
        byts += moved
    return {"bytes": int(byts), "flops": int(flops)}


# ------------------------------------------------------- the definition, 64 bits
def _round32(x):
    return x.float().double()


def _exact_rows(x):
    """s * (c - z) of each row, every rounding of the definition made explicitly on 64-bit numbers."""
    x = x.double()
    lo = torch.minimum(x.min(-1, keepdim=True)[0], torch.zeros((), dtype=torch.float64, device=x.device))
    hi = torch.maximum(x.max(-1, keepdim=True)[0], torch.zeros((), dtype=torch.float64, device=x.device))
    span = _round32(hi - lo)
    s = _round32(span / 15).bfloat16().double()
    r = _round32(1 / s)
    z = torch.round(_round32(-lo * r))
    c = torch.round(_round32(x * r)) + z
    c = torch.minimum(torch.maximum(c, torch.zeros_like(c)), torch.full_like(c, 15))
    y = s * (c - z)
    y = torch.where(s < 2.0 ** -126, torch.zeros_like(y), y)
    return torch.where(torch.isfinite(span), y, torch.full_like(y, math.nan))


def _exact_read(words, scale):
    """64-bit values of one row's positions: words [S, Hkv, d / 8], scale words [S, Hkv]."""
    w = words.long() & 0xFFFFFFFF
    even = [(w >> (4 * i)) & 15 for i in range(4)]
    odd = [(w >> (16 + 4 * i)) & 15 for i in range(4)]
    c = torch.stack([even[0], odd[0], even[1], odd[1], even[2], odd[2], even[3], odd[3]], -1).flatten(-2)
    u = scale.long() & 0xFFFFFFFF
    s = (u >> 16).to(torch.int32).to(torch.int16).view(torch.bfloat16).double()
    return s[..., None] * (c - (u & 0xFFFF)[..., None]).double()


def exact(case, seed):
    st = _inputs(case, seed)
    B, Hkv, G, d, T, W = (case[k] for k in ("B", "Hkv", "G", "d", "T", "window"))
    dev = st["q"].device
    new = []
    if case["op"] != "attend":
        for name in ("k_new", "v_new"):
            y = _exact_rows(st[name])
            gone = torch.arange(T, device=dev)[None, :] >= st["d_n_new"][:, None]
            y[gone[:, None, :].expand(B, Hkv, T)] = 0
            new.append(y)
        if case["op"] == "store":
            return tuple(new)
    out = torch.zeros((B, Hkv * G, T, d), dtype=torch.float64, device=dev)
    for b in range(B):
        L0, n = int(st["prior"][b]), int(st["n_new"][b])
        if n == 0:
            continue
        a0 = max(0, L0 - W + 1) if W else 0
        a = torch.arange(a0, L0 + n, device=dev)
        if case["layout"] == "paged":
            e, at = st["table"][b].long()[a // PAGE], a % PAGE
        else:
            e, at = torch.full_like(a, b), a % st["cap"]
        K, V = _exact_read(st["k"][e, :, at], st["ks"][e, :, at]), _exact_read(st["v"][e, :, at], st["vs"][e, :, at])
        if new:
            K[L0 - a0:], V[L0 - a0:] = new[0][b, :, :n].transpose(0, 1), new[1][b, :, :n].transpose(0, 1)
        pos = torch.arange(L0, L0 + n, device=dev)
        hide = a[None, :] > pos[:, None]
        if W:
            hide |= a[None, :] <= pos[:, None] - W
        for h in range(Hkv):
            x = st["q"][b, h * G:(h + 1) * G, :n].double() @ K[:, h].T / math.sqrt(d)
            out[b, h * G:(h + 1) * G, :n] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ V[:, h]
    return (out, *new) if new else out
