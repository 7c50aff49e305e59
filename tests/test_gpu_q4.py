"""The 4-bit cache on the GPU against the float64 oracle.

Stored codes and scale words must equal the oracle's bit for bit on every
path that writes them, rows read back must be the oracle's values rounded once
to bf16, and attention must stay within a bound worked out from the roundings
its kernels make (``_bound``).  Slots never written hold 0xFF bytes: code 15
and a NaN step, so a read of one shows.
"""

import math

import numpy as np
import pytest
import torch

import oracle.ref as ref
from gqa_attention_preallocated_gb300 import KVCache, KVCError, PagedKVCache
from gqa_attention_preallocated_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

U16, UB = 2.0 ** -11, 2.0 ** -8  # half a unit in the last place of f16, of bf16


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _bf(x):
    return wl.to_storage(x, torch.bfloat16)


def _attend(q, K, V, lens, n_new, window=0, parents=None):
    """(out, sum p |v| / sum p, largest sum |q k| / sqrt d over a query's keys, f32 sums' error) in float64.

    q [B, Hq, T, d]; K: per row values [Hkv, len, d], V: per row (values, steps [Hkv, len]), row b's tokens at
    their positions.

    The last is what adding in float32 may lose: out is sum p s c - sum p s z, both sums of terms up to
    15 p s, added 16 keys at a time by the tensor core (which may truncate: 2^-23 of the sum an addition)
    and a few keys a thread.  So each loses at most (L / 16 + 16) 2^-23 of 15 sum p s."""
    B, Hq, T, d = q.shape
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    dot, add = np.zeros((B, Hq, T, 1)), np.zeros((B, Hq, T, 1))
    for b in range(B):
        n, L = int(n_new[b]), int(lens[b])
        if n == 0:
            continue
        Hkv = K[b].shape[0]
        G = Hq // Hkv
        pos = L - n + np.arange(n)
        key = np.arange(L)
        see = key[None, :] <= pos[:, None]
        if window:
            see &= key[None, :] > pos[:, None] - window
        if parents is not None:
            for t in range(n):
                see[t, L - n:] = False
                for u in ref.tree_path(parents[b], t):
                    see[t, L - n + u] = True
        for h in range(Hkv):
            x = np.einsum("gtd,sd->gts", q[b, h * G:(h + 1) * G, :n], K[b][h]) / math.sqrt(d)
            x = np.where(see[None], x, -np.inf)
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            Vh = np.where(see.any(0)[:, None], V[b][0][h], 0.0)
            Sh = np.where(see.any(0), V[b][1][h], 0.0)
            add[b, h * G:(h + 1) * G, :n, 0] = (p @ Sh) * 15 * (L / 16 + 16) * 2.0 ** -22
            out[b, h * G:(h + 1) * G, :n] = p @ Vh
            mass[b, h * G:(h + 1) * G, :n] = p @ np.abs(Vh)
            a = np.einsum("gtd,sd->gts", np.abs(q[b, h * G:(h + 1) * G, :n]), np.abs(K[b][h])) / math.sqrt(d)
            dot[b, h * G:(h + 1) * G, :n, 0] = np.where(see[None], a, 0.0).max(-1)
    return out, mass, dot, add


def _bound(want, mass, dot, add, rows):
    """Largest |got - want| that the kernels' roundings allow.

    The output is rounded to bf16.  Up to 32 query rows per KV head (and in
    trees) the codes and queries enter the products exactly and only the softmax
    weights are rounded, to f16.  Above, the rows are rounded to f16 on their way
    to the tensor core (K: each score moves by at most U16 * sum |q k| / sqrt d,
    so each weight by twice that; V: by U16) and the weights too.  float32 sums,
    exp2 and the norm add 2^-16 of the mass, and 2^-20 * sum |q k| / sqrt d in
    the scores."""
    up, uv, uk = (U16, 0.0, 0.0) if rows <= 32 else (U16, U16, U16)
    shift = 2 * np.expm1((uk + 2.0 ** -20) * dot)
    return UB * np.abs(want) + mass * (1 + UB) * (up + uv + shift + 2.0 ** -16) + add + 1e-30


class Pair:
    """A 4-bit cache and the rows the oracle says it holds (per row b: [Hkv, len, d] values)."""

    def __init__(self, B, Hkv, d, max_len, window=0, ring=False, page=0, layers=1, layer=0, seed=0):
        self.B, self.Hkv, self.d, self.max_len, self.window, self.ring, self.page = B, Hkv, d, max_len, window, ring, page
        self.layer, self.rng, self.seed = layer, np.random.default_rng(seed + 1000), seed
        if page:
            mpr = max_len // page
            num = B * mpr + 3
            self.c = PagedKVCache(layers, B, Hkv, page, num, mpr, d, dtype="q4")
            self.table = self.rng.permutation(num)[: B * mpr].reshape(B, mpr)
            self.c.block_table.copy_(torch.as_tensor(self.table, dtype=torch.int32))
        else:
            self.c = KVCache(layers, B, Hkv, max_len, d, dtype="q4")
        for bufs in (self.c.k, self.c.v, self.c.k_scale, self.c.v_scale):
            for t in bufs:
                t.view(torch.uint8).fill_(0xFF)
        if window:
            self.c.set_window(window, ring=ring)
        self.x = [[np.zeros((Hkv, 0, d)) for _ in range(B)] for _ in range(2)]  # appended bf16 rows, K and V
        self.calls = 0

    @property
    def lens(self):
        return np.array([r.shape[1] for r in self.x[0]])

    def inputs(self, n_new, T, G, scale=1.0, spread=0.0):
        self.calls += 1
        s = self.seed * 100 + self.calls
        mk = lambda i, H: wl.normal(s, i, (self.B, H, T, self.d))  # noqa: E731
        bias = spread * wl.normal(s, 9, (1, 1, 1, self.d))
        return _bf(mk(1, self.Hkv * G)), _bf(mk(2, self.Hkv) * scale + bias), _bf(mk(3, self.Hkv) * scale)

    def note(self, k, v, n_new):
        for x, new in ((self.x[0], k), (self.x[1], v)):
            new = new.double().numpy()
            for b in range(self.B):
                x[b] = np.concatenate([x[b], new[b, :, : int(n_new[b])]], axis=1)

    def values(self):
        """K values, and V (values, steps), per row."""
        V = [ref.q4_quantize(r) for r in self.x[1]]
        return [ref.q4_store(r) for r in self.x[0]], [(ref.q4_values(*v), v[1]) for v in V]

    def check_out(self, out, q, n_new, T, parents=None, tag=""):
        K, V = self.values()
        want, *about = _attend(q.double().numpy(), K, V, self.lens, n_new, self.window, parents)
        got = out.double().cpu().numpy()
        for b in range(self.B):
            assert np.all(got[b, :, int(n_new[b]):] == 0.0), (tag, b)
        G = q.shape[1] // self.Hkv
        lim = _bound(want, *about, G * T)
        over = np.abs(got - want) - lim
        assert np.isfinite(got).all(), tag
        assert over.max() <= 0, (tag, float(over.max()), float(np.abs(got - want).max()))
        assert self.c.device_status() == 0

    def step(self, n_new, G, T=None, parents=None, split=False, **kw):
        """One chunk: append_attention (or append, then attention) against the oracle."""
        n_new = np.asarray(n_new)
        T = max(1, int(n_new.max())) if T is None else T
        q, k, v = self.inputs(n_new, T, G, **kw)
        if parents is not None:
            out = self.c.append_attention_tree(self.layer, q.cuda(), k.cuda(), v.cuda(), n_new, parents)
        elif split:
            self.c.append(self.layer, k.cuda(), v.cuda(), n_new)
            out = self.c.gqa_attention(self.layer, q.cuda(), n_new)
        else:
            out = self.c.append_attention(self.layer, q.cuda(), k.cuda(), v.cuda(), n_new)
        self.note(k, v, n_new)
        self.last_q = q.cuda()
        assert np.array_equal(self.c.lens(self.layer), self.lens)
        self.check_out(out, q, n_new, T, parents, tag=(self.calls, T, G))
        return out

    def check_store(self):
        """Codes and scale words of every stored position, bit for bit, and the rows read back."""
        kc, vc = (t[self.layer].cpu().numpy() for t in (self.c.k, self.c.v))
        ks, vs = (t[self.layer].cpu().numpy().view(np.uint32) for t in (self.c.k_scale, self.c.v_scale))
        lens = self.lens
        for codes, words, x in ((kc, ks, self.x[0]), (vc, vs, self.x[1])):
            used = np.zeros(words.shape, dtype=bool)
            for b in range(self.B):
                c, s, z = ref.q4_quantize(x[b])
                for a in range(max(0, lens[b] - self.max_len) if self.ring else 0, lens[b]):
                    e, at = (self.table[b, a // self.page], a % self.page) if self.page else (b, a % self.max_len)
                    assert np.array_equal(codes[e, :, at].view(np.uint32), ref.q4_pack(c[:, a])), (b, a)
                    assert np.array_equal(words[e, :, at], ref.q4_scale_words(s[:, a], z[:, a])), (b, a)
                    used[e, :, at] = True
            assert np.all(words[~used] == 0xFFFFFFFF) and np.all(codes[~used[..., : codes.shape[2]]] == 0xFF)
        first = np.maximum(0, lens - self.max_len) if self.ring else np.zeros(self.B, dtype=np.int64)
        K, V = self.c.read(self.layer, first, lens - first)
        for got, x in ((K, self.x[0]), (V, self.x[1])):
            got = got.double().cpu().numpy()
            for b in range(self.B):
                want = ref.bf16_round(ref.q4_store(x[b][:, first[b]:]).astype(np.float32))
                assert np.array_equal(got[b, :, : lens[b] - first[b]], want)
                assert not got[b, :, lens[b] - first[b]:].any()


# ------------------------------------------------------------------ storing
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 256])
def test_append_and_read(d):
    p = Pair(3, 2, d, 67, seed=d)  # an odd length: the scale words' stride is not max_len
    for n in ([1, 0, 1], [17, 64, 3], [0, 3, 40]):
        T = max(n) + 2
        q, k, v = p.inputs(n, T, 1, scale=2.5, spread=3.0)
        p.c.append(0, k.cuda(), v.cuda(), np.array(n))
        p.note(k, v, n)
    p.check_store()


def test_append_special_rows():
    """Rows of zeros, of one sign, of one value, tiny, huge, with NaN and infinities."""
    d, T = 128, 12
    x = wl.normal(5, 1, (1, 1, T, d)).float()
    x[0, 0, 0] = 0
    x[0, 0, 1] = x[0, 0, 1].abs() + 3
    x[0, 0, 2] = -x[0, 0, 2].abs() - 3
    x[0, 0, 3] = 0.75
    x[0, 0, 4] *= 2.0 ** -128
    x[0, 0, 5] *= 2.0 ** -122
    x[0, 0, 6] *= 2.0 ** 120
    x[0, 0, 7, 5] = math.nan
    x[0, 0, 8, 127] = math.inf
    x[0, 0, 9, 0] = -math.inf
    x[0, 0, 10, :2] = torch.tensor([3e38, -3e38])
    x = x.to(torch.bfloat16)
    c = KVCache(1, 1, 1, 16, d, dtype="q4")
    c.append(0, x.cuda(), x.flip(3).contiguous().cuda(), [T])
    codes, s, z = ref.q4_quantize(x.double().numpy()[0, 0])
    assert np.array_equal(c.k[0].cpu().numpy()[0, 0, :T].view(np.uint32), ref.q4_pack(codes))
    assert np.array_equal(c.k_scale[0].cpu().numpy().view(np.uint32)[0, 0, :T], ref.q4_scale_words(s, z))
    k, v = c.read(0, [0], [T])
    got, want = k.double().cpu().numpy()[0, 0], ref.q4_values(codes, s, z)
    want = ref.bf16_round(want.astype(np.float32))
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    assert np.isnan(got[7:11]).all() and np.isfinite(got[[0, 1, 2, 3, 4, 5, 6, 11]]).all()
    assert torch.equal(torch.nan_to_num(v.flip(3), nan=9.0), torch.nan_to_num(k, nan=9.0))


def test_codes_at_ties():
    """Values on the borders between codes round to the even code, as the definition says."""
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    x[0, 0, 0, :16] = torch.arange(16).to(torch.bfloat16) - 7       # range 15: step 1
    x[0, 0, 0, 16:31] = torch.arange(15).to(torch.bfloat16) - 6.5   # every border
    p = KVCache(1, 1, 1, 8, 64, dtype="q4")
    p.append(0, x.cuda(), x.cuda(), [1])
    k, _ = p.read(0, [0], [1])
    want = torch.arange(16).float() - 7
    assert torch.equal(k[0, 0, 0, :16].float().cpu(), want)
    assert torch.equal(k[0, 0, 0, 16:31].float().cpu(), torch.round(torch.arange(15).float() - 6.5))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("page", [0, 128])
def test_read_of_the_other_types(dtype, page):
    B, Hkv, d, L = 2, 2, 64 if dtype != torch.float8_e4m3fn else 128, 256
    io = torch.float32 if dtype == torch.float32 else torch.bfloat16
    if page:
        c = PagedKVCache(1, B, Hkv, page, 5, 2, d, dtype=dtype)
        c.block_table.copy_(torch.tensor([[4, 0], [2, 1]], dtype=torch.int32))
    else:
        c = KVCache(1, B, Hkv, L, d, dtype=dtype)
    ks, vs = np.array([0.01, 0.02], np.float32), np.array([0.5, 0.25], np.float32)
    if dtype == torch.float8_e4m3fn:
        c.set_kv_scales(0, ks, vs)
    k, v = (wl.to_storage(wl.normal(8, i, (B, Hkv, 200, d)), io) for i in (1, 2))
    c.append(0, k.cuda(), v.cuda(), [200, 131])
    out = [torch.full((B, Hkv, 77, d), 5.0, dtype=io, device="cuda") for _ in range(2)]
    c.read(0, [100, 60], [77, 71], k_out=out[0], v_out=out[1])
    for got, x, s in ((out[0], k, ks), (out[1], v, vs)):
        got = got.cpu()
        for b, (f, n) in enumerate(((100, 77), (60, 71))):
            want = x[b, :, f:f + n]
            if dtype == torch.float8_e4m3fn:
                want = np.stack([ref.e4m3_dequantize(ref.e4m3_quantize(want[h].double().numpy(), s[h]), s[h]) for h in range(Hkv)])
                want = torch.from_numpy(ref.bf16_round(want.astype(np.float32))).to(io)
            assert torch.equal(got[b, :, :n], want)
            assert torch.all(got[b, :, n:] == 5.0)


def test_read_through_a_bad_page_is_zeros():
    c = PagedKVCache(1, 1, 1, 128, 2, 2, 128, dtype="q4")
    x = torch.ones(1, 1, 256, 128, dtype=torch.bfloat16, device="cuda")
    c.append(0, x, x, [256])
    c.block_table[0, 1] = 2  # outside 0 .. num_pages - 1
    k, v = c.read(0, [0], [256])
    assert torch.all(k[0, 0, :128] == 1.0) and torch.all(k[0, 0, 128:] == 0.0) and torch.equal(k, v)


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("d", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("G,chunks", [
    (1, [[1, 1, 0], [1, 1, 1], [1, 0, 1]]),              # from empty rows on, single tokens
    (4, [[63, 1, 130], [1, 1, 1], [1, 0, 1], [1, 1, 1]]),  # decode around a tile's end
    (3, [[70, 128, 5], [4, 5, 1], [5, 5, 5]]),           # short verify: 12 to 15 rows per KV head
    (8, [[129, 64, 0], [2, 1, 2], [3, 4, 4]]),           # 16 to 32 rows
    (7, [[40, 90, 77], [9, 9, 8]]),                      # 63 rows
])
def test_chunks(d, G, chunks):
    p = Pair(3, 2, d, 203, seed=d + G)
    for i, n in enumerate(chunks):
        p.step(n, G, T=max(n) + (1 if i == 1 else 0), spread=1.0 if i == 0 else 0.0)
    p.check_store()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 5])
def test_prefill(d, G):
    p = Pair(2, 2, d, 700, seed=G)
    p.step([300, 129], G, spread=1.0)
    p.step([150, 200], G)
    p.step([0, 33], G, split=True)
    p.step([1, 1], G)
    p.check_store()


@pytest.mark.parametrize("d", [64, 128])
def test_pages(d):
    p = Pair(3, 2, d, 512, page=128, seed=4)
    for n, G in (([130, 0, 257], 4), ([1, 1, 1], 4), ([126, 5, 0], 4), ([4, 3, 4], 4), ([1, 1, 1], 8)):
        p.step(n, G)
    p.check_store()


def test_pages_of_odd_size():
    p = Pair(2, 2, 96, 90, page=18, seed=6)
    for n in ([19, 35], [1, 1], [5, 2], [17, 18]):
        p.step(n, 4)
    p.check_store()


@pytest.mark.parametrize("d,page", [(64, 0), (128, 0), (128, 128), (96, 0)])
@pytest.mark.parametrize("window", [1, 7, 64, 150])
def test_window(d, page, window):
    p = Pair(2, 2, d, 512, window=window, page=page, seed=window)
    for n in ([200, 3], [1, 1], [140, 129], [5, 4], [1, 0], [1, 1]):
        p.step(n, 4)


@pytest.mark.parametrize("d", [64, 96, 128])
def test_ring(d):
    p = Pair(2, 2, d, 256, window=100, ring=True, seed=d)
    for n in ([150, 157], [100, 1], [1, 1], [4, 3], [120, 157], [1, 1], [1, 0], [150, 60], [1, 1]):
        p.step(n, 4)
    p.check_store()


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("G,T", [(1, 6), (4, 4), (4, 7), (8, 8)])
def test_trees(d, G, T):
    rng = np.random.default_rng(G * T)
    p = Pair(3, 2, d, 300, seed=T)
    p.step([100, 0, 64], G)
    for n in ([T, T, T - 1], [T, 1, T]):
        parents = np.array([[rng.integers(-1, t) if t else -1 for t in range(T)] for _ in range(3)])
        p.step(n, G, T=T, parents=parents)
    p.check_store()


def test_scales_of_very_different_size():
    """Rows whose steps span 2^40, and queries of very different size, neither overflow nor vanish."""
    p = Pair(2, 1, 128, 300, seed=3)
    n = 120
    f = torch.tensor(2.0) ** torch.linspace(-20, 20, n)[None, None, :, None]
    q, k, v = p.inputs([n, n], n, 4)
    k = _bf(k.double() * 2.0 ** -3)
    v = _bf(v.double() * f.double())
    p.c.append(0, k.cuda(), v.cuda(), [n, n])
    p.note(k, v, [n, n])
    for T, scale in ((1, 1.0), (1, 2.0 ** -60), (1, 2.0 ** 4), (3, 1.0), (40, 1.0)):
        q, _, _ = p.inputs([T, T], T, 4)
        q = _bf(q.double() * scale)
        out = p.c.gqa_attention(0, q.cuda(), [T, T])
        p.check_out(out, q, [T, T], T, tag=(T, scale))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", [(4, 100), (2, 150), (8, 10)])
def test_steps_that_change_from_tile_to_tile(d, G, T):
    """V of some tiles is all zeros, of others 2^12 times the last tile's; K's too: the tiles' powers of two move."""
    p = Pair(2, 1, d, 1100, seed=d + T)
    n = 900
    q, k, v = p.inputs([n, n], n, 1)
    at = torch.arange(n)[None, None, :, None]
    v = _bf(torch.where(at < 256, torch.zeros(()), v.double() * 2.0 ** (4.0 * (at // 128)).double() * (at // 128 % 3 != 0)))
    k = _bf(k.double() * torch.where(at // 128 % 2 == 0, 2.0 ** -6, 1.0).double())
    p.c.append(0, k.cuda(), v.cuda(), [n, n])
    p.note(k, v, [n, n])
    p.step([T, T - 3], G, T=T)
    p.c.truncate([120, 240])  # nothing but zeros before the chunk
    for x in p.x:
        x[0], x[1] = x[0][:, :120], x[1][:, :240]
    p.step([T, 1], G, T=T)


def test_nan_rows_reach_their_queries_only():
    """A NaN row shows in the queries that see it and nowhere else (window, tree and causal masks)."""
    for d in (64, 96, 128):
        p = Pair(1, 1, d, 256, window=8, seed=d)
        q, k, v = p.inputs([40], 40, 2)
        v = v.clone()
        v[0, 0, 10, 3] = math.nan
        out = p.c.append_attention(0, q.cuda(), k.cuda(), v.cuda(), [40]).float().cpu()
        bad = torch.isnan(out).any(-1)[0]
        assert bad[:, 10:18].all() and not bad[:, :10].any() and not bad[:, 18:].any()
        # decode: the row has left the window
        q, k, v = p.inputs([1], 1, 2)
        assert torch.isfinite(p.c.append_attention(0, q.cuda(), k.cuda(), v.cuda(), [1])).all()
        t = Pair(1, 1, d, 64, seed=d)
        t.step([20], 2)
        q, k, v = t.inputs([3], 3, 2)
        k, v = k.clone(), v.clone()
        k[0, 0, 1, 0], v[0, 0, 1, 5] = math.inf, math.nan
        out = t.c.append_attention_tree(0, q.cuda(), k.cuda(), v.cuda(), [3], [[-1, 0, 0]]).float().cpu()
        bad = torch.isnan(out).any(-1)[0]
        assert bad[:, 1].all() and not bad[:, 0].any() and not bad[:, 2].any()


@pytest.mark.parametrize("d,T", [(64, 1), (128, 1), (128, 4), (64, 4), (96, 2), (128, 20)])
def test_queries_of_very_different_size_and_nan_queries(d, T):
    """Heads and tokens whose queries differ by 2^60 each keep their precision; a NaN or infinite query is NaN alone."""
    p = Pair(2, 2, d, 200, seed=d + T)
    p.step([150, 90], 4)
    q, k, v = p.inputs([T, T], T, 4)
    size = torch.tensor(2.0) ** torch.tensor([0.0, -40.0, 3.0, -60.0])
    q = _bf(q.double() * size.double().repeat(2)[None, :, None, None])
    p.c.append(0, k.cuda(), v.cuda(), [T, T])
    p.note(k, v, [T, T])
    out = p.c.gqa_attention(0, q.cuda(), [T, T])
    p.check_out(out, q, [T, T], T)
    bad = q.clone()
    bad[0, 1, 0, 5], bad[1, 6, T - 1, 0] = math.nan, math.inf
    got = p.c.gqa_attention(0, bad.cuda(), [T, T])
    lost = torch.isnan(got).all(-1).cpu()
    assert lost[0, 1, 0] and lost[1, 6, T - 1]
    lost[0, 1, 0] = lost[1, 6, T - 1] = False
    assert not lost.any()
    keep = torch.ones_like(lost)
    keep[0, 1, 0] = keep[1, 6, T - 1] = False
    assert torch.equal(got.cpu()[keep], out.cpu()[keep])


def test_layers_truncate_and_host_buffers():
    p = Pair(2, 2, 128, 256, layers=2, layer=1, seed=2)
    p.step([70, 33], 4)
    p.c.append(0, *(t.cuda() for t in p.inputs([70, 33], 70, 4)[1:]), [70, 33])
    p.c.truncate([50, 33])
    for x in p.x:
        x[0] = x[0][:, :50]
    p.step([1, 1], 4)
    q, k, v = (t.pin_memory() for t in p.inputs([2, 1], 3, 4))
    out = torch.zeros(q.shape, dtype=torch.bfloat16).pin_memory()
    p.c.append_attention_host(1, q, k, v, [2, 1], out)
    p.c.host_copies_done()
    torch.cuda.synchronize()
    p.note(k, v, [2, 1])
    p.check_out(out, q, [2, 1], 3)


@pytest.mark.parametrize("d,G,page,T", [(128, 4, 0, 2), (64, 4, 0, 2), (128, 8, 128, 1), (128, 3, 0, 2), (128, 4, 0, 6),
                                        (64, 8, 128, 4), (128, 16, 0, 2)])
def test_device_steps_and_graph(d, G, page, T):
    """Device-resident lengths: steps run eagerly and replayed from a graph, a rejected step, and the lengths back."""
    p = Pair(3, 2, d, 256, page=page, seed=d + G)
    p.step([100, 0, 126], G)
    q, k, v = (torch.zeros(3, H, T, d, dtype=torch.bfloat16, device="cuda") for H in (2 * G, 2, 2))
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, ws = torch.zeros_like(q), torch.zeros(p.c.workspace_bytes(2 * G, T), dtype=torch.uint8, device="cuda")
    p.c.lens_to_device()

    def feed(n_new):
        i = p.inputs(n_new, T, G)
        for dst, src in zip((q, k, v), i):
            dst.copy_(src)
        n.copy_(torch.tensor(n_new, dtype=torch.int32))
        return i

    def check(i, n_new):
        p.note(i[1], i[2], n_new)
        K, V = p.values()
        want, *about = _attend(i[0].double().numpy(), K, V, p.lens, n_new)
        got = out.double().cpu().numpy()
        assert (np.abs(got - want) - _bound(want, *about, G * T)).max() <= 0
        assert p.c.device_status(ws) == 0

    i = feed([T, 1, 0])
    p.c.decode_step(0, q, k, v, n, out, ws)
    check(i, [T, 1, 0])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    feed([0, 0, 0])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        p.c.decode_step(0, q, k, v, n, out, ws)
    for n_new in ([1, 1, T], [T, 0, 1], [0, T, T]):
        i = feed(n_new)
        graph.replay()
        check(i, n_new)
    feed([200, 0, 0] if T >= 200 else [T + 1, 0, 0])  # n_new outside 0 .. T: the whole step is rejected
    graph.replay()
    with pytest.raises(KVCError):
        p.c.device_status(ws)
    with pytest.raises(KVCError):
        p.c.read(0, [0, 0, 0], [1, 1, 1])
    p.c.lens_from_device()
    assert np.array_equal(p.c.lens(0), p.lens)
    p.check_store()
    p.step([1, 1, 1], G)


@pytest.mark.parametrize("d", [64, 128])
def test_allocation_free_call(d):
    p = Pair(3, 2, d, 300, seed=d)
    p.step([100, 1, 260], 4)
    for T in (1, 4, 30):
        q, k, v = p.inputs([T, 0, T], T, 4)
        p.c.append(0, k.cuda(), v.cuda(), [T, 0, T])
        p.note(k, v, [T, 0, T])
        out = torch.empty_like(q, device="cuda")
        p.c.gqa_attention_noalloc(0, q.cuda(), [T, 0, T], out=out)
        assert p.c.noalloc_status() == 0
        p.check_out(out, q, [T, 0, T], T)
    c = KVCache(1, 1, 1, 64, 96, dtype="q4")
    q = torch.zeros(1, 1, 1, 96, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(KVCError):  # the generic kernel's head widths have no such call, as for the other types
        c.gqa_attention_noalloc(0, q, [0], out=q.clone())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hkv,G,L", [(1, 1, 8, 20000), (2, 8, 4, 5000), (40, 4, 2, 700), (5, 2, 16, 3001)])
def test_longer_decode(d, B, Hkv, G, L):
    """Units cut across many CTAs, whole units, and several units in one CTA."""
    rng = np.random.default_rng(L)
    p = Pair(B, Hkv, d, L + 8, seed=L)
    n = rng.integers(L // 2, L + 1, size=B)
    n[0] = L
    if B > 2:
        n[1] = 0
    q, k, v = p.inputs(n, L, 1)
    p.c.append(0, k.cuda(), v.cuda(), n)
    p.note(k, v, n)
    out = p.step(np.ones(B, dtype=np.int64), G)
    p.c.truncate(p.lens)
    q = p.inputs(np.ones(B), 1, G)[0].cuda()
    a = p.c.gqa_attention(0, q, np.ones(B))
    for _ in range(3):  # the same bits every time
        assert torch.equal(a, p.c.gqa_attention(0, q, np.ones(B)))


@pytest.mark.parametrize("d,G,T,page,window", [(128, 4, 1, 0, 0), (128, 4, 4, 0, 0), (128, 5, 4, 128, 0), (128, 8, 4, 0, 0),
                                               (128, 3, 3, 0, 200), (64, 4, 1, 128, 0), (64, 4, 4, 0, 0), (64, 5, 4, 0, 0),
                                               (64, 8, 4, 0, 0), (128, 8, 1, 0, 130)])
def test_units_for_every_sm(d, G, T, page, window):
    """Rows times KV heads at least the SMs (156 units): each warp group takes units of its own, of one tile to
    seven; then device-resident steps, with every row, with few, and with none."""
    B, Hkv = 39, 4
    p = Pair(B, Hkv, d, 896, window=window, page=page, seed=d + G + T)
    n = p.rng.integers(0, 860, size=B)
    n[:4] = 0, 1, 128, 860
    q, k, v = p.inputs(n, 860, 1)
    p.c.append(0, k.cuda(), v.cuda(), n)
    p.note(k, v, n)
    some = np.where(np.arange(B) % 5 == 2, 0, p.rng.integers(1, T + 1, size=B))
    out = p.step(some, G, T=T)
    again = p.c.gqa_attention(0, p.last_q, some)
    assert torch.equal(out, again) and torch.equal(out, p.c.gqa_attention(0, p.last_q, some))
    few = np.where(np.arange(B) % 9 == 1, T, 0)  # (units with tiles are fewer than the SMs: the groups work together)
    p.step(few, G, T=T)
    ws = torch.zeros(p.c.workspace_bytes(Hkv * G, T), dtype=torch.uint8, device="cuda")
    p.c.lens_to_device()
    one = np.zeros(B, dtype=np.int64)
    one[3] = 1
    for n_new in (some, one, np.zeros(B, dtype=np.int64), np.minimum(some, 1)):
        q, k, v = p.inputs(n_new, T, G)
        out = torch.full_like(q, 7, device="cuda")
        p.c.decode_step(0, q.cuda(), k.cuda(), v.cuda(), torch.as_tensor(n_new, dtype=torch.int32, device="cuda"), out, ws)
        p.note(k, v, n_new)
        assert p.c.device_status(ws) == 0
        p.check_out(out, q, n_new, T)
    p.c.lens_from_device()
    p.check_store()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,G,window", [(200, 3, 0), (40, 4, 0), (9, 4, 0), (150, 4, 3000)])
def test_long_prefill(d, T, G, window):
    """Many key tiles a block, blocks cut into pieces, ragged priors and chunks: the converters' slots turn over often."""
    p = Pair(3, 2, d, 8300, window=window, seed=T + G)
    n = [8011, 3000, 5557]
    q, k, v = p.inputs(n, 8011, 1)
    p.c.append(0, k.cuda(), v.cuda(), n)
    p.note(k, v, n)
    for n_new in ([T, T - 1, T // 2], [1, T, T]):
        out = p.step(n_new, G, T=T)
        for _ in range(3):
            again = p.c.gqa_attention(0, p.last_q, n_new)
            assert torch.equal(out, again)


@pytest.mark.parametrize("d,G,T", [(64, 4, 1), (128, 4, 1), (128, 4, 4), (64, 4, 4)])
def test_more_units_than_the_workspace_counts(d, G, T):
    """9000 units: the separate merge, with units for every SM and with a few; host and device plans."""
    rows, Hkv, L = 20, 9, 300
    p = Pair(rows, Hkv, d, L + 20, seed=d + T)
    n = p.rng.integers(L // 2, L + 1, size=rows)
    q, k, v = p.inputs(n, L, 1)
    p.c.append(0, k.cuda(), v.cuda(), n)
    p.note(k, v, n)
    big = KVCache(1, 1000, Hkv, L + 20, d, dtype="q4")
    for to, src in ((big.k, p.c.k), (big.v, p.c.v), (big.k_scale, p.c.k_scale), (big.v_scale, p.c.v_scale)):
        to[0][:rows].copy_(src[0])
    big.set_lens(0, np.concatenate([n, np.zeros(1000 - rows, dtype=np.int64)]))
    assert big.B * big.Hkv > 8192
    for live in (rows, 3):
        n_new = np.where(np.arange(1000) < live, T, 0)
        q = torch.zeros(1000, Hkv * G, T, d, dtype=torch.bfloat16)
        q[:rows] = p.inputs(n_new[:rows], T, G)[0]
        out = big.gqa_attention(0, q.cuda(), n_new)
        assert not out[rows:].any() and big.device_status() == 0
        p.check_out(out[:rows], q[:rows], n_new[:rows], T)
    ws = torch.zeros(big.workspace_bytes(Hkv * G, T), dtype=torch.uint8, device="cuda")
    big.lens_to_device()
    q, k, v = (torch.zeros(1000, H, T, d, dtype=torch.bfloat16) for H in (Hkv * G, Hkv, Hkv))
    n_new = np.where(np.arange(1000) < rows, T, 0)
    for to, src in zip((q, k, v), p.inputs(n_new[:rows], T, G)):
        to[:rows] = src
    out = torch.full_like(q, 7, device="cuda")
    big.decode_step(0, q.cuda(), k.cuda(), v.cuda(), torch.as_tensor(n_new, dtype=torch.int32, device="cuda"), out, ws)
    p.note(k[:rows], v[:rows], n_new[:rows])
    assert big.device_status(ws) == 0 and not out[rows:].any()
    p.check_out(out[:rows], q[:rows], n_new[:rows], T)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T,window", [(3, 130, 0), (1, 260, 0), (5, 200, 90), (4, 129, 0)])
def test_long_ragged_chunks_of_packed_rows(d, G, T, window):
    """Chunks of 128 queries and more whose heads' rows share tiles; what stands in padded queries does not matter."""
    p = Pair(4, 2, d, 700, window=window, seed=d + T)
    p.step([300, 0, 257, 400], G, T=400)
    n_new = [T, T - 3, 0, 70]
    q, k, v = p.inputs(n_new, T, G)
    for b in range(4):
        for x in (q, k, v):
            x[b, :, n_new[b]:] = float("nan")
    out = p.c.append_attention(0, q.cuda(), k.cuda(), v.cuda(), n_new)
    p.note(k, v, n_new)
    for b in range(4):
        assert not out[b, :, n_new[b]:].any()
        q[b, :, n_new[b]:] = 0
    p.check_out(out, q, n_new, T)
    p.check_store()


def test_streams_and_two_caches():
    """Calls of two caches on two streams at once, each with its own workspace."""
    a, b = Pair(2, 2, 128, 600, seed=1), Pair(2, 2, 64, 600, seed=2)
    for p in (a, b):
        p.step([500, 333], 4)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = []
    for p, s in zip((a, b), streams):
        i = p.inputs([1, 1], 1, 4)
        gpu = [t.cuda() for t in i]
        ws = torch.zeros(p.c.workspace_bytes(8, 1), dtype=torch.uint8, device="cuda")
        work.append((p, s, i, gpu, ws, torch.empty_like(gpu[0])))
    torch.cuda.synchronize()
    for p, s, i, gpu, ws, out in work:
        p.c.append_attention(0, *gpu, [1, 1], out=out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for p, s, i, gpu, ws, out in work:
        p.note(i[1], i[2], [1, 1])
        p.check_out(out, i[0], [1, 1], 1)


def test_refusals():
    c = KVCache(1, 1, 1, 64, 128, dtype="q4")
    q = torch.zeros(1, 2, 1, 128, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (q.float(), q[..., :64], q.transpose(1, 2)):
        with pytest.raises(KVCError):
            c.append_attention(0, bad, kv, kv, [1])
    with pytest.raises(KVCError):
        c.set_kv_scales(0, [1.0], [1.0])
    with pytest.raises(KVCError):
        KVCache(1, 1, 1, 64, 128, dtype=torch.bfloat16, k_scales=[q])
    with pytest.raises(KVCError):
        KVCache(1, 1, 1, 64, 128, dtype="q4", k_bufs=[torch.zeros(1, 1, 64, 128, dtype=torch.uint8, device="cuda")])
    with pytest.raises(KVCError):
        c.read(0, [0], [1])
    with pytest.raises(KVCError):
        c.read(0, [0], [0], k_out=kv)
    with pytest.raises(KVCError):
        c.append(0, kv.expand(1, 1, 65, 128).contiguous(), kv.expand(1, 1, 65, 128).contiguous(), [65])
    assert c.lens(0)[0] == 0
