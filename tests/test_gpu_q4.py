"""The 4-bit cache on the GPU: what it holds, the attention over it, and its pages back as bf16."""
import numpy as np
import pytest
import torch

import q4_ref as ref
import sparse_paged_kv_score_gb300 as spkv
from helpers import DEV, bf, f32, host_bits, i32

pytestmark = pytest.mark.gpu


def u8(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.uint8)).to(DEV)


class Cache:
    """A 4-bit cache of N(0, 1) rows with its handle; page p of request b is page_table[b, p]."""

    def __init__(self, Hk, B, np_max, seq_len, seed=0, junk=False, sums=True, ksum_dtype=torch.float32, key_scale=1.0):
        rng = np.random.default_rng(seed)
        self.Hk, self.B, self.np_max = Hk, B, np_max
        self.n_phys = B * np_max + 1
        self.gk = (rng.uniform(0.5, 2, Hk) * 5 / 2688).astype(np.float32)
        self.gv = (rng.uniform(0.5, 2, Hk) * 5 / 2688).astype(np.float32)
        shape = (Hk, self.n_phys, 64, 128)
        self.blob = ref.pool_of(ref.bf16(rng.standard_normal(shape) * key_scale), ref.bf16(rng.standard_normal(shape)),
                                self.gk, self.gv)
        self.pt = rng.permutation(self.n_phys)[:B * np_max].reshape(B, np_max).astype(np.int32)
        self.L = np.asarray(seq_len, np.int32)
        self.cnt = np.zeros(self.n_phys, np.int32)
        for b in range(B):
            for p in range((int(self.L[b]) + 63) // 64):
                self.cnt[self.pt[b, p]] = min(64, self.L[b] - 64 * p)
        if junk:   # bytes behind a page's last token: every scale NaN, codes all ones
            for p in range(self.n_phys):
                for t in range(self.cnt[p], 64):
                    for at in (ref.KC, ref.VC, ref.KS, ref.VS):
                        self.blob[:, p, at[t]] = 0xFF
        self.pool = u8(self.blob)
        self.ksum = torch.zeros(Hk, self.n_phys, 4, 128, dtype=ksum_dtype, device=DEV) if sums else None
        self.cnt_d = i32(self.cnt) if sums else None
        self.gk_d, self.gv_d = f32(self.gk), f32(self.gv)
        self.handle = spkv.paged_kv_create_q4(self.pool, self.gk_d, self.gv_d, self.ksum, self.cnt_d, max_units=B * Hk)

    def select(self, stride, rng, counts=None):
        """Random ascending selections; each ends with the local page unless counts says how many."""
        sel = np.full((self.B, self.Hk, stride), -1, np.int32)
        n = np.zeros((self.B, self.Hk), np.int32)
        for b in range(self.B):
            pages = (int(self.L[b]) + 63) // 64
            for h in range(self.Hk):
                k = min(stride, pages) if counts is None else min(stride, pages, int(counts[b, h]))
                x = rng.permutation(pages - 1)[:max(0, k - 1)] if pages > 1 else np.zeros(0, int)
                lst = sorted(list(x) + [pages - 1])[:k]
                sel[b, h, :k], n[b, h] = lst[:k], k
        return sel, n

    def attend(self, q, sel, n, **kw):
        B, Hq = q.shape[:2]
        out = torch.full((B, Hq, 128), 7.0, device=DEV)
        lse = torch.full((B, Hq), 7.0, device=DEV)
        spkv.sparse_decode_attn(self.handle, q, i32(self.pt), i32(sel), i32(n), i32(self.L), out, lse, **kw)
        return out, lse


def queries(B, Hq, seed=1, scale=1.0):
    x = ref.bf16(np.random.default_rng(seed).standard_normal((B, Hq, 128)) * scale)
    return x, bf(ref.bf16_bits(x))


def check(out, lse, want):
    o, l, eo, el = want
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(l)
    assert np.array_equal(empty, np.isneginf(lse))
    assert np.all(out[empty] == 0)
    d = np.abs(out - o).max(-1)
    assert np.all(d <= eo), (d / np.maximum(eo, 1e-30)).max()
    d = np.abs(lse[~empty] - l[~empty])
    assert np.all(d <= el[~empty]), (d / el[~empty]).max()


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (1, 1), (3, 3), (6, 2), (5, 1), (8, 1), (18, 2), (16, 1)])
@pytest.mark.parametrize("L", [1, 15, 64, 65, 400])
def test_attention_sizes(Hq, Hk, L):
    B = 3
    c = Cache(Hk, B, (L + 63) // 64 + 1, [L, max(1, L - 1), max(1, L // 2)], seed=L, junk=True)
    rng = np.random.default_rng(L)
    sel, n = c.select(max(1, (L + 63) // 64), rng)
    qx, q = queries(B, Hq)
    out, lse = c.attend(q, sel, n)
    assert spkv.get_device_error(c.handle) == (0, 0)
    check(out, lse, ref.attention(qx, c.blob, c.gk, c.gv, c.pt, sel, n, c.L))


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (10, 2), (16, 1)])
def test_attention_ragged_selections(Hq, Hk):
    """Selections of every length, empty ones too, many pages in one of them."""
    B = 9
    c = Cache(Hk, B, 70, [4480, 1, 64, 100, 900, 4000, 65, 2222, 4410], seed=5, junk=True)
    rng = np.random.default_rng(2)
    counts = rng.integers(0, 68, (B, Hk))
    counts[0], counts[1], counts[4] = 67, 0, 0
    sel, n = c.select(67, rng, counts)
    qx, q = queries(B, Hq)
    out, lse = c.attend(q, sel, n)
    assert spkv.get_device_error(c.handle) == (0, 0)
    check(out, lse, ref.attention(qx, c.blob, c.gk, c.gv, c.pt, sel, n, c.L))


@pytest.mark.parametrize("Hq,Hk,B,pages", [(8, 2, 8, 1200), (16, 1, 9, 2000), (6, 1, 3, 7000), (32, 8, 32, 65), (40, 8, 30, 70),
                                             (16, 1, 200, 60)])
def test_attention_long_lists(Hq, Hk, B, pages):
    """More pages to a CTA than its rings hold, from few physical pages that repeat (a repeated page's
    weights count as often as it is listed); an odd number of units of uneven lengths."""
    c = Cache(Hk, 1, 12, [768], seed=21)
    rng = np.random.default_rng(7)
    which = rng.integers(0, 12, (B, pages))
    pt = c.pt[0][which].astype(np.int32)
    n = rng.integers(pages // 2, pages + 1, (B, Hk)).astype(np.int32)
    n[0, 0] = pages
    sel = np.tile(np.arange(pages, dtype=np.int32), (B, Hk, 1))
    qx, q = queries(B, Hq)
    out, lse = torch.zeros(B, Hq, 128, device=DEV), torch.zeros(B, Hq, device=DEV)
    L = i32(np.full(B, 64 * pages))
    h = spkv.paged_kv_create_q4(c.pool, c.gk_d, c.gv_d, None, None, max_units=B * Hk)
    spkv.sparse_decode_attn(h, q, i32(pt), i32(sel), i32(n), L, out, lse)
    assert spkv.get_device_error(h) == (0, 0)
    G = Hq // Hk
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for b in range(B):
        for g in range(Hq):
            kv = g // G
            k = ref.rows(c.blob[kv, c.pt[0]], True).reshape(-1, 128) * float(c.gk[kv])
            v = ref.rows(c.blob[kv, c.pt[0]], False).reshape(-1, 128) * float(c.gv[kv])
            times = np.repeat(np.bincount(which[b, :n[b, kv]], minlength=12), 64)
            x = k @ qx[b, g].astype(np.float64) / np.sqrt(128)
            p = times * np.exp(x - x.max())
            want, wl = p @ v / p.sum(), x.max() + np.log(p.sum())
            # as ref.attention, and the fp32 sums of up to 64 pages / 14 terms a lane, rounded to nearest
            dx = 136 * 2.0 ** -23 * (np.abs(k) @ np.abs(qx[b, g].astype(np.float64))).max() / np.sqrt(128)
            dx += 2.0 ** -19 + pages * 4 * 2.0 ** -24
            assert np.abs(out[b, g] - want).max() <= 2 * dx * np.abs(v).max()
            assert abs(lse[b, g] - wl) <= dx * (1 + abs(wl))


@pytest.mark.parametrize("B,Hk,G,most", [(100, 3, 2, 7), (257, 1, 9, 3), (512, 8, 1, 2), (300, 2, 4, 12)])
@pytest.mark.parametrize("empty", [0.0, 0.5, 0.99])
def test_attention_many_units(B, Hk, G, most, empty):
    """More units than are looked up at a time, most of them short or empty, and two long ones."""
    rng = np.random.default_rng(B + most)
    c = Cache(Hk, 2, 40, [2560, 2500], seed=B)
    c.handle = spkv.paged_kv_create_q4(c.pool, c.gk_d, c.gv_d, c.ksum, c.cnt_d, max_units=B * Hk)
    full = c.pt[0][:39]      # pages of 64 tokens; requests share them
    c.B, c.np_max, c.L = B, 39, np.full(B, 39 * 64, np.int32)
    c.pt = np.stack([rng.permutation(full) for _ in range(B)]).astype(np.int32)
    n = rng.integers(1, most + 1, (B, Hk)).astype(np.int32)
    n[rng.random((B, Hk)) < empty] = 0
    n[B // 3, 0], n[B - 2, Hk - 1] = 39, 31
    sel = np.tile(np.arange(39, dtype=np.int32), (B, Hk, 1))
    x, q = queries(B, G * Hk, seed=B)
    out, lse = c.attend(q, sel, n)
    assert spkv.get_device_error(c.handle) == (0, 0)
    check(out, lse, ref.attention(x, c.blob, c.gk, c.gv, c.pt, sel, n, c.L))


@pytest.mark.parametrize("B,Hk,G,pages", [(1, 1, 4, 2000), (61, 1, 9, 129), (40, 2, 5, 300), (200, 1, 2, 40), (3, 1, 1, 20000),
                                           (64, 2, 16, 70), (128, 2, 1, 9), (300, 1, 4, 17)])
@pytest.mark.parametrize("short", [0, 1, 2])
def test_attention_dealing(B, Hk, G, pages, short):
    """Lists of one length, lists a little shorter (dealt by unit as well), and lists of every length, over few physical
    pages: for each list the mean of its pages' weighted values."""
    rng = np.random.default_rng(pages + short)
    c = Cache(Hk, 1, 12, [768], seed=B)
    h = spkv.paged_kv_create_q4(c.pool, c.gk_d, c.gv_d, None, None, max_units=B * Hk)
    which = rng.integers(0, 12, (B, pages))
    pt = c.pt[0][which].astype(np.int32)
    n = np.full((B, Hk), pages, np.int32)
    if short:
        n -= rng.integers(0, (pages // 20 if short == 1 else pages) + 1, (B, Hk)).astype(np.int32)
    sel = np.tile(np.arange(pages, dtype=np.int32), (B, Hk, 1))
    x, q = queries(B, G * Hk, seed=pages)
    out, lse = torch.zeros(B, G * Hk, 128, device=DEV), torch.zeros(B, G * Hk, device=DEV)
    for _ in range(2):     # the second call finds the workspace as the first left it
        spkv.sparse_decode_attn(h, q, i32(pt), i32(sel), i32(n), i32(np.full(B, 64 * pages)), out.fill_(7), lse.fill_(7))
        assert spkv.get_device_error(h) == (0, 0)
        o, l = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        for kv in range(Hk):
            k = ref.rows(c.blob[kv, c.pt[0]], True).reshape(-1, 128) * float(c.gk[kv])
            v = ref.rows(c.blob[kv, c.pt[0]], False).reshape(12, 64, 128) * float(c.gv[kv])
            for g in range(kv * G, kv * G + G):
                y = x[:, g].astype(np.float64) @ k.T / np.sqrt(128)       # [B][12 * 64]
                dx = 136 * 2.0 ** -23 * (np.abs(x[:, g].astype(np.float64)) @ np.abs(k).T).max() / np.sqrt(128)
                m = y.max(1)
                w = np.exp(y - m[:, None]).reshape(B, 12, 64)
                num, den = np.einsum("bpt,ptd->bpd", w, v), w.sum(2)
                for b in range(B):
                    times = np.bincount(which[b, :n[b, kv]], minlength=12)
                    if n[b, kv] == 0:
                        assert np.all(o[b, g] == 0) and np.isneginf(l[b, g])
                        continue
                    s = times @ den[b]
                    assert np.abs(o[b, g] - times @ num[b] / s).max() <= 2 * (dx + 2.0 ** -19) * np.abs(v).max()
                    assert abs(l[b, g] - m[b] - np.log(s)) <= dx + 2.0 ** -19 * (1 + abs(l[b, g]))


@pytest.mark.parametrize("q_scale,key_scale", [(1e-6, 1.0), (30.0, 1.0), (1e4, 1e-3), (1.0, 0.0)])
def test_attention_score_ranges(q_scale, key_scale):
    """Flat and peaked weights, queries outside f16's range, keys of zeros: the running maximum rises."""
    c = Cache(2, 2, 9, [530, 77], seed=7, key_scale=key_scale)
    sel, n = c.select(9, np.random.default_rng(3))
    qx, q = queries(2, 8, scale=q_scale)
    out, lse = c.attend(q, sel, n)
    check(out, lse, ref.attention(qx, c.blob, c.gk, c.gv, c.pt, sel, n, c.L))


def test_attention_rising_scores():
    """Each page's keys score far above the last one's, so the reference moves at every page."""
    c = Cache(1, 1, 12, [12 * 64 - 5], seed=8)
    k = np.zeros((1, c.n_phys, 64, 128), np.float32)
    qx, q = queries(1, 4, seed=9)
    for p in range(12):
        k[0, c.pt[0, p]] = ref.bf16(qx[0, 0] * (0.02 * (p + 1) ** 2))
    v = ref.bf16(np.random.default_rng(4).standard_normal(k.shape))
    c.blob[:] = ref.pool_of(k, v, c.gk, c.gv)
    c.pool.copy_(u8(c.blob))
    sel, n = c.select(12, np.random.default_rng(3))
    out, lse = c.attend(q, sel, n)
    check(out, lse, ref.attention(qx, c.blob, c.gk, c.gv, c.pt, sel, n, c.L))


def test_attention_passes_nan_on():
    """A NaN key scale of an attended token makes its unit's outputs NaN, and no other unit's."""
    c = Cache(2, 2, 3, [150, 150], seed=11)
    c.blob[0, c.pt[0, 1], ref.KS[5]] = 0x7F
    c.pool.copy_(u8(c.blob))
    sel, n = c.select(3, np.random.default_rng(3))
    _, q = queries(2, 8)
    out, lse = c.attend(q, sel, n)
    assert torch.isnan(out[0, :4]).all() and torch.isnan(lse[0, :4]).all()
    assert torch.isfinite(out[0, 4:]).all() and torch.isfinite(out[1]).all()


def test_attention_bad_entries_are_skipped():
    """Page ids and physical pages out of range are flagged and left out; the others attend."""
    c = Cache(2, 2, 6, [380, 200], seed=12)
    sel, n = c.select(4, np.random.default_rng(3))
    good, gn = sel.copy(), n.copy()
    sel[0, 1, 1] = 6            # past the table
    good[0, 1], gn[0, 1] = np.concatenate([np.delete(good[0, 1], 1), [-1]]), n[0, 1] - 1
    pt = c.pt.copy()
    dead = int(sel[1, 0, 0])
    pt[1, dead] = c.n_phys
    for h in range(2):
        keep = [x for x in good[1, h, :gn[1, h]] if x != dead]
        good[1, h, :], gn[1, h] = -1, len(keep)
        good[1, h, :len(keep)] = keep
    qx, q = queries(2, 8)
    out, lse = torch.zeros(2, 8, 128, device=DEV), torch.zeros(2, 8, device=DEV)
    spkv.sparse_decode_attn(c.handle, q, i32(pt), i32(sel), i32(n), i32(c.L), out, lse)
    st, bits = spkv.get_device_error(c.handle)
    assert st == -4 and bits == spkv.DEVERR["PAGE_ID"] | spkv.DEVERR["PHYS"]
    check(out, lse, ref.attention(qx, c.blob, c.gk, c.gv, c.pt, good, gn, c.L))


def test_attention_page_tables_past_the_positions():
    """A table with more pages than positions below 2^31 is refused, one with as many is not."""
    c = Cache(1, 1, 1, [64], seed=23)
    x, q = queries(1, 4)
    wide = torch.zeros(1, (1 << 25) + 1, dtype=torch.int32, device=DEV)
    out, lse = torch.zeros(1, 4, 128, device=DEV), torch.zeros(1, 4, device=DEV)
    with pytest.raises(spkv.SpkvError) as e:
        spkv.sparse_decode_attn(c.handle, q, wide, i32([[[0]]]), i32([[1]]), i32([64]), out, lse)
    assert e.value.status == -1
    wide = wide[:, 1:].contiguous()
    spkv.sparse_decode_attn(c.handle, q, wide, i32([[[0, (1 << 25) - 1, 1 << 25]]]), i32([[3]]), i32([64]), out, lse)
    assert spkv.get_device_error(c.handle)[1] == spkv.DEVERR["PAGE_ID"]
    c.pt[:] = 0
    check(out, lse, ref.attention(x, c.blob, c.gk, c.gv, c.pt, np.zeros((1, 1, 1), int), np.array([[1]]), c.L))


def test_attention_runs_of_bad_entries():
    """Runs of bad entries longer than any ring of stages, between good ones."""
    c = Cache(1, 2, 8, [512, 450], seed=22)
    good = np.stack([np.arange(7), np.arange(7)])
    sel = np.full((2, 1, 400), 9, np.int32)      # past the table
    at = [0, 1, 150, 151, 153, 300, 399]
    for b in range(2):
        sel[b, 0, at] = good[b]
    n = np.full((2, 1), 400, np.int32)
    qx, q = queries(2, 4)
    out, lse = c.attend(q, sel, n)
    assert spkv.get_device_error(c.handle)[1] == spkv.DEVERR["PAGE_ID"]
    short = np.full((2, 1, 7), 0, np.int32)
    short[:, 0] = good
    check(out, lse, ref.attention(qx, c.blob, c.gk, c.gv, c.pt, short, np.full((2, 1), 7), c.L))


def test_attention_through_slots_and_directory():
    """The slot and page-directory forms give bit for bit what the flat table gives."""
    B, Hk, Hq = 3, 2, 8
    c = Cache(Hk, B, 20, [1280, 900, 70], seed=13)
    rng = np.random.default_rng(5)
    sel, n = c.select(7, rng)
    _, q = queries(B, Hq)
    out, lse = c.attend(q, sel, n)
    pm = spkv.PageMap(B, 20, seg_shift=4, n_dev_segs=2)
    for b in range(B):
        pm.map(b, 0, c.pt[b])
    pm.promote(0, 3)
    pm.sync()
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    spkv.sparse_decode_attn_dir(c.handle, q, pm, i32(sel), i32(n), i32(c.L), o2, l2)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    # a pool of slots: unit (b, h)'s i-th page in slot 6 - i
    slots = torch.zeros(Hk, B * 8, 9216, dtype=torch.uint8, device=DEV)
    slot = np.full_like(sel, -1)
    for b in range(B):
        for h in range(Hk):
            for i in range(n[b, h]):
                slot[b, h, i] = 6 - i
                slots[h, b * 8 + 6 - i] = c.pool[h, int(c.pt[b, sel[b, h, i]])]
    s = spkv.paged_kv_create_q4(slots, c.gk_d, c.gv_d, None, None, max_units=B * Hk)
    o3, l3 = torch.zeros_like(out), torch.zeros_like(lse)
    spkv.sparse_decode_attn_slots(s, q, i32(sel), i32(slot), i32(n), 8, i32(c.L), o3, l3)
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    slot[1, 0, 0] = 8
    spkv.sparse_decode_attn_slots(s, q, i32(sel), i32(slot), i32(n), 8, i32(c.L), o3, l3)
    assert spkv.get_device_error(s)[1] == spkv.DEVERR["SLOT"]
    pm.close()


def test_attention_page_order_and_repeats():
    """Any order of pages gives the same result to rounding, and the same call the same bits."""
    c = Cache(2, 2, 40, [2560, 2000], seed=14)
    rng = np.random.default_rng(6)
    sel, n = c.select(30, rng)
    qx, q = queries(2, 8)
    a, b = c.attend(q, sel, n), c.attend(q, sel, n)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_replayed_graph_and_other_stream():
    c = Cache(2, 4, 40, [2560, 2000, 100, 5], seed=15)
    sel, n = c.select(30, np.random.default_rng(6))
    qx, q = queries(4, 8)
    want = c.attend(q, sel, n)
    pt, s, m, L = i32(c.pt), i32(sel), i32(n), i32(c.L)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        spkv.sparse_decode_attn(c.handle, q, pt, s, m, L, out, lse)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spkv.sparse_decode_attn(c.handle, q, pt, s, m, L, out, lse)
        spkv.sparse_decode_attn(c.handle, q, pt, s, m, L, out, lse)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_sums_at_creation():
    """The pooled sums: valid tokens' codes times scales in order, the head's factor once."""
    for dtype in (torch.float32, torch.bfloat16):
        c = Cache(2, 2, 3, [130, 33], seed=16, ksum_dtype=dtype)
        k = ref.rows(c.blob, True).astype(np.float32)
        want = np.zeros((2, c.n_phys, 4, 128), np.float32)
        for p in range(c.n_phys):
            for t in range(c.cnt[p]):
                want[:, p, t // 16] += k[:, p, t]
        want *= c.gk[:, None, None, None]
        got = c.ksum.float().cpu().numpy()
        assert np.array_equal(got, want if dtype == torch.float32 else ref.bf16(want))


@pytest.mark.parametrize("Hk,sums", [(1, True), (3, False)])
def test_unpack(Hk, sums):
    """Listed pages in any order, twice too; rows behind the count and bad pages stay."""
    c = Cache(Hk, 2, 4, [250, 64], seed=17, junk=True, sums=sums)
    if not sums:    # counts alone
        c.handle = spkv.paged_kv_create_q4(c.pool, c.gk_d, c.gv_d, None, i32(c.cnt), max_units=8)
    pages = np.concatenate([c.pt[0], c.pt[1, :2], c.pt[0, :1], [c.n_phys, -1, c.n_phys - 1]]).astype(np.int32)
    k = torch.full((Hk, len(pages), 64, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    spkv.paged_kv_unpack_q4(c.handle, i32(pages), k, v)
    assert spkv.get_device_error(c.handle)[1] == spkv.DEVERR["PHYS"]
    for out, g, keys in ((k, c.gk, True), (v, c.gv, False)):
        x = (ref.rows(c.blob, keys).astype(np.float32) * g[:, None, None, None])
        for i, p in enumerate(pages):
            m = c.cnt[p] if 0 <= p < c.n_phys else 0
            got = host_bits(out[:, i])
            assert np.array_equal(got[:, :m], ref.bf16_bits(x[:, p, :m]) if m else got[:, :0])
            assert np.all(got[:, m:] == 0x4040)


def test_unpack_without_counts_and_every_code():
    """Every code with every finite scale comes back as code * scale * g rounded to bf16."""
    rng = np.random.default_rng(18)
    blob = rng.integers(0, 256, (1, 8, 9216), dtype=np.uint8)
    scales = np.concatenate([np.arange(127), 128 + np.arange(127)]).astype(np.uint8)   # no NaN
    blob[:, :, 8192:] = scales[rng.integers(0, len(scales), (1, 8, 1024))]
    g = np.array([0.37], np.float32)
    h = spkv.paged_kv_create_q4(u8(blob), f32(g), f32(g), None, None, max_units=1)
    k = torch.zeros(1, 8, 64, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    spkv.paged_kv_unpack_q4(h, i32(np.arange(8)), k, v)
    for out, keys in ((k, True), (v, False)):
        want = ref.rows(blob, keys).astype(np.float32) * g[0]
        assert np.array_equal(out.float().cpu().numpy(), ref.bf16(want))


def test_refused_calls():
    """Calls for bf16 pools refuse a 4-bit handle before anything runs."""
    c = Cache(2, 1, 2, [100], seed=19)
    U = -6
    rows = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=DEV)
    _, q = queries(1, 8)
    one = i32([0])
    out, lse = torch.zeros(1, 8, 128, device=DEV), torch.zeros(1, 8, device=DEV)
    word = i32([[0, 0]])
    calls = [
        lambda: spkv.paged_kv_append(c.handle, one, one, rows, rows),
        lambda: spkv.decode_append_score(c.handle, rows, rows, q, i32(c.pt), i32(c.L), torch.zeros(1, 2, 2, device=DEV)),
        lambda: spkv.lazy_rope_decode_attn(c.handle, q, one, word, one, one.view(1, 1), 1e4, out, lse),
        lambda: spkv.lazy_rope_prefill_attn(c.handle, q[:, None], one, word, one, one.view(1, 1), 1e4, out[:, None], lse[:, None]),
        lambda: spkv.lazy_alibi_prefill_attn(c.handle, q[:, None], one, word, one, word, one.view(1, 1),
                                             torch.zeros(8, device=DEV), out[:, None], lse[:, None]),
        lambda: spkv.attn_column_scores(c.handle, q[:, None], i32(c.pt), i32(c.L), torch.zeros(1, 8, 128, device=DEV)),
        lambda: spkv.DocPlan(c.handle, 8, np.zeros((1, 1), np.int32), np.array([0, 1], np.int32)),
    ]
    for f in calls:
        with pytest.raises(spkv.SpkvError) as e:
            f()
        assert e.value.status == U
    bfc = spkv.paged_kv_create(torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device=DEV),
                               torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device=DEV), None, None, max_units=1)
    with pytest.raises(spkv.SpkvError) as e:
        spkv.paged_kv_unpack_q4(bfc, one, torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device=DEV),
                                torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device=DEV))
    assert e.value.status == U
    # an output whose rows begin between two pairs of values
    odd = torch.zeros(8 * 128 + 1, device=DEV)[1:].view(1, 8, 128)
    with pytest.raises(spkv.SpkvError) as e:
        spkv.sparse_decode_attn(c.handle, q, i32(c.pt), i32(np.zeros((1, 2, 1))), i32([[1, 1]]), i32(c.L), odd, lse)
    assert e.value.status == -1
    assert spkv.get_device_error(c.handle) == (0, 0)


def test_wait_limit_then_recovery():
    """With no time to wait a call may give up (status and flag, nothing else), the next one is right again."""
    c = Cache(2, 3, 60, [60 * 64, 64 * 60 - 5, 700], seed=20)
    x, q = queries(3, 8)
    sel, n = c.select(48, np.random.default_rng(0))
    c.handle.set_wait_limit(0)
    for _ in range(3):
        c.attend(q, sel, n)
        st, bits = spkv.get_device_error(c.handle)
        assert (st, bits) in ((0, 0), (-5, spkv.DEVERR["TIMEOUT"]))
    c.handle.set_wait_limit(1_000_000_000)
    for _ in range(2):
        out, lse = c.attend(q, sel, n)
        assert spkv.get_device_error(c.handle) == (0, 0)
        check(out, lse, ref.attention(x, c.blob, c.gk, c.gv, c.pt, sel, n, c.L))


def test_two_handles_in_two_graphs():
    """Two caches' attention captured, and replayed on two streams at once: each has its own workspace."""
    work = []
    for seed in (21, 22):
        c = Cache(2, 2, 150, [9600, 9001], seed=seed)
        x, q = queries(2, 8, seed=seed)
        sel, n = c.select(140, np.random.default_rng(seed))
        d = i32(c.pt), i32(sel), i32(n), i32(c.L)
        out, lse = torch.zeros(2, 8, 128, device=DEV), torch.zeros(2, 8, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            spkv.sparse_decode_attn(c.handle, q, *d, out, lse)
        work.append((c, x, q, sel, n, d, out, lse, g, torch.cuda.Stream()))
    for _ in range(10):
        for w in work:
            with torch.cuda.stream(w[9]):
                w[8].replay()
    torch.cuda.synchronize()
    for c, x, q, sel, n, d, out, lse, g, s in work:
        assert spkv.get_device_error(c.handle) == (0, 0)
        check(out, lse, ref.attention(x, c.blob, c.gk, c.gv, c.pt, sel, n, c.L))
