"""The 8-bit cache on the GPU: what appends leave in it bit for bit, the attention over it, its pages back as bf16."""
import numpy as np
import pytest
import torch

import q4_ref
import q8_ref as ref
import sparse_paged_kv_score_gb300 as spkv
from helpers import DEV, bf, f32, host_bits, i32
from q4_ref import bf16, bf16_bits

pytestmark = pytest.mark.gpu


def u8(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.uint8)).to(DEV)


class Cache:
    """An 8-bit cache of N(0, 1) rows of uneven sizes with its handle; page p of request b is page_table[b, p]."""

    def __init__(self, Hk, B, np_max, seq_len, seed=0, junk=True, sums=True, ksum_dtype=torch.float32, key_scale=1.0):
        rng = np.random.default_rng(seed)
        self.Hk, self.B, self.np_max = Hk, B, np_max
        self.n_phys = B * np_max + 1
        shape = (Hk, self.n_phys, 64, 128)
        size = 2.0 ** rng.integers(-2, 3, (Hk, self.n_phys, 64, 1))
        self.blob = ref.pool_of(bf16(rng.standard_normal(shape) * size * key_scale), bf16(rng.standard_normal(shape) * size[::-1]))
        self.pt = rng.permutation(self.n_phys)[:B * np_max].reshape(B, np_max).astype(np.int32)
        self.L = np.asarray(seq_len, np.int32)
        self.cnt = np.zeros(self.n_phys, np.int32)
        for b in range(B):
            for p in range((int(self.L[b]) + 63) // 64):
                self.cnt[self.pt[b, p]] = min(64, self.L[b] - 64 * p)
        if junk:   # bytes behind a page's last token all ones, scales of sub-blocks without tokens NaN
            for p in range(self.n_phys):
                c = self.cnt[p]
                for at, keys in ((ref.KC, True), (ref.VC, False)):
                    self.blob[:, p, at[c:].flatten()] = 0xFF
                    for j in range((c + 15) // 16, 4):
                        ref.set_scale(self.blob[:, p], keys, j, np.nan)
        self.pool = u8(self.blob)
        self.ksum = torch.zeros(Hk, self.n_phys, 4, 128, dtype=ksum_dtype, device=DEV) if sums else None
        self.cnt_d = i32(self.cnt) if sums else None
        self.handle = spkv.paged_kv_create_q8(self.pool, self.ksum, self.cnt_d, max_units=B * Hk)

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
    x = bf16(np.random.default_rng(seed).standard_normal((B, Hq, 128)) * scale)
    return x, bf(bf16_bits(x))


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


# ---------------------------------------------------------------------------------------------- append


class Batch:
    """An 8-bit cache with earlier rows, and new rows for some requests."""

    def __init__(self, past, lens, Hq, Hk, axes=1, seed=0, sum16=False, rope=True, pad=0, fused=False, uneven=True):
        rng = np.random.default_rng(seed)
        self.Hq, self.Hk, self.B, self.rope, self.axes = Hq, Hk, len(past), rope, axes
        self.past, self.lens = np.asarray(past), np.asarray(lens)
        self.n = int(self.lens.sum()) + pad
        self.np_max = int((self.past + self.lens).max() + 63) // 64 + 1
        self.n_phys = self.B * self.np_max + 2
        self.pt = rng.permutation(self.n_phys)[:self.B * self.np_max].reshape(self.B, self.np_max).astype(np.int32)
        self.cnt = np.zeros(self.n_phys, np.int32)
        for b in range(self.B):
            for p in range((self.past[b] + 63) // 64):
                self.cnt[self.pt[b, p]] = min(64, self.past[b] - 64 * p)
        shape = (Hk, self.n_phys, 64, 128)
        self.blob = ref.pool_of(bf16(rng.standard_normal(shape)), bf16(rng.standard_normal(shape)))
        self.ksum = torch.zeros(Hk, self.n_phys, 4, 128, dtype=torch.bfloat16 if sum16 else torch.float32, device=DEV)
        self.cnt_d = i32(self.cnt)
        self.pool = u8(self.blob)
        self.cache = spkv.paged_kv_create_q8(self.pool, self.ksum, self.cnt_d, max_units=64)
        w = rng.standard_normal((self.n, Hq + 2 * Hk, 128))
        if uneven:   # rows of very different sizes: scales rise inside a sub-block
            w *= 2.0 ** rng.integers(-6, 7, (self.n, Hq + 2 * Hk, 1))
        w = bf16(w)
        if seed % 2:
            w[:, :, ::7] = 0
            w[: self.n // 3, Hq:] = 0
        self.set_rows(w, fused)
        self.first = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
        self.L = (self.past + self.lens).astype(np.int32)
        self.pos, self.pair_axis = None, None
        self.n_pos = int(self.L.max()) + 70
        if axes > 1:
            self.pos = rng.integers(0, self.n_pos, (self.n, axes)).astype(np.int32)
            self.pair_axis = [int(a) for a in rng.integers(0, axes, 64)]
        self.tab = q4_ref.table(self.n_pos)
        self.q_out = torch.full((self.n, Hq, 128), 3.0, dtype=torch.bfloat16, device=DEV)

    def set_rows(self, w, fused=False):
        self.x = w
        d = bf(q4_ref.bf16_bits_special(w))
        Hq, Hk = self.Hq, self.Hk
        parts = d[:, :Hq], d[:, Hq:Hq + Hk], d[:, Hq + Hk:]
        self.qd, self.kd, self.vd = parts if fused else (t.contiguous() for t in parts)

    def call(self, **kw):
        a = dict(row_first=i32(self.first))
        if self.rope:
            a.update(q=self.qd, q_out=self.q_out, cos_sin=f32(self.tab), pos=None if self.pos is None else i32(self.pos),
                     pair_axis=self.pair_axis)
        a.update(kw)
        spkv.paged_kv_append_rope(self.cache, self.kd, self.vd, i32(self.L), i32(self.pt), **a)

    def expect(self, skip=()):
        """The pool's bytes, counts and queries after the call, by the formula, a sub-block at a time."""
        Hq, Hk = self.Hq, self.Hk
        q_out = np.full((self.n, Hq, 128), 0x4040, np.uint16)
        old = self.cnt.copy()
        for b in range(self.B):
            blocks = {}
            for i in range(self.first[b], self.first[b + 1]):
                m = int(self.L[b] - (self.first[b + 1] - i))
                k, q = self.x[i, Hq:Hq + Hk], self.x[i, :Hq]
                blocks.setdefault(m // 16, {})
                if i in skip:
                    continue
                if self.rope:
                    where = np.full(64, m) if self.pos is None else self.pos[i, self.pair_axis] if self.axes > 1 else \
                        np.full(64, self.pos[i])
                    c, s = self.tab[where, np.arange(64)], self.tab[where, 64 + np.arange(64)]
                    with np.errstate(invalid="ignore"):
                        k, q = q4_ref.rotate(k, c, s), q4_ref.rotate(q, c, s)
                    q_out[i] = bf16_bits(q)
                blocks[m // 16][m % 16] = (k, self.x[i, Hq + Hk:])
                self.cnt[self.pt[b, m // 64]] = max(self.cnt[self.pt[b, m // 64]], m % 64 + 1)
            begin, end = int(self.L[b] - self.lens[b]), int(self.L[b])
            for blk, new in blocks.items():
                p, j = int(self.pt[b, blk // 4]), blk % 4
                held = [t for t in range(16) if 16 * blk + t < begin or (16 * blk + t >= end and 16 * j + t < old[p])]
                for h in range(Hk):
                    ref.put(self.blob[h, p], j, {t: x[0][h] for t, x in new.items()}, held, True)
                    ref.put(self.blob[h, p], j, {t: x[1][h] for t, x in new.items()}, held, False)
        return q_out

    def check(self, q_out, without=None):
        assert np.array_equal(self.cnt_d.cpu().numpy(), self.cnt)
        got = self.pool.cpu().numpy()
        bad = np.argwhere(got != self.blob)
        assert len(bad) == 0, (len(bad), bad[:5])
        if self.rope:
            assert np.array_equal(host_bits(self.q_out), q_out)
        # the sums are exact, and those that a new handle over the same rows forms (which counts the rows of
        # `without`, [(page, token)], that were left out)
        live = np.arange(64) < self.cnt[:, None]
        for page, t in without or ():
            live[page, t] = False
        k = np.where(live[None, :, :, None], ref.rows(self.blob, True), 0)
        want = k.reshape(self.Hk, self.n_phys, 4, 16, 128).sum(3)
        with np.errstate(invalid="ignore", over="ignore"):
            want = bf16(want) if self.ksum.dtype == torch.bfloat16 else want.astype(np.float32)
        assert np.array_equal(self.ksum.float().cpu().numpy(), want, equal_nan=True)
        if not without:
            fresh = torch.zeros_like(self.ksum)
            spkv.paged_kv_create_q8(self.pool, fresh, self.cnt_d, max_units=64)
            assert np.array_equal(fresh.float().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (3, 3), (16, 1), (10, 2)])
@pytest.mark.parametrize("past,lens", [
    ([0], [1]), ([63], [2]), ([64], [1]), ([5, 0, 200], [1, 1, 1]), ([0], [130]), ([7, 100, 0, 61], [40, 0, 17, 66]),
    ([3] * 20, [1, 2] * 10), ([15, 31, 14], [1, 17, 18])])
def test_append(Hq, Hk, past, lens):
    b = Batch(past, lens, Hq, Hk, seed=len(past) + Hk)
    b.call()
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.check(b.expect())


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("sum16", [False, True])
def test_append_axes_strides_padding(axes, sum16):
    b = Batch([30, 0, 77], [33, 5, 90], 8, 2, axes=axes, seed=axes, sum16=sum16, pad=9, fused=True)
    b.call()
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.check(b.expect())


def test_append_decode_rows_and_no_rotation():
    b = Batch([0, 17, 63, 64, 1000], [1] * 5, 4, 2, seed=3)
    b.call(row_first=None)
    b.check(b.expect())
    b = Batch([9, 0], [40, 3], 4, 2, seed=4, rope=False)
    b.call()
    b.check(b.expect())


@pytest.mark.parametrize("lens", [[700, 300, 1, 999], [1] * 300, [2, 15, 16, 17, 33] * 12])
def test_append_many_rows(lens):
    rng = np.random.default_rng(1)
    b = Batch(rng.integers(0, 90, len(lens)), lens, 8, 8, seed=6)
    b.call()
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.check(b.expect())


@pytest.mark.parametrize("Hq,Hk", [(40, 8), (6, 6), (22, 2), (16, 1), (3, 3)])
@pytest.mark.parametrize("pad,fused,axes", [(0, False, 1), (37, True, 3)])
def test_append_many_rows_heads(Hq, Hk, pad, fused, axes):
    """Query heads that slices do not divide, kv heads that CTAs do not, rows behind the last request's, strided rows."""
    n = 2700 // Hk + 100
    b = Batch([5, 0, 63], [n // 2, 17, n // 3], Hq, Hk, seed=19, pad=pad, fused=fused, axes=axes, sum16=bool(pad))
    b.call()
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.check(b.expect())


@pytest.mark.parametrize("cuts", [[1] * 70, [3] * 23 + [1], [16, 16, 16, 22], [33, 37], [69, 1]])
def test_append_in_any_pieces(cuts):
    """However a prompt is cut into calls, the cache holds the same bytes: floors compose."""
    whole = Batch([21], [70], 4, 2, seed=8)
    whole.call()
    pieces = Batch([21], [70], 4, 2, seed=8)
    for n, end in zip(cuts, np.cumsum(cuts)):
        spkv.paged_kv_append_rope(pieces.cache, pieces.kd[end - n:end], pieces.vd[end - n:end], i32([21 + end]), i32(pieces.pt),
                                  row_first=i32([0, n]), q=pieces.qd[end - n:end].contiguous(),
                                  q_out=torch.zeros(n, 4, 128, dtype=torch.bfloat16, device=DEV), cos_sin=f32(pieces.tab))
    assert torch.equal(whole.pool, pieces.pool) and torch.equal(whole.ksum, pieces.ksum)
    assert torch.equal(whole.cnt_d, pieces.cnt_d)
    whole.check(whole.expect())


def test_append_again_and_overwriting():
    """The same rows again leave everything as it is; others in their place keep the scale that rows beside them need."""
    b = Batch([40, 5], [7, 30], 4, 2, seed=10)
    b.call()
    b.check(b.expect())
    b.call()
    b.check(b.expect())
    # one token back: the row before the last is written again, the rows behind it count as far as page_cnt says
    b.lens, b.L = np.array([3, 20]), b.L - np.array([2, 4])
    b.n = 23
    b.first = np.array([0, 3, 23], np.int32)
    rng = np.random.default_rng(0)
    b.set_rows(bf16(rng.standard_normal((23, 8, 128)) * 0.01))
    b.q_out = torch.full((23, 4, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    b.call()
    b.check(b.expect())


@pytest.mark.parametrize("special", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("decode", [False, True])
def test_append_special_values(special, decode):
    """A NaN or an infinity makes its sub-block of its head NaN, keys or values, and no other; a page begun again is whole."""
    past, lens = ([20], [1]) if decode else ([20], [40])
    b = Batch(past, lens, 4, 2, seed=12, uneven=False)
    w = b.x.copy()
    w[0, 4, 5] = special          # a key of head 0 at position 20
    w[-1, 7, 100] = special       # a value of head 1 at the last position
    b.set_rows(w)
    b.call()
    q = b.expect()
    b.check(q)
    s = ref.scales(b.pool.cpu().numpy(), True)[:, b.pt[0, 0]]
    assert np.isnan(s[0, 1]) and np.isfinite(s[0, 0]) and np.all(np.isfinite(s[1, :2]))
    b.lens, b.L, b.n, b.first = np.array([30]), np.array([30], np.int32), 30, np.array([0, 30], np.int32)
    b.cnt[:] = 0
    b.cnt_d.zero_()
    b.ksum.zero_()      # sums of sub-blocks without rows are not looked at (here: are what a new handle writes)
    b.set_rows(bf16(np.random.default_rng(1).standard_normal((30, 8, 128))))
    b.q_out = torch.full((30, 4, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    b.call()
    b.check(b.expect())
    assert np.all(np.isfinite(ref.scales(b.pool.cpu().numpy(), True)[:, b.pt[0, 0], :2]))


def test_append_ends_of_the_range():
    """Zeros, subnormals, the largest bf16 values, powers of two and their neighbours, negative zero."""
    b = Batch([0], [128], 1, 1, seed=14, rope=False)
    w = np.zeros((128, 3, 128), np.float32)
    big = np.float32(2.0 ** 127 * (2 - 2.0 ** -7))
    ladder = [0.0, -0.0, 2.0 ** -133, -2.0 ** -133, 2.0 ** -126, 2.0 ** -120, -2.0 ** -120, 1.0, -1.0, 2.0, -2.0, 1.9921875, big, -big]
    rng = np.random.default_rng(2)
    for blk in range(8):
        top = ladder[blk + 6] if blk else 0.0
        for t in range(16):
            w[16 * blk + t, 1:] = np.array(ladder, np.float32)[rng.integers(0, len(ladder), (2, 128))]
            w[16 * blk + t, 1:][np.abs(w[16 * blk + t, 1:]) > abs(top)] = top
    b.set_rows(bf16(w))
    b.call()
    b.check(b.expect())
    for t in range(128):      # the same one by one
        spkv.paged_kv_append_rope(b.cache, b.kd[t:t + 1], b.vd[t:t + 1], i32([t + 1]), i32(b.pt))
    b.check(None)
    k = torch.zeros(1, 2, 64, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    spkv.paged_kv_unpack_q8(b.cache, i32(b.pt[0, :2]), k, v)
    for out, keys in ((k, True), (v, False)):
        assert np.array_equal(out.double().cpu().numpy(), ref.rows(b.blob[:, b.pt[0, :2]], keys))


def test_append_bad_rows_are_skipped():
    """Rows outside the table or the pool and positions outside the rotation's are left out and flagged; rows of the same
    sub-blocks are appended."""
    b = Batch([10, 0, 30], [9, 40, 20], 4, 2, seed=16, axes=2)
    b.pos[[2, 12, 60], [0, 1, 1]] = [b.n_pos, -1, 1 << 30]
    b.call()
    assert spkv.get_device_error(b.cache) == (-4, spkv.DEVERR["POS"])
    b.check(b.expect(skip={2, 12, 60}), [(b.pt[0, 0], 12), (b.pt[1, 0], 3), (b.pt[2, 0], 41)])
    b = Batch([10, 0, 30], [9, 40, 20], 4, 2, seed=16)
    keep = b.blob.copy()
    pt = b.pt.copy()
    b.pt[1, 0] = b.n_phys
    b.call()
    assert spkv.get_device_error(b.cache) == (-4, spkv.DEVERR["PHYS"])
    b.pt = pt
    q = b.expect()
    b.blob[:, pt[1, 0]] = keep[:, pt[1, 0]]
    b.cnt[pt[1, 0]] = 0
    assert np.array_equal(b.pool.cpu().numpy(), b.blob) and np.array_equal(b.cnt_d.cpu().numpy(), b.cnt)
    assert np.array_equal(host_bits(b.q_out), q)      # their queries have positions


def test_append_rows_of_a_sub_block_that_are_all_bad():
    b = Batch([8], [4], 4, 1, seed=17, axes=2)
    b.pos[:, 0] = -1
    b.call()
    assert spkv.get_device_error(b.cache) == (-4, spkv.DEVERR["POS"])
    b.check(b.expect(skip={0, 1, 2, 3}))


def test_append_graph_and_other_stream():
    b = Batch([30, 61, 200], [1, 1, 1], 8, 2, seed=18)
    first, L, pt, tab = i32(b.first), i32(b.L), i32(b.pt), f32(b.tab)
    pool0, cnt0, sum0 = b.pool.clone(), b.cnt_d.clone(), b.ksum.clone()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        spkv.paged_kv_append_rope(b.cache, b.kd, b.vd, L, pt, row_first=first, q=b.qd, q_out=b.q_out, cos_sin=tab)
    q = b.expect()
    g.replay()
    b.check(q)
    for dst, src in ((b.pool, pool0), (b.cnt_d, cnt0), (b.ksum, sum0)):
        dst.copy_(src)
    b.q_out.fill_(3)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        spkv.paged_kv_append_rope(b.cache, b.kd, b.vd, L, pt, row_first=first, q=b.qd, q_out=b.q_out, cos_sin=tab)
    side.synchronize()
    b.check(q)


# ---------------------------------------------------------------------------------------------- attention


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (1, 1), (3, 3), (6, 2), (5, 1), (8, 1), (18, 2), (16, 1)])
@pytest.mark.parametrize("L", [1, 15, 16, 17, 48, 49, 64, 65, 400])
def test_attention_sizes(Hq, Hk, L):
    B = 3
    c = Cache(Hk, B, (L + 63) // 64 + 1, [L, max(1, L - 1), max(1, L // 2)], seed=L)
    rng = np.random.default_rng(L)
    sel, n = c.select(max(1, (L + 63) // 64), rng)
    qx, q = queries(B, Hq)
    out, lse = c.attend(q, sel, n)
    assert spkv.get_device_error(c.handle) == (0, 0)
    check(out, lse, ref.attention(qx, c.blob, c.pt, sel, n, c.L))


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (10, 2), (16, 1), (13, 1)])
def test_attention_ragged_selections(Hq, Hk):
    """Selections of every length, empty ones too, many pages in one of them."""
    B = 9
    c = Cache(Hk, B, 70, [4480, 1, 64, 100, 900, 4000, 65, 2222, 4410], seed=5)
    rng = np.random.default_rng(2)
    counts = rng.integers(0, 68, (B, Hk))
    counts[0], counts[1], counts[4] = 67, 0, 0
    sel, n = c.select(67, rng, counts)
    qx, q = queries(B, Hq)
    out, lse = c.attend(q, sel, n)
    assert spkv.get_device_error(c.handle) == (0, 0)
    check(out, lse, ref.attention(qx, c.blob, c.pt, sel, n, c.L))


@pytest.mark.parametrize("B,Hk,G,pages", [(1, 1, 4, 2000), (61, 1, 9, 129), (40, 2, 5, 300), (200, 1, 2, 40), (3, 1, 1, 20000),
                                           (64, 2, 16, 70), (128, 2, 1, 9), (300, 1, 4, 17), (32, 8, 4, 65), (9, 1, 16, 2000)])
@pytest.mark.parametrize("short", [0, 1, 2])
def test_attention_dealing(B, Hk, G, pages, short):
    """Lists of one length, lists a little shorter, and lists of every length, over few physical pages that repeat: for each
    list the mean of its pages' weighted values."""
    rng = np.random.default_rng(pages + short)
    c = Cache(Hk, 1, 12, [768], seed=B)
    h = spkv.paged_kv_create_q8(c.pool, None, None, max_units=B * Hk)
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
            k, v = ref.rows(c.blob[kv, c.pt[0]], True).reshape(-1, 128), ref.rows(c.blob[kv, c.pt[0]], False).reshape(12, 64, 128)
            ks, vs = (np.repeat(ref.scales(c.blob[kv, c.pt[0]], s).astype(np.float64).flatten(), 16) for s in (True, False))
            for g in range(kv * G, kv * G + G):
                qr = x[:, g].astype(np.float64)
                y = qr @ k.T / np.sqrt(128)                                   # [B][12 * 64]
                m = y.max(1)
                w = np.exp(y - m[:, None]).reshape(B, 12, 64)
                num, den = np.einsum("bpt,ptd->bpd", w, v), w.sum(2)
                for b in range(B):
                    times = np.bincount(which[b, :n[b, kv]], minlength=12)
                    if n[b, kv] == 0:
                        assert np.all(o[b, g] == 0) and np.isneginf(l[b, g])
                        continue
                    # a lane adds its CTA's pages / 4, and the parts' sums are merged
                    dx, dw, vmax = ref.error_bounds(qr[b], k, ks, v.reshape(-1, 128), vs, 4 * pages)
                    s = times @ den[b]
                    assert np.abs(o[b, g] - times @ num[b] / s).max() <= 2 * dw * vmax
                    assert abs(l[b, g] - m[b] - np.log(s)) <= dw + 2.0 ** -19 * (1 + abs(l[b, g]))


@pytest.mark.parametrize("B,Hk,G,most", [(100, 3, 2, 7), (257, 1, 9, 3), (512, 8, 1, 2), (300, 2, 4, 12)])
@pytest.mark.parametrize("empty", [0.0, 0.5, 0.99])
def test_attention_many_units(B, Hk, G, most, empty):
    """More units than are looked up at a time, most of them short or empty, and two long ones."""
    rng = np.random.default_rng(B + most)
    c = Cache(Hk, 2, 40, [2560, 2500], seed=B)
    c.handle = spkv.paged_kv_create_q8(c.pool, c.ksum, c.cnt_d, max_units=B * Hk)
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
    check(out, lse, ref.attention(x, c.blob, c.pt, sel, n, c.L))


@pytest.mark.parametrize("q_scale,key_scale", [(1e-6, 1.0), (30.0, 1.0), (1e4, 1e-3), (1.0, 0.0)])
def test_attention_score_ranges(q_scale, key_scale):
    """Flat and peaked weights, queries outside f16's range, keys of zeros: the running maximum rises."""
    c = Cache(2, 2, 9, [530, 77], seed=7, key_scale=key_scale)
    sel, n = c.select(9, np.random.default_rng(3))
    qx, q = queries(2, 8, scale=q_scale)
    out, lse = c.attend(q, sel, n)
    check(out, lse, ref.attention(qx, c.blob, c.pt, sel, n, c.L))


@pytest.mark.parametrize("G", [4, 7, 12])
def test_attention_rising_scores(G):
    """Each page's keys score far above the last one's, so the reference moves at every page; values of every size."""
    c = Cache(1, 1, 12, [12 * 64 - 5], seed=8)
    rng = np.random.default_rng(4)
    k = np.zeros((1, c.n_phys, 64, 128), np.float32)
    qx, q = queries(1, G, seed=9)
    for p in range(12):
        k[0, c.pt[0, p]] = bf16(qx[0, 0] * (0.02 * (p + 1) ** 2))
    v = bf16(rng.standard_normal(k.shape) * 2.0 ** np.repeat(rng.integers(-20, 20, (1, c.n_phys, 4, 1)), 16, 2))
    c.blob[:] = ref.pool_of(k, v)
    c.pool.copy_(u8(c.blob))
    sel, n = c.select(12, np.random.default_rng(3))
    out, lse = c.attend(q, sel, n)
    check(out, lse, ref.attention(qx, c.blob, c.pt, sel, n, c.L))


@pytest.mark.parametrize("keys", [True, False])
def test_attention_passes_nan_on(keys):
    """A NaN scale of an attended sub-block makes its unit's outputs NaN, and no other unit's."""
    c = Cache(2, 2, 3, [150, 150], seed=11)
    ref.set_scale(c.blob[0, c.pt[0, 1]], keys, 1, np.nan)
    c.pool.copy_(u8(c.blob))
    sel, n = c.select(3, np.random.default_rng(3))
    _, q = queries(2, 8)
    out, lse = c.attend(q, sel, n)
    assert torch.isnan(out[0, :4]).all() and torch.isnan(lse[0, :4]).all() == keys
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
    check(out, lse, ref.attention(qx, c.blob, c.pt, good, gn, c.L))


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
    check(out, lse, ref.attention(qx, c.blob, c.pt, short, np.full((2, 1), 7), c.L))


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
    slots = torch.zeros(Hk, B * 8, spkv.Q8_PAGE_BYTES, dtype=torch.uint8, device=DEV)
    slot = np.full_like(sel, -1)
    for b in range(B):
        for h in range(Hk):
            for i in range(n[b, h]):
                slot[b, h, i] = 6 - i
                slots[h, b * 8 + 6 - i] = c.pool[h, int(c.pt[b, sel[b, h, i]])]
    s = spkv.paged_kv_create_q8(slots, None, None, max_units=B * Hk)
    o3, l3 = torch.zeros_like(out), torch.zeros_like(lse)
    spkv.sparse_decode_attn_slots(s, q, i32(sel), i32(slot), i32(n), 8, i32(c.L), o3, l3)
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    slot[1, 0, 0] = 8
    spkv.sparse_decode_attn_slots(s, q, i32(sel), i32(slot), i32(n), 8, i32(c.L), o3, l3)
    assert spkv.get_device_error(s)[1] == spkv.DEVERR["SLOT"]
    pm.close()


def test_attention_same_bits_in_graphs_and_on_other_streams():
    c = Cache(2, 4, 40, [2560, 2000, 100, 5], seed=15)
    sel, n = c.select(30, np.random.default_rng(6))
    qx, q = queries(4, 8)
    want = c.attend(q, sel, n)
    again = c.attend(q, sel, n)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
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
        work.append((c, x, sel, n, d, out, lse, g, torch.cuda.Stream(), q))
    for _ in range(10):
        for w in work:
            with torch.cuda.stream(w[8]):
                w[7].replay()
    torch.cuda.synchronize()
    for c, x, sel, n, d, out, lse, g, s, q in work:
        assert spkv.get_device_error(c.handle) == (0, 0)
        check(out, lse, ref.attention(x, c.blob, c.pt, sel, n, c.L))


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
        check(out, lse, ref.attention(x, c.blob, c.pt, sel, n, c.L))


# ---------------------------------------------------------------------------------------------- pages back


@pytest.mark.parametrize("Hk,sums", [(1, True), (3, False)])
def test_unpack(Hk, sums):
    """Listed pages in any order, twice too; rows behind the count and bad pages stay."""
    c = Cache(Hk, 2, 5, [250, 65], seed=17, sums=sums)
    if not sums:    # counts alone
        c.handle = spkv.paged_kv_create_q8(c.pool, None, i32(c.cnt), max_units=8)
    pages = np.concatenate([c.pt[0], c.pt[1, :2], c.pt[0, :1], [c.n_phys, -1, c.n_phys - 1]]).astype(np.int32)
    k = torch.full((Hk, len(pages), 64, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    spkv.paged_kv_unpack_q8(c.handle, i32(pages), k, v)
    assert spkv.get_device_error(c.handle)[1] == spkv.DEVERR["PHYS"]
    for out, keys in ((k, True), (v, False)):
        x = ref.rows(c.blob, keys)
        for i, p in enumerate(pages):
            m = c.cnt[p] if 0 <= p < c.n_phys else 0
            got = out[:, i].double().cpu().numpy()
            assert np.array_equal(got[:, :m], x[:, p, :m] if m else got[:, :0])
            assert np.all(got[:, m:] == 3)


def test_unpack_every_code_and_scale():
    """Every code with every kind of scale comes back exactly; a handle without counts gives whole pages."""
    rng = np.random.default_rng(18)
    blob = rng.integers(0, 256, (1, 70, ref.BLOB), dtype=np.uint8)
    s = 2.0 ** np.concatenate([[-126, -125, 121], rng.integers(-126, 122, 70 * 8 - 3)]).astype(np.float32)
    s[3], s[4] = 0, np.nan
    blob[0, :, 16384:] = s.astype(np.float32).reshape(70, 8).view(np.uint8)
    h = spkv.paged_kv_create_q8(u8(blob), None, None, max_units=1)
    k = torch.zeros(1, 70, 64, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    spkv.paged_kv_unpack_q8(h, i32(np.arange(70)), k, v)
    for out, keys in ((k, True), (v, False)):
        assert np.array_equal(out.double().cpu().numpy(), ref.rows(blob, keys), equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sums_at_creation(dtype):
    c = Cache(2, 2, 3, [130, 33], seed=16, ksum_dtype=dtype)
    k = np.where((np.arange(64) < c.cnt[:, None])[None, :, :, None], ref.rows(c.blob, True), 0)
    want = k.reshape(2, c.n_phys, 4, 16, 128).sum(3)
    assert np.array_equal(c.ksum.double().cpu().numpy(), want if dtype == torch.float32 else bf16(want))


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: pages at both ends appended to, attended and unpacked."""
    n_phys = (1 << 32) // ref.BLOB + 40
    pool = torch.zeros(1, n_phys, ref.BLOB, dtype=torch.uint8, device=DEV)
    cnt = torch.zeros(n_phys, dtype=torch.int32, device=DEV)
    ksum = torch.zeros(1, n_phys, 4, 128, device=DEV, dtype=torch.bfloat16)
    h = spkv.paged_kv_create_q8(pool, ksum, cnt, max_units=4)
    rng = np.random.default_rng(0)
    x = bf16(rng.standard_normal((80, 2, 1, 128)))
    k, v = bf(bf16_bits(x[:, 0])), bf(bf16_bits(x[:, 1]))
    pt = np.array([[n_phys - 1, 3], [5, n_phys - 2]], np.int32)
    spkv.paged_kv_append_rope(h, k, v, i32([70, 10]), i32(pt), row_first=i32([0, 70, 80]))
    blob = {}
    want = np.zeros((1, 4, ref.BLOB), np.uint8)
    for b, (i0, n) in enumerate(((0, 70), (70, 10))):
        for j in range((n + 15) // 16):
            rows = range(16 * j, min(n, 16 * j + 16))
            for keys, side in ((True, 0), (False, 1)):
                ref.put(want[0, 2 * b + j // 4], j % 4, {t % 16: x[i0 + t, side, 0] for t in rows}, [], keys)
    got = pool[0, torch.tensor([n_phys - 1, 3, 5], device=DEV)].cpu().numpy()
    assert np.array_equal(got, want[0, :3])
    qx, q = queries(2, 4)
    sel, n = np.array([[[0, 1]], [[0, -1]]], np.int32), np.array([[2], [1]], np.int32)
    out, lse = torch.zeros(2, 4, 128, device=DEV), torch.zeros(2, 4, device=DEV)
    spkv.sparse_decode_attn(h, q, i32(pt), i32(sel), i32(n), i32([70, 10]), out, lse)
    assert spkv.get_device_error(h) == (0, 0)
    check(out, lse, ref.attention(qx, want, np.array([[0, 1], [2, 3]]), sel, n, np.array([70, 10])))
    ko = torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device=DEV)
    vo = torch.zeros_like(ko)
    spkv.paged_kv_unpack_q8(h, i32([n_phys - 1]), ko, vo)
    assert np.array_equal(ko.double().cpu().numpy()[0], ref.rows(want[0, :1], True))


def test_decode_steps_on_an_8bit_cache():
    """A prompt and decode steps: append, block scores, selection of all pages, attention, as they are used."""
    B, Hq, Hk, past, steps = 2, 8, 2, 100, 5
    rng = np.random.default_rng(30)
    np_max, n_phys = 3, 7
    pool = torch.zeros(Hk, n_phys, ref.BLOB, dtype=torch.uint8, device=DEV)
    cnt, ksum = torch.zeros(n_phys, dtype=torch.int32, device=DEV), torch.zeros(Hk, n_phys, 4, 128, device=DEV)
    h = spkv.paged_kv_create_q8(pool, ksum, cnt, max_units=B * Hk)
    pt = rng.permutation(n_phys)[:B * np_max].reshape(B, np_max).astype(np.int32)
    tab = f32(q4_ref.table(200))
    k, v = (torch.randn(B * past, Hk, 128, device=DEV).bfloat16() for _ in range(2))
    spkv.paged_kv_append_rope(h, k, v, i32([past] * B), i32(pt), row_first=i32([0, past, 2 * past]),
                              q=torch.zeros(B * past, Hq, 128, dtype=torch.bfloat16, device=DEV),
                              q_out=torch.zeros(B * past, Hq, 128, dtype=torch.bfloat16, device=DEV), cos_sin=tab)
    scores = torch.zeros(B, Hk, np_max, device=DEV)
    evict = torch.zeros(B, Hk, np_max, device=DEV)
    sel, n = torch.zeros(B, Hk, 4, dtype=torch.int32, device=DEV), torch.zeros(B, Hk, dtype=torch.int32, device=DEV)
    for step in range(steps):
        L = i32([past + step + 1] * B)
        k, v, q = (torch.randn(B, x, 128, device=DEV).bfloat16() for x in (Hk, Hk, Hq))
        q_rot, out, lse = torch.zeros_like(q), torch.zeros(B, Hq, 128, device=DEV), torch.zeros(B, Hq, device=DEV)
        spkv.paged_kv_append_rope(h, k, v, L, i32(pt), q=q, q_out=q_rot, cos_sin=tab)
        spkv.score_blocks(h, q_rot, i32(pt), L, scores)
        alive = torch.full((B, Hk, 1), -1, dtype=torch.int32, device=DEV)
        spkv.select_topk(h, scores, evict, alive, L, 3, 0, sel, n)
        spkv.sparse_decode_attn(h, q_rot, i32(pt), sel, n, L, out, lse)
        assert spkv.get_device_error(h) == (0, 0)
        blob = pool.cpu().numpy()
        qx = q4_ref.from_bf16_bits(host_bits(q_rot))
        check(out, lse, ref.attention(qx, blob, pt, sel.cpu().numpy(), n.cpu().numpy(), L.cpu().numpy()))
        # block scores from the sums of the values that the cache holds
        m = ref.rows(blob[:, pt[:, :1]], True).reshape(Hk, B, 4, 16, 128).mean(3)
        s = np.einsum("bhd,hbjd->bhj", qx.reshape(B, Hk, 4, 128).sum(2).astype(np.float64), m) / np.sqrt(128)
        bound = 2e-5 * np.einsum("bhd,hbjd->bhj", np.abs(qx.reshape(B, Hk, 4, 128).sum(2)).astype(np.float64), np.abs(m)).max()
        assert np.abs(scores[:, :, 0].cpu().numpy() - s.max(-1)).max() <= bound
