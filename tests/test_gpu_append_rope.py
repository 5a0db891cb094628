"""The rotating append, into bf16 and 4-bit caches: bit for bit the formula's rows, sums and counts."""
import numpy as np
import pytest
import torch

import q4_ref as ref
import sparse_paged_kv_score_gb300 as spkv
from helpers import DEV, bf, f32, host_bits, i32

pytestmark = pytest.mark.gpu


class Batch:
    """A cache (bf16 or 4-bit) with earlier rows, and new rows for some requests."""

    def __init__(self, q4, past, lens, Hq, Hk, axes=1, seed=0, sum16=False, rope=True, pad=0, fused=False, n_pos=None,
                 spare_full=False):
        rng = np.random.default_rng(seed)
        self.q4, self.Hq, self.Hk, self.B, self.rope = q4, Hq, Hk, len(past), rope
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
        k0, v0 = ref.bf16(rng.standard_normal(shape)), ref.bf16(rng.standard_normal(shape))
        self.gk = (rng.uniform(0.5, 2, Hk) * 5 / 2688).astype(np.float32)
        self.gv = (rng.uniform(0.5, 2, Hk) * 5 / 2688).astype(np.float32)
        self.ksum = torch.zeros(Hk, self.n_phys, 4, 128, dtype=torch.bfloat16 if sum16 else torch.float32, device=DEV)
        self.cnt_d = i32(self.cnt)
        if q4:
            self.blob = ref.pool_of(k0, v0, self.gk, self.gv)
            self.pool = torch.from_numpy(self.blob.copy()).to(DEV)
            self.cache = spkv.paged_kv_create_q4(self.pool, f32(self.gk), f32(self.gv), self.ksum, self.cnt_d, max_units=64)
        else:
            self.kb, self.vb = ref.bf16_bits(k0), ref.bf16_bits(v0)
            self.kp, self.vp = bf(self.kb), bf(self.vb)
            self.cache = spkv.paged_kv_create(self.kp, self.vp, self.ksum, self.cnt_d, max_units=64)
        w = ref.bf16(rng.standard_normal((self.n, Hq + 2 * Hk, 128)))
        if seed % 2:
            w[:, :, ::7] = 0     # zeros, and blocks of nothing but zeros
            w[: self.n // 3, Hq:, 16:32] = 0
        self.x = w
        d = bf(ref.bf16_bits(w))
        parts = d[:, :Hq], d[:, Hq:Hq + Hk], d[:, Hq + Hk:]
        self.qd, self.kd, self.vd = parts if fused else (t.contiguous() for t in parts)
        self.first = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
        self.L = (self.past + self.lens).astype(np.int32)
        self.axes = axes
        self.pos, self.pair_axis = None, None
        self.n_pos = n_pos or int(self.L.max()) + 70
        if axes > 1:
            self.pos = rng.integers(0, self.n_pos, (self.n, axes)).astype(np.int32)
            self.pair_axis = [int(a) for a in rng.integers(0, axes, 64)]
        self.tab = ref.table(self.n_pos)
        self.q_out = torch.full((self.n, Hq, 128), 3.0, dtype=torch.bfloat16, device=DEV)

    def call(self, **kw):
        a = dict(row_first=i32(self.first))
        if self.rope:
            a.update(q=self.qd, q_out=self.q_out, cos_sin=f32(self.tab), pos=None if self.pos is None else i32(self.pos),
                     pair_axis=self.pair_axis)
        a.update(kw)
        spkv.paged_kv_append_rope(self.cache, self.kd, self.vd, i32(self.L), i32(self.pt), **a)

    def expect(self, skip=()):
        """Cache, counts and queries after the call, by the formula."""
        Hq, Hk = self.Hq, self.Hk
        q_out = np.full((self.n, Hq, 128), 0x4040, np.uint16)
        for b in range(self.B):
            for i in range(self.first[b], self.first[b + 1]):
                if i in skip:
                    continue
                m = int(self.L[b] - (self.first[b + 1] - i))
                k, q = self.x[i, Hq:Hq + Hk], self.x[i, :Hq]
                if self.rope:
                    where = np.full(64, m) if self.pos is None else self.pos[i, self.pair_axis] if self.axes > 1 else \
                        np.full(64, self.pos[i])
                    c, s = self.tab[where, np.arange(64)], self.tab[where, 64 + np.arange(64)]
                    k, q = ref.rotate(k, c, s), ref.rotate(q, c, s)
                    q_out[i] = ref.bf16_bits(q)
                p, t = int(self.pt[b, m // 64]), m % 64
                for h in range(Hk):
                    if self.q4:
                        ref.put(self.blob[h, p], t, k[h], self.gk[h], True)
                        ref.put(self.blob[h, p], t, self.x[i, Hq + Hk + h], self.gv[h], False)
                    else:
                        self.kb[h, p, t] = ref.bf16_bits(k[h])
                        self.vb[h, p, t] = ref.bf16_bits(self.x[i, Hq + Hk + h])
                self.cnt[p] = max(self.cnt[p], t + 1)
        return q_out

    def expect_none(self):
        """After a call whose rows are no request's: as the call before left it."""
        return host_bits(self.q_out)

    def check(self, q_out):
        assert np.array_equal(self.cnt_d.cpu().numpy(), self.cnt)
        if self.q4:
            assert np.array_equal(self.pool.cpu().numpy(), self.blob)
        else:
            assert np.array_equal(host_bits(self.kp), self.kb) and np.array_equal(host_bits(self.vp), self.vb)
        if self.rope:
            assert np.array_equal(host_bits(self.q_out), q_out)
        # the sums are those that a new handle over the same rows forms
        fresh = torch.zeros_like(self.ksum)
        if self.q4:
            spkv.paged_kv_create_q4(self.pool, f32(self.gk), f32(self.gv), fresh, self.cnt_d, max_units=64)
        else:
            spkv.paged_kv_create(self.kp, self.vp, fresh, self.cnt_d, max_units=64)
        torch.cuda.synchronize()
        assert torch.equal(fresh, self.ksum)


FORMATS = [pytest.param(False, id="bf16"), pytest.param(True, id="q4")]


@pytest.mark.parametrize("q4", FORMATS)
@pytest.mark.parametrize("Hq,Hk", [(8, 2), (3, 3), (16, 1), (10, 2)])
@pytest.mark.parametrize("past,lens", [
    ([0], [1]), ([63], [2]), ([64], [1]), ([5, 0, 200], [1, 1, 1]), ([0], [130]), ([7, 100, 0, 61], [40, 0, 17, 66]),
    ([3] * 20, [1, 2] * 10)])
def test_rows_sums_counts(q4, Hq, Hk, past, lens):
    b = Batch(q4, past, lens, Hq, Hk, seed=len(past) + Hk)
    b.call()
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("sum16", [False, True])
def test_axes_strides_padding(q4, axes, sum16):
    """Several axes in any order of pairs, rows inside a wider projection, padding rows behind the last."""
    b = Batch(q4, [30, 0, 77], [33, 5, 90], 8, 2, axes=axes, seed=axes, sum16=sum16, pad=9, fused=True)
    b.call()
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
def test_one_axis_given_positions(q4):
    """A document's own positions, not the context's (deferred rotation)."""
    b = Batch(q4, [100, 0], [20, 50], 8, 2, seed=3)
    b.pos = np.arange(70, dtype=np.int32)[::-1].copy()
    b.call()
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
def test_no_rotation(q4):
    b = Batch(q4, [10, 64], [60, 3], 4, 2, seed=4, rope=False)
    b.call()
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
def test_decode_rows_without_row_first_and_in_place(q4):
    """One row a request; the queries rotated in place."""
    b = Batch(q4, [0, 15, 16, 63, 64, 1000], [1] * 6, 8, 2, seed=6)
    b.q_out = b.qd
    b.call(row_first=None, q_out=b.qd)
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
def test_many_rows(q4):
    """Enough rows for the widest windows, lengths that leave a sub-block in two of them."""
    b = Batch(q4, [5, 0, 33], [1300, 7, 1501], 2, 2, seed=7)
    b.call()
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
def test_called_again_and_overwriting(q4):
    """The same rows twice leave the same cache; rows inside a filled page are replaced."""
    b = Batch(q4, [90], [20], 4, 1, seed=8)
    b.call()
    b.call()
    b.check(b.expect())
    b.L, b.first = np.array([70], np.int32), np.array([0, 20], np.int32)    # positions 50 .. 69, both pages hold more
    b.call()
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
def test_bad_rows_are_skipped(q4):
    """A page outside the pool, a position past the table: flagged, the other rows are appended."""
    b = Batch(q4, [10, 0, 0], [3, 2, 2], 8, 2, seed=9)
    pt = b.pt.copy()
    b.pt = pt.copy()
    b.pt[1, 0] = b.n_phys
    b.call()
    assert spkv.get_device_error(b.cache)[1] == spkv.DEVERR["PHYS"]
    b.pt = pt
    q = b.expect(skip=(3, 4))
    c = [b.tab[[0, 1], :64], b.tab[[0, 1], 64:]]
    q[3:5] = ref.bf16_bits(ref.rotate(b.x[3:5, :8], c[0][:, None], c[1][:, None]))   # a query needs no page
    b.check(q)
    b = Batch(q4, [10, 0], [3, 18], 8, 2, seed=9)
    b.pos = np.arange(21, dtype=np.int32)
    b.pos[20], b.pos[4] = b.n_pos, -1
    b.call()
    assert spkv.get_device_error(b.cache)[1] == spkv.DEVERR["POS"]
    q = b.expect(skip=(20, 4))
    assert np.array_equal(host_bits(b.q_out), q)
    assert np.array_equal(b.cnt_d.cpu().numpy(), b.cnt)
    if q4:
        assert np.array_equal(b.pool.cpu().numpy(), b.blob)
    else:
        assert np.array_equal(host_bits(b.kp), b.kb)
    b = Batch(q4, [64 * 3 - 1], [1], 8, 2, seed=9, n_pos=4096)
    b.L = np.array([64 * b.np_max + 1], np.int32)
    b.call()
    assert spkv.get_device_error(b.cache)[1] == spkv.DEVERR["PAGE_ID"]


@pytest.mark.parametrize("special", [np.nan, np.inf, -np.inf])
def test_q4_special_values(special):
    """A NaN makes its block NaN, an infinity saturates, other blocks are as ever."""
    b = Batch(True, [0], [3], 4, 1, seed=10, rope=False)
    b.x[1, 4, 20] = special
    b.x[2, 5, 127] = special
    b.kd, b.vd = bf(ref.bf16_bits_special(b.x[:, 4:5])), bf(ref.bf16_bits_special(b.x[:, 5:6]))
    b.call()
    b.expect()
    assert np.array_equal(b.pool.cpu().numpy(), b.blob)


def test_q4_tiny_and_huge_values():
    """Blocks below the smallest scale hold zeros, above the largest they saturate; factors far from one."""
    for g in (2.0 ** -64, 1.0, 2.0 ** 60):
        b = Batch(True, [0], [4], 2, 1, seed=11, rope=False)
        b.gk[:] = b.gv[:] = g
        b.cache = spkv.paged_kv_create_q4(b.pool, f32(b.gk), f32(b.gv), b.ksum, b.cnt_d, max_units=64)
        mag = np.exp2(np.linspace(-30, 30, 8)).astype(np.float32) * np.float32(g)
        b.x[:, 2:4] *= np.repeat(mag, 16)
        b.x = ref.bf16(b.x)
        b.kd, b.vd = bf(ref.bf16_bits(b.x[:, 2:3])), bf(ref.bf16_bits(b.x[:, 3:4]))
        b.call()
        b.expect()
        assert np.array_equal(b.pool.cpu().numpy(), b.blob)


@pytest.mark.parametrize("g", [2.0 ** -118, 2.0 ** -102, 2.0 ** -97, 1.0, 0.7, 2.0 ** 95, 2.0 ** 101])
def test_q4_ties(g):
    """Values on the ties between codes, and a bf16 step beside them, for factors up to the ends of fp32."""
    b = Batch(True, [0], [64], 2, 1, seed=31, rope=False)
    b.gk[:] = b.gv[:] = g
    b.cache = spkv.paged_kv_create_q4(b.pool, f32(b.gk), f32(b.gv), b.ksum, b.cnt_d, max_units=64)
    rng = np.random.default_rng(5)
    ties = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6])
    x = rng.permuted(np.tile(ties, (64, 3, 8)).reshape(64, 3, 8, 16), axis=-1) * rng.choice([-1, 1], (64, 3, 8, 16))
    x = x * 2.0 ** rng.integers(-6, 6, (64, 3, 8, 1)) * np.float64(np.float32(g))
    x = x.reshape(64, 3, 128) * (1 + rng.choice([-2.0 ** -8, 0, 0, 0, 2.0 ** -7], (64, 3, 128)))
    b.x[:, 1:] = 0
    b.x[:, 2:4] = ref.bf16(x[:, :2].astype(np.float32))
    b.kd, b.vd = bf(ref.bf16_bits(b.x[:, 2:3])), bf(ref.bf16_bits(b.x[:, 3:4]))
    b.call()
    b.expect()
    assert np.array_equal(b.pool.cpu().numpy(), b.blob)


def test_q4_held_values_are_near():
    """In 64 bits: a held value is off by at most half the code's step and the scale's rounding.

    With a = max |x| of the block and t = a / 6g, s is off t by at most half an e4m3 step (2^-4 s, or 2^-10
    below the normal numbers), codes by at most half a step (1 at the widest) of s g, and the largest
    value may saturate by the scale's error: |value - x| <= s g + 6 g |s - t|."""
    b = Batch(True, [0], [64], 2, 2, seed=12, rope=False)
    b.call()
    blob = b.pool.cpu().numpy()
    for keys, x, g in ((True, b.x[:, 2:4], b.gk), (False, b.x[:, 4:6], b.gv)):
        for h in range(2):
            p = int(b.pt[0, 0])
            held = ref.rows(blob[h, p], keys) * float(g[h])
            s = ref.E4M3[blob[h, p][ref.KS if keys else ref.VS]] * float(g[h])
            a = np.abs(x[:, h].astype(np.float64)).reshape(64, 8, 16)
            t = a.max(-1) / 6
            bound = (s + 6 * np.abs(s - t)) * (1 + 2.0 ** -20)
            assert np.all(np.abs(held - x[:, h]).reshape(64, 8, 16) <= bound[..., None])
            small = a <= 2 * s[..., None]     # codes up to 2 are half a unit apart
            assert np.all((np.abs(held - x[:, h]).reshape(64, 8, 16) <= 0.25 * (1 + 2.0 ** -20) * s[..., None])[small])


def test_graph_replay_and_other_stream():
    b = Batch(True, [40, 3], [1, 1], 8, 2, seed=13)
    L, pt, tab, first = i32(b.L), i32(b.pt), f32(b.tab), i32(b.first)
    run = lambda: spkv.paged_kv_append_rope(b.cache, b.kd, b.vd, L, pt, row_first=first, q=b.qd, q_out=b.q_out, cos_sin=tab)  # noqa: E731
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    g.replay()
    torch.cuda.synchronize()
    b.check(b.expect())
    L += 1      # the next step through the same graph
    g.replay()
    torch.cuda.synchronize()
    b.L = b.L + 1
    b.check(b.expect())


@pytest.mark.parametrize("steps", [3])
def test_prompt_then_decode_on_a_q4_cache(steps):
    """Prompts, then decode steps: append, block scores, selection, attention, all on the 4-bit cache."""
    Hq, Hk, B = 8, 2, 3
    b = Batch(True, [0, 0, 0], [300, 64, 131], Hq, Hk, seed=14)
    b.call()
    q = b.expect()
    b.check(q)
    k_q, k_e, npm = 2, 1, b.np_max
    alive = torch.full((B, Hk, (npm + 31) // 32), -1, dtype=torch.int32, device=DEV)
    rng = np.random.default_rng(1)
    ev = f32(rng.standard_normal((B, Hk, npm)))
    for step in range(steps):
        w = ref.bf16(rng.standard_normal((B, Hq + 2 * Hk, 128)))
        b.x, b.n, b.lens = w, B, np.ones(B, int)
        b.first, b.L = np.arange(B + 1, dtype=np.int32), b.L + 1
        d = bf(ref.bf16_bits(w))
        b.qd, b.kd, b.vd = d[:, :Hq], d[:, Hq:Hq + Hk], d[:, Hq + Hk:]
        b.q_out = torch.full((B, Hq, 128), 3.0, dtype=torch.bfloat16, device=DEV)
        b.call(row_first=None)
        b.check(b.expect())
        scores = torch.empty(B, Hk, npm, device=DEV)
        L, pt = i32(b.L), i32(b.pt)
        spkv.score_blocks(b.cache, b.q_out, pt, L, scores)
        sel = torch.empty(B, Hk, k_q + k_e + 1, dtype=torch.int32, device=DEV)
        n_sel = torch.empty(B, Hk, dtype=torch.int32, device=DEV)
        spkv.select_topk(b.cache, scores, ev, alive, L, k_q, k_e, sel, n_sel)
        out, lse = torch.empty(B, Hq, 128, device=DEV), torch.empty(B, Hq, device=DEV)
        spkv.sparse_decode_attn(b.cache, b.q_out, pt, sel, n_sel, L, out, lse)
        assert spkv.get_device_error(b.cache) == (0, 0)
        qx = ref.from_bf16_bits(host_bits(b.q_out))
        # block scores of complete pages: products with the sums, the largest sub-block
        k = ref.rows(b.blob, True) * b.gk[:, None, None, None].astype(np.float64)
        s = scores.cpu().numpy()
        for r in range(B):
            for h in range(Hk):
                qs = qx[r, 4 * h:4 * h + 4].astype(np.float64).sum(0)
                for p in range((int(b.L[r]) - 1) // 64):
                    sums = k[h, b.pt[r, p]].reshape(4, 16, 128).sum(1)
                    x = (sums @ qs).max() / (16 * np.sqrt(128))
                    bound = 140 * 2.0 ** -23 * (np.abs(sums) @ np.abs(qs)).max() / (16 * np.sqrt(128))
                    assert abs(s[r, h, p] - x) <= bound
        o, l, eo, el = ref.attention(qx, b.blob, b.gk, b.gv, b.pt, sel.cpu().numpy(), n_sel.cpu().numpy(), b.L)
        assert np.all(np.abs(out.cpu().numpy() - o).max(-1) <= eo)
        assert np.all(np.abs(lse.cpu().numpy() - l) <= el)


def test_unpacked_pages_feed_the_prefill():
    """A chunk into the 4-bit cache, its pages unpacked, and the bf16 prefill over them: the attention of the
    values that the cache holds (their bf16 rounding is the prefill's operand rounding: 2^-8 a weight and a
    value, the score off by 2^-8 sum |q k| / sqrt(128) at most)."""
    Hq, Hk = 4, 2
    b = Batch(True, [0], [150], Hq, Hk, seed=15)
    b.call()
    b.expect()
    pages = i32(b.pt[0, :3])
    k = torch.zeros(Hk, 3, 64, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    spkv.paged_kv_unpack_q4(b.cache, pages, k, v)
    stage = spkv.paged_kv_create(k, v, None, None, max_units=64)
    words = spkv.pack_page_words([0, 1, 2], [64, 64, 22], [0, 0, 0])
    T = 5
    qx = ref.bf16(np.random.default_rng(3).standard_normal((1, T, Hq, 128)))
    out, lse = torch.zeros(1, T, Hq, 128, device=DEV), torch.zeros(1, T, Hq, device=DEV)
    meta = torch.from_numpy(words.view(np.int32).reshape(1, 1, 3)).to(DEV)
    # every position the same as the document's start plus 150: rows of one request, offsets as stored keys
    spkv.lazy_rope_prefill_attn(stage, bf(ref.bf16_bits(qx)), i32([150]), meta, i32([3]), i32([[0]]), 500000.0, out, lse)
    assert spkv.get_device_error(stage) == (0, 0)
    tab = ref.table(200)
    for h in range(Hk):
        kk = np.concatenate([ref.rows(b.blob[h, p], True) for p in b.pt[0, :3]])[:150] * float(b.gk[h])
        vv = np.concatenate([ref.rows(b.blob[h, p], False) for p in b.pt[0, :3]])[:150] * float(b.gv[h])
        for t in range(T):
            c, s = tab[150 + t, :64].astype(np.float64), tab[150 + t, 64:].astype(np.float64)
            for g in range(h * 2, h * 2 + 2):
                x = qx[0, t, g].astype(np.float64)
                r = np.concatenate([x[:64] * c - x[64:] * s, x[64:] * c + x[:64] * s])
                sc = kk @ r / np.sqrt(128)
                p = np.exp(sc - sc.max())
                want = p @ vv / p.sum()
                dx = 2.0 ** -7 * (np.abs(kk) @ np.abs(r)).max() / np.sqrt(128)
                assert np.abs(out[0, t, g].cpu().numpy() - want).max() <= 2 * (dx + 2.0 ** -7) * np.abs(vv).max()


@pytest.mark.parametrize("q4", FORMATS)
def test_rows_in_front_count_as_held(q4):
    """A page whose count is behind the request's first new row: the rows in front are summed, as
    paged_kv_append sums them; what a count tells behind the last new row is summed too."""
    b = Batch(q4, [37, 100], [6, 2], 4, 2, seed=16)
    b.cnt[b.pt[0, 0]], b.cnt[b.pt[1, 1]] = 3, 45    # request 1's new rows are 36 and 37 of its page
    b.cnt_d.copy_(i32(b.cnt))
    b.call()
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
@pytest.mark.parametrize("B", [31, 32, 33, 70, 1100])
def test_many_requests(q4, B):
    """More requests than a warp looks through at once, most of them with a row or two or none."""
    rng = np.random.default_rng(B)
    lens = rng.choice([0, 0, 1, 1, 2, 19], B)
    lens[B // 2: B // 2 + 40] = 0
    lens[-1] = 3
    b = Batch(q4, rng.integers(0, 40, B), lens, 2, 1, seed=B)
    b.call(pair_axis=np.zeros(64, np.int64))
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
def test_rows_of_no_request(q4):
    """Rows before the first request, empty requests, and a call of nothing."""
    b = Batch(q4, [0, 9, 64], [5, 0, 4], 4, 2, seed=17, pad=6)
    b.first = b.first + 3      # rows 0 .. 2 and the last three belong to no request
    b.call()
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.check(b.expect())
    b.call(row_first=i32([3, 3, 3, 3]))
    b.check(b.expect_none())
    none = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=DEV)
    spkv.paged_kv_append_rope(b.cache, none, none, i32(np.zeros(0)), i32(np.zeros((0, 4))))


def test_two_handles_in_two_graphs():
    """Each handle has its own workspace: graphs of two, replayed on two streams at once."""
    caches = [Batch(q4, [40, 3], [1, 1], 8, 2, seed=18 + q4) for q4 in (True, False)]
    graphs = []
    keep = []
    for b in caches:
        a = i32(b.L), i32(b.pt)
        kw = dict(row_first=i32(b.first), q=b.qd, q_out=b.q_out, cos_sin=f32(b.tab))
        keep.append((a, kw))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            spkv.paged_kv_append_rope(b.cache, b.kd, b.vd, *a, **kw)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for b in caches:
        b.check(b.expect())


def test_refused_arguments():
    b = Batch(True, [5, 7], [1, 1], 8, 2, seed=19)
    wide = torch.zeros(2, 3, 130, dtype=torch.bfloat16, device=DEV)
    L, pt, tab = i32(b.L), i32(b.pt), f32(b.tab)
    rot = dict(q=b.qd, q_out=b.q_out, cos_sin=tab)

    def refused(error, *, k=b.kd, v=b.vd, L=L, pt=pt, cache=b.cache, **kw):
        with pytest.raises(error) as e:
            spkv.paged_kv_append_rope(cache, k, v, L, pt, **kw)
        return e.value

    E, A = ValueError, spkv.SpkvError
    refused(E, k=wide[:, :2, :128])                                  # heads apart
    refused(E, k=b.kd[:1])                                           # another number of rows
    assert refused(A, k=b.kd[:1].expand(2, 2, 128)).status == -1     # one row for all
    odd = torch.zeros(2, 2 * 128 + 4, dtype=torch.bfloat16, device=DEV)[:, :256].view(2, 2, 128)
    assert refused(A, v=odd).status == -1                            # rows 8 bytes off
    assert refused(A, k=torch.zeros(2 * 256 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(2, 2, 128)).status == -1
    assert refused(A, L=L[:1], pt=pt[:1]).status == -1               # two rows, one request, no row_first
    refused(E, q=b.qd, q_out=b.q_out)                                # queries are rotated or not given
    refused(E, q=b.qd, cos_sin=tab)                                  # nowhere to write them
    refused(E, pos=i32([1, 2]))
    refused(E, cos_sin=tab, pos=i32(1))
    refused(E, cos_sin=tab, pos=i32([[[1], [2]]]), pair_axis=[0] * 64)
    refused(E, cos_sin=tab, pos=i32([[1, 2], [3, 4]]))               # which axis turns which pair?
    refused(E, cos_sin=tab, pos=i32([[1, 2], [3, 4]]), pair_axis=[0] * 63)
    refused(E, cos_sin=tab, pos=i32([[1, 2], [3, 4]]), pair_axis=[2] * 64)
    refused(E, cos_sin=tab, pos=i32([[1, 2], [3, 4]]), pair_axis=[-1] * 64)
    refused(E, cos_sin=tab, pos=i32([[1, 2], [3, 4]]), pair_axis=np.full(64, 2))
    assert refused(A, cos_sin=tab, pos=i32(np.zeros((2, 5))), pair_axis=[4] * 64).status == -1   # five axes
    assert refused(A, q=b.qd[:, :7].contiguous(), q_out=b.q_out[:, :7].contiguous(), cos_sin=tab).status == -1
    many = torch.zeros(2, 34, 128, dtype=torch.bfloat16, device=DEV)
    assert refused(A, q=many, q_out=many, cos_sin=tab).status == -6  # more than 16 heads a group
    assert refused(A, pt=pt[:, :0], **rot).status == -1              # a table of no pages
    refused(TypeError, q=b.qd.half(), q_out=b.q_out, cos_sin=tab)
    refused(TypeError, L=L.long())
    bare = spkv.paged_kv_create_q4(b.pool, f32(b.gk), f32(b.gv), None, None, max_units=4)
    assert refused(A, cache=bare, **rot).status == -1                # no sums to keep
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.call(**rot)
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
def test_offsets_past_32_bits(q4):
    """A pool of more than 2^32 bytes, its last pages used: bit for bit what a small pool holds, gives and attends."""
    b = Batch(q4, [70], [130], 8, 1, seed=30, fused=True)
    n = (1 << 32) // (9216 if q4 else 16384) + 40
    pt = n - 1 - np.arange(b.np_max, dtype=np.int32)[None]
    cnt = torch.zeros(n, dtype=torch.int32, device=DEV)
    ksum = torch.zeros(1, n, 4, 128, device=DEV)
    old, new = torch.from_numpy(b.pt[0].astype(np.int64)).to(DEV), torch.from_numpy(pt[0].astype(np.int64)).to(DEV)
    cnt[new] = b.cnt_d[old]
    if q4:
        pools = [torch.zeros(1, n, 9216, dtype=torch.uint8, device=DEV)]
        small = [b.pool]
    else:
        pools = [torch.zeros(1, n, 64, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        small = [b.kp, b.vp]
    for big, sm in zip(pools, small):
        big[:, new] = sm[:, old]
    if q4:
        cache = spkv.paged_kv_create_q4(pools[0], f32(b.gk), f32(b.gv), ksum, cnt, max_units=4)
    else:
        cache = spkv.paged_kv_create(*pools, ksum, cnt, max_units=4)
    q_out = torch.zeros_like(b.q_out)
    spkv.paged_kv_append_rope(cache, b.kd, b.vd, i32(b.L), i32(pt), row_first=i32(b.first), q=b.qd, q_out=q_out, cos_sin=f32(b.tab))
    b.call()
    assert spkv.get_device_error(cache) == (0, 0)
    b.check(b.expect())
    assert torch.equal(q_out, b.q_out) and torch.equal(ksum[:, new], b.ksum[:, old]) and torch.equal(cnt[new], b.cnt_d[old])
    for big, sm in zip(pools, small):
        assert torch.equal(big[:, new], sm[:, old])
    outs = []
    for c, table in ((cache, pt), (b.cache, b.pt)):
        out, lse = torch.zeros(1, 8, 128, device=DEV), torch.zeros(1, 8, device=DEV)
        spkv.sparse_decode_attn(c, q_out[-1:].contiguous(), i32(table), i32([[[0, 1, 2, 3]]]), i32([[4]]), i32(b.L), out, lse)
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    if q4:
        pages = [torch.zeros(1, 4, 64, 128, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
        spkv.paged_kv_unpack_q4(cache, i32(pt[0, :4]), pages[0], pages[1])
        spkv.paged_kv_unpack_q4(b.cache, i32(b.pt[0, :4]), pages[2], pages[3])
        assert torch.equal(pages[0], pages[2]) and torch.equal(pages[1], pages[3])
