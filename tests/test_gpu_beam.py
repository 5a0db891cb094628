"""Beam search over paged caches on the GPU: selection, reordering, and both with a decode step."""
import numpy as np
import pytest
import torch

import beam_ref as ref
import q4_ref
import q8_ref
import sparse_paged_kv_score_gb300 as spkv
from helpers import DEV, bf, f32, host_bits, i32
from q4_ref import bf16, bf16_bits

pytestmark = pytest.mark.gpu

TYPES = [pytest.param(torch.float32, id="fp32"), pytest.param(torch.bfloat16, id="bf16"), pytest.param(torch.float16, id="fp16")]


def small_cache(max_units=4096):
    page = torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device=DEV)
    return spkv.paged_kv_create(page, page.clone(), None, None, max_units=max_units)


class Select:
    """Selection on logits [B][W][V], rows `pad` elements further apart, the first `shift` elements into their storage."""

    def __init__(self, x, cum, K, pad=0, shift=0, cache=None, plan=None):
        self.cache = cache or small_cache()
        self.B, self.W, self.V = x.shape
        store = torch.full((self.B * self.W * (self.V + pad) + shift + pad,), 77.0, dtype=x.dtype, device=DEV)
        rows = store[shift:shift + self.B * self.W * (self.V + pad)].view(self.B, self.W, self.V + pad)
        rows[..., :self.V] = x.to(DEV)
        self.x = rows[..., :self.V]
        self.host = x.double().cpu().numpy()
        self.cum = np.asarray(cum, np.float32)
        self.cum_d = f32(self.cum)
        self.plan = plan or spkv.BeamPlan(self.cache, self.B * self.W, self.V)
        self.tokens, self.parents = (torch.full((self.B, K), 7, dtype=torch.int32, device=DEV) for _ in range(2))
        self.scores = torch.full((self.B, K), 7.0, device=DEV)
        self.K = K

    def call(self, **kw):
        spkv.beam_select(self.cache, self.plan, self.x, self.cum_d, self.tokens, self.parents, self.scores, **kw)

    def check(self, bits=0):
        assert spkv.get_device_error(self.cache)[1] == bits
        t, p, s = self.tokens.cpu().numpy(), self.parents.cpu().numpy(), self.scores.cpu().numpy().astype(np.float64)
        for b in range(self.B):
            ref.check_best(self.host[b], self.cum[b], self.K, t[b], p[b], s[b])
        return t, p, s


def logits(B, W, V, dtype, seed=0, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, W, V, generator=g) * scale
    x.scatter_(2, torch.randint(0, V, (B, W, 5), generator=g), 4 + 6 * torch.rand(B, W, 5, generator=g))
    return x.to(dtype)


def cums(B, W, seed=0):
    return -np.sort(np.random.default_rng(seed).uniform(0, 9, (B, W)).astype(np.float32), 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,W,V,K", [(1, 1, 1, 1), (1, 1, 1, 3), (2, 1, 5, 2), (1, 4, 32000, 8), (3, 2, 1024, 4), (2, 3, 2047, 6),
                                     (5, 5, 10007, 10), (1, 64, 700, 128), (2, 16, 4099, 33), (1, 2, 200001, 64)])
def test_select(dtype, B, W, V, K):
    s = Select(logits(B, W, V, dtype, seed=V), cums(B, W, V), K)
    s.call()
    s.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 1, 3, 64])
@pytest.mark.parametrize("shift", [0, 1, 5, 37, 63])
def test_select_rows_anywhere(dtype, pad, shift):
    """Rows that begin at any element of a 128-byte line, and lie apart; what lies between them (the largest numbers) is not
    looked at."""
    s = Select(logits(2, 3, 1500 + 7 * shift, dtype, seed=pad), cums(2, 3), 6, pad=pad, shift=shift)
    s.call()
    s.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_select_ties(dtype):
    """Equal logits: the lower token of a beam; equal beams: the lower beam."""
    for x in (torch.zeros(2, 3, 5000), torch.zeros(1, 2, 40), logits(2, 3, 5000, torch.float32).round()):
        s = Select(x.to(dtype), np.zeros(x.shape[:2]) - 1, 16)
        s.call()
        t, p, _ = s.check()
        if not x.any():     # all alike
            V = x.shape[2]
            assert np.array_equal(t[0], np.arange(16) % V) and np.all(p[0] == 0)
    x = logits(1, 1, 3001, dtype).expand(1, 4, 3001).contiguous()     # four beams alike, each K-th best four times
    s = Select(x, np.zeros((1, 4)), 10)
    s.call()
    t, p, v = s.check()
    assert np.array_equal(p[0], [0, 1, 2, 3, 0, 1, 2, 3, 0, 1])
    assert np.array_equal(t[0, ::4][:2], t[0, 1::4][:2])


@pytest.mark.parametrize("order", ["up", "down", "one_line", "lines"])
def test_select_orders(order):
    """The best ones beside one another or far apart."""
    V, K = 70000, 32
    x = torch.zeros(1, 2, V)
    if order == "up":
        x[:] = torch.arange(V) * 1e-4
    elif order == "down":
        x[:] = -torch.arange(V) * 1e-4
    elif order == "one_line":
        x[0, 1, 32 * 100:32 * 101] = 5 + torch.rand(32)
    else:
        x[0, 0, ::1024][:K] = 5 + torch.rand(K)
    s = Select(x, [[0.0, -0.25]], K)
    s.call()
    s.check()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype,e", [(t, e) for t, es in ((torch.float32, (10, 20, 23, 24, 25, 29, 30, 31, 32, 40, 64, 100, 125, 126, 127)),
                                                           (torch.bfloat16, (7, 15, 23, 24, 30, 31, 33, 64, 126, 127)),
                                                           (torch.float16, (7, 11, 15))) for e in es])
def test_select_sizes(dtype, e, sign):
    """Logits of magnitude 2^e, some of them steps of their type apart, and far smaller ones."""
    V, step = 5000, torch.finfo(dtype).eps * 2.0 ** e
    x = 2.0 ** e + step * torch.randint(0, 9, (2, 3, V), generator=torch.Generator().manual_seed(e)).double()
    x[:, :, ::7] = torch.randn(2, 3, x[:, :, ::7].shape[2], dtype=torch.float64) if sign > 0 else 1.5 * 2.0 ** e
    s = Select((sign * x).to(dtype), cums(2, 3, e), 12)
    s.call()
    s.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_select_masks(dtype):
    """-infinity and the type's lowest value as masks; rows with nothing left, few tokens left; beams that ended."""
    low = torch.finfo(dtype).min
    x = logits(4, 4, 3000, torch.float32, seed=3)
    x[:, :, 100:] = -np.inf
    x[0, 1] = -np.inf                 # nothing left
    x[0, 2, 3:] = -np.inf             # three tokens
    x = x.to(dtype)
    x[1, :, 1:] = low                 # one token, and the rest at the lowest value
    x[2, 0] = low                     # nothing but the lowest value: all alike
    cum = cums(4, 4)
    cum[1, 2] = cum[2, 1] = cum[2, 3] = -np.inf
    cum[3] = -np.inf                  # no beam at all
    s = Select(x, cum, 12)
    s.call()
    t, p, v = s.check()
    assert np.all(t[3] == -1) and np.all(np.isneginf(v[3]))
    assert 1 not in p[0] and 2 not in p[1]
    s = Select(x[:1, 1:3], [[0, 0]], 12)     # three candidates in all
    s.call()
    t, p, v = s.check()
    assert np.array_equal(t[0, 3:], [-1] * 9) and np.all(p[0, :3] == 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("special", [np.nan, np.inf])
def test_select_special_values(dtype, special):
    """A NaN or +infinity among a beam's logits, or as its score: no candidates from it, flagged; the others are chosen from."""
    x = logits(2, 3, 4000, dtype, seed=5)
    x[0, 1, 1234] = special
    s = Select(x, cums(2, 3), 6)
    s.call()
    _, p, _ = s.check(spkv.DEVERR["BEAM"])
    assert 1 not in p[0]
    cum = cums(2, 3)
    cum[1, 0] = special
    s = Select(logits(2, 3, 4000, dtype, seed=5), cum, 6)
    s.call()
    _, p, _ = s.check(spkv.DEVERR["BEAM"])
    assert 0 not in p[1]


def test_select_ended_beams_are_not_read():
    """A beam whose score is -infinity may have anything as logits."""
    x = logits(1, 3, 5000, torch.float32)
    x[0, 1] = np.nan
    cum = cums(1, 3)
    cum[0, 1] = -np.inf
    s = Select(x, cum, 6)
    s.call()
    s.check()


def test_select_extreme_scores():
    """Large logits, large negative scores, a beam far behind."""
    x = logits(2, 3, 3000, torch.float32, scale=1000.0)
    s = Select(x, [[-1e6, -2.0, -1e-30], [0, -1e30, -5]], 6)
    s.call()
    s.check()
    x = torch.full((1, 2, 600), -3.0e38)
    x[0, 0, 5], x[0, 1, 7] = 3.0e38, 3.2e38
    s = Select(x, [[0, -1]], 4)
    s.call()
    t, p, _ = s.check()
    assert (t[0, 0], p[0, 0], t[0, 1], p[0, 1]) == (5, 0, 7, 1)


def test_select_plan_for_smaller_calls_and_in_graphs():
    """One plan for calls of any size that fit; a replayed graph of two calls; another stream; the same bits each time."""
    cache = small_cache()
    plan = spkv.BeamPlan(cache, 32, 20000)
    runs = []
    for B, W, V, dtype in ((8, 4, 20000, torch.float32), (1, 2, 50, torch.bfloat16), (2, 16, 9999, torch.float16)):
        s = Select(logits(B, W, V, dtype, seed=B), cums(B, W, B), 2 * W, cache=cache, plan=plan)
        s.call()
        s.check()
        runs.append((s, s.tokens.clone(), s.scores.clone()))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for s, _, _ in runs:
            s.call()
    side = torch.cuda.Stream()
    for how in (g.replay, g.replay, lambda: [s.call(stream=side) for s, _, _ in runs]):
        for s, _, _ in runs:
            s.tokens.fill_(7)
            s.scores.fill_(7)
        torch.cuda.synchronize()
        how()
        torch.cuda.synchronize()
        for s, t, v in runs:
            assert torch.equal(s.tokens, t) and torch.equal(s.scores, v)
    with pytest.raises(spkv.SpkvError):
        Select(logits(1, 33, 100, torch.float32), cums(1, 33), 4, cache=cache, plan=plan).call()
    with pytest.raises(spkv.SpkvError):
        Select(logits(1, 2, 20001, torch.float32), cums(1, 2), 4, cache=cache, plan=plan).call()


# ---------------------------------------------------------------------------------------------- reordering


class Beams:
    """A cache of any format with tables of B requests' W beams; rows of random bytes (codes) or numbers."""

    def __init__(self, fmt, B, W, Hk, L, np_max=None, seed=0, sums=True):
        rng = np.random.default_rng(seed)
        self.fmt, self.B, self.W, self.Hk = fmt, B, W, Hk
        self.L = np.asarray(L, np.int32)
        self.np_max = np_max or int(self.L.max()) // 64 + 2
        self.n_phys = B * (W * 2 + 3) + 1
        ids = rng.permutation(self.n_phys - 1).reshape(B, -1)
        self.pt = np.stack([ids[b, W:][rng.integers(0, W + 3, (W, self.np_max))] for b in range(B)]).astype(np.int32)
        self.cnt = np.full(self.n_phys, 64, np.int32)
        for b in range(B):
            full = self.L[b] // 64
            self.pt[b, :, full:] = ids[b, :W, None]
            self.cnt[ids[b, :W]] = self.L[b] % 64 + rng.integers(0, 2, W) * (64 - self.L[b] % 64 > 3) * 3   # some hold rows behind
        self.pt = self.pt.reshape(B * W, self.np_max)
        self.seq = np.repeat(self.L, W).astype(np.int32)
        self.cnt_d = i32(self.cnt) if sums else None
        self.ksum = torch.zeros(Hk, self.n_phys, 4, 128, device=DEV, dtype=torch.bfloat16 if fmt == "q4" else torch.float32) if sums else None
        if fmt == "bf16":
            self.pools = [bf(bf16_bits(rng.standard_normal((Hk, self.n_phys, 64, 128)))) for _ in range(2)]
            self.cache = spkv.paged_kv_create(*self.pools, self.ksum, self.cnt_d, max_units=max(1, B * W * Hk))
        else:
            size = 9216 if fmt == "q4" else 16416
            blob = rng.integers(0, 120, (Hk, self.n_phys, size), dtype=np.uint8)
            if fmt == "q8":
                blob[..., 16384:] = np.full(8, 0.25, np.float32).view(np.uint8)
            self.pools = [torch.from_numpy(blob).to(DEV)]
            one = torch.ones(Hk, device=DEV)
            args = (self.pools[0], one, one) if fmt == "q4" else (self.pools[0],)
            create = spkv.paged_kv_create_q4 if fmt == "q4" else spkv.paged_kv_create_q8
            self.cache = create(*args, self.ksum, self.cnt_d, max_units=max(1, B * W * Hk))
        self.table = i32(self.pt)

    def expect(self, parents, bad=()):
        new, copies = ref.reorder(np.asarray(parents), self.pt, self.seq)
        pools = [p.clone() for p in self.pools]
        ksum = None if self.ksum is None else self.ksum.clone()
        cnt = self.cnt.copy()
        for b, src, dst in copies:
            if b in bad:
                continue
            n = 64 if self.cnt_d is None else int(self.cnt[src])
            for p in pools:
                if self.fmt == "bf16":
                    p[:, dst, :n] = p[:, src, :n]
                else:
                    p[:, dst] = p[:, src]
            if ksum is not None:
                ksum[:, dst] = ksum[:, src]
            cnt[dst] = cnt[src]
        return new, pools, ksum, cnt

    def check(self, want):
        new, pools, ksum, cnt = want
        assert np.array_equal(self.table.cpu().numpy(), new)
        for p, w in zip(self.pools, pools):
            assert torch.equal(p.view(torch.uint8), w.view(torch.uint8))
        if ksum is not None:
            assert torch.equal(self.ksum, ksum) and np.array_equal(self.cnt_d.cpu().numpy(), cnt)
        self.pt, self.cnt = new, cnt

    def call(self, parents, **kw):
        spkv.beam_reorder(self.cache, i32(parents), self.table, i32(self.seq), **kw)


FORMATS = ["bf16", "q4", "q8"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,W,Hk,L", [(1, 1, 1, [5]), (1, 4, 2, [1000]), (3, 5, 2, [64, 1, 130]), (2, 64, 1, [500, 63]), (7, 33, 1, [66] * 7),
                                      (1, 2, 8, [7000]), (4, 3, 2, [0, 128, 64 * 70 + 1, 2])])
def test_reorder(fmt, B, W, Hk, L):
    s = Beams(fmt, B, W, Hk, L, seed=W)
    rng = np.random.default_rng(B)
    for step in range(4):      # one after another, in place
        parents = rng.integers(0, W, (B, W)) if step else np.zeros((B, W), int)
        want = s.expect(parents)
        s.call(parents)
        assert spkv.get_device_error(s.cache) == (0, 0)
        s.check(want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sums", [True, False])
def test_reorder_parents(fmt, sums):
    """Every beam its own parent (nothing moves), a rotation (nothing is copied), all of one, beams that stop, no parents."""
    W = 6
    for parents in ([0, 1, 2, 3, 4, 5], [1, 2, 3, 4, 5, 0], [3] * 6, [5, 5, -1, 5, 0, 0], [-1] * 6, [-1, 0, -1, 0, 2, -1]):
        s = Beams(fmt, 2, W, 2, [200, 77], seed=3, sums=sums)
        p = np.array([parents, parents[::-1]])
        want = s.expect(p)
        s.call(p)
        assert spkv.get_device_error(s.cache) == (0, 0)
        s.check(want)
        if parents == list(range(W)):
            assert np.array_equal(want[0][:W], s.pt[:W])


def test_reorder_bad_requests_are_left_alone():
    s = Beams("bf16", 5, 3, 2, [200, 300, 100, 250, 90], seed=5)
    par = np.array([[0, 0, 1], [0, 3, 0], [2, 2, 2], [1, 0, -2], [1, 1, 0]])
    s.seq[2 * 3 + 1] += 1                     # beams of different lengths
    good = np.array([[0, 0, 1], [0, 1, 2], [0, 1, 2], [0, 1, 2], [1, 1, 0]])
    seq = s.seq.copy()
    s.seq[7] -= 1
    want = s.expect(good)
    s.seq = seq
    s.call(par)
    assert spkv.get_device_error(s.cache) == (-4, spkv.DEVERR["BEAM"])
    s.check(want)
    # a column outside the table, a negative length
    s = Beams("bf16", 3, 2, 1, [100, 140, 70], seed=6, np_max=3)
    want = s.expect(np.array([[0, 1], [0, 1], [1, 1]]))
    s.seq[:4] = [193, 193, -1, -1]
    s.call(np.array([[0, 0], [1, 1], [1, 1]]))
    assert spkv.get_device_error(s.cache) == (-4, spkv.DEVERR["PAGE_ID"])
    s.check(want)
    # part-filled pages outside the pool: tables follow, nothing is copied
    s = Beams("bf16", 2, 2, 2, [100, 140], seed=7)
    s.pt[1, 1:] = s.n_phys
    s.pt[0 + 2, 2:] = -5
    s.table = i32(s.pt)
    par = np.array([[0, 0], [0, 0]])
    new, copies = ref.reorder(par, s.pt, s.seq)
    pools = [p.clone() for p in s.pools]
    s.call(par)
    assert spkv.get_device_error(s.cache) == (-4, spkv.DEVERR["PHYS"])
    assert np.array_equal(s.table.cpu().numpy(), new) and all(torch.equal(a, b) for a, b in zip(s.pools, pools))


def test_reorder_in_a_graph_and_on_another_stream():
    par = np.array([[1, 1, 0], [2, 2, 2]])
    s = Beams("q8", 2, 3, 2, [200, 77], seed=8)
    p, n = i32(par), i32(s.seq)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        spkv.beam_reorder(s.cache, p, s.table, n)
    for _ in range(3):
        want = s.expect(par)
        g.replay()
        s.check(want)
    side = torch.cuda.Stream()
    want = s.expect(par)
    torch.cuda.synchronize()
    s.call(par, stream=side)
    side.synchronize()
    s.check(want)


def test_refused_arguments():
    cache = small_cache(max_units=8)
    plan = spkv.BeamPlan(cache, 8, 100)
    s = Select(logits(2, 4, 100, torch.float32), cums(2, 4), 8, cache=cache, plan=plan)
    bad = [
        (TypeError, dict(x=s.x.double())), (TypeError, dict(x=None)), (ValueError, dict(x=s.x.cpu())), (ValueError, dict(x=s.x[0])),
        (ValueError, dict(x=s.x.transpose(1, 2).contiguous().transpose(1, 2))), (ValueError, dict(x=s.x[:, :3])),
        (ValueError, dict(x=s.x[:, :1].expand(2, 4, 100))), (ValueError, dict(cum_d=s.cum_d[:1])), (TypeError, dict(cum_d=s.cum_d.double())),
        (ValueError, dict(tokens=s.tokens[:, :3])), (ValueError, dict(scores=s.scores.cpu())), (TypeError, dict(parents=s.parents.long())),
    ]
    for kind, change in bad:
        old = {k: getattr(s, k) for k in change}
        for k, v in change.items():
            setattr(s, k, v)
        with pytest.raises(kind):
            s.call()
        for k, v in old.items():
            setattr(s, k, v)
    s.call()
    s.check()
    t = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    n = torch.zeros(8, dtype=torch.int32, device=DEV)
    par = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    for args in ((par.long(), t, n), (par, t[:7], n), (par, t, n[:7]), (par.cpu(), t, n), (par, t.float(), n)):
        with pytest.raises((TypeError, ValueError)):
            spkv.beam_reorder(cache, *args)
    with pytest.raises(spkv.SpkvError):      # more beams and heads than the handle's units
        spkv.beam_reorder(cache, par.expand(2, 4).repeat(2, 1), t.repeat(2, 1), n.repeat(2))
    spkv.beam_reorder(cache, par, t, n)
    assert spkv.get_device_error(cache) == (0, 0)


# ---------------------------------------------------------------------------------------------- as they are used


@pytest.mark.parametrize("B,W,past", [(2, 3, 50), (1, 4, 64), (3, 2, 5)])
def test_beam_search_on_an_8bit_cache(B, W, past):
    """A prompt forked to beams, then steps of append, attention, selection and reordering over two page borders: every
    beam's pages hold bit for bit what its own history gives, attention and selection are right at every step."""
    Hq, Hk, V, steps = 4, 2, 1111, 80
    rng = np.random.default_rng(past)
    N = B * W
    np_max = (past + steps) // 64 + 1
    n_phys = B + N * (np_max + 1)
    pool = torch.zeros(Hk, n_phys, q8_ref.BLOB, dtype=torch.uint8, device=DEV)
    cnt, ksum = torch.zeros(n_phys, dtype=torch.int32, device=DEV), torch.zeros(Hk, n_phys, 4, 128, device=DEV)
    cache = spkv.paged_kv_create_q8(pool, ksum, cnt, max_units=N * Hk)
    plan = spkv.BeamPlan(cache, N, V)
    tab = f32(q4_ref.table(past + steps + 1))
    table_h = q4_ref.table(past + steps + 1)
    spare = iter(rng.permutation(n_phys).tolist())
    pt = np.zeros((N, np_max), np.int32)
    for n in range(N):
        for p in range((past + 63) // 64):
            pt[n, p] = next(spare) if n % W == 0 or (past % 64 and p == past // 64) else 0
    # the prompt, in each request's beam 0
    kp, vp = bf16(rng.standard_normal((B * past, Hk, 128))), bf16(rng.standard_normal((B * past, Hk, 128)))
    spkv.paged_kv_append_rope(cache, bf(bf16_bits(kp)), bf(bf16_bits(vp)), i32([past] * B), i32(pt[::W]),
                              row_first=i32(np.arange(B + 1) * past), q=torch.zeros(B * past, Hq, 128, dtype=torch.bfloat16, device=DEV),
                              q_out=torch.zeros(B * past, Hq, 128, dtype=torch.bfloat16, device=DEV), cos_sin=tab)
    table = i32(pt)
    spkv.beam_reorder(cache, i32(np.zeros((B, W))), table, i32([past] * N))
    history = [[(kp[b * past + i], vp[b * past + i]) for i in range(past)] for b in range(B) for _ in range(W)]
    cum = np.full((B, W), -np.inf, np.float32)
    cum[:, 0] = 0
    cum_d = f32(cum)
    weight = torch.randn(V, Hq * 128, device=DEV) * 0.6
    embed = rng.standard_normal((V, Hq + 2 * Hk, 128))
    token = np.zeros((B, W), int)
    for step in range(steps):
        L = past + step + 1
        if (L - 1) % 64 == 0:       # a new page for each beam
            t = table.cpu().numpy()
            t[:, (L - 1) // 64] = [next(spare) for _ in range(N)]
            table.copy_(i32(t))
        x = bf16(embed[token.reshape(-1)] + 0.1 * rng.standard_normal((N, Hq + 2 * Hk, 128)))
        d = bf(bf16_bits(x))
        q, k, v = d[:, :Hq], d[:, Hq:Hq + Hk], d[:, Hq + Hk:]
        q_rot = torch.zeros(N, Hq, 128, dtype=torch.bfloat16, device=DEV)
        seq = i32([L] * N)
        spkv.paged_kv_append_rope(cache, k, v, seq, table, q=q, q_out=q_rot, cos_sin=tab)
        pages = (L + 63) // 64
        sel = i32(np.tile(np.arange(pages), (N, Hk, 1)))
        n_sel = i32(np.full((N, Hk), pages))
        out, lse = torch.zeros(N, Hq, 128, device=DEV), torch.zeros(N, Hq, device=DEV)
        spkv.sparse_decode_attn(cache, q_rot, table, sel, n_sel, seq, out, lse)
        logit = (out.flatten(1) @ weight.T).view(B, W, V)
        K = 2 * W
        tokens, parents, scores = (torch.zeros(B, K, dtype=t, device=DEV) for t in (torch.int32, torch.int32, torch.float32))
        spkv.beam_select(cache, plan, logit, cum_d, tokens, parents, scores)
        for n in range(N):
            history[n] = history[n] + [(x[n, Hq:Hq + Hk], x[n, Hq + Hk:])]
        if step % 13 == 0 or step == steps - 1:
            blob, t = pool.cpu().numpy(), table.cpu().numpy()
            for n in range(N):
                for j in range((L + 15) // 16):
                    rows = range(16 * j, min(L, 16 * j + 16))
                    ang = table_h[list(rows)]
                    want = np.zeros((Hk, q8_ref.BLOB), np.uint8)
                    for h in range(Hk):
                        kk = q4_ref.rotate(np.stack([history[n][i][0][h] for i in rows]), ang[:, :64], ang[:, 64:])
                        q8_ref.put(want[h], j % 4, {i % 16: kk[e] for e, i in enumerate(rows)}, [], True)
                        q8_ref.put(want[h], j % 4, {i % 16: history[n][i][1][h] for i in rows}, [], False)
                    got = blob[:, t[n, j // 4]]
                    for at in (q8_ref.KC, q8_ref.VC):
                        where = at[[i % 64 for i in rows]]
                        assert np.array_equal(got[:, where], want[:, where]), (n, j)
                    for keys in (True, False):
                        assert np.array_equal(q8_ref.scales(got, keys)[:, j % 4], q8_ref.scales(want, keys)[:, j % 4])
            qx = q4_ref.from_bf16_bits(host_bits(q_rot))
            o, l, eo, el = q8_ref.attention(qx, blob, t, sel.cpu().numpy(), n_sel.cpu().numpy(), seq.cpu().numpy())
            assert np.all(np.abs(out.cpu().numpy() - o).max(-1) <= eo) and np.all(np.abs(lse.cpu().numpy() - l) <= el)
            for b in range(B):
                ref.check_best(logit[b].double().cpu().numpy(), cum[b], K, tokens[b].cpu().numpy(), parents[b].cpu().numpy(),
                               scores[b].cpu().numpy().astype(np.float64))
        # the first W go on
        token, par, cum = tokens[:, :W].cpu().numpy(), parents[:, :W].cpu().numpy(), scores[:, :W].cpu().numpy()
        cum_d = f32(cum)
        spkv.beam_reorder(cache, i32(par), table, seq)
        history = [history[b * W + par[b, w]] for b in range(B) for w in range(W)]
    assert spkv.get_device_error(cache) == (0, 0)
