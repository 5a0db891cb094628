"""The 4-bit attention: every group size, lists in any order, queries that hold infinities and NaN; and the calls
around it (block scores through a directory, selection, residency) on a 4-bit handle."""
import numpy as np
import pytest
import torch

import q4_ref as ref
import sparse_paged_kv_score_gb300 as spkv
from helpers import DEV, bf, f32, i32
from test_gpu_q4 import Cache, check, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,Hk", [(2, 3), (6, 2), (7, 4), (9, 1), (10, 1), (11, 2), (12, 1), (13, 1), (14, 1), (15, 1), (15, 3)])
@pytest.mark.parametrize("L", [1, 65, 900])
def test_group_sizes(G, Hk, L):
    """Groups that leave query columns, a second half of them, or none unused; lists of all pages and of any."""
    B = 5
    c = Cache(Hk, B, (L + 63) // 64 + 1, [L, max(1, L - 1), max(1, L // 2), 1, max(1, L // 3)], seed=G + L, junk=True)
    rng = np.random.default_rng(G)
    qx, q = queries(B, G * Hk, seed=G)
    pages = (L + 63) // 64
    for counts in (None, rng.integers(0, pages + 1, (B, Hk))):
        sel, n = c.select(pages, rng, counts)
        out, lse = c.attend(q, sel, n)
        assert spkv.get_device_error(c.handle) == (0, 0)
        check(out, lse, ref.attention(qx, c.blob, c.gk, c.gv, c.pt, sel, n, c.L))


@pytest.mark.parametrize("Hq,Hk,pages", [(8, 2, 40), (7, 1, 40), (16, 1, 23), (2, 2, 5), (4, 1, 130)])
def test_lists_in_any_order(Hq, Hk, pages):
    """The local, incomplete page first, last or between; each order against the 64-bit form, a repeat bit for bit."""
    c = Cache(Hk, 3, pages, [64 * pages - 9, 64 * pages - 63, 64 * (pages // 2) + 30], seed=pages, junk=True)
    rng = np.random.default_rng(pages)
    sel, n = c.select(pages, rng, rng.integers(1, pages + 1, (3, Hk)))
    qx, q = queries(3, Hq, seed=2)
    want = ref.attention(qx, c.blob, c.gk, c.gv, c.pt, sel, n, c.L)
    orders = [sel.copy() for _ in range(4)]
    for b in range(3):
        for h in range(Hk):
            k = n[b, h]
            orders[1][b, h, :k] = sel[b, h, :k][::-1]
            orders[2][b, h, :k] = rng.permutation(sel[b, h, :k])
            orders[3][b, h, :k] = np.roll(sel[b, h, :k], k // 2)
    for o in orders:
        first, again = c.attend(q, o, n), c.attend(q, o, n)
        assert spkv.get_device_error(c.handle) == (0, 0)
        check(*first, want)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("Hq,Hk", [(4, 1), (12, 1)])
@pytest.mark.parametrize("wide,exact", [(30, True), (34, False), (44, False)])
def test_queries_of_a_wide_range(Hq, Hk, wide, exact):
    """Sixteen dims 2^wide times the others, where the keys are zero.  A query row goes into f16 with its largest dim in
    [2^13, 2^14): dims within 30 powers of two of that one keep all 8 bits (f16 holds 8 bits down to 2^-17), a smaller one
    is off by half of f16's smallest number, 2^-25, at most: 2^-38 of the largest."""
    c = Cache(Hk, 2, 6, [380, 200], seed=51, junk=True)
    c.blob[:, :, ref.KC[:, :8]] = 0
    c.pool.copy_(torch.from_numpy(c.blob))
    sel, n = c.select(6, np.random.default_rng(3))
    rng = np.random.default_rng(wide)
    qx = rng.choice([-1, 1], (2, Hq, 128)) * (rng.uniform(1, 1.9, (2, Hq, 128)) if exact else rng.standard_normal((2, Hq, 128)))
    qx[:, :, :16] *= 2.0 ** wide
    qx[:, :, 3] = 2.0 ** wide
    qx = ref.bf16(qx.astype(np.float32))
    out, lse = c.attend(bf(ref.bf16_bits(qx)), sel, n)
    o, l, eo, el = ref.attention(qx, c.blob, c.gk, c.gv, c.pt, sel, n, c.L)
    if not exact:
        k, v = (np.abs(np.nan_to_num(ref.rows(c.blob, keys))) for keys in (True, False))
        dx = 2.0 ** -38 * np.abs(qx).max() * (k * c.gk[:, None, None, None]).sum(-1).max() / np.sqrt(128)
        eo, el = eo + 2 * dx * (v * c.gv[:, None, None, None]).max(), el + dx
    check(out, lse, (o, l, eo, el))


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (6, 1), (16, 1), (13, 1)])
@pytest.mark.parametrize("special", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("L", [3, 700])
def test_queries_with_infinities_and_nan(Hq, Hk, special, L):
    """A query head with one has infinite or NaN scores for every token, so its softmax, and its outputs, are NaN; the
    other heads of its group, which share its products, are as ever, and so are empty lists."""
    B, pages = 3, (L + 63) // 64
    c = Cache(Hk, B, pages, [L, L, L], seed=L, junk=True)
    sel, n = c.select(pages, np.random.default_rng(1))
    n[2, 0] = 0
    qx, _ = queries(B, Hq, seed=4)
    bad = [(0, 0), (1, Hq - 1), (2, 0)]
    for k, (b, g) in enumerate(bad):
        qx[b, g, 5 + 60 * k] = special
        qx[b, g, 7] = 3e38          # past f16 beside it
    q = bf(ref.bf16_bits_special(qx))
    out, lse = c.attend(q, sel, n)
    assert spkv.get_device_error(c.handle) == (0, 0)
    for b, g in bad[:2]:
        assert torch.isnan(out[b, g]).all() and torch.isnan(lse[b, g])
        qx[b, g] = 0
        out[b, g], lse[b, g] = 0, 0
    qx[2, 0] = 0
    o, l, eo, el = ref.attention(qx, c.blob, c.gk, c.gv, c.pt, sel, n, c.L)
    for b, g in bad[:2]:
        o[b, g], l[b, g] = 0, 0
    check(out, lse, (o, l, eo, el))


@pytest.mark.parametrize("ksum_dtype", [torch.float32, torch.bfloat16])
def test_scores_selection_residency_on_a_4bit_handle(ksum_dtype):
    """The calls that read pooled sums or no pool at all: bit for bit what a bf16 handle with the same sums gives, through
    the flat table and the directory."""
    B, Hk, Hq, npm = 3, 2, 8, 20
    c = Cache(Hk, B, npm, [1280, 900, 70], seed=41, ksum_dtype=ksum_dtype)
    pages = torch.zeros(Hk, c.n_phys, 64, 128, dtype=torch.bfloat16, device=DEV)
    other = spkv.paged_kv_create(pages, pages.clone(), torch.zeros_like(c.ksum), c.cnt_d, max_units=B * Hk)
    torch.cuda.synchronize()
    other.tensors[2].copy_(c.ksum)      # that handle's sums are now the 4-bit one's
    _, q = queries(B, Hq, seed=5)
    pt, L = i32(c.pt), i32(c.L)
    pm = spkv.PageMap(B, npm, seg_shift=4, n_dev_segs=2)
    for b in range(B):
        pm.map(b, 0, c.pt[b])
    pm.promote(1, 1)
    pm.sync()
    ev = f32(np.random.default_rng(2).standard_normal((B, Hk, npm)))
    k_q, k_e = 5, 2
    stride, U, slots = k_q + k_e + 1, B * Hk, 10
    results = []
    for h in (other, c.handle):
        r = {}
        r["scores"] = torch.full((B, Hk, npm), 3.0, device=DEV)
        spkv.score_blocks(h, q, pt, L, r["scores"])
        r["scores_dir"] = torch.full((B, Hk, npm), 3.0, device=DEV)
        spkv.score_blocks_dir(h, q, pm, L, r["scores_dir"])
        assert torch.equal(r["scores"], r["scores_dir"])
        ints = lambda *s: torch.full(s, -1, dtype=torch.int32, device=DEV)  # noqa: E731
        r["alive"], r["sel"], r["n_sel"] = ints(B, Hk, 1), ints(B, Hk, stride), ints(B, Hk)
        spkv.select_topk(h, r["scores"], ev, r["alive"], L, k_q, k_e, r["sel"], r["n_sel"])
        r["resident"], r["ts"] = ints(U, slots), ints(U, slots).fill_(-2 ** 31)
        r["missing"], r["n_missing"], r["slot"] = ints(U, stride), ints(U), ints(U, stride)
        spkv.resident_setdiff(h, r["resident"], r["sel"], r["n_sel"], r["missing"], r["n_missing"], r["slot"])
        r["victims"], r["hist"] = ints(U, stride), ints(U, 64)
        spkv.lru_bucket_update(h, r["resident"], r["ts"], r["slot"], r["n_sel"].view(U), r["missing"], r["n_missing"], 0, 1,
                               r["victims"], r["hist"])
        r["alive2"], r["sel2"], r["n_sel2"] = ints(B, Hk, 1), ints(B, Hk, stride), ints(B, Hk)
        r["resident2"], r["ts2"] = ints(U, slots), ints(U, slots).fill_(-2 ** 31)
        r["missing2"], r["n_missing2"], r["slot2"] = ints(U, stride), ints(U), ints(U, stride)
        r["victims2"], r["hist2"] = ints(U, stride), ints(U, 64)
        spkv.select_resident_update(h, r["scores"], ev, r["alive2"], L, k_q, k_e, r["sel2"], r["n_sel2"], r["resident2"],
                                    r["ts2"], 0, 1, r["missing2"], r["n_missing2"], r["slot2"], r["victims2"], r["hist2"])
        assert spkv.get_device_error(h) == (0, 0)
        results.append(r)
    a, b = results
    for name in a:
        assert torch.equal(a[name], b[name]), name
    assert int(a["n_sel"].max()) > 1
    pm.close()


def test_unpack_in_a_graph_and_on_another_stream():
    """The unpacking captured and replayed after the pages changed, and eagerly on a side stream."""
    c = Cache(2, 2, 4, [250, 64], seed=42)
    pages = i32(np.concatenate([c.pt[0], c.pt[1, :1]]))
    n = pages.numel()
    k, v = (torch.zeros(2, n, 64, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        spkv.paged_kv_unpack_q4(c.handle, pages, k, v)
    side.synchronize()
    want = k.clone(), v.clone()
    assert float(want[0].float().abs().max()) > 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spkv.paged_kv_unpack_q4(c.handle, pages, k, v)
    for flip in (False, True):
        if flip:        # the same pages listed backwards
            pages.copy_(pages.flip(0).clone())
        k.zero_(), v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for out, w in zip((k, v), want):
            if flip:    # rows behind a page's count stay zero wherever the page is listed
                assert torch.equal(out.flip(1), w)
            else:
                assert torch.equal(out, w)
    empty = torch.zeros(2, 0, 64, 128, dtype=torch.bfloat16, device=DEV)
    spkv.paged_kv_unpack_q4(c.handle, i32(np.zeros(0)), empty, empty)
    assert spkv.get_device_error(c.handle) == (0, 0)


def test_slots_that_the_caller_fills():
    """Decode steps over a 4-bit slot pool: the missing pages' bytes copied to their victim slots and the slot list
    completed by the caller; bit for bit the attention over the whole pool."""
    B, Hk, Hq, npm, slots, stride = 2, 2, 8, 30, 9, 6
    U = B * Hk
    c = Cache(Hk, B, npm, [30 * 64 - 3, 25 * 64 + 1], seed=43)
    pool = torch.zeros(Hk, B * slots, 9216, dtype=torch.uint8, device=DEV)
    s = spkv.paged_kv_create_q4(pool, c.gk_d, c.gv_d, None, None, max_units=U)
    resident = torch.full((U, slots), -1, dtype=torch.int32, device=DEV)
    ts = torch.full((U, slots), -2 ** 31, dtype=torch.int32, device=DEV)
    rng = np.random.default_rng(4)
    brought = 0
    for t in range(5):
        sel, n = c.select(stride, rng, rng.integers(1, stride + 1, (B, Hk)))
        _, q = queries(B, Hq, seed=60 + t)
        sel_d, n_d = i32(sel), i32(n)
        missing, slot, victims = (torch.full((U, stride), -1, dtype=torch.int32, device=DEV) for _ in range(3))
        n_missing, hist = torch.zeros(U, dtype=torch.int32, device=DEV), torch.zeros(U, 64, dtype=torch.int32, device=DEV)
        spkv.resident_setdiff(s, resident, sel_d, n_d, missing, n_missing, slot)
        spkv.lru_bucket_update(s, resident, ts, slot, n_d.view(U), missing, n_missing, t, 1, victims, hist)
        for u in range(U):
            b, h, k = u // Hk, u % Hk, int(n_missing[u])
            brought += k
            to, page = victims[u, :k].long(), missing[u, :k].cpu().numpy()
            pool[h, b * slots + to] = c.pool[h, torch.from_numpy(c.pt[b, page].astype(np.int64)).to(DEV)]
            row = slot[u, :int(n[b, h])]
            row[row < 0] = victims[u, :k]
        out, lse = torch.zeros(B, Hq, 128, device=DEV), torch.zeros(B, Hq, device=DEV)
        spkv.sparse_decode_attn_slots(s, q, sel_d, slot.view(B, Hk, stride), n_d, slots, i32(c.L), out, lse)
        assert spkv.get_device_error(s) == (0, 0)
        want = c.attend(q, sel, n)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert brought > 0
