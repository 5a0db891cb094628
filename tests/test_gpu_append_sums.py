"""The rotating append's pooled sums where rows are skipped, in front of the new ones and behind them: bit for bit
the sums that the formula gives from the rows it keeps."""
import numpy as np
import pytest

import q4_ref as ref
import sparse_paged_kv_score_gb300 as spkv
from helpers import host_bits, i32
from test_gpu_append_rope import FORMATS, Batch

pytestmark = pytest.mark.gpu


def held_rows(b):
    """fp32 keys [Hk][n_phys][64][128] of the cache as `b` expects it, 4-bit: without the head's factor."""
    return ref.rows(b.blob, True).astype(np.float32) if b.q4 else ref.from_bf16_bits(b.kb)


def expected_sums(b, sums, counts, skip):
    """`sums` (fp32) with those formed again that the call touches: of a sub-block's rows in token order, those in
    front of the request's new ones, the new ones that are not skipped, and those behind that `counts` tells."""
    keys, out = held_rows(b), sums.copy()
    for r in range(b.B):
        first, last, end = b.first[r], b.first[r + 1], int(b.L[r])
        start = end - (last - first)
        for m0 in range(start // 16 * 16, end, 16) if last > first else ():
            p, t0 = int(b.pt[r, m0 // 64]), m0 % 64
            s = np.zeros((b.Hk, 128), np.float32)
            for m in range(m0, m0 + 16):
                i = last - (end - m)
                there = m < start or (i not in skip if m < end else m % 64 < counts[p])
                if there:
                    s += keys[:, p, m % 64]
            out[:, p, t0 // 16] = s * b.gk[:, None] if b.q4 else s
    return out


def check_all(b, q_out, sums, dtype16):
    assert np.array_equal(b.cnt_d.cpu().numpy(), b.cnt)
    assert np.array_equal(host_bits(b.q_out), q_out)
    if b.q4:
        assert np.array_equal(b.pool.cpu().numpy(), b.blob)
    else:
        assert np.array_equal(host_bits(b.kp), b.kb) and np.array_equal(host_bits(b.vp), b.vb)
    got = b.ksum.float().cpu().numpy()
    assert np.array_equal(got, ref.bf16(sums) if dtype16 else sums)


# rows of a request whose new rows begin at position 10 of its context: places 10, 15 | 16, 20, 31 | ..
@pytest.mark.parametrize("q4", FORMATS)
@pytest.mark.parametrize("sum16", [False, True])
@pytest.mark.parametrize("skip", [
    [0], [5], [6], [10], [21], [0, 5, 6, 21], list(range(6, 22)), list(range(0, 6)), [53, 54], [59], list(range(60)),
    [60, 63, 66], list(range(60, 68)), [2, 61, 62, 70]])
def test_rows_with_a_position_outside_the_table(q4, sum16, skip):
    """Left out of the cache, the counts, the queries and their sub-block's sums, at its first, a middle and its last
    place and where none of its new rows is left; the windows' sizes vary with the rows behind."""
    for more in (0, 700):
        b = Batch(q4, [10, 61, 3], [60, 8, 6 + more], 8, 2, seed=33 + len(skip), sum16=sum16)
        b.pos = np.arange(b.n, dtype=np.int32) % b.n_pos
        for k, i in enumerate(skip):
            b.pos[i] = (-1, b.n_pos, -2 ** 31, 2 ** 31 - 1)[k % 4]
        sums, counts = b.ksum.float().cpu().numpy(), b.cnt.copy()
        b.call()
        assert spkv.get_device_error(b.cache)[1] == spkv.DEVERR["POS"]
        q_out = b.expect(skip=set(skip))
        check_all(b, q_out, expected_sums(b, sums, counts, set(skip)), sum16)


@pytest.mark.parametrize("q4", FORMATS)
@pytest.mark.parametrize("axis", [0, 1, 2])
def test_one_axis_outside_the_table(q4, axis):
    """A row is left out for one of its axes; what the caches' rows behind the new ones hold is summed."""
    b = Batch(q4, [20, 40], [7, 30], 4, 2, axes=3, seed=35)
    for p, c in ((0, 30), (1, 50)):     # counts behind the new rows: places 27 .. 29; 6 .. 49 of the second page
        b.cnt[b.pt[p, p]] = c
    b.cnt_d.copy_(i32(b.cnt))
    b.pos[3, axis], b.pos[20, axis] = b.n_pos, -7
    sums, counts = b.ksum.float().cpu().numpy(), b.cnt.copy()
    b.call()
    assert spkv.get_device_error(b.cache)[1] == spkv.DEVERR["POS"]
    q_out = b.expect(skip={3, 20})
    check_all(b, q_out, expected_sums(b, sums, counts, {3, 20}), False)


@pytest.mark.parametrize("q4", FORMATS)
def test_rows_past_the_table_of_pages(q4):
    """A request longer than its page table: its rows in the table are appended, the others change nothing; one whose
    length is below its new rows likewise."""
    b = Batch(q4, [200, 50, 30], [90, 9, 20], 4, 2, seed=36)
    wide, b.pt = b.pt, np.ascontiguousarray(b.pt[:, :4])      # 256 positions: rows 56 .. 89 of request 0 are outside
    b.L[2] = 12                                               # rows 0 .. 7 of request 2 before its context
    skip = set(range(56, 90)) | set(range(99, 107))
    sums, counts = b.ksum.float().cpu().numpy(), b.cnt.copy()
    b.call()
    assert spkv.get_device_error(b.cache)[1] == spkv.DEVERR["PAGE_ID"] | spkv.DEVERR["POS"]
    b.pt = wide
    # what is before its context has no position either; what is past the table has one, and queries out
    x, first, L, n = b.x, b.first, b.L, b.n
    q_past = [ref.bf16_bits(ref.rotate(x[i, :4], b.tab[[200 + i], :64], b.tab[[200 + i], 64:])) for i in range(56, 90)]
    keep = [i for i in range(n) if i not in skip]
    b.x, b.first, b.L, b.n = x[keep], np.array([0, 56, 65, 77], np.int32), np.array([256, 59, 12], np.int32), 77
    q_kept = b.expect()
    sums = expected_sums(b, sums, counts, set())
    b.x, b.first, b.L, b.n = x, first, L, n
    q_out = np.full((n, 4, 128), 0x4040, np.uint16)
    q_out[keep] = q_kept
    q_out[56:90] = q_past
    check_all(b, q_out, sums, False)


@pytest.mark.parametrize("q4", FORMATS)
def test_a_page_outside_the_pool(q4):
    """Its rows change no row, sum or count; their queries come out."""
    b = Batch(q4, [60, 5], [40, 3], 4, 2, seed=37)
    good = int(b.pt[0, 1])
    for bad in (b.n_phys, -1, 2 ** 31 - 1, -2 ** 31):
        b.pt[0, 1] = bad
        sums, counts = b.ksum.float().cpu().numpy(), b.cnt.copy()
        b.call()
        assert spkv.get_device_error(b.cache)[1] == spkv.DEVERR["PHYS"]
        skip = set(range(4, 40))
        x, first, L, n = b.x, b.first, b.L, b.n
        keep = [0, 1, 2, 3, 40, 41, 42]
        b.x, b.first, b.L, b.n = x[keep], np.array([0, 4, 7], np.int32), np.array([64, 8], np.int32), 7
        q_kept = b.expect()
        sums = expected_sums(b, sums, counts, set())
        b.x, b.first, b.L, b.n = x, first, L, n
        q_out = np.zeros((n, 4, 128), np.uint16)
        q_out[keep] = q_kept
        for i in skip:
            q_out[i] = ref.bf16_bits(ref.rotate(x[i, :4], b.tab[[60 + i], :64], b.tab[[60 + i], 64:]))
        check_all(b, q_out, sums, False)
    b.pt[0, 1] = good
    b.call()
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.check(b.expect())


@pytest.mark.parametrize("q4", FORMATS)
def test_keys_rotated_without_queries(q4):
    """Keys and values alone: a cache filled where no query is asked."""
    b = Batch(q4, [9, 0], [40, 21], 8, 2, axes=2, seed=38, fused=True)
    b.call(q=None, q_out=None)
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.expect()
    b.check(np.full((b.n, 8, 128), 0x4040, np.uint16))
