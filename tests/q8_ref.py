"""Plain numpy forms of the 8-bit cache, for the tests: its bytes by the format's definition, one token and dim at a time,
and the attention in 64 bits from the values that those bytes stand for."""
from __future__ import annotations

import numpy as np

PAGE, D, BLOB, SUB = 64, 128, 16416, 16


def places():
    """Byte of token t, dim d [64][128]: keys, values."""
    t, d = np.arange(64)[:, None], np.arange(128)[None]
    kc = 1024 * (t // 8) + 512 * ((d // 16) % 2) + 64 * (t % 8) + 16 * (d // 32) + d % 16
    vc = 8192 + 1024 * (t // 8) + 512 * ((d // 8) % 2) + 64 * (d // 16) + 16 * ((t % 8) // 2) + 2 * (d % 8) + t % 2
    return kc, vc


KC, VC = places()
NAN_BITS = 0x7FFFFFFF


def scales(blob, keys):
    """fp32 scales [..., 4] of page-heads [..., 16416]."""
    at = 16384 if keys else 16400
    return np.ascontiguousarray(blob[..., at:at + 16]).view(np.float32)


def set_scale(blob, keys, j, s):
    at = (16384 if keys else 16400) + 4 * j
    blob[..., at:at + 4] = np.array([s], np.float32).view(np.uint8)


def scale_of(a):
    """The scale of a sub-block whose largest magnitude is a (fp32)."""
    a = np.float32(a)
    if a == 0:
        return np.float32(0)
    if not np.isfinite(a):
        return np.array(NAN_BITS, np.uint32).view(np.float32)[()]
    return np.float32(2.0 ** max(int(np.frexp(np.float64(a))[1]) - 7, -126))


def codes(x, s):
    """floor(x / s) as bytes."""
    with np.errstate(all="ignore"):
        c = np.floor(np.asarray(x, np.float64) / np.float64(s)) if np.isfinite(s) and s > 0 else np.zeros(np.shape(x))
    return (c + 128).astype(np.uint8)


def put(blob, j, new, held, keys):
    """Rows `new` ({token of the sub-block: fp32 [128]}) into sub-block j of the page-head bytes `blob`, which holds the
    tokens `held` of it beside them."""
    at = KC if keys else VC
    was = scales(blob, keys)[j] if held else np.float32(0)
    need = np.float32(0)
    for x in new.values():
        a = np.abs(np.asarray(x, np.float32))
        need = np.maximum(need, np.float32(np.inf) if np.isnan(a).any() else a.max())
    if not new:
        return
    is_ = scale_of(need)
    if np.isnan(was) or was > is_:
        is_ = was
    if not np.isnan(is_):
        for t in held:
            c = blob[at[16 * j + t]].astype(np.float64) - 128
            blob[at[16 * j + t]] = (np.floor(c * (np.float64(was) / np.float64(is_))) if is_ > 0 else c) + 128
    for t, x in new.items():
        blob[at[16 * j + t]] = codes(x, is_)
    set_scale(blob, keys, j, is_)


def pool_of(k, v):
    """Page-head bytes [Hk][n][16416] of rows fp32 [Hk][n][64][128]."""
    Hk, n = k.shape[:2]
    out = np.zeros((Hk, n, BLOB), np.uint8)
    for x, at, start in ((k, KC, 16384), (v, VC, 16400)):
        x = np.asarray(x, np.float64).reshape(Hk, n, 4, SUB, D)
        a = np.abs(x).max((3, 4))
        s = np.where(a > 0, 2.0 ** np.maximum(np.frexp(a)[1] - 7, -126), 0)
        c = np.floor(np.divide(x, s[..., None, None], out=np.zeros_like(x), where=s[..., None, None] > 0))
        out[:, :, at] = (c + 128).reshape(Hk, n, PAGE, D)
        out[:, :, start:start + 16] = np.ascontiguousarray(s.astype(np.float32)).view(np.uint8)
    return out


def rows(blob, keys):
    """Values (exact, in 64 bits) of page-heads [..., 16416]: [..., 64, 128]."""
    c = blob[..., KC if keys else VC].astype(np.float64) - 128
    return (c + 0.5) * np.repeat(scales(blob, keys).astype(np.float64), SUB, -1)[..., None]


def error_bounds(qrow, k, ks, v, vs, tiles):
    """Bounds on the fp32 kernel's error of scores (absolute) and of weights (relative), and the values' largest magnitude.

    Products of a query dim (8 bits) and a code (8 bits) are exact.  A score's error is that of its fp32 sum of 128 terms
    |q_i c_i| (a step of 2^-23 where an addition truncates), of the sum of q (the half of each code), and of a few scalings:
    (128 + 16) 2^-23 s sum |q_i| (|c_i| + 1/2) / sqrt(128), where |c| s <= |k| + s / 2; then the reference is taken off in two
    roundings of numbers as large as the scores: 2^-22 (1.45 |x| + 16) in log2 units.  A weight is off by that (relative),
    by its split and exp2, 2^-19 in all, and by the sums over the tiles, 2^-24 each."""
    big = ((np.abs(k) + ks[:, None]) @ np.abs(qrow)) / np.sqrt(D)
    dx = 144 * 2.0 ** -23 * big.max() + 2.0 ** -22 * (big.max() + 16)
    return dx, dx + 2.0 ** -19 + 4 * tiles * 2.0 ** -24, (np.abs(v) + vs[:, None]).max()


def attention(q, blob, page_table, sel, n_sel, seq_len):
    """64-bit (out [B][Hq][128], lse [B][Hq], bound on the fp32 kernel's output error, bound on its lse error)."""
    B, Hq = q.shape[:2]
    Hk = blob.shape[0]
    G = Hq // Hk
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    e_out, e_lse = np.zeros((B, Hq)), np.zeros((B, Hq))
    for b in range(B):
        for h in range(Hk):
            lp = [int(x) for x in sel[b, h, :n_sel[b, h]]]
            if not lp:
                continue
            ph = [int(page_table[b, x]) for x in lp]
            n = [min(64, int(seq_len[b]) - 64 * x) for x in lp]
            k, v = (np.concatenate([rows(blob[h, p], s)[:m] for p, m in zip(ph, n)]) for s in (True, False))
            ks, vs = (np.concatenate([np.repeat(scales(blob[h, p], s).astype(np.float64), SUB)[:m] for p, m in zip(ph, n)])
                      for s in (True, False))
            for g in range(h * G, (h + 1) * G):
                qr = q[b, g].astype(np.float64)
                with np.errstate(invalid="ignore"):
                    x = k @ qr / np.sqrt(D)
                    dx, dw, vmax = error_bounds(qr, k, ks, v, vs, 4 * len(lp))
                    m = x.max()
                    p = np.exp(x - m)
                    out[b, g] = p @ v / p.sum()
                    lse[b, g] = m + np.log(p.sum())
                    e_out[b, g] = 2 * dw * vmax
                    e_lse[b, g] = dw + 2.0 ** -19 * (1 + abs(lse[b, g]))
    return out, lse, e_out, e_lse
