"""Plain numpy forms of the 4-bit cache and of the rotating append, for the tests.

The format's arithmetic is written twice: in fp32, operation by operation as spkv.h gives it (its results
are the bytes that the cache holds), and the attention in 64 bits from the values that those bytes stand for."""
from __future__ import annotations

import numpy as np

PAGE, D, BLOB = 64, 128, 9216
LEVELS = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float64)


def bf16(x):
    """fp32 rounded to bf16 (nearest even), as fp32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return np.where(np.isnan(x), np.float32(np.nan), r.view(np.float32)).astype(np.float32)


def bf16_bits(x):
    return (bf16(x).view(np.uint32) >> 16).astype(np.uint16)


def bf16_bits_special(x):
    """bf16_bits that keeps infinities and NaN."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return np.where(np.isfinite(x), bf16_bits(np.where(np.isfinite(x), x, 0)), (b >> 16) | np.where(np.isnan(x), 0x40, 0)).astype(np.uint16)


def from_bf16_bits(u):
    return (np.asarray(u, np.uint16).astype(np.uint32) << 16).view(np.float32)


def e4m3_values():
    v = np.empty(256, np.float64)
    for i in range(256):
        e, m = (i >> 3) & 15, i & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[i] = -x if i & 128 else x
    v[127] = v[255] = np.nan
    return v


E4M3 = e4m3_values()
FINITE = E4M3[:127]


def e4m3_byte(x):
    """Nearest e4m3 byte (ties to even, saturating) of fp32 x >= 0; NaN gives 127."""
    x = np.asarray(x, np.float64)
    y = np.where(np.isnan(x), 0, np.minimum(x, 448))
    hi = np.clip(np.searchsorted(FINITE, y), 1, 126)
    lo = hi - 1
    dl, dh = y - FINITE[lo], FINITE[hi] - y
    pick = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(x), 127, pick).astype(np.uint8)


def encode(x, g):
    """Rows fp32 [..., 128] and g fp32 [...]: codes uint8 [..., 128], scale bytes uint8 [..., 8]."""
    x = np.asarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], 8, 16)
    g = np.asarray(g, np.float32)[..., None]
    with np.errstate(all="ignore"):
        a = np.abs(b).max(-1)                       # a NaN is the largest
        a = np.where(np.isnan(b).any(-1), np.float32(np.nan), a)
        s = e4m3_byte(a / (np.float32(6) * g))
        d = (E4M3[s].astype(np.float32) * g)[..., None]
        y = np.where(d > 0, b / d, np.float32(0)).astype(np.float32)
    m = np.minimum(np.abs(y), np.float32(6)).astype(np.float64)
    c = np.zeros(m.shape, np.uint8)
    for edge, even in ((.25, 0), (.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5, 0)):
        c += (m >= edge) if even else (m > edge)
    c = np.where(np.isnan(y), 0, c + 8 * np.signbit(y)).astype(np.uint8)
    return c.reshape(x.shape), s


def places():
    """Byte of each token's code bytes [64][64] and scales [64][8], keys then values."""
    t, b, k = np.arange(64)[:, None], np.arange(64)[None], np.arange(8)[None]
    kc = 64 * t + b
    vc = 4096 + 512 * (t // 8) + 64 * (b // 8) + 8 * (t % 8) + b % 8
    ks = 8192 + 16 * (4 * (t % 8) + k // 2) + 4 * (t // 16) + 2 * ((t // 8) % 2) + k % 2
    vs = 8704 + 16 * (4 * k + (t % 8) // 2) + 4 * (t // 16) + 2 * ((t // 8) % 2) + t % 2
    return kc, vc, ks, vs


KC, VC, KS, VS = places()


def put(blob, t, row, g, keys):
    """Row fp32 [128] into token t of the page-head bytes `blob`."""
    c, s = encode(row, g)
    blob[(KC if keys else VC)[t]] = c[0::2] | (c[1::2] << 4)
    blob[(KS if keys else VS)[t]] = s


def pool_of(k, v, gk, gv):
    """Page-head bytes [Hk][n][9216] of rows fp32 [Hk][n][64][128]."""
    Hk, n = k.shape[:2]
    out = np.empty((Hk, n, BLOB), np.uint8)
    for x, g, ci, si in ((k, gk, KC, KS), (v, gv, VC, VS)):
        c, s = encode(x, np.broadcast_to(np.asarray(g, np.float32)[:, None, None], x.shape[:3]))
        out[:, :, ci] = c[..., 0::2] | (c[..., 1::2] << 4)
        out[:, :, si] = s
    return out


def rows(blob, keys):
    """code * scale (exact, in 64 bits) of page-heads [..., 9216]: [..., 64, 128]."""
    b = blob[..., KC if keys else VC]
    c = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], 128)
    v = np.where(c & 8, -1.0, 1.0) * LEVELS[c & 7]
    s = E4M3[blob[..., KS if keys else VS]]
    return (v.reshape(*v.shape[:-1], 8, 16) * s[..., None]).reshape(v.shape)


def rotate(x, c, s):
    """fp32 rows [..., 128] by fp32 cos and sin [..., 64], products and sums rounded one by one."""
    lo, hi = np.float32(x[..., :64]), np.float32(x[..., 64:])
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], -1).astype(np.float32)


def table(n_pos, theta=500000.0):
    a = np.arange(n_pos, dtype=np.float64)[:, None] * theta ** (-np.arange(64) / 64)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def attention(q, blob, gk, gv, page_table, sel, n_sel, seq_len):
    """64-bit (out [B][Hq][128], lse [B][Hq], bound on the fp32 kernel's output error, bound on its lse error).

    The bounds: products of at most 8-bit and 6-bit significands are exact, so a score's error is that of
    its fp32 sum of 128 terms and of a few scalings: (128 + 8) 2^-23 sum |q_i k_i| / sqrt(128) (a step of
    2^-23 where an addition truncates).  A weight is off by that (relative) and by its split and exp2, 2^-19
    in all, and so are the weighted mean (twice: weights and their sum) and the log of the sum."""
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
            k = np.concatenate([rows(blob[h, p], True)[:min(64, seq_len[b] - 64 * x)] for p, x in zip(ph, lp)]) * float(gk[h])
            v = np.concatenate([rows(blob[h, p], False)[:min(64, seq_len[b] - 64 * x)] for p, x in zip(ph, lp)]) * float(gv[h])
            for g in range(h * G, (h + 1) * G):
                with np.errstate(invalid="ignore"):
                    x = k @ q[b, g].astype(np.float64) / np.sqrt(D)
                    dx = 136 * 2.0 ** -23 * (np.abs(k) @ np.abs(q[b, g].astype(np.float64))).max() / np.sqrt(D)
                    m = x.max()
                    p = np.exp(x - m)
                    out[b, g] = p @ v / p.sum()
                    lse[b, g] = m + np.log(p.sum())
                    e_out[b, g] = 2 * (dx + 2.0 ** -19) * np.abs(v).max()
                    e_lse[b, g] = dx + 2.0 ** -19 * (1 + abs(lse[b, g]))
    return out, lse, e_out, e_lse
