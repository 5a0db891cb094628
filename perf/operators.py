"""Cases of the 4-bit paged KV cache and of the append that rotates, each in a plain form of elementary torch
operations and through this library's entry points.

A page-head (one page of 64 tokens of one kv head) of the 4-bit pool is 9216 bytes: 4096 of key codes, 4096 of
value codes, 512 of key scales, 512 of value scales.  A value is code * scale * g with a 4-bit code
(0, .5, 1, 1.5, 2, 3, 4, 6 and a sign), one e4m3 scale for 16 dims of a token and one fp32 g for a kv head.
"""
import math

import torch

own = False

DEV = torch.device("cuda" if torch.cuda.is_available() else "cpu")
D, PAGE, SUB, BLOB = 128, 64, 16, 9216
THETA = 500000.0

# Places inside a page-head: token t, byte b of a row's 64 code bytes (dims 2b, 2b + 1), block k of 16 dims.
_t, _b, _k = torch.arange(64)[:, None], torch.arange(64)[None, :], torch.arange(8)[None, :]
_r, _tg = _t % 16, _t // 16
K_CODE = (_t * 64 + _b).to(DEV)
V_CODE = (4096 + (_t // 8) * 512 + (_b // 8) * 64 + (_t % 8) * 8 + _b % 8).to(DEV)
K_SCALE = (8192 + (4 * (_r % 8) + _k // 2) * 16 + _tg * 4 + (_r // 8) * 2 + _k % 2).to(DEV)
V_SCALE = (8704 + (4 * _k + (_r % 8) // 2) * 16 + _tg * 4 + (_r // 8) * 2 + _r % 2).to(DEV)
LEVELS = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)


def listed():
    return [
        # the new token of every request of a decode batch: latency
        dict(name="append decode", kind="append", B=32, rows=32, Hq=32, Hk=8, axes=1, fused=False, sum16=False, ctx=32768),
        # prompts of several lengths, queries, keys and values as slices of one projection's output
        dict(name="append prompts", kind="append", B=6, rows=8192, Hq=32, Hk=8, axes=1, fused=True, sum16=True, ctx=4096),
        # a video's tokens with positions of time, height and width
        dict(name="append video", kind="append", B=2, rows=2501, Hq=40, Hk=8, axes=3, fused=True, sum16=True, ctx=0),
        # a chunk of a prompt into the 4-bit cache, and its pages back as bf16 for the prefill: a short question
        dict(name="chunk short", kind="chunk", B=1, rows=77, Hq=8, Hk=2, axes=1, fused=False, sum16=True, ctx=1000),
        # the same for a batch of prompts
        dict(name="chunk prompts", kind="chunk", B=4, rows=6000, Hq=32, Hk=8, axes=1, fused=True, sum16=True, ctx=2048),
        # one context's pages, and a batch's, unpacked for a bf16 kernel
        dict(name="unpack context", kind="unpack", pages=17, Hk=2),
        dict(name="unpack batch", kind="unpack", pages=2048, Hk=8),
        # decode attention over selected pages of the 4-bit cache: one request
        dict(name="attend tiny", kind="attend", B=1, Hq=8, Hk=2, sel=17, ctx=4096, ragged=False),
        # a decode batch
        dict(name="attend batch", kind="attend", B=32, Hq=32, Hk=8, sel=65, ctx=32768, ragged=False),
        # few requests with long contexts
        dict(name="attend long", kind="attend", B=8, Hq=40, Hk=8, sel=129, ctx=262144, ragged=False),
        # one kv head for all query heads, selections of every length, empty ones too
        dict(name="attend ragged", kind="attend", B=61, Hq=16, Hk=1, sel=129, ctx=10000, ragged=True),
        # a decode step: the new token rotated and appended, then attended with the selected pages
        dict(name="step batch", kind="step", B=16, Hq=32, Hk=8, sel=65, ctx=65536, ragged=False),
    ]


HEADS = [(8, 2), (32, 8), (40, 8), (16, 1), (6, 6), (28, 4), (22, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "append", "chunk", "unpack", "attend", "attend", "step"])
    Hq, Hk = rng.choice(HEADS)
    if kind in ("append", "chunk"):
        decode = rng.random() < 0.4
        rows = _log(rng, 1, 200) if decode else _log(rng, 20, 5000)
        B = rows if decode else min(rows, _log(rng, 1, 12))
        return dict(kind=kind, B=B, rows=rows, Hq=Hq, Hk=Hk, axes=rng.choice([1, 1, 2, 3, 4]), fused=rng.random() < 0.5,
                    sum16=True, ctx=rng.randint(0, 30000) if decode else rng.randint(0, 3000))
    if kind == "unpack":
        return dict(kind=kind, pages=_log(rng, 1, 12000 // Hk), Hk=Hk)
    sel = _log(rng, 1, 140)
    B = _log(rng, 1, max(1, min(64, 14000 // (Hk * sel))))
    return dict(kind=kind, B=B, Hq=Hq, Hk=Hk, sel=sel, ctx=rng.randint(64 * sel + 64, 64 * sel + 40000),
                ragged=kind == "attend" and rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------- inputs


def _quantise(x, g):
    """fp32 rows [..., 128] and g (broadcasting to [..., 1]): code bytes [..., 64], scale bytes [..., 8]."""
    y = x.unflatten(-1, (8, 16))
    g = g.unsqueeze(-1)
    s = (y.abs().amax(-1, keepdim=True) / (6 * g)).clamp(max=448).to(torch.float8_e4m3fn)
    d = s.float() * g
    y = torch.where(d > 0, y / d, 0.)
    m = y.abs()
    c = (m > .25).to(torch.uint8)
    for edge, even in ((.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5., False)):
        c += (m >= edge) if even else (m > edge)
    c = (c + 8 * (y < 0).to(torch.uint8)).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.squeeze(-1).view(torch.uint8)


def _pool4(gen, Hk, n_phys, gk, gv):
    """A 4-bit pool of N(0, 1) rows, one key row in a hundred four times as large."""
    pool = torch.empty(Hk, n_phys, BLOB, dtype=torch.uint8, device=DEV)
    for h in range(Hk):
        for x0 in range(0, n_phys, 2048):
            n = min(2048, n_phys - x0)
            k = torch.randn(n, PAGE, D, generator=gen, device=DEV)
            k *= 1 + 3 * (torch.rand(n, PAGE, 1, generator=gen, device=DEV) < 0.01)
            v = torch.randn(n, PAGE, D, generator=gen, device=DEV)
            for x, g, ci, si in ((k, gk, K_CODE, K_SCALE), (v, gv, V_CODE, V_SCALE)):
                c, s = _quantise(x.bfloat16().float(), g[h].reshape(1, 1, 1))
                pool[h, x0:x0 + n, ci.flatten()] = c.flatten(1)
                pool[h, x0:x0 + n, si.flatten()] = s.flatten(1)
    return pool


def _table(n_pos):
    """cos (64 pairs) and sin (64 pairs) of every position, angles in 64 bits."""
    f = THETA ** (-torch.arange(64, dtype=torch.float64, device=DEV) / 64)
    a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _scales(gen, Hk):
    return (20 / 2688) * (1 + 0.2 * torch.rand(Hk, generator=gen, device=DEV))


def _sums(state):
    """Pooled sums of every page from the pool, by the page counts."""
    k = _page_keys(state, slice(None))
    live = torch.arange(PAGE, device=DEV) < state["page_cnt"][:, None]
    s = (k * live[None, :, :, None]).unflatten(2, (4, SUB)).sum(3)
    state["ksum"].copy_(s.to(state["ksum"].dtype))


def _int(x):
    return torch.as_tensor(x, device=DEV).to(torch.int32)


def _prepare_append(case, gen):
    B, n, Hq, Hk, ctx, axes = (case[k] for k in ("B", "rows", "Hq", "Hk", "ctx", "axes"))
    cpu = torch.Generator().manual_seed(int(torch.randint(1 << 30, (1,), generator=gen, device=DEV)))
    if B == n:
        lens = torch.ones(B, dtype=torch.int64)
    else:   # ragged prompts
        cut = torch.sort(torch.randint(0, n + 1, (B - 1,), generator=cpu)).values
        lens = torch.diff(cut, prepend=torch.zeros(1, dtype=torch.int64), append=torch.tensor([n]))
    past = torch.randint(0, ctx + 1, (B,), generator=cpu)
    first_page, last_page = past // PAGE, (past + lens - 1).clamp(min=0) // PAGE
    np_max = int(last_page.max()) + 1
    touched = [(b, p) for b in range(B) if lens[b] > 0 for p in range(int(first_page[b]), int(last_page[b]) + 1)]
    # as many pages whatever the lengths: those that the append does not touch are full
    n_pages = B if B == n else n // PAGE + 2 * B
    n_phys = n_pages + max(2, n_pages // 8)
    perm = torch.randperm(n_phys, generator=cpu)
    pt = perm[-1].repeat(B, np_max)
    cnt = torch.full((n_phys,), PAGE, dtype=torch.int64)
    for i, (b, p) in enumerate(touched):
        pt[b, p] = perm[i]
        cnt[perm[i]] = max(0, int(past[b]) - PAGE * p)
    s = dict(row_first=_int(torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])), seq_len=_int(past + lens),
             page_table=_int(pt), page_cnt=_int(cnt), pages=_int(perm[:n_pages]))
    width = (Hq + 2 * Hk) * D
    if case["fused"]:   # one projection's output, sliced
        qkv = torch.randn(n, width, generator=gen, device=DEV).bfloat16()
        q, k, v = qkv.split([Hq * D, Hk * D, Hk * D], 1)
    else:
        q, k, v = (torch.randn(n, h * D, generator=gen, device=DEV).bfloat16() for h in (Hq, Hk, Hk))
    s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in (q, k, v))
    s["q_out"] = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device=DEV)
    n_pos = int((past + lens).max()) + 1
    s["pos"], s["pair_axis"] = None, None
    if axes > 1:        # time, height, width of a frame's patches, placed after the context
        i = torch.arange(n, device=DEV)
        p = torch.stack([i // 400, i // 20 % 20, i % 20, i % 7], 1)[:, :axes] + ctx
        s["pos"] = _int(p).contiguous()
        cuts = [0, 16, 40, 52, 64] if axes == 4 else [0, 16, 40, 64] if axes == 3 else [0, 32, 64]
        s["pair_axis"] = [sum(j >= c for c in cuts[1:-1]) for j in range(64)]
        n_pos = int(p.max()) + 1
    s["cos_sin"], s["axis_of"] = _table(n_pos), torch.tensor(s["pair_axis"] or [0] * 64, device=DEV)
    return s, n_phys


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    kind, Hk = case["kind"], case["Hk"]
    if kind in ("append", "chunk"):
        s, n_phys = _prepare_append(case, gen)
        s["ksum"] = torch.zeros(Hk, n_phys, 4, D, dtype=torch.bfloat16 if case["sum16"] else torch.float32, device=DEV)
    elif kind == "unpack":
        n = case["pages"]
        n_phys = n + max(1, n // 8)
        cnt = torch.where(torch.rand(n_phys, generator=gen, device=DEV) < 0.9, PAGE,
                          torch.randint(0, PAGE + 1, (n_phys,), generator=gen, device=DEV))
        s = dict(page_cnt=_int(cnt), pages=_int(torch.randperm(n_phys, generator=gen, device=DEV)[:n]), ksum=None)
    else:
        s, n_phys = _prepare_attend(case, gen)
    s["kind"] = kind
    if kind == "append":
        s["k_pool"], s["v_pool"] = (torch.randn(Hk, n_phys, PAGE, D, generator=gen, device=DEV).bfloat16() for _ in range(2))
    else:
        s["k_scale"], s["v_scale"] = _scales(gen, Hk), _scales(gen, Hk)
        s["pool"] = _pool4(gen, Hk, n_phys, s["k_scale"], s["v_scale"])
    if kind in ("chunk", "unpack"):
        shape = (Hk, s["pages"].numel(), PAGE, D)
        s["k_out"], s["v_out"] = (torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    if s["ksum"] is not None:
        _sums(s)
    if own:
        import sparse_paged_kv_score_gb300 as spkv
        units = case.get("B", 1) * Hk
        cnt, ksum = (s["page_cnt"], s["ksum"]) if s["ksum"] is not None else (s["page_cnt"], None)
        if kind == "append":
            s["cache"] = spkv.paged_kv_create(s["k_pool"], s["v_pool"], ksum, cnt, max_units=min(4096, units))
        else:
            s["cache"] = spkv.paged_kv_create_q4(s["pool"], s["k_scale"], s["v_scale"], ksum, cnt,
                                                 max_units=min(4096, units))
    return s


def _prepare_attend(case, gen):
    B, Hq, Hk, S, ctx = (case[k] for k in ("B", "Hq", "Hk", "sel", "ctx"))
    L = torch.randint(max(1, ctx - ctx // 8), ctx + 1, (B,), generator=gen, device=DEV)
    local = (L - 1) // PAGE
    np_max = (ctx + PAGE - 1) // PAGE
    held = min(np_max - np_max // 8, S + S // 2)        # logical pages of a request that the pool holds
    # `held` logical pages of each request: its local page, the others drawn from the pages before it
    r = torch.rand(B, np_max, generator=gen, device=DEV)
    r = torch.where(torch.arange(np_max, device=DEV) < local[:, None], r, 2.)
    r.scatter_(1, local[:, None], -1.)
    held = min(held, int(local.min()) + 1)
    logical = r.argsort(1)[:, :held]                    # [B][held], the local page first
    n_phys = B * held + 1
    pt = torch.full((B, np_max), -1, dtype=torch.int64, device=DEV)
    pt.scatter_(1, logical, torch.randperm(n_phys, generator=gen, device=DEV)[:B * held].reshape(B, held))
    cnt = torch.full((n_phys,), PAGE, dtype=torch.int64, device=DEV)
    step = case["kind"] == "step"
    cnt[pt.gather(1, local[:, None]).flatten()] = L - PAGE * local - (1 if step else 0)
    n = min(S, held)
    w = torch.rand(B, Hk, held, generator=gen, device=DEV)
    w[:, :, 0] = -1
    pick = logical[:, None].expand(B, Hk, held).gather(2, w.argsort(2)[:, :, :n])
    n_sel = torch.full((B, Hk), n, dtype=torch.int64, device=DEV)
    if case["ragged"]:
        n_sel = torch.randint(0, n + 1, (B, Hk), generator=gen, device=DEV)
    pick = torch.where(torch.arange(n, device=DEV) < n_sel[..., None], pick, np_max)
    pick = pick.sort(2).values
    sel = torch.full((B, Hk, S), -1, dtype=torch.int64, device=DEV)
    sel[:, :, :n] = torch.where(pick < np_max, pick, -1)
    q = torch.randn(B, Hq, D, generator=gen, device=DEV).bfloat16()
    s = dict(seq_len=_int(L), page_table=_int(pt), page_cnt=_int(cnt), sel=_int(sel), n_sel=_int(n_sel), q=q, ksum=None,
             out=torch.zeros(B, Hq, D, device=DEV), lse=torch.zeros(B, Hq, device=DEV))
    if step:
        s["ksum"] = torch.zeros(Hk, n_phys, 4, D, dtype=torch.bfloat16, device=DEV)
        s["k"], s["v"] = (torch.randn(B, Hk, D, generator=gen, device=DEV).bfloat16() for _ in range(2))
        s["row_first"], s["pos"], s["pair_axis"], s["q_out"] = None, None, None, torch.zeros_like(q)
        s["cos_sin"], s["axis_of"] = _table(int(L.max()) + 1), torch.zeros(64, dtype=torch.int64, device=DEV)
        s["pages"] = _int(pt.gather(1, local[:, None]).flatten())
    return s, n_phys


# ---------------------------------------------------------------------------------------------- plain forms


def _values(blob, code_at, scale_at, g):
    """Rows [..., 64, 128] of page-heads [..., 9216]; g broadcasts to them."""
    b = blob[..., code_at]
    c = LEVELS[torch.stack([b & 15, b >> 4], -1).flatten(-2).int()]
    s = blob[..., scale_at].view(torch.float8_e4m3fn).float()
    return (c.unflatten(-1, (8, 16)) * s[..., None]).flatten(-2) * g


def _page_keys(s, pages):
    """fp32 keys [Hk][pages][64][128] that the pool holds."""
    if "pool" in s:
        return _values(s["pool"][:, pages], K_CODE, K_SCALE, s["k_scale"][:, None, None, None])
    return s["k_pool"][:, pages].float()


def _rotate(x, cs):
    """Rows [n][H][128] by the cos and sin [n][64] of their positions (pairs j, j + 64)."""
    lo, hi = x.float().split(64, -1)
    c, sn = (y[:, None] for y in cs)
    return torch.cat([lo * c - hi * sn, hi * c + lo * sn], -1)


def _plain_append(s):
    n = s["k"].shape[0]
    B = s["seq_len"].shape[0]
    first = torch.arange(B + 1, device=DEV) if s["row_first"] is None else s["row_first"].long()
    lens = first.diff()
    b = torch.repeat_interleave(torch.arange(B, device=DEV), lens, output_size=n)
    at = s["seq_len"].long()[b] - lens[b] + torch.arange(n, device=DEV) - first[b]
    page, tok = s["page_table"].long()[b, at // PAGE], at % PAGE
    pos = at[:, None] if s["pos"] is None else s["pos"].long()
    pos, j = pos[:, s["axis_of"]], torch.arange(64, device=DEV)
    cs = s["cos_sin"][pos, j], s["cos_sin"][pos, j + 64]
    s["q_out"].copy_(_rotate(s["q"], cs))
    k, v = _rotate(s["k"], cs).transpose(0, 1), s["v"].transpose(0, 1)
    if "pool" in s:
        for x, g, ci, si in ((k, s["k_scale"], K_CODE, K_SCALE), (v.float(), s["v_scale"], V_CODE, V_SCALE)):
            c, sc = _quantise(x, g[:, None, None])
            s["pool"][:, page[:, None], ci[tok]] = c
            s["pool"][:, page[:, None], si[tok]] = sc
    else:
        s["k_pool"][:, page, tok] = k.bfloat16()
        s["v_pool"][:, page, tok] = v
    s["page_cnt"].scatter_reduce_(0, page, (tok + 1).int(), "amax")
    pages = s["pages"].long()
    keys = _page_keys(s, pages)
    live = torch.arange(PAGE, device=DEV) < s["page_cnt"][pages][:, None]
    sums = (keys * live[None, :, :, None]).unflatten(2, (4, SUB)).sum(3)
    s["ksum"][:, pages] = sums.to(s["ksum"].dtype)


def _plain_unpack(s):
    pages = s["pages"].long()
    live = (torch.arange(PAGE, device=DEV) < s["page_cnt"][pages][:, None])[None, :, :, None]
    blob = s["pool"][:, pages]
    for out, g, ci, si in ((s["k_out"], s["k_scale"], K_CODE, K_SCALE), (s["v_out"], s["v_scale"], V_CODE, V_SCALE)):
        out.copy_(torch.where(live, _values(blob, ci, si, g[:, None, None, None]).bfloat16(), out))


def _plain_attend(s, q):
    B, Hq = q.shape[:2]
    sel = s["sel"].long()
    Hk, S = sel.shape[1:]
    taken = torch.arange(S, device=DEV) < s["n_sel"][..., None]
    sel = torch.where(taken, sel, 0)
    page = s["page_table"].long()[torch.arange(B, device=DEV)[:, None, None], sel].clamp(min=0)
    h = torch.arange(Hk, device=DEV)[None, :, None]
    blob = s["pool"][h, page]
    k = _values(blob, K_CODE, K_SCALE, s["k_scale"][:, None, None, None]).flatten(2, 3)
    at = sel[..., None] * PAGE + torch.arange(PAGE, device=DEV)
    live = (taken[..., None] & (at < s["seq_len"][:, None, None, None])).flatten(2)[:, :, None]
    x = (q.float().unflatten(1, (Hk, -1)) @ k.transpose(2, 3)) / math.sqrt(D)
    del k
    v = _values(blob, V_CODE, V_SCALE, s["v_scale"][:, None, None, None]).flatten(2, 3)
    x = torch.where(live, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.where(live, (x - m).exp(), 0.)
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, (p @ v) / l, 0.)
    s["out"].copy_(o.flatten(1, 2))
    s["lse"].copy_((m + l.log()).flatten(1) if S else torch.full_like(s["lse"], -math.inf))


def run(state):
    s, kind = state, state["kind"]
    if own:
        import sparse_paged_kv_score_gb300 as spkv
        if kind in ("append", "chunk", "step"):
            spkv.paged_kv_append_rope(s["cache"], s["k"], s["v"], s["seq_len"], s["page_table"], row_first=s["row_first"],
                                      q=s["q"], q_out=s["q_out"], cos_sin=s["cos_sin"], pos=s["pos"], pair_axis=s["pair_axis"])
        if kind in ("chunk", "unpack"):
            spkv.paged_kv_unpack_q4(s["cache"], s["pages"], s["k_out"], s["v_out"])
        if kind in ("attend", "step"):
            spkv.sparse_decode_attn(s["cache"], s["q"] if kind == "attend" else s["q_out"], s["page_table"], s["sel"],
                                    s["n_sel"], s["seq_len"], s["out"], s["lse"])
    else:
        if kind in ("append", "chunk", "step"):
            _plain_append(s)
        if kind in ("chunk", "unpack"):
            _plain_unpack(s)
        if kind in ("attend", "step"):
            _plain_attend(s, s["q"] if kind == "attend" else s["q_out"])
    names = {"append": ("k_pool", "v_pool", "ksum", "page_cnt", "q_out"),
             "chunk": ("k_out", "v_out", "ksum", "page_cnt", "q_out"), "unpack": ("k_out", "v_out"),
             "attend": ("out", "lse"), "step": ("out", "lse", "ksum", "page_cnt", "q_out")}[kind]
    return {k: s[k] for k in names}


def work(case):
    kind, Hk = case["kind"], case["Hk"]
    if kind == "unpack":
        return dict(bytes=case["pages"] * Hk * (BLOB + 2 * PAGE * D * 2), flops=2 * case["pages"] * Hk * PAGE * D * 2)
    n, Hq = case.get("rows", case["B"]), case["Hq"]
    bytes_, flops = 0, 0
    if kind != "attend":    # q in and out, k and v in, the cos and sin of a position, the cache's rows and sums out
        held = 512 if kind == "append" else 144
        sums = max(case["B"], n // SUB) * Hk * D * (2 if case.get("sum16", True) else 4)
        bytes_ += n * (Hq * 512 + Hk * (512 + held) + 512) + sums
        flops += n * (Hq + Hk) * 64 * 6
    if kind == "chunk":
        bytes_ += n * Hk * 512
        flops += n * Hk * 2 * D * 2
    if kind in ("attend", "step"):
        pages = case["B"] * Hk * case["sel"] * (0.5 if case["ragged"] else 1)
        bytes_ += pages * BLOB + case["B"] * Hq * (256 + 512 + 4)
        flops += pages * PAGE * (Hq // Hk) * 4 * D
    return dict(bytes=bytes_, flops=flops)


# ---------------------------------------------------------------------------------------------- in 64 bits


def _bits(byte_, exponent_bits, bias):
    """Numbers of a sign, exponent_bits and the rest of mantissa, from their bits (no infinities here)."""
    width = 8 if exponent_bits == 4 else 4
    man = width - 1 - exponent_bits
    x = byte_.int()
    e, m = (x >> man) & ((1 << exponent_bits) - 1), x & ((1 << man) - 1)
    v = torch.where(e > 0, (2 ** man + m).double() * torch.exp2((e - bias - man).double()), m.double() * 2.0 ** (1 - bias - man))
    return torch.where((x >> (width - 1)) > 0, -v, v)


def _open(blob, g, keys):
    """64-bit rows [..., 64, 128] of page-heads, walked in storage order."""
    lead = blob.shape[:-1]
    g = g.double()
    code, scale = (blob[..., :4096], blob[..., 8192:8704]) if keys else (blob[..., 4096:8192], blob[..., 8704:])
    v = torch.stack([_bits(code & 15, 2, 1), _bits(code >> 4, 2, 1)], -1)
    sc = _bits(scale, 4, 7)
    if keys:
        v = v.reshape(*lead, 64, 8, 16)
        # [row in 8][block pair][tile][half][block in pair] -> [tile][half][row][block]
        sc = sc.reshape(*lead, 8, 4, 4, 2, 2)
        i = len(lead)
        sc = sc.permute(*range(i), i + 2, i + 3, i, i + 1, i + 4).reshape(*lead, 64, 8)
    else:
        i = len(lead)
        v = v.reshape(*lead, 8, 8, 8, 16).transpose(i + 1, i + 2).reshape(*lead, 64, 8, 16)
        # [block][row pair][tile][half][row in pair] -> [tile][half][row pair][row in pair][block]
        sc = sc.reshape(*lead, 8, 4, 4, 2, 2).permute(*range(i), i + 2, i + 3, i + 1, i + 4, i).reshape(*lead, 64, 8)
    return (v * sc[..., None]).reshape(*lead, 64, 128) * g


def _held(x, g):
    """What the 4-bit cache holds for 64-bit rows [..., 128]."""
    y = x.reshape(*x.shape[:-1], 8, 16)
    g = g.double()[..., None]
    t = y.abs().amax(-1, keepdim=True) / (6 * g)
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
    d = ((t / step).round() * step).clamp(max=448) * g
    z = torch.where(d > 0, y / d, 0.)
    m = z.abs()
    step = torch.where(m < 2, .5, torch.where(m < 4, 1., 2.)).double()
    return (((m / step).round() * step).clamp(max=6) * z.sign() * d).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    kind, Hk = case["kind"], case["Hk"]
    got = {}
    if "pool" in s:
        gk, gv = s["k_scale"][:, None, None, None], s["v_scale"][:, None, None, None]
    if kind == "unpack":
        blob = s["pool"][:, s["pages"].long()]
        valid = s["page_cnt"].long()[s["pages"].long()][:, None] > torch.arange(64, device=DEV)
        return {"k_out": _open(blob, gk, True) * valid[..., None], "v_out": _open(blob, gv, False) * valid[..., None]}
    B = case["B"]
    q = s["q"].double()
    if kind != "attend":
        n = case.get("rows", B)
        first = s["row_first"].tolist() if s["row_first"] is not None else list(range(B + 1))
        L = s["seq_len"].tolist()
        at = torch.tensor([L[b] - first[b + 1] + i for b in range(B) for i in range(first[b], first[b + 1])], device=DEV)
        req = torch.tensor([b for b in range(B) for i in range(first[b], first[b + 1])], device=DEV)
        where = s["pos"].long() if s["pos"] is not None else at[:, None]
        ax = torch.tensor(s["pair_axis"] if s["pair_axis"] is not None else [0] * 64, device=DEV)
        cs = torch.stack([s["cos_sin"][where[:, a]] for a in range(where.shape[1])], 1).double()     # [n][axes][128]
        c, sn = (cs[:, ax, torch.arange(64, device=DEV) + o][:, None] for o in (0, 64))

        def turn(x):
            z = torch.complex(x[..., :64], x[..., 64:]) * torch.complex(c, sn)
            return torch.cat([z.real, z.imag], -1)

        got["q_out"] = turn(q)
        kr, vr = turn(s["k"].double()), s["v"].double()
        phys, tok = s["page_table"].long()[req, at // 64], at % 64
        cnt = s["page_cnt"].long().scatter_reduce(0, phys, tok + 1, "amax")
        got["page_cnt"] = None
        if kind == "append":
            kp, vp = s["k_pool"].double(), s["v_pool"].double()
            kp[:, phys, tok], vp[:, phys, tok] = kr.transpose(0, 1).bfloat16().double(), vr.transpose(0, 1)
            got["k_pool"], got["v_pool"] = kp, vp
        else:
            pages = s["pages"].long()
            slot = torch.zeros(cnt.numel(), dtype=torch.long, device=DEV)
            slot[pages] = torch.arange(pages.numel(), device=DEV)
            kp, vp = _open(s["pool"][:, pages], gk, True), _open(s["pool"][:, pages], gv, False)
            kp[:, slot[phys], tok] = _held(kr.transpose(0, 1), s["k_scale"][:, None, None])
            vp[:, slot[phys], tok] = _held(vr.transpose(0, 1), s["v_scale"][:, None, None])
            if kind == "chunk":
                valid = (cnt[pages][:, None] > torch.arange(64, device=DEV))[..., None]
                got["k_out"], got["v_out"] = kp * valid, vp * valid
        if case.get("sum16", True):
            ks = s["ksum"].double()
            pages = s["pages"].long()
            rows = kp[:, pages] if kind == "append" else kp
            valid = (cnt[pages][:, None] > torch.arange(64, device=DEV))[..., None]
            ks[:, pages] = (rows * valid).reshape(Hk, -1, 4, 16, 128).sum(3)
            got["ksum"] = ks
        else:
            got["ksum"] = None
    if kind == "step":  # attends with what was rounded to 16 and 4 bits on the way, where 64 bits now and then round otherwise
        got["out"] = got["lse"] = None
    if kind == "attend":
        Hq, G = case["Hq"], case["Hq"] // Hk
        outs, lses = [], []
        for b in range(B):      # one request at a time keeps the 64-bit pages small
            idx = s["sel"][b].long()
            ok = torch.arange(idx.shape[1], device=DEV) < s["n_sel"][b][:, None]
            idx = idx.clamp(min=0)
            pg = s["page_table"][b].long()[idx].clamp(min=0)
            blob = s["pool"][torch.arange(Hk, device=DEV)[:, None], pg]
            k, v = _open(blob, gk, True), _open(blob, gv, False)
            keep = (ok[..., None] & (idx[..., None] * 64 + torch.arange(64, device=DEV) < s["seq_len"][b])).reshape(Hk, 1, -1)
            x = torch.einsum("hgd,htd->hgt", q[b].reshape(Hk, G, 128), k.reshape(Hk, -1, 128)) / 128 ** .5
            x = x.masked_fill(~keep, -math.inf)
            lse = x.logsumexp(-1)
            p = (x - lse[..., None]).exp().nan_to_num(0.).masked_fill(~keep, 0.)
            outs.append(torch.einsum("hgt,htd->hgd", p, v.reshape(Hk, -1, 128)).reshape(Hq, 128))
            lses.append(lse.reshape(Hq))
        got["out"], got["lse"] = torch.stack(outs), torch.stack(lses)
    return got
