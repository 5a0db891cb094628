"""Cases of the 8-bit paged KV cache and of beam search over paged caches, each in a plain form of elementary torch
operations and through this library's entry points.

A page-head (one page of 64 tokens of one kv head) of the 8-bit pool is 16416 bytes: 8192 of key codes, 8192 of value
codes, four fp32 scales of the keys' sub-blocks (16 tokens each) and four of the values'.  A value is (c + 1/2) s with
c = byte - 128 and the sub-block's scale s, a power of two: s = 2^(E - 6) with E the exponent of the sub-block's largest
magnitude, c = floor(x / s).
"""
import math

import torch

own = False

DEV = torch.device("cuda" if torch.cuda.is_available() else "cpu")
D, PAGE, SUB, BLOB = 128, 64, 16, 16416
THETA = 500000.0
INF = math.inf

# Places inside a page-head: token t, dim d; four key scales and four value scales as fp32 behind the codes.
_t, _d = torch.arange(64)[:, None], torch.arange(128)[None, :]
K_CODE = (_t // 8 * 1024 + _d // 16 % 2 * 512 + _t % 8 * 64 + _d // 32 * 16 + _d % 16).to(DEV)
V_CODE = (8192 + _t // 8 * 1024 + _d // 8 % 2 * 512 + _d // 16 * 64 + _t % 8 // 2 * 16 + _d % 8 * 2 + _t % 2).to(DEV)


def listed():
    return [
        # a short question into the 8-bit cache, behind a context, and its pages back as bf16 for the prefill
        dict(name="chunk short", kind="chunk", B=1, rows=77, Hq=8, Hk=2, axes=1, fused=False, ctx=1000),
        # the same for a batch of prompts, queries, keys and values as slices of one projection's output
        dict(name="chunk prompts", kind="chunk", B=4, rows=6000, Hq=32, Hk=8, axes=1, fused=True, ctx=2048),
        # one context's pages, and a batch's, unpacked for a bf16 kernel
        dict(name="unpack context", kind="unpack", pages=17, Hk=2),
        dict(name="unpack batch", kind="unpack", pages=2048, Hk=8),
        # decode attention over selected pages of the 8-bit cache: one request
        dict(name="attend tiny", kind="attend", B=1, Hq=8, Hk=2, sel=17, ctx=4096, ragged=False),
        # a decode batch
        dict(name="attend batch", kind="attend", B=32, Hq=32, Hk=8, sel=65, ctx=32768, ragged=False),
        # one kv head for all query heads, selections of every length, empty ones too
        dict(name="attend ragged", kind="attend", B=61, Hq=16, Hk=1, sel=129, ctx=10000, ragged=True),
        # a decode step: the new token rotated and appended, then attended with the selected pages
        dict(name="step batch", kind="step", B=16, Hq=32, Hk=8, sel=65, ctx=65536, ragged=False),
        # the next tokens of one request's beams: latency
        dict(name="select one", kind="select", B=1, W=4, V=32000, K=8, dtype="fp32", pad=0, dead=False),
        # of a batch's, with a vocabulary as large as they get; twice as many as there are beams, some of which end
        dict(name="select batch", kind="select", B=32, W=8, V=128256, K=16, dtype="bf16", pad=0, dead=False),
        # beams that follow their parents: one request's
        dict(name="reorder one", kind="reorder", B=1, W=4, Hk=2, ctx=1000),
        # a batch's
        dict(name="reorder batch", kind="reorder", B=32, W=8, Hk=8, ctx=4000),
    ]


HEADS = [(8, 2), (32, 8), (40, 8), (16, 1), (6, 6), (28, 4), (22, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["chunk", "chunk", "unpack", "attend", "attend", "step", "select", "select", "reorder"])
    if kind == "select":
        W = rng.choice([1, 2, 3, 4, 5, 8, 10, 16])
        B = _log(rng, 1, 64 // W if W < 16 else 4)
        dtype = rng.choice(["fp32", "bf16", "fp16"])
        V = _log(rng, 500, min(200000, 16000000 // (B * W)))
        return dict(kind=kind, B=B, W=W, V=V, K=rng.randint(1, 2 * W), dtype=dtype, pad=rng.choice([0, 1, 40]),
                    dead=rng.random() < 0.5)
    if kind == "reorder":
        return dict(kind=kind, B=_log(rng, 1, 24), W=rng.randint(1, 12), Hk=rng.choice([1, 2, 4, 8]), ctx=_log(rng, 1, 6000))
    Hq, Hk = rng.choice(HEADS)
    if kind == "chunk":
        decode = rng.random() < 0.4
        rows = _log(rng, 1, 200) if decode else _log(rng, 20, 5000)
        B = rows if decode else min(rows, _log(rng, 1, 12))
        return dict(kind=kind, B=B, rows=rows, Hq=Hq, Hk=Hk, axes=rng.choice([1, 1, 2, 3, 4]), fused=rng.random() < 0.5,
                    ctx=rng.randint(0, 30000) if decode else rng.randint(0, 3000))
    if kind == "unpack":
        return dict(kind=kind, pages=_log(rng, 1, 12000 // Hk), Hk=Hk)
    sel = _log(rng, 1, 140)
    B = _log(rng, 1, max(1, min(64, 14000 // (Hk * sel))))
    return dict(kind=kind, B=B, Hq=Hq, Hk=Hk, sel=sel, ctx=rng.randint(64 * sel + 64, 64 * sel + 40000),
                ragged=kind == "attend" and rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------- inputs


def _scale(a):
    """Scales of sub-blocks whose largest magnitudes are a (fp32)."""
    e = torch.frexp(a).exponent - 7
    s = torch.ldexp(torch.ones_like(a), e.clamp(min=-126))
    return torch.where(a == 0, 0., torch.where(a.isfinite(), s, math.nan))


def _pool8(gen, Hk, n_phys):
    """An 8-bit pool of N(0, 1) rows, one key row in a hundred four times as large."""
    pool = torch.empty(Hk, n_phys, BLOB, dtype=torch.uint8, device=DEV)
    for h in range(Hk):
        for x0 in range(0, n_phys, 2048):
            n = min(2048, n_phys - x0)
            k = torch.randn(n, PAGE, D, generator=gen, device=DEV)
            k *= 1 + 3 * (torch.rand(n, PAGE, 1, generator=gen, device=DEV) < 0.01)
            v = torch.randn(n, PAGE, D, generator=gen, device=DEV)
            scales = []
            for x, at in ((k, K_CODE), (v, V_CODE)):
                x = x.bfloat16().float().unflatten(1, (4, SUB))
                s = _scale(x.abs().amax((2, 3)))
                c = torch.floor(x / s[:, :, None, None])
                pool[h, x0:x0 + n, at.flatten()] = (c + 128).to(torch.uint8).flatten(1)
                scales.append(s)
            pool[h, x0:x0 + n, 16384:] = torch.cat(scales, 1).contiguous().view(torch.uint8)
    return pool


def _table(n_pos):
    """cos (64 pairs) and sin (64 pairs) of every position, angles in 64 bits."""
    f = THETA ** (-torch.arange(64, dtype=torch.float64, device=DEV) / 64)
    a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


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


def _prepare_select(case, gen):
    B, W, V, K = (case[k] for k in ("B", "W", "V", "K"))
    dtype = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[case["dtype"]]
    x = torch.empty(B * W, V + case["pad"], dtype=dtype, device=DEV)
    for r0 in range(0, B * W, 32):
        x[r0:r0 + 32] = (2.5 * torch.randn(min(32, B * W - r0), V + case["pad"], generator=gen, device=DEV) - 2).to(dtype)
    # a few tokens of each beam stand out
    few = torch.randint(0, V, (B * W, 6), generator=gen, device=DEV)
    x.scatter_(1, few, (5 + 8 * torch.rand(B * W, 6, generator=gen, device=DEV)).to(dtype))
    x = x[:, :V].unflatten(0, (B, W))
    x[..., V - V // 500:] = -INF                        # padding of the vocabulary
    cum = -(12 * torch.rand(B, W, generator=gen, device=DEV)).sort(1).values
    if case["dead"]:                                    # beams that ended, a beam with few tokens allowed
        cum[:, W - W // 3:] = -INF
        x[0, 0, 3 * W:] = -INF
    return dict(logits=x, cum=cum, tokens=torch.zeros(B, K, dtype=torch.int32, device=DEV),
                parents=torch.zeros(B, K, dtype=torch.int32, device=DEV), scores=torch.zeros(B, K, device=DEV))


def _prepare_reorder(case, gen):
    B, W, Hk, ctx = (case[k] for k in ("B", "W", "Hk", "ctx"))
    L = torch.randint(ctx - ctx // 8, ctx + 1, (B,), generator=gen, device=DEV)
    full, np_max = L // PAGE, ctx // PAGE + 4
    n_phys = B * (W + 4)
    ids = torch.randperm(n_phys, generator=gen, device=DEV).reshape(B, W + 4)
    # complete pages: the prompt's shared ones, then a page of the beams; each beam's own pages from its last one on
    pt = ids.gather(1, torch.randint(0, 4, (B, W * np_max), generator=gen, device=DEV)).reshape(B, W, np_max)
    pt[..., :np_max // 2] = pt[:, :1, :np_max // 2]
    own_page = torch.where(torch.arange(np_max, device=DEV) >= full[:, None, None], ids[:, 4:, None], pt)
    cnt = torch.full((n_phys,), PAGE, dtype=torch.int64, device=DEV)
    cnt[ids[:, 4:]] = (L % PAGE)[:, None].expand(B, W)
    s = dict(page_table=_int(own_page).reshape(B * W, np_max), page_cnt=_int(cnt), seq_len=_int(L.repeat_interleave(W)),
             parents=_int(torch.randint(0, W, (B, W), generator=gen, device=DEV)),
             ksum=torch.zeros(Hk, n_phys, 4, D, device=DEV))
    return s, n_phys


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    kind = case["kind"]
    if kind == "select":
        s = _prepare_select(case, gen)
        s["kind"] = kind
        if own:
            import sparse_paged_kv_score_gb300 as spkv
            page = torch.zeros(1, 1, PAGE, D, dtype=torch.bfloat16, device=DEV)
            s["cache"] = spkv.paged_kv_create(page, page.clone(), None, None, max_units=1)
            s["plan"] = spkv.BeamPlan(s["cache"], case["B"] * case["W"], case["V"])
        return s
    Hk = case["Hk"]
    if kind == "chunk":
        s, n_phys = _prepare_append(case, gen)
        s["ksum"] = torch.zeros(Hk, n_phys, 4, D, dtype=torch.bfloat16, device=DEV)
    elif kind == "unpack":
        n = case["pages"]
        n_phys = n + max(1, n // 8)
        cnt = torch.where(torch.rand(n_phys, generator=gen, device=DEV) < 0.9, PAGE,
                          torch.randint(0, PAGE + 1, (n_phys,), generator=gen, device=DEV))
        s = dict(page_cnt=_int(cnt), pages=_int(torch.randperm(n_phys, generator=gen, device=DEV)[:n]), ksum=None)
    elif kind == "reorder":
        s, n_phys = _prepare_reorder(case, gen)
    else:
        s, n_phys = _prepare_attend(case, gen)
    s["kind"] = kind
    if kind == "reorder":
        s["k_pool"], s["v_pool"] = (torch.randn(Hk, n_phys, PAGE, D, generator=gen, device=DEV).bfloat16() for _ in range(2))
    else:
        s["pool"] = _pool8(gen, Hk, n_phys)
    if kind in ("chunk", "unpack"):
        shape = (Hk, s["pages"].numel(), PAGE, D)
        s["k_out"], s["v_out"] = (torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    if s["ksum"] is not None:
        _sums(s)
    if own:
        import sparse_paged_kv_score_gb300 as spkv
        units = min(4096, case.get("B", 1) * case.get("W", 1) * Hk)
        if kind == "reorder":
            s["cache"] = spkv.paged_kv_create(s["k_pool"], s["v_pool"], s["ksum"], s["page_cnt"], max_units=units)
        else:
            s["cache"] = spkv.paged_kv_create_q8(s["pool"], s["ksum"], s["page_cnt"], max_units=units)
    return s


# ---------------------------------------------------------------------------------------------- plain forms


def _codes(blob, keys):
    """fp32 codes [..., 64, 128] and scales [..., 4] of page-heads [..., 16416]."""
    at = 16384 if keys else 16400
    return blob[..., K_CODE if keys else V_CODE].float() - 128, blob[..., at:at + 16].contiguous().view(torch.float32)


def _values(blob, keys):
    """fp32 rows [..., 64, 128] of page-heads [..., 16416]."""
    c, s = _codes(blob, keys)
    return (c + 0.5) * s.repeat_interleave(SUB, -1)[..., None]


def _page_keys(s, pages):
    """fp32 keys [Hk][pages][64][128] that the pool holds."""
    return _values(s["pool"][:, pages], True) if "pool" in s else s["k_pool"][:, pages].float()


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
    # the touched pages opened, the new rows put among the rows they hold, and written back
    pages = s["pages"].long()
    place = torch.zeros(s["page_cnt"].numel(), dtype=torch.long, device=DEV)
    place[pages] = torch.arange(pages.numel(), device=DEV)
    i = place[page]
    new = torch.zeros(pages.numel(), PAGE, dtype=torch.bool, device=DEV)
    new[i, tok] = True
    held = (torch.arange(PAGE, device=DEV) < s["page_cnt"][pages][:, None]) & ~new
    some, old_rows = new.unflatten(1, (4, SUB)).any(2), held.unflatten(1, (4, SUB)).any(2)
    blob = s["pool"][:, pages]
    for x, at8, keys in ((_rotate(s["k"], cs), K_CODE, True), (s["v"].float(), V_CODE, False)):
        c, scale = _codes(blob, keys)                                           # [Hk][pages][64][128], [Hk][pages][4]
        rows = torch.zeros_like(c)
        rows[:, i, tok] = x.transpose(0, 1)
        need = _scale(rows.unflatten(2, (4, SUB)).abs().amax((3, 4)))
        to = torch.where(old_rows, torch.maximum(need, scale), need)
        to = torch.where(some, to, scale)
        step = to.repeat_interleave(SUB, -1)[..., None]
        c = torch.where(held[None, :, :, None] & (step > 0), torch.floor(c * (scale.repeat_interleave(SUB, -1)[..., None] / step)), c)
        c = torch.where(new[None, :, :, None], torch.where(step > 0, torch.floor(rows / step), 0.), c)
        blob[..., at8] = (c + 128).to(torch.uint8)
        start = 16384 if keys else 16400
        blob[..., start:start + 16] = to.contiguous().view(torch.uint8)
    s["pool"][:, pages] = blob
    s["page_cnt"].scatter_reduce_(0, page, (tok + 1).int(), "amax")
    keys = _page_keys(s, pages)
    live = torch.arange(PAGE, device=DEV) < s["page_cnt"][pages][:, None]
    sums = (keys * live[None, :, :, None]).unflatten(2, (4, SUB)).sum(3)
    s["ksum"][:, pages] = sums.to(s["ksum"].dtype)


def _plain_unpack(s):
    pages = s["pages"].long()
    live = (torch.arange(PAGE, device=DEV) < s["page_cnt"][pages][:, None])[None, :, :, None]
    blob = s["pool"][:, pages]
    for out, keys in ((s["k_out"], True), (s["v_out"], False)):
        out.copy_(torch.where(live, _values(blob, keys).bfloat16(), out))


def _plain_attend(s, q):
    B, Hq = q.shape[:2]
    sel = s["sel"].long()
    Hk, S = sel.shape[1:]
    taken = torch.arange(S, device=DEV) < s["n_sel"][..., None]
    sel = torch.where(taken, sel, 0)
    page = s["page_table"].long()[torch.arange(B, device=DEV)[:, None, None], sel].clamp(min=0)
    h = torch.arange(Hk, device=DEV)[None, :, None]
    blob = s["pool"][h, page]
    k = _values(blob, True).flatten(2, 3)
    at = sel[..., None] * PAGE + torch.arange(PAGE, device=DEV)
    live = (taken[..., None] & (at < s["seq_len"][:, None, None, None])).flatten(2)[:, :, None]
    x = (q.float().unflatten(1, (Hk, -1)) @ k.transpose(2, 3)) / math.sqrt(D)
    del k
    v = _values(blob, False).flatten(2, 3)
    x = torch.where(live, x, -INF)
    m = x.amax(-1, keepdim=True)
    p = torch.where(live, (x - m).exp(), 0.)
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, (p @ v) / l, 0.)
    s["out"].copy_(o.flatten(1, 2))
    s["lse"].copy_((m + l.log()).flatten(1) if S else torch.full_like(s["lse"], -INF))


def _plain_select(s):
    """Each beam's best tokens (the larger logit first, then the lower token), then the best of all beams by score (then
    the lower beam).  In 64 bits: scores of different beams may lie close together."""
    B, W, V = s["logits"].shape
    K = s["tokens"].shape[1]
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    off = s["cum"].double() - (m + (x - m).exp().sum(-1, keepdim=True).log()).squeeze(-1)
    top, token = x.sort(dim=-1, descending=True, stable=True)
    n = min(K, V)
    score = top[..., :n] + off[..., None]
    score = torch.where(score.isnan(), -INF, score).flatten(1)
    score, at = score.sort(dim=1, descending=True, stable=True)
    n = min(K, score.shape[1])
    score, at = score[:, :n], at[:, :n]
    some, each = score > -INF, min(K, V)
    for name, x, none in (("tokens", token[..., :each].flatten(1).gather(1, at), -1), ("parents", at // each, -1), ("scores", score, -INF)):
        s[name].fill_(none)
        s[name][:, :n] = torch.where(some, x, none).to(s[name].dtype)


def _plain_reorder(s):
    B, W = s["parents"].shape
    np_max = s["page_table"].shape[1]
    pt, par = s["page_table"].long().unflatten(0, (B, W)), s["parents"].long()
    beam = torch.arange(W, device=DEV)
    L = s["seq_len"].long().unflatten(0, (B, W))[:, 0]
    full, part = L // PAGE, L % PAGE > 0
    src = torch.where(par >= 0, par, beam)
    moved = pt.gather(1, src[..., None].expand(B, W, np_max))
    new = torch.where(torch.arange(np_max, device=DEV) < full[:, None, None], moved, pt)
    # part pages: of a parent's children itself, else the first one, keeps its page
    child = par[:, :, None] == beam                                                  # [B][child][parent]
    itself = child & torch.eye(W, dtype=torch.bool, device=DEV)
    first = torch.where(itself.any(1, keepdim=True), itself, child & (child.cumsum(1) == 1))
    keeps, used = first.any(2), child.any(1)
    column = full.clamp(max=np_max - 1)[:, None, None].expand(B, W, 1)
    mine = pt.gather(2, column).squeeze(2)
    others, free = keeps.int().sort(dim=1, stable=True).indices, used.int().sort(dim=1, stable=True).indices
    got = torch.where(keeps.gather(1, others), mine.gather(1, src.gather(1, others)), mine.gather(1, free))
    to = torch.empty_like(mine).scatter_(1, others, got)
    s["page_table"].copy_(torch.where(part[:, None, None], new.scatter(2, column, to[..., None]), new).flatten(0, 1))
    # contents (a page that is kept, or given to a beam without a parent, onto itself)
    frm = torch.where(par >= 0, mine.gather(1, src), to)
    frm, to = (torch.where(part[:, None], x, mine).flatten() for x in (frm, to))
    live = (torch.arange(PAGE, device=DEV) < s["page_cnt"][frm][:, None])[None, :, :, None]
    for name in ("k_pool", "v_pool"):
        s[name][:, to] = torch.where(live, s[name][:, frm], s[name][:, to])
    s["ksum"][:, to] = s["ksum"][:, frm]
    s["page_cnt"][to] = s["page_cnt"][frm]


def run(state):
    s, kind = state, state["kind"]
    if own:
        import sparse_paged_kv_score_gb300 as spkv
        if kind in ("chunk", "step"):
            spkv.paged_kv_append_rope(s["cache"], s["k"], s["v"], s["seq_len"], s["page_table"], row_first=s["row_first"],
                                      q=s["q"], q_out=s["q_out"], cos_sin=s["cos_sin"], pos=s["pos"], pair_axis=s["pair_axis"])
        if kind in ("chunk", "unpack"):
            spkv.paged_kv_unpack_q8(s["cache"], s["pages"], s["k_out"], s["v_out"])
        if kind in ("attend", "step"):
            spkv.sparse_decode_attn(s["cache"], s["q"] if kind == "attend" else s["q_out"], s["page_table"], s["sel"],
                                    s["n_sel"], s["seq_len"], s["out"], s["lse"])
        if kind == "select":
            spkv.beam_select(s["cache"], s["plan"], s["logits"], s["cum"], s["tokens"], s["parents"], s["scores"])
        if kind == "reorder":
            spkv.beam_reorder(s["cache"], s["parents"], s["page_table"], s["seq_len"])
    else:
        if kind in ("chunk", "step"):
            _plain_append(s)
        if kind in ("chunk", "unpack"):
            _plain_unpack(s)
        if kind in ("attend", "step"):
            _plain_attend(s, s["q"] if kind == "attend" else s["q_out"])
        if kind == "select":
            _plain_select(s)
        if kind == "reorder":
            _plain_reorder(s)
    names = {"chunk": ("k_out", "v_out", "ksum", "page_cnt", "q_out"), "unpack": ("k_out", "v_out"), "attend": ("out", "lse"),
             "step": ("out", "lse", "ksum", "page_cnt", "q_out"), "select": ("tokens", "parents", "scores"),
             "reorder": ("page_table", "page_cnt", "k_pool", "v_pool", "ksum")}[kind]
    return {k: s[k] for k in names}


def work(case):
    kind = case["kind"]
    if kind == "select":
        n = case["B"] * case["W"] * case["V"]
        return dict(bytes=n * (4 if case["dtype"] == "fp32" else 2) + case["B"] * (case["W"] * 4 + case["K"] * 12), flops=3 * n)
    Hk = case["Hk"]
    if kind == "reorder":   # with random parents (1 - 1/W)^W of the beams have no child, so as many pages are copied
        B, W, ctx = case["B"], case["W"], case["ctx"]
        copies = B * W * (1 - 1 / W) ** W
        return dict(bytes=int(copies * Hk * 2 * (32 * 512 + 4 * D * 4)) + B * W * (8 + 2 * 4 * (ctx // PAGE + 1)), flops=0)
    if kind == "unpack":
        return dict(bytes=case["pages"] * Hk * (BLOB + 2 * PAGE * D * 2), flops=2 * case["pages"] * Hk * PAGE * D * 2)
    n, Hq = case.get("rows", case["B"]), case["Hq"]
    bytes_, flops = 0, 0
    if kind != "attend":    # q in and out, k and v in, the cos and sin of a position, the cache's rows, scales and sums out
        sums = max(case["B"], n // SUB) * Hk * (D * 2 + 8)
        bytes_ += n * (Hq * 512 + Hk * (512 + 256) + 512) + sums
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


def _open(blob, keys):
    """64-bit codes [..., 64, 128] and scales [..., 4] of page-heads, walked in storage order."""
    lead, i = blob.shape[:-1], blob.dim() - 1
    c = (blob[..., :8192] if keys else blob[..., 8192:16384]).double() - 128
    if keys:    # [eight tokens][half][token][four][sixteen dims] -> token, four, half, dims
        c = c.reshape(*lead, 8, 2, 8, 4, 16).permute(*range(i), i, i + 2, i + 3, i + 1, i + 4)
    else:       # [eight tokens][half][block][pair][dim][token of the pair] -> pair, token, block, half, dim
        c = c.reshape(*lead, 8, 2, 8, 4, 8, 2).permute(*range(i), i, i + 3, i + 5, i + 2, i + 1, i + 4)
    s = blob[..., 16384:].contiguous().view(torch.float32).double().unflatten(-1, (2, 4))[..., 0 if keys else 1, :]
    return c.reshape(*lead, 64, 128), s


def _rows64(blob, keys):
    c, s = _open(blob, keys)
    return ((2 * c + 1).unflatten(-2, (4, 16)) * (s / 2)[..., None, None]).flatten(-3, -2)


def _exact_chunk(case, s):
    B, n, Hk = case["B"], case.get("rows", case["B"]), case["Hk"]
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

    got = dict(q_out=turn(s["q"].double()), page_cnt=None)
    kr, vr = turn(s["k"].double()), s["v"].double()
    phys, tok = s["page_table"].long()[req, at // 64], at % 64
    before = s["page_cnt"].long()
    cnt = before.scatter_reduce(0, phys, tok + 1, "amax")
    pages = s["pages"].long()
    slot = torch.zeros(cnt.numel(), dtype=torch.long, device=DEV)
    slot[pages] = torch.arange(pages.numel(), device=DEV)
    fresh = torch.zeros(pages.numel(), 64, dtype=torch.bool, device=DEV)
    fresh[slot[phys], tok] = True
    kept = (torch.arange(64, device=DEV) < before[pages][:, None]) & ~fresh
    for name, x, keys in (("k", kr, True), ("v", vr, False)):
        code, sc = _open(s["pool"][:, pages], keys)
        rows = torch.zeros_like(code)
        rows[:, slot[phys], tok] = x.transpose(0, 1)
        big = rows.abs().reshape(Hk, -1, 4, 16 * 128).amax(3)
        want = torch.where(big > 0, torch.exp2(torch.floor(torch.log2(big.clamp(min=2.0 ** -120))) - 6), 0.)
        has, any_new = kept.reshape(-1, 4, 16).any(2), fresh.reshape(-1, 4, 16).any(2)
        now = torch.where(any_new, torch.where(has, torch.maximum(want, sc), want), sc)
        per = now.repeat_interleave(16, 2)[..., None]
        ratio = torch.where(per > 0, sc.repeat_interleave(16, 2)[..., None] / per, 1.)
        code = torch.where(kept[None, ..., None], torch.floor(code * ratio), code)
        code = torch.where(fresh[None, ..., None], torch.where(per > 0, torch.floor(rows / per), 0.), code)
        got[name] = (code + 0.5) * per
    valid = (cnt[pages][:, None] > torch.arange(64, device=DEV))[..., None]
    ks = s["ksum"].double()
    ks[:, pages] = (got["k"] * valid).reshape(Hk, -1, 4, 16, 128).sum(3)
    return dict(k_out=got["k"] * valid, v_out=got["v"] * valid, ksum=ks, page_cnt=None, q_out=got["q_out"])


def _exact_select(case, s):
    B, W, V, K = (case[k] for k in ("B", "W", "V", "K"))
    tokens, parents, scores = (torch.full((B, K), x, dtype=t) for x, t in ((-1, torch.int64), (-1, torch.int64), (-INF, torch.float64)))
    for b in range(B):
        x = s["logits"][b].double()
        y = (x - x.logsumexp(-1, keepdim=True) + s["cum"][b].double()[:, None]).nan_to_num(-INF, neginf=-INF).flatten()
        y, at = y.sort(descending=True, stable=True)
        n = min(K, int((y[:K] > -INF).sum()))
        tokens[b, :n], parents[b, :n], scores[b, :n] = at[:n].cpu() % V, at[:n].cpu() // V, y[:n].cpu()
    return dict(tokens=tokens.int().to(DEV), parents=parents.int().to(DEV), scores=scores.to(DEV))


def _exact_reorder(case, s):
    B, W = case["B"], case["W"]
    old = s["page_table"].cpu().reshape(B, W, -1)
    new = old.clone()
    k, v, ks, cnt = s["k_pool"].double(), s["v_pool"].double(), s["ksum"].double(), s["page_cnt"].clone()
    for b, par in enumerate(s["parents"].tolist()):
        L = int(s["seq_len"][b * W])
        full, rows = L // PAGE, L % PAGE
        for w, p in enumerate(par):
            if p >= 0:
                new[b, w, :full] = old[b, p, :full]
        if rows == 0:
            continue
        free = [p for p in range(W) if p not in par]
        for w, p in enumerate(par):
            if p >= 0 and w == (p if par[p] == p else par.index(p)):
                new[b, w, full] = old[b, p, full]
                continue
            to = int(old[b, free.pop(0), full])
            new[b, w, full] = to
            if p >= 0:
                frm = int(old[b, p, full])
                n = int(cnt[frm])
                k[:, to, :n], v[:, to, :n], ks[:, to], cnt[to] = k[:, frm, :n], v[:, frm, :n], ks[:, frm], cnt[frm]
    return dict(page_table=new.reshape(B * W, -1).to(DEV), page_cnt=cnt, k_pool=k, v_pool=v, ksum=ks)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "unpack":
        blob = s["pool"][:, s["pages"].long()]
        valid = s["page_cnt"].long()[s["pages"].long()][:, None] > torch.arange(64, device=DEV)
        return {"k_out": _rows64(blob, True) * valid[..., None], "v_out": _rows64(blob, False) * valid[..., None]}
    if kind == "select":
        return _exact_select(case, s)
    if kind == "reorder":
        return _exact_reorder(case, s)
    if kind == "chunk":
        return _exact_chunk(case, s)
    if kind == "step":  # attends with what was rounded to 16 and 8 bits on the way, where 64 bits now and then round otherwise
        got = _exact_chunk(case, s)
        return dict(out=None, lse=None, ksum=got["ksum"], page_cnt=None, q_out=got["q_out"])
    B, Hq, Hk = case["B"], case["Hq"], case["Hk"]
    q = s["q"].double()
    outs, lses = [], []
    for b in range(B):      # one request at a time keeps the 64-bit pages small
        idx = s["sel"][b].long()
        ok = torch.arange(idx.shape[1], device=DEV) < s["n_sel"][b][:, None]
        idx = idx.clamp(min=0)
        pg = s["page_table"][b].long()[idx].clamp(min=0)
        blob = s["pool"][torch.arange(Hk, device=DEV)[:, None], pg]
        k, v = _rows64(blob, True), _rows64(blob, False)
        keep = (ok[..., None] & (idx[..., None] * 64 + torch.arange(64, device=DEV) < s["seq_len"][b])).reshape(Hk, 1, -1)
        x = torch.einsum("hgd,htd->hgt", q[b].reshape(Hk, Hq // Hk, 128), k.reshape(Hk, -1, 128)) / 128 ** .5
        x = x.masked_fill(~keep, -INF)
        lse = x.logsumexp(-1)
        p = (x - lse[..., None]).exp().nan_to_num(0.).masked_fill(~keep, 0.)
        outs.append(torch.einsum("hgt,htd->hgd", p, v.reshape(Hk, -1, 128)).reshape(Hq, 128))
        lses.append(lse.reshape(Hq))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
