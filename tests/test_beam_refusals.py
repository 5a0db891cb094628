"""What beam search's calls refuse on the host, what they launch, and the tests' own forms of them."""
import ctypes
import json

import numpy as np
import pytest
import torch

import beam_ref as ref
import fake_cuda


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from sparse_paged_kv_score_gb300 import build
    build.build()
    return fake_cuda.build(str(tmp_path_factory.mktemp("fake")))


def test_refusals_and_launches(fake):
    program = """
import ctypes, json
P = 4096
h = f.handle(False, 2, max_units=64)
plan = ctypes.c_void_p()
def create(cache=h, rows=8, vocab=1000, out=ctypes.byref(plan)):
    return f.lib.beam_plan_create(cache, rows, vocab, out)
plans = [create(cache=None), create(rows=0), create(vocab=0), create(rows=65537), create(vocab=(1 << 24) + 1), create(out=None), create()]
f.events()
def select(cache=h, plan=plan, logits=P, kind=0, stride=1000, B=2, W=4, V=1000, cum=P, K=8, tokens=P, parents=P, scores=P):
    return f.lib.beam_select(cache, plan, logits, kind, stride, B, W, V, cum, K, tokens, parents, scores, None)
selects = dict(
    cache=select(cache=None), plan=select(plan=None), logits=select(logits=None), odd=select(logits=P + 2), odd16=select(logits=P + 1, kind=1),
    kind=select(kind=3), stride=select(stride=999), negative=select(B=-1), beams=select(W=0), vocab=select(V=0), best=select(K=0),
    cum=select(cum=None), tokens=select(tokens=None), parents=select(parents=None), scores=select(scores=None),
    rows=select(B=3), wide=select(V=1001, stride=1001), many_beams=select(W=65, B=0), many_best=select(K=129))
none = [f.events(), select(B=0), f.events()]
runs = [[select(kind=k, logits=P + (4 if k == 0 else 2)), f.events()] for k in range(3)]
def reorder(cache=h, parents=P, B=2, W=4, table=P, np_max=100, seq_len=P):
    return f.lib.beam_reorder(cache, parents, B, W, table, np_max, seq_len, None)
reorders = dict(cache=reorder(cache=None), parents=reorder(parents=None), table=reorder(table=None), seq_len=reorder(seq_len=None),
                np_max=reorder(np_max=0), negative=reorder(B=-1), beams=reorder(W=0), many=reorder(W=65), units=reorder(B=9))
none2 = [f.events(), reorder(B=0), f.events()]
run2 = [reorder(), f.events()]
print(json.dumps([plans, selects, none, runs, reorders, none2, run2, f.lib.beam_plan_destroy(plan), f.lib.beam_plan_destroy(None)]))
"""
    plans, selects, none, runs, reorders, none2, run2, done, again = json.loads(fake_cuda.run(fake, program))
    assert plans == [-1, -1, -1, -6, -6, -1, 0] and done == 0 and again == -1
    six = {"many_beams", "many_best", "many"}
    assert all(v == (-6 if k in six else -1) for k, v in {**selects, **reorders}.items()), (selects, reorders)
    assert none == [[], 0, []] and none2 == [[], 0, []]
    for r in runs:
        assert r[0] == 0 and len(r[1]) == 2 and "beam_groups_kernel" in r[1][0] and "beam_best_kernel" in r[1][1]
    assert run2[0] == 0 and len(run2[1]) == 1 and "beam_reorder_kernel" in run2[1][0]


def test_arguments_on_the_host():
    import sparse_paged_kv_score_gb300 as spkv
    from types import SimpleNamespace
    cache = SimpleNamespace(handle=None, tensors=[torch.zeros(1)])
    x = torch.zeros(1, 2, 3)
    t = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        spkv.beam_select(cache, None, x, x[:, :, 0], t, t, x[0])
    with pytest.raises(TypeError, match="bfloat16"):
        spkv.beam_select(cache, None, x.double(), x[:, :, 0], t, t, x[0])
    with pytest.raises(ValueError):
        spkv.beam_reorder(cache, t, t, t[0])


def test_reference_pins():
    """The tests' own forms: definitions on small cases."""
    rng = np.random.default_rng(0)
    x, cum = rng.standard_normal((3, 7)), np.array([-1.0, -np.inf, 0.5])
    s = ref.scores64(x, cum)
    p = np.exp(x) / np.exp(x).sum(1, keepdims=True)
    assert np.allclose(s[[0, 2]], np.log(p[[0, 2]]) + cum[[0, 2], None]) and np.all(np.isneginf(s[1]))
    t, par, v = ref.best(s, 20)
    assert np.array_equal(v[:14], np.sort(s[[0, 2]].ravel())[::-1]) and np.all(t[14:] == -1)
    assert np.array_equal(s[par[:14], t[:14]], v[:14])
    ref.check_best(x, cum, 20, t, par, v)
    t, par, _ = ref.best(np.zeros((2, 3)), 4)      # equal ones: the lower beam, then the lower token
    assert t.tolist() == [0, 1, 2, 0] and par.tolist() == [0, 0, 0, 1]
    # histories of letters follow the parents, whatever the parents are
    for _ in range(200):
        W, L = int(rng.integers(1, 7)), int(rng.integers(0, 200))
        pages = {}
        table = np.zeros((W, 5), int)
        for w in range(W):
            for j in range(5):
                table[w, j] = 10 * w + j if j >= L // 64 else 100 + int(rng.integers(0, 9))
                pages.setdefault(table[w, j], f"{table[w, j]}")
        par = rng.integers(-1, W, (1, W))
        before = [[pages[table[w, j]] for j in range((L + 63) // 64)] for w in range(W)]
        new, copies = ref.reorder(par, table, [L] * W)
        for _, a, b in copies:
            pages[b] = pages[a]
        for w in range(W):
            if par[0, w] >= 0:
                assert [pages[new[w, j]] for j in range((L + 63) // 64)] == before[par[0, w]]
        assert sorted(new[:, L // 64:].ravel()) == sorted(table[:, L // 64:].ravel())      # no page is lost, none is shared
