"""Pins of the paged-cache and tree-attention oracle (CPU only)."""
import numpy as np
import pytest

import oracle
import workloads
from oracle import kvcache as okv


def _setup(seed, batch=3, n=12, hq=4, hkv=2, d=8, page=4, ctx_hi=13):
    rng = np.random.default_rng(seed)
    tok, par, dep, cnt = workloads.random_tree(batch, n, 50, 5, seed=seed)
    ctx = rng.integers(0, ctx_hi, batch)
    width = -(-(ctx_hi + n) // page)
    n_pages = batch * width + 2
    table = rng.permutation(n_pages)[: batch * width].reshape(batch, width)
    k, v = rng.normal(size=(2, n_pages, page, hkv, d))
    q = rng.normal(size=(batch, n, hq, d))
    return dict(par=par, dep=dep, cnt=cnt, ctx=ctx, table=table, k=k, v=v, q=q, page=page, n_pages=n_pages)


def _token(s, b, t):
    return int(s["table"][b, t // s["page"]]), t % s["page"]


@pytest.mark.parametrize("seed", range(4))
def test_a_node_attends_its_own_root_path_as_a_sequence(seed):
    """Tree attention of node i is ordinary attention of the sequence context + root path."""
    s = _setup(seed)
    B, n, hq, d = s["q"].shape
    mask = oracle.tree_ancestor_mask(s["par"], s["cnt"], n)
    r = okv.tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["cnt"], mask, d ** -0.5)
    for b in range(B):
        for i in range(int(s["cnt"][b])):
            path, u = [], i
            while u >= 0:
                path.append(u)
                u = int(s["par"][b, u])
            tokens = list(range(int(s["ctx"][b]))) + [int(s["ctx"][b]) + j for j in reversed(path)]
            for h in range(hq):
                rows = [_token(s, b, t) for t in tokens]
                w = np.array([np.exp(s["q"][b, i, h] @ s["k"][p, o, h // 2] * d ** -0.5) for p, o in rows])
                want = sum(x * s["v"][p, o, h // 2] for x, (p, o) in zip(w, rows)) / w.sum()
                np.testing.assert_allclose(r.out[b, i, h], want, rtol=1e-12, atol=1e-13)
                np.testing.assert_allclose(r.lse[b, i, h], np.log(w.sum()), rtol=1e-12)
        assert (r.out[b, int(s["cnt"][b]):] == 0).all() and np.isneginf(r.lse[b, int(s["cnt"][b]):]).all()


def test_no_mask_is_a_causal_chain():
    s = _setup(9)
    B, n = s["cnt"].shape[0], s["q"].shape[1]
    chain = np.tile(np.arange(-1, n - 1), (B, 1))
    m = oracle.tree_ancestor_mask(chain, s["cnt"], n)
    a = okv.tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["cnt"], m, 0.3)
    b = okv.tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["cnt"], None, 0.3)
    np.testing.assert_array_equal(a.out, b.out)


@pytest.mark.parametrize("seed", range(6))
def test_resize_conserves_pages_and_undoes_itself(seed):
    rng = np.random.default_rng(seed)
    B, page, width, n_pages = 7, 3, 9, 60
    held = rng.integers(0, 5, B)
    order = rng.permutation(n_pages)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, : held[b]] = order[at: at + held[b]]
        at += held[b]
    free = list(order[at:])
    length = rng.integers(0, width * page + 1, B)
    t, h, f, st = okv.pages_resize(length, table, held, free, page, n_pages)
    owned = [int(x) for b in range(B) for x in t[b, : h[b]]]
    assert sorted(owned + f) == list(range(n_pages))
    assert (st == 0).all() and (h == -(-length // page)).all()
    assert (t[np.arange(width)[None, :] >= h[:, None]] == -1).all()
    # growth alone, then back: the list and the tables are what they were
    up = np.maximum(length, held * page)
    t2, h2, f2, _ = okv.pages_resize(up, table, held, free, page, n_pages)
    t3, h3, f3, _ = okv.pages_resize(held * page, t2, h2, f2, page, n_pages)
    assert f3 == [int(x) for x in free] and (t3 == table).all() and (h3 == held).all()


def test_resize_serves_in_order_until_one_does_not_fit():
    table = np.full((4, 8), -1)
    t, h, f, st = okv.pages_resize([4, 0, 12, 2], table, [0, 0, 0, 0], [5, 6, 7, 8], 2, 10)
    assert st.tolist() == [0, 0, okv.NO_PAGE, okv.NO_PAGE]
    assert h.tolist() == [2, 0, 0, 0] and t[0, :2].tolist() == [8, 7] and f == [5, 6]


@pytest.mark.parametrize("seed", range(4))
def test_append_then_commit_reads_back_as_the_accepted_sequence(seed):
    s = _setup(seed)
    B, n = s["cnt"].shape[0], s["q"].shape[1]
    rng = np.random.default_rng(seed + 50)
    kn, vn = rng.normal(size=(2, B, n) + s["k"].shape[2:])
    slot, pos, st = okv.tree_slots(s["ctx"], s["cnt"], s["dep"], s["table"], n, s["page"], s["n_pages"])
    assert (st == 0).all()
    k, v, _ = okv.append(kn, vn, slot, s["k"], s["v"])
    alen = np.array([min(3, int(c) - 1) for c in s["cnt"]])
    path = np.full((B, 5), -1)
    for b in range(B):
        path[b, : alen[b]] = np.sort(rng.permutation(np.arange(1, s["cnt"][b]))[: alen[b]])
    ck, cv, new_len, st = okv.commit(k[None], v[None], s["table"], s["ctx"], s["cnt"], alen, path)
    assert (st == 0).all() and (new_len == s["ctx"] + 1 + alen).all()
    for b in range(B):
        want = [0] + list(path[b, : alen[b]])
        for i, node in enumerate(want):
            p, o = _token(s, b, int(s["ctx"][b]) + i)
            np.testing.assert_array_equal(ck[0, p, o], kn[b, node])
            np.testing.assert_array_equal(cv[0, p, o], vn[b, node])
        for t in range(int(s["ctx"][b])):                       # the context is untouched
            p, o = _token(s, b, t)
            np.testing.assert_array_equal(ck[0, p, o], s["k"][p, o])
        assert (pos[b, : s["cnt"][b]] == s["ctx"][b] + s["dep"][b, : s["cnt"][b]]).all()
