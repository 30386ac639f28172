"""GPU parity of the paged-cache operators and tree attention with the oracle.

Bounds. With p the exact softmax weights of a row, W = sum_t p_t |v_t| and
S = max_t scale sum_d |q_d k_td|: a score is a sum of d products in fp32 (off by
at most d 2^-24 S, in any order; bf16 products are exact), so a weight is off by
a factor of 1 + 2 d 2^-24 S, plus a few steps for the exponential; sums over
tokens run over at most 128 values of a tile and then over tiles and pieces
(T / 32 at most). That is r = 2^-24 (2 d S + T / 32 + 256), once in the numerator and
once in the denominator. In bf16 each weight is rounded by at most 2^-8 before
the second product, and every output by at most 2^-8 (bf16) or 2^-24 (fp32).
So |out - exact| <= (2 r + u) W + u |out| with u = 2^-8 or 2^-24, and
|lse - exact| <= r + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_draft_07_b200 as pct
import workloads
from gpu_util import f64, host
from oracle import kvcache as okv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _cache(n_pages, page, hkv, d, dtype, layout="nhd", fill=None):
    """K and V [n_pages][page][hkv][d] in a memory order: nhd, hnd, or kv (interleaved by page)."""
    dt = DT[dtype]
    if layout == "nhd":
        k, v = (torch.empty((n_pages, page, hkv, d), dtype=dt, device=DEV) for _ in range(2))
    elif layout == "hnd":
        k, v = (torch.empty((n_pages, hkv, page, d), dtype=dt, device=DEV).transpose(1, 2) for _ in range(2))
    else:
        kv = torch.empty((n_pages, 2, page, hkv, d), dtype=dt, device=DEV)
        k, v = kv[:, 0], kv[:, 1]
    for t in (k, v):
        if fill is None:
            t.copy_(torch.randn(t.shape, device=DEV))
        else:
            t.fill_(fill)
    return k, v


def _case(seed, dtype="bf16", hq=8, hkv=2, d=64, page=16, n=6, ctx=(5, 40), layout="nhd", mask="tree",
          counts=None, fill=None, q_sigma=2.0):
    torch.manual_seed(seed)
    rng = np.random.default_rng(seed)
    B = len(ctx)
    counts = [n] * B if counts is None else counts
    width = max(max(-(-(c + m) // page) for c, m in zip(ctx, counts)), 1) + 1
    n_pages = B * width + 1
    table = rng.permutation(n_pages)[: B * width].reshape(B, width).astype(np.int32)
    k, v = _cache(n_pages, page, hkv, d, dtype, layout, fill)
    if fill is not None:                        # only the tokens that exist hold numbers
        for b in range(B):
            for t in range(ctx[b] + counts[b]):
                p, o = int(table[b, t // page]), t % page
                k[p, o], v[p, o] = torch.randn((2, hkv, d), device=DEV).to(DT[dtype])
    for b in range(B):                          # entries past a request's pages are never read
        used = -(-(ctx[b] + counts[b]) // page)
        table[b, used:] = -7
    q = (torch.randn((B, n, hq, d), device=DEV) * q_sigma).to(DT[dtype])
    words = (n + 31) // 32
    if mask == "tree":
        par = np.full((B, n), -1, np.int32)
        for b in range(B):
            for i in range(1, n):
                par[b, i] = rng.integers(max(0, i - 9), i)
        m = oracle.tree_ancestor_mask(par, counts, n)
    elif mask == "random":                      # any bits: above the diagonal too, empty rows too
        m = rng.integers(0, 1 << 32, (B, n, words), dtype=np.uint64).astype(np.uint32)
        m[:, ::3] = 0
    else:
        m = None
    g = dict(q=q, k=k, v=v, table=torch.from_numpy(table).to(DEV),
             ctx=torch.tensor(ctx, dtype=torch.int64, device=DEV),
             count=torch.tensor(counts, dtype=torch.int32, device=DEV),
             mask=None if m is None else torch.from_numpy(m.view(np.int32)).to(DEV))
    return g, table, list(ctx), list(counts), m


def _run(g, **kw):
    return pct.tree_attention(g["q"], g["k"], g["v"], g["table"], g["ctx"], g["count"], mask=g["mask"], **kw)


def _check(r, g, table, ctx, counts, m, scale=None):
    d = g["q"].shape[3]
    ref = okv.tree_attention(f64(g["q"]), f64(g["k"]), f64(g["v"]), table, ctx, counts, m,
                             d ** -0.5 if scale is None else scale)
    torch.cuda.synchronize()
    out, lse = f64(r.out), f64(r.lse)
    np.testing.assert_array_equal(host(r.status), ref.status)
    u = 2.0 ** -8 if g["q"].dtype == torch.bfloat16 else 2.0 ** -24
    T = max([c + n for c, n in zip(ctx, counts)] + [1])
    rel = 2.0 ** -24 * (2 * d * ref.size + T / 32 + 256)
    np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(ref.lse))
    empty = np.isneginf(ref.lse)
    assert (out[empty] == 0).all()
    err = np.abs(out - ref.out)
    tol = (2 * rel[..., None] + u) * ref.weight + u * np.abs(ref.out)
    assert (err <= tol).all(), (np.nanmax(err - tol), np.argwhere(~(err <= tol))[:4])
    e = np.abs(lse[~empty] - ref.lse[~empty])
    t = rel[~empty] + 2.0 ** -22 * np.abs(ref.lse[~empty])
    assert (e <= t).all(), (e - t).max()
    return ref


SHAPES = [
    dict(n=1, ctx=(0,), mask=None), dict(n=1, ctx=(1, 31, 32, 33, 500), mask=None),
    dict(n=1, ctx=(2000, 0, 7, 129), mask=None, hq=4, hkv=4, d=128, page=8),
    dict(n=1, ctx=(20000,), mask=None, hq=8, hkv=1, d=128, page=64),
    dict(n=2, ctx=(15, 16), mask="tree", page=1), dict(n=7, ctx=(3, 100, 61), page=5),
    dict(n=33, ctx=(0, 64, 95), hq=7, hkv=1, d=72), dict(n=33, ctx=(130, 0), hq=6, hkv=6, d=96, page=24),
    dict(n=64, ctx=(1000,), hq=8, hkv=2, d=128, page=32), dict(n=130, ctx=(300, 1), hq=4, hkv=2, d=128, page=256),
    dict(n=130, ctx=(77, 256), hq=16, hkv=1, d=64, page=16, mask=None),
    dict(n=20, ctx=(150, 9), hq=2, hkv=1, d=256, page=16), dict(n=5, ctx=(40,), hq=3, hkv=1, d=200, page=7),
    dict(n=12, ctx=(40, 3), hq=1, hkv=1, d=8, page=4), dict(n=40, ctx=(0, 12, 100), mask="random", d=128),
    dict(n=100, ctx=(0, 129), mask="random", hq=8, hkv=4, page=128, d=128),
    dict(n=9, ctx=(8, 30, 64, 0), counts=[9, 0, 1, 4]), dict(n=70, ctx=(513, 127, 0), counts=[70, 3, 64], hq=8, hkv=2, d=128, page=128),
    dict(n=3, ctx=(60,), hq=64, hkv=1, d=64), dict(n=5, ctx=(90, 0), hq=48, hkv=1, d=128),
    dict(n=400, ctx=(150, 0), hq=2, hkv=1, d=64, mask=None), dict(n=50, ctx=(200, 3), hq=2, hkv=2, d=112, page=8),
    dict(n=70, ctx=(300, 5), hq=4, hkv=2, d=200), dict(n=40, ctx=(64, 700), hq=3, hkv=1, d=136, page=40),
    dict(n=300, ctx=(0, 20), hq=2, hkv=1, d=256, page=64, mask=None),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "n%d-t%s-%s" % (s["n"], max(s["ctx"]), s.get("d", 64)))
def test_attention_matches_the_oracle(shape, dtype):
    c = _case(11, dtype=dtype, **shape)
    _check(_run(c[0]), *c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["hnd", "kv"])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_cache_layouts_and_fused_queries(layout, n, dtype):
    c = _case(5, dtype=dtype, n=n, ctx=(50, 200), layout=layout, d=128)
    g = c[0]
    B, _, hq, d = g["q"].shape
    qkv = torch.zeros((B, n, hq + 4, d), dtype=g["q"].dtype, device=DEV)
    qkv[:, :, :hq] = g["q"]
    g["q"] = qkv[:, :, :hq]
    assert not g["q"].is_contiguous()
    _check(_run(g), *c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,page,hq", [(1, 16, 8), (37, 16, 8), (100, 64, 8), (100, 24, 8), (3, 16, 32)])
def test_places_past_the_end_do_not_enter(n, page, hq, dtype):
    """The whole cache but the requests' own tokens is NaN, also behind the end in their last pages."""
    c = _case(6, dtype=dtype, n=n, ctx=(33, 0, 118), page=page, hq=hq, d=128, fill=float("nan"))
    _check(_run(c[0]), c[0] | {"k": torch.nan_to_num(c[0]["k"]), "v": torch.nan_to_num(c[0]["v"])}, *c[1:])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n,hq", [(6, 8), (60, 8), (100, 16)])
def test_keys_of_unseen_nodes_do_not_enter(n, hq, bad):
    """Node 1's K is not finite and only node 1 sees it: every other row is as if it were not there."""
    c = _case(7, n=n, hq=hq, ctx=(33, 100), d=128, mask="random")
    g, table, ctx, counts, m = c
    m &= np.uint32(0xffffffff ^ 2)              # bit 1 of word 0 off for all rows: nobody sees node 1
    m[:, :, 1:] = m[:, :, 1:]
    g["mask"] = torch.from_numpy(m.view(np.int32)).to(DEV)
    clean = _run(g)
    torch.cuda.synchronize()
    want, wl = clean.out.clone(), clean.lse.clone()
    for b in range(2):
        t = ctx[b] + 1
        g["k"][int(table[b, t // 16]), t % 16] = bad
    r = _run(g)
    torch.cuda.synchronize()
    assert torch.equal(r.out, want) and torch.equal(r.lse, wl)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq", [(1, 8), (60, 8), (100, 32)])
def test_non_finite_keys_that_are_seen(n, hq, dtype):
    """A NaN in a context key makes every row that sees it NaN, and only those; where every key a row
    sees scores -inf the row is empty; one key at -inf has no weight."""
    c = _case(13, dtype=dtype, n=n, hq=hq, ctx=(70, 70, 70, 70), d=64)
    g, table, ctx, counts, m = c
    g["q"] = g["q"].abs() + 0.5
    clean = _run(g)
    torch.cuda.synchronize()
    want, wl = clean.out.clone(), clean.lse.clone()
    at = lambda b, t: (int(table[b, t // 16]), t % 16)       # noqa: E731
    g["k"][at(0, 40)][..., 3] = float("nan")
    for t in range(ctx[1] + counts[1]):
        g["k"][at(1, t)] = float("-inf")
    g["k"][at(2, 69)] = float("-inf")
    r = _run(g)
    torch.cuda.synchronize()
    assert torch.isnan(r.out[0]).all() and torch.isnan(r.lse[0]).all()
    assert (r.out[1] == 0).all() and torch.isneginf(r.lse[1]).all()
    # leaving out weight p lowers the lse by -ln(1 - p), which vanishes in fp32 for p < 2^-24; each side
    # is off by at most 256 steps of 2^-24 besides (the sums' order may differ)
    assert torch.isfinite(r.out[2].float()).all() and (r.lse[2] <= wl[2] + 2.0 ** -16).all()
    assert (r.lse[2] < wl[2]).any()
    assert torch.equal(r.out[3], want[3]) and torch.equal(r.lse[3], wl[3])


def test_large_scores_and_a_given_scale():
    """Scores far from 0 and a scale that is not 1 / sqrt(d), negative too."""
    for scale in (1.0, -0.7, 3e-3):
        c = _case(8, dtype="f32", n=9, ctx=(70, 3), q_sigma=6.0)
        _check(_run(c[0], scale=scale), *c, scale=scale)


def test_refused_requests_and_bad_pages():
    c = _case(9, n=8, ctx=(20, 20, 20, 20, 20), counts=[8] * 5)
    g, table, ctx, counts, m = c
    width = table.shape[1]
    ctx = [20, -1, width * 16 - 7, 20, 20]
    counts = [9, 8, 8, 8, -1]
    table[3, 1] = 10 ** 6                       # tokens 16..31 of request 3
    g["table"].copy_(torch.from_numpy(table))
    g["ctx"].copy_(torch.tensor(ctx))
    g["count"].copy_(torch.tensor(counts))
    r = _run(g)
    ref = _check(r, g, table, ctx, counts, m)
    assert ref.status.tolist() == [okv.BAD_COUNT, okv.BAD_LENGTH, okv.BAD_LENGTH, okv.BAD_PAGE, okv.BAD_COUNT]


def test_lengths_far_outside_are_refused():
    """Lengths at the ends of 64 bits: every call answers PCT_DEV_BAD_LENGTH and touches nothing of the request."""
    far = [2 ** 63 - 1, -2 ** 63, 2 ** 62, 2 ** 32 + 5, 5]
    c = _case(14, n=4, ctx=(5,) * 5)
    g, table = c[0], c[1]
    g["ctx"].copy_(torch.tensor(far))
    r = _run(g)
    slot, pos, st = pct.kv_tree_slots(g["ctx"], g["count"], g["table"], 4, 16, g["k"].shape[0])
    before = g["k"].clone()
    new_len, st2 = pct.kv_commit(g["k"], g["v"], g["table"], g["ctx"], g["count"],
                                 torch.full((5,), 1, dtype=torch.int32, device=DEV),
                                 torch.full((5, 2), 2, dtype=torch.int32, device=DEV))
    want, held, free, nfree = g["table"].clone(), *(torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([1] * 5, list(range(99)), [0]))
    st3 = pct.kv_pages_resize(g["ctx"], g["table"], held, free, nfree, 16, count=g["count"])
    torch.cuda.synchronize()
    for s in (r.status, st, st2, st3):
        assert host(s).tolist() == [okv.BAD_LENGTH] * 4 + [0]
    assert (r.out[:4] == 0).all() and torch.isneginf(r.lse[:4]).all() and (r.out[4] != 0).any()
    assert (slot[:4] == -1).all() and (pos[:4] == -1).all() and host(new_len).tolist() == far[:4] + [7]
    assert torch.equal(g["table"][:4], want[:4]) and torch.equal(host_rows(g["k"], table, 4), host_rows(before, table, 4))


def host_rows(k, table, requests):
    used = torch.from_numpy(table[:requests][table[:requests] >= 0].astype(np.int64)).to(DEV)
    return k[used]


@pytest.mark.parametrize("dtype,n,hq,batch", [("bf16", 1, 8, 300), ("bf16", 70, 16, 3), ("f32", 5, 8, 40)])
def test_results_repeat_and_do_not_depend_on_the_workspace(dtype, n, hq, batch):
    rng = np.random.default_rng(3)
    c = _case(10, dtype=dtype, n=n, hq=hq, d=128, ctx=[int(x) for x in rng.integers(0, 400, batch)])
    g = c[0]
    a = _run(g)
    nbytes = pct.tree_attention_workspace(g["k"], g["v"], g["table"].shape[1], batch, n, hq)
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)
    out = pct.AttnOut(torch.full_like(a.out, 7), torch.full_like(a.lse, 7), torch.full_like(a.status, 7))
    b = _run(g, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse) and torch.equal(a.status, b.status)
    _check(a, *c) if batch < 100 else None


@pytest.mark.parametrize("d,longest", [(96, 63), (64, 63), (128, 400), (64, 700), (200, 63)])
def test_many_short_items_of_both_kinds(d, longest):
    """A block's share mixes row tiles with one and with two halves, of one key tile and of several,
    so that a tile's place in the load ring passes between readers that do and do not use it."""
    rng = np.random.default_rng(d + longest)
    B, n, page = 64, 257, 192
    ctx = [int(x) for x in rng.integers(0, longest + 1, B)]
    counts = [int(rng.choice([n, 0, 1, rng.integers(0, n + 1), rng.integers(0, 40)])) for _ in range(B)]
    g, table, _, _, _ = _case(21, hq=32, hkv=8, d=d, page=page, n=n, ctx=ctx, counts=counts, mask=None)
    first = _run(g)
    torch.cuda.synchronize()
    assert not host(first.status).any()
    want, wl = first.out.clone(), first.lse.clone()
    for _ in range(20):
        r = _run(g)
        torch.cuda.synchronize()
        assert torch.equal(r.out, want) and torch.equal(r.lse, wl) and not host(r.status).any()
    for b in range(0, B, 9):
        one = g | {"q": g["q"][b:b + 1], "ctx": g["ctx"][b:b + 1], "count": g["count"][b:b + 1]}
        _check(pct.AttnOut(want[b:b + 1], wl[b:b + 1], first.status[b:b + 1]), one, table[b:b + 1],
               ctx[b:b + 1], counts[b:b + 1], None)


def test_many_requests_one_token():
    rng = np.random.default_rng(4)
    c = _case(12, n=1, hq=4, hkv=2, ctx=[int(x) for x in rng.integers(0, 90, 400)], mask=None, page=8)
    _check(_run(c[0]), *c)


def test_cache_offsets_past_32_bits():
    """A cache of more than 2^32 elements; the pages in use lie at its end."""
    page, hkv, d = 64, 8, 128
    n_pages = (1 << 32) // (page * hkv * d) + 40
    k = torch.empty((n_pages, page, hkv, d), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    B, n, ctx = 2, 9, [200, 70]
    torch.manual_seed(1)
    small = [torch.randn((16, page, hkv, d), device=DEV).to(torch.bfloat16) for _ in range(2)]
    k[-16:], v[-16:] = small
    rng = np.random.default_rng(1)
    local = rng.permutation(16).reshape(2, 8).astype(np.int32)
    table = torch.from_numpy(local + n_pages - 16).to(DEV)
    q = torch.randn((B, n, 32, d), device=DEV).to(torch.bfloat16)
    ct, cn = torch.tensor(ctx, device=DEV), torch.full((B,), n, dtype=torch.int32, device=DEV)
    for kk, rows in ((1, 1), (9, 9)):
        a = pct.tree_attention(q[:, :rows], k, v, table, ct, cn.clamp(max=rows))
        b = pct.tree_attention(q[:, :rows], small[0], small[1], torch.from_numpy(local).to(DEV), ct, cn.clamp(max=rows))
        torch.cuda.synchronize()
        assert torch.equal(a.out, b.out) and (host(a.status) == 0).all()
    slot, pos, st = pct.kv_tree_slots(ct, cn, table, n, page, n_pages)
    new = torch.randn((2, B, n, hkv, d), device=DEV).to(torch.bfloat16)
    pct.kv_append(new[0], new[1], slot, k, v)
    got = k.view(-1, hkv, d)[slot.view(-1)].view(B, n, hkv, d)
    assert torch.equal(got, new[0]) and int(slot.max()) * hkv * d > 1 << 32
    path = torch.tensor([[2, 5, 8], [1, 3, -1]], dtype=torch.int32, device=DEV)
    new_len, st = pct.kv_commit(k, v, table, ct, cn, torch.tensor([3, 2], dtype=torch.int32, device=DEV), path)
    torch.cuda.synchronize()
    assert host(new_len).tolist() == [204, 73] and (host(st) == 0).all()
    assert torch.equal(v.view(-1, hkv, d)[slot[0, 3]], new[1, 0, 8])
    del k, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,hq", [(1, 8), (50, 8), (100, 32)])
def test_capture_replay_and_two_streams(n, hq):
    """Two captured graphs of different lengths, replayed in turn; and calls on two streams at once."""
    cs = [_case(20 + i, n=n, hq=hq, d=128, ctx=(300 * i + 30, 5)) for i in range(2)]
    want = []
    for c in cs:
        r = _run(c[0])
        torch.cuda.synchronize()
        want.append((r.out.clone(), r.lse.clone()))
    graphs = []
    for c in cs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            r = _run(c[0])
        graphs.append((gr, r))
    for _ in range(3):
        for (gr, r), w in zip(graphs, want):
            r.out.zero_()
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(r.out, w[0]) and torch.equal(r.lse, w[1])
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    rs = [_run(c[0], stream=s) for _ in range(5) for c, s in zip(cs, streams)]
    torch.cuda.synchronize()
    for i, r in enumerate(rs):
        assert torch.equal(r.out, want[i % 2][0])


# ---------------------------------------------------------------------------------------------------
# page bookkeeping
def _pool(seed, B, width, n_pages, page, most):
    rng = np.random.default_rng(seed)
    held = rng.integers(0, most + 1, B).astype(np.int32)
    order = rng.permutation(n_pages)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, : held[b]] = order[at: at + held[b]]
        at += held[b]
    free = np.full(n_pages, -1, np.int32)
    free[: n_pages - at] = order[at:]
    return rng, table, held, free, n_pages - at


def _resize(length, table, held, free, nfree, page, count=None):
    t = [torch.from_numpy(np.array(x)).to(DEV) for x in (table, held, free)]
    fc = torch.tensor([nfree], dtype=torch.int32, device=DEV)
    st = pct.kv_pages_resize(torch.tensor(np.array(length), dtype=torch.int64, device=DEV), t[0], t[1], t[2], fc, page,
                             count=None if count is None else torch.tensor(np.array(count), dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    n = int(fc[0])
    return host(t[0]), host(t[1]), host(t[2])[:n], host(st), n


@pytest.mark.parametrize("B,width,page,tight", [(1, 4, 16, 0), (5, 1, 1, 0), (33, 40, 3, 0), (1000, 30, 16, 0),
                                                (1024, 9, 7, 40), (2500, 12, 64, 0), (2500, 12, 64, 900), (3, 5000, 2, 0)])
@pytest.mark.parametrize("seed", [0, 1])
def test_pages_resize_matches_the_oracle(B, width, page, tight, seed):
    n_pages = B * width
    rng, table, held, free, nfree = _pool(seed, B, width, n_pages, page, width // 2)
    if tight:
        nfree = tight
    length = rng.integers(0, width * page + 1, B)
    count = np.minimum(rng.integers(0, 9, B), width * page - length)
    want = okv.pages_resize(length + count, table, held, free[:nfree], page, n_pages)
    got = _resize(length, table, held, free, nfree, page, count)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)
    assert (want[3] != 0).any() == bool(tight)


def test_pages_resize_refusals():
    B, width, page, n_pages = 6, 4, 8, 40
    _, table, held, free, nfree = _pool(2, B, width, n_pages, page, 0)
    held[:] = 2
    table[:, :2] = np.arange(12).reshape(6, 2) + 28
    nfree = 20
    free[:20] = np.arange(20)
    table[4, 1] = 77                       # an entry to return that is no page
    held[5] = 9                            # more than there are columns
    length = [-1, 8 * 5, 0, 32, 3, 8]
    want = okv.pages_resize(length, table, held, free[:nfree], page, n_pages)
    got = _resize(length, table, held, free, nfree, page)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)
    assert got[3].tolist() == [okv.BAD_LENGTH, okv.BAD_LENGTH, 0, 0, okv.BAD_PAGE, okv.BAD_LENGTH]
    for nf in (-1, 41, 39):                # 39: what comes back does not fit the list
        got = _resize(length, table, held, free, nf, page)
        np.testing.assert_array_equal(got[0], table)
        np.testing.assert_array_equal(got[1], held)
        assert (got[3] == okv.BAD_COUNT).all() and got[4] == nf


@pytest.mark.parametrize("B,n,page", [(1, 1, 16), (3, 33, 5), (7, 300, 64), (400, 17, 1), (2, 5000, 16)])
def test_tree_slots_match_the_oracle(B, n, page):
    rng = np.random.default_rng(B + n)
    ctx = rng.integers(0, 100, B)
    count = rng.integers(0, n + 1, B)
    width = -(-(100 + n) // page)
    n_pages = B * width
    table = rng.permutation(n_pages).reshape(B, width).astype(np.int32)
    if B > 2:
        table[1, int(ctx[1]) // page] = -3
        count[1] = max(count[1], 1)
        ctx[2], count[0] = -5, n + 1
    depth = rng.integers(0, 16, (B, n)).astype(np.int32)
    for dep in (depth, None):
        want = okv.tree_slots(ctx, count, dep, table, n, page, n_pages)
        got = pct.kv_tree_slots(torch.from_numpy(ctx).to(DEV), torch.from_numpy(count.astype(np.int32)).to(DEV),
                                torch.from_numpy(table).to(DEV), n, page, n_pages,
                                depth=None if dep is None else torch.from_numpy(dep).to(DEV))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            np.testing.assert_array_equal(host(a), b)


# ---------------------------------------------------------------------------------------------------
# rows into the cache, and the accepted path's rows
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n,hkv,d,page,layout", [(1, 1, 1, 8, 16, "nhd"), (3, 7, 2, 64, 5, "hnd"), (4, 50, 8, 128, 16, "kv"),
                                                   (2, 300, 3, 72, 64, "nhd"), (3, 2500, 1, 64, 16, "nhd")])
def test_append_matches_the_oracle(B, n, hkv, d, page, layout, dtype):
    torch.manual_seed(B)
    rng = np.random.default_rng(n)
    n_pages = -(-2 * B * n // page) + 1
    k, v = _cache(n_pages, page, hkv, d, dtype, layout)
    slot = rng.permutation(n_pages * page)[: B * n].reshape(B, n)
    slot[rng.random((B, n)) < 0.2] = -1
    if B > 1:
        slot[1, 0] = n_pages * page
    new = torch.randn((B, n, 2 * hkv + 1, d), device=DEV).to(DT[dtype])     # slices of one projection
    kn, vn = new[:, :, :hkv], new[:, :, hkv: 2 * hkv]
    want = okv.append(f64(kn), f64(vn), slot, f64(k), f64(v))
    st = pct.kv_append(kn, vn, torch.from_numpy(slot).to(DEV), k, v)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(f64(k), want[0])
    np.testing.assert_array_equal(f64(v), want[1])
    np.testing.assert_array_equal(host(st), want[2])


@pytest.mark.parametrize("dtype,layout", [("bf16", "nhd"), ("f32", "hnd"), ("bf16", "kv")])
@pytest.mark.parametrize("B,n,depth,layers,page", [(1, 2, 1, 1, 16), (5, 40, 15, 3, 8), (3, 700, 600, 2, 5), (64, 20, 7, 1, 64)])
def test_commit_matches_the_oracle(B, n, depth, layers, page, dtype, layout):
    torch.manual_seed(n)
    rng = np.random.default_rng(depth)
    hkv, d = 2, 24
    ctx = rng.integers(0, 50, B)
    width = -(-(50 + n) // page)
    n_pages = B * width
    table = rng.permutation(n_pages).reshape(B, width).astype(np.int32)
    kv = [torch.stack(x) for x in zip(*[_cache(n_pages, page, hkv, d, dtype) for _ in range(layers)])]
    if layout == "hnd":
        kv = [x.transpose(2, 3).contiguous().transpose(2, 3) for x in kv]
    elif layout == "kv":
        both = torch.stack(kv, dim=2)
        kv = [both[:, :, 0], both[:, :, 1]]
    k, v = kv
    count = rng.integers(max(1, n // 2), n + 1, B)
    alen = np.array([int(rng.integers(0, min(depth, c - 1) + 1)) for c in count])
    alen[0] = min(depth, count[0] - 1)                       # the longest path there is
    path = np.full((B, depth), -1, np.int32)
    for b in range(B):
        path[b, : alen[b]] = np.sort(rng.permutation(np.arange(1, count[b]))[: alen[b]])
    if B > 4:
        path[1, :2], alen[1], count[1] = [3, 3], 2, n        # does not rise
        alen[2] = depth + 1
        ctx[3] = -1
        count[4] = 0
    if B > 5:
        table[5, int(ctx[5]) // page] = n_pages
        alen[5], path[5, 0] = max(alen[5], 1), max(path[5, 0], 1)
    want = okv.commit(f64(k), f64(v), table, ctx, count, alen, path)
    arg = [torch.from_numpy(np.ascontiguousarray(x.astype(np.int32))).to(DEV) for x in (table, count, alen, path)]
    args = (k, v) if layers > 1 else (k[0], v[0])
    new_len, st = pct.kv_commit(*args, arg[0], torch.from_numpy(ctx).to(DEV), arg[1], arg[2], arg[3])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host(st), want[3])
    np.testing.assert_array_equal(host(new_len), want[2])
    gk, gv = f64(k), f64(v)
    for b in range(B):                                       # up to the new length; behind it nothing is promised
        for t in range(int(want[2][b])):
            p, o = int(table[b, t // page]), t % page
            if not 0 <= p < n_pages:
                continue
            np.testing.assert_array_equal(gk[:, p, o], want[0][:, p, o])
            np.testing.assert_array_equal(gv[:, p, o], want[1][:, p, o])


# ---------------------------------------------------------------------------------------------------
def test_rounds_together_decode_what_plain_decoding_decodes():
    """Several rounds of a one-layer toy target as they would be used: pages grow, the tree's K and V go
    in, tree attention, greedy verification, the accepted path is kept, pages shrink. The tokens are those
    of plain greedy decoding, one token at a time, of the same target in float64."""
    torch.manual_seed(0)
    rng = np.random.default_rng(0)
    B, V, hq, hkv, d, page, N, D = 3, 64, 4, 2, 64, 8, 24, 6
    dm = hq * d
    emb = torch.randn((V, dm), device=DEV)
    wq, wk, wv = (torch.randn((dm, h * d), device=DEV) / dm ** 0.5 for h in (hq, hkv, hkv))
    wo = torch.randn((dm, V), device=DEV)

    def greedy(seq, steps):                                  # float64, positions by a phase on the embedding
        seq = list(seq)
        E, Q, K, Vv, O = (x.double() for x in (emb, wq, wk, wv, wo))
        gaps = []
        for _ in range(steps):
            x = torch.stack([E[t] * np.cos(0.3 * i) for i, t in enumerate(seq)])
            q, k, v = (x[-1] @ Q).view(hq, d), (x @ K).view(-1, hkv, d), (x @ Vv).view(-1, hkv, d)
            o = []
            for h in range(hq):
                a = torch.softmax(k[:, h // 2] @ q[h] * d ** -0.5, 0)
                o.append(a @ v[:, h // 2])
            y = torch.cat(o) @ O
            top = torch.topk(y, 2).values
            gaps.append(float(top[0] - top[1]))
            seq.append(int(y.argmax()))
        return seq, min(gaps)

    prompt = [list(rng.integers(0, V, 5 + 4 * b)) for b in range(B)]
    plain = [greedy(p, 24) for p in prompt]
    assert min(g for _, g in plain) > 1e-3                   # fp32 cannot flip an argmax
    n_pages, width = 60, 20
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    held = torch.zeros(B, dtype=torch.int32, device=DEV)
    free = torch.arange(n_pages, dtype=torch.int32, device=DEV)
    nfree = torch.tensor([n_pages], dtype=torch.int32, device=DEV)
    k, v = _cache(n_pages, page, hkv, d, "f32", fill=float("nan"))
    ctx = torch.zeros(B, dtype=torch.int64, device=DEV)

    def forward(tok, depth, cnt, mask):
        st = pct.kv_pages_resize(ctx, table, held, free, nfree, page, count=cnt)
        slot, pos, st2 = pct.kv_tree_slots(ctx, cnt, table, tok.shape[1], page, n_pages, depth=depth)
        x = emb[tok.long().clamp(min=0)] * torch.cos(0.3 * pos.double())[..., None].float()
        shape = lambda w, h: (x @ w).view(B, -1, h, d)       # noqa: E731
        st3 = pct.kv_append(shape(wk, hkv), shape(wv, hkv), slot, k, v)
        r = pct.tree_attention(shape(wq, hq), k, v, table, ctx, cnt, mask=mask)
        for s in (st, st2, st3, r.status):
            assert (host(s) == 0).all()
        return (r.out.reshape(B, -1, dm) @ wo).contiguous()

    n = max(len(p) for p in prompt)                          # the prompts but their last token, as a chunk
    tok = torch.zeros((B, n), dtype=torch.int32, device=DEV)
    cnt = torch.tensor([len(p) - 1 for p in prompt], dtype=torch.int32, device=DEV)
    for b, p in enumerate(prompt):
        tok[b, : len(p)] = torch.tensor(p)
    forward(tok, None, cnt, None)
    ctx = ctx + cnt
    seqs, accepted = [list(p) for p in prompt], 0
    while min(len(s) - len(p) for s, p in zip(seqs, prompt)) < 18:
        # drafts: a random tree whose nodes follow the true continuation half of the time
        tok_h, par, dep, cnt_h = workloads.random_tree(B, N, V, D, seed=int(rng.integers(1 << 30)))
        for b in range(B):
            tok_h[b, 0] = seqs[b][-1]
            on = {0}
            for i in range(1, int(cnt_h[b])):
                at = len(seqs[b]) + int(dep[b, i]) - 1
                twin = any(par[b, j] == par[b, i] and j in on for j in range(1, i))
                if par[b, i] in on and not twin and rng.random() < 0.8 and at < len(plain[b][0]):
                    tok_h[b, i] = plain[b][0][at]
                    on.add(i)
        tok, parent, depth, cnt = (torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in (tok_h, par, dep, cnt_h))
        mask, _ = pct.tree_ancestor_mask(parent, cnt)
        target = forward(tok, depth, cnt, mask)
        ver = pct.tree_verify_accept(tok, parent, cnt, target, max_depth=D)
        ctx2, st = pct.kv_commit(k, v, table, ctx, cnt, ver.accept_len, ver.accept_path)
        st2 = pct.kv_pages_resize(ctx2, table, held, free, nfree, page)
        assert (host(st) == 0).all() and (host(st2) == 0).all()
        for b in range(B):
            a = int(ver.accept_len[b])
            seqs[b] += [int(tok_h[b, i]) for i in host(ver.accept_path)[b, :a]] + [int(ver.correction[b])]
            accepted += a
        ctx = ctx2
        assert host(held).tolist() == [-(-int(c) // page) for c in ctx] and int(nfree) + int(held.sum()) == n_pages
    assert accepted > 0
    for s, (p, _) in zip(seqs, plain):
        m = min(len(s), len(p))
        assert s[:m] == p[:m]
