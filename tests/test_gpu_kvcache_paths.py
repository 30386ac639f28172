"""Tree attention on each of its kernels and row groups: bad pages, the calls that the tcgen05
kernel cannot take, and optional arguments. Bounds are those of ``test_gpu_kvcache``."""
import numpy as np
import pytest
import torch

import speculative_decoding_draft_07_b200 as pct
from gpu_util import host
from oracle import kvcache as okv
from test_gpu_kvcache import DEV, _case, _check, _run

pytestmark = pytest.mark.gpu

# query heads over 2 kv heads: 32 rows a head (warp-level kernels), 80 (tcgen05: one row tile, its
# key tiles dealt to two streams), 280 (two row tiles a block, and a last one alone)
ROWS = [(8, 8), (20, 8), (70, 8)]


def _bad_pages(table, ctx, counts, n_pages, page):
    """Requests in turn: a page inside a key tile, all pages of a tile, the last page (nodes), every
    other page, all pages, none."""
    for b in range(table.shape[0]):
        used = -(-(ctx[b] + counts[b]) // page)
        cols = {0: [1], 1: range(64 // page, 128 // page), 2: [used - 1], 3: range(0, used, 2),
                4: range(used), 5: []}[b % 6]
        for i, c in enumerate(cols):
            table[b, c] = (10 ** 6, -1, n_pages, -(1 << 31), (1 << 31) - 1)[(b + i) % 5]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 32), (200, 8)])
@pytest.mark.parametrize("n,hq", ROWS)
def test_bad_pages(n, hq, d, page, dtype):
    g, table, ctx, counts, m = _case(40, dtype=dtype, n=n, hq=hq, d=d, page=page, ctx=(70, 200, 130, 257, 90, 150))
    _bad_pages(table, ctx, counts, g["k"].shape[0], page)
    g["table"].copy_(torch.from_numpy(table))
    ref = _check(_run(g), g, table, ctx, counts, m)
    assert ref.status.tolist() == [okv.BAD_PAGE] * 5 + [0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq", ROWS)
def test_bad_pages_in_later_pieces(n, hq, dtype):
    """One request cut over many blocks: bad pages that only some pieces meet."""
    g, table, ctx, counts, m = _case(41, dtype=dtype, n=n, hq=hq, d=128, page=16, ctx=(3000,))
    table[0, 100:120:3] = -1
    table[0, 150] = 10 ** 6
    g["table"].copy_(torch.from_numpy(table))
    ref = _check(_run(g), g, table, ctx, counts, m)
    assert ref.status.tolist() == [okv.BAD_PAGE]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,hq,hkv", [(33, 2, 2), (16, 8, 2), (50, 8, 2)])
@pytest.mark.parametrize("page,scale", [(5, None), (7, None), (16, -0.7), (16, 0.0)])
def test_bf16_calls_the_tcgen05_kernel_cannot_take(page, scale, n, hq, hkv, d):
    """33, 64 and 200 rows a kv head with pages that are no multiple of 8 tokens or a scale that is
    not positive."""
    c = _case(42, n=n, hq=hq, hkv=hkv, d=d, page=page, ctx=(150, 0, 63))
    _check(_run(c[0], scale=scale), *c, scale=scale)


@pytest.mark.parametrize("how", ["heads", "nodes", "batch", "transposed"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq", ROWS)
def test_query_strides(n, hq, dtype, how):
    """Queries broadcast along an axis (stride 0, which no tensor map takes) or laid out head first."""
    c = _case(43, dtype=dtype, n=n, hq=hq, d=128, ctx=(100, 31))
    g = c[0]
    q = g["q"]
    if how == "transposed":
        g["q"] = q.transpose(1, 2).contiguous().transpose(1, 2)
    else:
        axis = {"batch": 0, "nodes": 1, "heads": 2}[how]
        g["q"] = q.narrow(axis, 0, 1).expand_as(q)
        assert g["q"].stride(axis) == 0
    assert not g["q"].is_contiguous()
    _check(_run(g), *c)


@pytest.mark.parametrize("axis", [0, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq", ROWS)
def test_broadcast_caches_are_read(n, hq, dtype, axis):
    """A cache expanded over its heads or pages (read only): one kv head, or one page, for all."""
    c = _case(44, dtype=dtype, n=n, hq=hq, d=64, ctx=(40, 77))
    g = c[0]
    for x in ("k", "v"):
        g[x] = g[x].narrow(axis, 0, 1).expand_as(g[x])
    _check(_run(g), *c)
    with pytest.raises(pct.PctError):
        pct.kv_append(g["k"][:1, :1], g["v"][:1, :1], torch.zeros((1, 1), dtype=torch.int64, device=DEV), g["k"], g["v"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq,page", [r + (16,) for r in ROWS] + [(70, 8, 5)])
def test_no_count_and_no_lse(n, hq, page, dtype):
    c = _case(45, dtype=dtype, n=n, hq=hq, d=128, page=page, ctx=(100, 0, 31))
    g = c[0]
    want = _run(g)
    _check(want, *c)
    r = pct.tree_attention(g["q"], g["k"], g["v"], g["table"], g["ctx"], None, mask=g["mask"])
    out = pct.AttnOut(torch.full_like(want.out, 7), None, torch.full_like(want.status, 7))
    s = _run(g, out=out)
    torch.cuda.synchronize()
    assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse) and not host(r.status).any()
    assert s.lse is None and torch.equal(s.out, want.out) and not host(s.status).any()


def test_workspaces_of_two_captured_graphs_may_be_one():
    """Two captured calls over one workspace, replayed one after the other on a stream."""
    cs = [_case(46 + i, n=20, hq=8, d=128, ctx=(900 * i + 30, 5)) for i in range(2)]
    need = max(pct.tree_attention_workspace(c[0]["k"], c[0]["v"], c[0]["table"].shape[1], 2, 20, 8) for c in cs)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    want = [_run(c[0]).out.clone() for c in cs]
    graphs = []
    for c in cs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            r = _run(c[0], workspace=ws)
        graphs.append((gr, r))
    for _ in range(3):
        for gr, r in graphs:
            r.out.zero_()
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(r.out, w) for (_, r), w in zip(graphs, want))


def test_new_lengths_over_old_ones_are_refused():
    """kv_commit with new lengths shifted by a request over the old ones."""
    g, table, ctx, counts, _ = _case(48, n=4, ctx=(5, 9))
    buf = torch.zeros(3, dtype=torch.int64, device=DEV)
    one = torch.ones(2, dtype=torch.int32, device=DEV)
    path = torch.ones((2, 2), dtype=torch.int32, device=DEV)
    with pytest.raises(pct.PctError):
        pct.kv_commit(g["k"], g["v"], g["table"], buf[:2], g["count"], one, path, new_len=buf[1:])
    np.testing.assert_array_equal(host(buf), 0)
