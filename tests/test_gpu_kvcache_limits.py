"""The paged-cache calls at the ends of their ranges, and a whole round as one captured graph whose
lengths change between replays. Rows are compared with 64-bit attention of that row alone, within the
bound of ``test_gpu_kvcache``."""
import pytest
import torch

import speculative_decoding_draft_07_b200 as pct
from test_gpu_kvcache import DEV, DT

pytestmark = pytest.mark.gpu


def _lengths(batch, hi):
    return [(b * 7919) % hi for b in range(batch)]


# (requests, nodes, query heads, kv heads, head_dim, page, context lengths, rows looked at)
LIMITS = {
    "3 million tokens": (1, 1, 2, 1, 8, 64, [3000000], [(0, 0)]),
    "2 million tokens, many rows": (1, 40, 2, 1, 8, 64, [2000001], [(0, 0), (0, 39)]),
    "most requests": (65535, 1, 2, 1, 8, 16, _lengths(65535, 16), [(0, 0), (65534, 0), (777, 0)]),
    "many requests, many rows": (20000, 40, 1, 1, 16, 16, _lengths(20000, 70), [(0, 39), (19999, 0), (777, 20)]),
    "most nodes": (1, 65536, 1, 1, 16, 128, [5], [(0, 0), (0, 65535), (0, 30000)]),
    "most heads, largest group": (2, 3, 65536, 1024, 8, 16, [20, 5], [(0, 2), (1, 0)]),
    "largest page": (2, 5, 4, 2, 64, 65536, [70000, 5], [(0, 4), (1, 0)]),
    "largest page, many rows": (2, 50, 4, 2, 64, 65536, [70000, 5], [(0, 49), (1, 0)]),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", LIMITS)
def test_attention_at_its_limits(name, dtype):
    B, n, hq, hkv, d, page, ctx, rows = LIMITS[name]
    torch.manual_seed(1)
    width = -(-(max(ctx) + n) // page)
    k, v = (torch.randn((B * width, page, hkv, d), device=DEV).to(DT[dtype]) for _ in range(2))
    table = torch.randperm(B * width, device=DEV).view(B, width).to(torch.int32)
    q = torch.randn((B, n, hq, d), device=DEV).to(DT[dtype])
    r = pct.tree_attention(q, k, v, table, torch.tensor(ctx, device=DEV))
    torch.cuda.synchronize()
    assert not r.status.any()
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for b, i in rows:
        T = ctx[b] + i + 1
        kk, vv = (x[table[b].long()].view(-1, hkv, d)[:T].double() for x in (k, v))
        qq = q[b, i].double().view(hkv, hq // hkv, d) * d ** -0.5
        s = torch.einsum("hgd,thd->hgt", qq, kk)
        w = torch.softmax(s, -1)
        want, weight = (torch.einsum("hgt,thd->hgd", w, x).reshape(hq, d) for x in (vv, vv.abs()))
        size = torch.einsum("hgd,thd->hgt", qq.abs(), kk.abs()).amax(-1).view(hq, 1)
        rel = 2.0 ** -24 * (2 * d * size + T / 32 + 256)
        err = (r.out[b, i].double() - want).abs()
        assert (err <= (2 * rel + u) * weight + u * want.abs()).all(), (b, i)
        lse = torch.logsumexp(s, -1).view(hq, 1)
        assert ((r.lse[b, i].double().view(hq, 1) - lse).abs() <= rel + 2.0 ** -22 * lse.abs()).all(), (b, i)


def test_slots_rows_and_paths_at_their_limits():
    """2^20 tokens a request, a path of 4096 nodes."""
    B, n, page, depth = 3, 1 << 20, 16, 4096
    width = (n + 100) // page + 1
    n_pages = B * width
    torch.manual_seed(2)
    table = torch.randperm(n_pages, device=DEV).view(B, width).to(torch.int32)
    ctx, cnt = torch.tensor([0, 7, 99], device=DEV), torch.tensor([n, n - 5, 1], dtype=torch.int32, device=DEV)
    place = lambda b, t: table[b].long()[t // page] * page + t % page        # noqa: E731
    slot, pos, st = pct.kv_tree_slots(ctx, cnt, table, n, page, n_pages)
    for b in range(B):
        i = torch.arange(int(cnt[b]), device=DEV)
        assert torch.equal(slot[b, : i.numel()], place(b, ctx[b] + i)) and (slot[b, i.numel():] == -1).all()
        assert torch.equal(pos[b, : i.numel()], ctx[b] + i) and (pos[b, i.numel():] == -1).all()
    new = torch.randn((2, B, n, 1, 8), device=DEV).bfloat16()
    k, v = torch.zeros((2, n_pages, page, 1, 8), dtype=torch.bfloat16, device=DEV)
    st2 = pct.kv_append(new[0], new[1], slot, k, v)
    assert not st.any() and not st2.any()
    for b in range(B):
        m = int(cnt[b])
        assert torch.equal(k.view(-1, 8)[slot[b, :m]], new[0, b, :m, 0]) and torch.equal(v.view(-1, 8)[slot[b, :m]], new[1, b, :m, 0])
    path = (torch.arange(1, depth + 1, device=DEV) * 3).to(torch.int32).repeat(B, 1)
    alen = torch.tensor([depth, 1000, 0], dtype=torch.int32, device=DEV)
    was = k.clone()
    new_len, st = pct.kv_commit(k, v, table, ctx, cnt, alen, path)
    assert not st.any() and new_len.tolist() == [4097, 1008, 100]
    for b in range(2):
        i = torch.arange(int(alen[b]), device=DEV)
        assert torch.equal(k.view(-1, 8)[place(b, ctx[b] + 1 + i)], was.view(-1, 8)[place(b, ctx[b] + path[b, i].long())])


def test_pages_of_the_most_requests():
    B, width, page = 65535, 40, 16
    table, held = torch.full((B, width), -1, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    free = torch.arange(B * width, dtype=torch.int32, device=DEV)
    nfree = torch.tensor([B * width], dtype=torch.int32, device=DEV)
    torch.manual_seed(3)
    length = torch.randint(0, width * page + 1, (B,), device=DEV)
    st = pct.kv_pages_resize(length, table, held, free, nfree, page)
    assert not st.any() and torch.equal(held.long(), (length + page - 1) // page)
    got = table[table >= 0]
    assert got.unique().numel() == got.numel() == int(held.sum()) == B * width - int(nfree)
    st = pct.kv_pages_resize(torch.zeros_like(length), table, held, free, nfree, page)
    assert not st.any() and int(nfree) == B * width and (table == -1).all()
    assert torch.equal(free, torch.arange(B * width, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("n,hq", [(4, 4), (24, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_round_captured_once_and_replayed(dtype, n, hq):
    """Pages, slots, append, attention, commit and pages again in one graph; the lengths move on from
    replay to replay. State and outputs are those of the same calls made one by one."""
    B, hkv, d, page, width, depth = 4, 2, 64, 8, 40, 3
    torch.manual_seed(4)
    n_pages = B * width

    def state():
        return dict(ctx=torch.tensor([5, 0, 60, 17], device=DEV), table=torch.full((B, width), -1, dtype=torch.int32, device=DEV),
                    held=torch.zeros(B, dtype=torch.int32, device=DEV), free=torch.arange(n_pages, dtype=torch.int32, device=DEV),
                    nfree=torch.tensor([n_pages], dtype=torch.int32, device=DEV),
                    k=torch.zeros((2, n_pages, page, hkv, d), dtype=DT[dtype], device=DEV),
                    v=torch.zeros((2, n_pages, page, hkv, d), dtype=DT[dtype], device=DEV))

    # what changes from round to round, in the buffers that the graph reads
    buf = dict(q=torch.empty((B, n, hq, d), dtype=DT[dtype], device=DEV), kn=torch.empty((B, n, hkv, d), dtype=DT[dtype], device=DEV),
               vn=torch.empty((B, n, hkv, d), dtype=DT[dtype], device=DEV), parent=torch.zeros((B, n), dtype=torch.int32, device=DEV),
               cnt=torch.ones(B, dtype=torch.int32, device=DEV), alen=torch.zeros(B, dtype=torch.int32, device=DEV),
               path=torch.zeros((B, depth), dtype=torch.int32, device=DEV))

    def fill(r):
        g = torch.Generator().manual_seed(100 + r)
        for x in ("q", "kn", "vn"):
            buf[x].copy_(torch.randn(buf[x].shape, generator=g))
        par = (torch.rand((B, n), generator=g) * torch.arange(n)).long()
        par[:, 0] = -1
        cnt = torch.randint(1, n + 1, (B,), generator=g)
        path = torch.full((B, depth), -1)
        alen = torch.zeros(B, dtype=torch.long)
        for b in range(B):
            alen[b] = min(int(torch.randint(0, depth + 1, (1,), generator=g)), int(cnt[b]) - 1)
            path[b, : alen[b]] = (torch.randperm(int(cnt[b]) - 1, generator=g)[: alen[b]] + 1).sort().values
        for x, t in (("parent", par), ("cnt", cnt), ("alen", alen), ("path", path)):
            buf[x].copy_(t)

    def round_(s):
        st = [pct.kv_pages_resize(s["ctx"], s["table"], s["held"], s["free"], s["nfree"], page, count=buf["cnt"])]
        slot, pos, x = pct.kv_tree_slots(s["ctx"], buf["cnt"], s["table"], n, page, n_pages)
        st.append(x)
        mask, _ = pct.tree_ancestor_mask(buf["parent"], buf["cnt"])
        out = []
        for layer in range(2):
            st.append(pct.kv_append(buf["kn"], buf["vn"], slot, s["k"][layer], s["v"][layer]))
            out.append(pct.tree_attention(buf["q"], s["k"][layer], s["v"][layer], s["table"], s["ctx"], buf["cnt"], mask=mask))
            st.append(out[-1].status)
        new_len, x = pct.kv_commit(s["k"], s["v"], s["table"], s["ctx"], buf["cnt"], buf["alen"], buf["path"])
        st += [x, pct.kv_pages_resize(new_len, s["table"], s["held"], s["free"], s["nfree"], page)]
        s["ctx"].copy_(new_len)
        return [o.out for o in out] + [o.lse for o in out], torch.cat(st)

    a, b = state(), state()
    for s in (a, b):                                     # pages of the contexts the requests start with
        pct.kv_pages_resize(s["ctx"], s["table"], s["held"], s["free"], s["nfree"], page)
    fill(0)
    spare = state()
    round_(spare)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, gst = round_(b)
    for r in range(8):
        fill(r)
        want, wst = round_(a)
        g.replay()
        torch.cuda.synchronize()
        assert not wst.any() and not gst.any()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        for key in a:
            assert torch.equal(a[key], b[key]), key
