"""The paged key-value operators around draft-tree verification, as calls to measure.

Four operators, each in its plain form (elementary torch operations in 32 bits, ``own = False``) and
as the calls a user makes of the library (``own = True``):

* ``pages``  -- one round's page bookkeeping on the GPU: the block tables grow to hold the tree's
  nodes, slots and positions of the nodes are written, and after the accept walk the tables shrink
  to the accepted length (``kv_pages_resize``, ``kv_tree_slots``, ``kv_pages_resize``).
* ``append`` -- the nodes' new K and V rows go into the pages at their slots (``kv_append``).
* ``attend`` -- attention of the tree's nodes over the paged cache with the ancestor bitmask, or a
  causal chain without it; one node per request is the decode step (``tree_attention``).
* ``commit`` -- the accepted path's K and V rows move behind the context in every layer
  (``kv_commit``).
"""
import random

import torch

own = False


def listed():
    return [
        # one round of 8 requests with 32-node trees: bookkeeping is pure latency
        dict(name="pages b8 n32", op="pages", batch=8, n=32, page=16, ctx_lo=40, ctx_hi=900, depth=7),
        # a full serving batch with uneven contexts
        dict(name="pages b1000 n64", op="pages", batch=1000, n=64, page=32, ctx_lo=1, ctx_hi=6000, depth=15),
        # a 7-token chain of one request, fp32 cache
        dict(name="append b1 n7 f32", op="append", batch=1, n=7, hkv=4, d=64, page=16, ctx_lo=99, ctx_hi=99, dtype="f32", fused=False),
        # prompt chunks of 32 requests, K and V as slices of a fused projection
        dict(name="append b32 n1000", op="append", batch=32, n=1000, hkv=8, d=128, page=64, ctx_lo=0, ctx_hi=500, dtype="bf16", fused=True),
        # decode of one short request: the smallest call
        dict(name="decode b1 t500", op="attend", batch=1, n=1, hq=32, hkv=8, d=128, page=16, ctx_lo=500, ctx_hi=500, dtype="bf16", tree=False),
        # decode of 32 requests over long uneven contexts: the cache's bytes
        dict(name="decode b32 t32768", op="attend", batch=32, n=1, hq=32, hkv=8, d=128, page=64, ctx_lo=500, ctx_hi=32768, dtype="bf16", tree=False),
        # fp32 tree of the tiny configuration, odd page size, every head its own K and V
        dict(name="tree b4 n32 f32", op="attend", batch=4, n=32, hq=8, hkv=8, d=64, page=24, ctx_lo=301, ctx_hi=1777, dtype="f32", tree=True),
        # one request, 64 nodes, a long context
        dict(name="tree b1 n64 t8000", op="attend", batch=1, n=64, hq=32, hkv=8, d=128, page=32, ctx_lo=8000, ctx_hi=8000, dtype="bf16", tree=True),
        # 32 requests, 128 nodes
        dict(name="tree b32 n128", op="attend", batch=32, n=128, hq=16, hkv=4, d=128, page=16, ctx_lo=200, ctx_hi=2500, dtype="bf16", tree=True),
        # 64 requests, 256 nodes: the full round, the largest call
        dict(name="tree b64 n256", op="attend", batch=64, n=256, hq=32, hkv=8, d=128, page=64, ctx_lo=512, ctx_hi=4096, dtype="bf16", tree=True),
        # one request's accepted path in 4 layers
        dict(name="commit b1 l4", op="commit", batch=1, n=32, hkv=4, d=64, page=16, ctx_lo=99, ctx_hi=99, dtype="bf16", layers=4, depth=7),
        # the full round's accepted paths in 16 layers
        dict(name="commit b64 l16", op="commit", batch=64, n=256, hkv=8, d=128, page=64, ctx_lo=50, ctx_hi=500, dtype="bf16", layers=16, depth=15),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["pages", "append", "attend", "attend", "attend", "attend", "commit"])
    if op == "pages":
        hi = _log(rng, 20, 8000)
        return dict(op=op, batch=_log(rng, 1, 1000), n=_log(rng, 1, 300), page=rng.choice([8, 16, 24, 32, 64, 128]),
                    ctx_lo=rng.randrange(hi), ctx_hi=hi, depth=rng.randint(1, 15))
    hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 64, 96, 128, 128, 128, 256])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "append":
        batch = _log(rng, 1, 64)
        return dict(op=op, batch=batch, n=_log(rng, 1, 30000 // batch), hkv=hkv, d=d, page=page, ctx_lo=0, ctx_hi=_log(rng, 1, 1000),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), fused=rng.random() < 0.5)
    if op == "commit":
        batch = _log(rng, 1, 64)
        return dict(op=op, batch=batch, n=_log(rng, 2, 256), hkv=min(hkv, 8), d=min(d, 128), page=page, ctx_lo=0,
                    ctx_hi=_log(rng, 1, 500), dtype=rng.choice(["bf16", "bf16", "f32"]), layers=_log(rng, 1, 8), depth=rng.randint(1, 15))
    dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
    g = rng.choice([1, 2, 4, 7, 8])
    kind = rng.choice(["decode", "tree", "tree", "chunk"])
    batch = _log(rng, 1, 64)
    n = 1 if kind == "decode" else _log(rng, 2, 256) if kind == "tree" else _log(rng, 64, 1500)
    # the largest listed case bounds a draw: the cache's bytes and the products
    most = min(32768, 500000 * 8 * 128 // (batch * hkv * d), 4 * 10**10 // (batch * n * g * hkv * d))
    if dtype == "f32":
        most = min(most, 4 * 10**9 // (batch * n * g * hkv * d))
    if most < 64:
        batch, most = 1, max(64, min(32768, 4 * 10**9 // (n * g * hkv * d)))
    hi = _log(rng, 32, most)
    return dict(op=op, batch=batch, n=n, hq=g * hkv, hkv=hkv, d=d, page=page, ctx_lo=rng.randrange(hi), ctx_hi=hi, dtype=dtype, tree=kind == "tree")


# ---- sizes of a case, from the case alone ---------------------------------------------------------
def _sizes(case):
    """ctx[b] spread over [ctx_lo, ctx_hi]; count[b] from n down to about three quarters of it."""
    B, n, lo, hi = case["batch"], case["n"], case["ctx_lo"], case["ctx_hi"]
    ctx = [lo + int((hi - lo) * ((b * 0.6180339887 + 1.0) % 1.0 if B > 1 else 1.0)) for b in range(B)]
    ctx[0] = hi
    count = [n - (b * 7) % (n // 4 + 1) for b in range(B)]
    return ctx, count


def _pages(tokens, page):
    return -(-tokens // page)


def _paths(case):
    """Accepted path lengths, 0 up to depth (and up to the nodes there are)."""
    _, count = _sizes(case)
    return [min((b * 5 + 2) % (case["depth"] + 1), max(0, count[b] // 2 - 1)) for b in range(case["batch"])]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ---- inputs ---------------------------------------------------------------------------------------
def _table(case, gen, spare):
    """Block tables of ctx + count tokens per request over shuffled pages."""
    ctx, count = _sizes(case)
    need = [_pages(c + m, case["page"]) for c, m in zip(ctx, count)]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64)
    width = max(need)
    need_t = torch.tensor(need, device="cuda")
    start = torch.cumsum(need_t, 0) - need_t
    col = torch.arange(width, device="cuda")
    table = order[(start[:, None] + col).clamp(max=total - 1)]
    table = torch.where(col < need_t[:, None], table, torch.full_like(table, -1))
    return ctx, count, table.to(torch.int32).contiguous(), order, total


def _tree(B, n, gen):
    """parent [B][n]: nodes in breadth-first order, depth of about 3 log2 n at most."""
    u = torch.rand((B, n), generator=gen, device="cuda").sort(dim=1).values * 0.75
    p = (u * torch.arange(n, device="cuda")).floor().to(torch.int64)
    p[:, 0] = -1
    return p


def _ancestors(parent):
    """Bitmask words [B][n][ceil(n / 32)] of self and ancestors."""
    B, n = parent.shape
    bits = torch.zeros((B, n, _pages(n, 32) * 32), dtype=torch.bool, device="cuda")
    at = torch.arange(n, device="cuda").expand(B, n).clone()
    while bool((at >= 0).any()):
        bits.scatter_(2, at.clamp(min=0)[..., None], torch.ones((B, n, 1), dtype=torch.bool, device="cuda") & (at >= 0)[..., None] | bits.gather(2, at.clamp(min=0)[..., None]))
        at = torch.where(at >= 0, parent.gather(1, at.clamp(min=0)), at)
    w = (bits.view(B, n, -1, 32).to(torch.int64) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, B, n, page = case["op"], case["batch"], case["n"], case["page"]
    st = dict(case)
    if op == "pages":
        ctx, count, table, order, total = _table(case, gen, spare=B)
        acc = _paths(case)
        held = [_pages(c, page) for c in ctx]
        held_t = torch.tensor(held, device="cuda")
        keep = torch.arange(table.shape[1], device="cuda") < held_t[:, None]
        taken = torch.zeros(total, dtype=torch.bool, device="cuda")
        taken[table[keep].long()] = True
        rest = order[~taken[order]]
        free = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        free[: rest.numel()] = rest.to(torch.int32)
        parent = _tree(B, n, gen)
        depth, at = torch.zeros((B, n), dtype=torch.int32, device="cuda"), parent.clone()
        while bool((at >= 0).any()):
            depth += (at >= 0).to(torch.int32)
            at = torch.where(at >= 0, parent.gather(1, at.clamp(min=0)), at)
        st.update(table=torch.where(keep, table, torch.full_like(table, -1)).contiguous(), held=held_t.to(torch.int32), free=free,
                  free_count=torch.tensor([rest.numel()], dtype=torch.int32, device="cuda"),
                  ctx=torch.tensor(ctx, dtype=torch.int64, device="cuda"), count=torch.tensor(count, dtype=torch.int32, device="cuda"),
                  depths=depth, kept=torch.tensor([c + 1 + a for c, a in zip(ctx, acc)], dtype=torch.int64, device="cuda"), total=total)
        return st
    hkv, d, dt = case["hkv"], case["d"], _dtype(case)
    ctx, count, table, order, total = _table(case, gen, spare=3)
    layers = case.get("layers", 1)
    shape = (layers, total, page, hkv, d) if op == "commit" else (total, page, hkv, d)
    st.update(table=table, total=total, ctx=torch.tensor(ctx, dtype=torch.int64, device="cuda"), count=torch.tensor(count, dtype=torch.int32, device="cuda"),
              k=torch.empty(shape, dtype=dt, device="cuda").normal_(generator=gen), v=torch.empty(shape, dtype=dt, device="cuda").normal_(generator=gen))
    node = torch.arange(n, device="cuda")
    if op == "append":
        if case["fused"]:  # K and V as slices of one projection's output, beside 4 hkv query heads
            qkv = torch.empty((B, n, 6 * hkv, d), dtype=dt, device="cuda").normal_(generator=gen)
            st.update(k_new=qkv[:, :, 4 * hkv: 5 * hkv], v_new=qkv[:, :, 5 * hkv:])
        else:
            st.update(k_new=torch.empty((B, n, hkv, d), dtype=dt, device="cuda").normal_(generator=gen),
                      v_new=torch.empty((B, n, hkv, d), dtype=dt, device="cuda").normal_(generator=gen))
        t = st["ctx"][:, None] + node
        p = table.long().gather(1, (t // page).clamp(max=table.shape[1] - 1))
        st["slot"] = torch.where(node < st["count"][:, None], p * page + t % page, torch.full_like(t, -1)).contiguous()
    elif op == "attend":
        # queries of twice the keys' scale: a softmax with a few large weights, as trained heads have
        st["q"] = (torch.randn((B, n, case["hq"], d), generator=gen, device="cuda") * 2).to(dt)
        st["mask"] = _ancestors(_tree(B, n, gen)) if case["tree"] else None
    else:
        acc = _paths(case)
        path = torch.full((B, case["depth"]), -1, dtype=torch.int32)
        rng = random.Random(int(seed))
        for b, a in enumerate(acc):
            path[b, :a] = torch.tensor(sorted(rng.sample(range(1, count[b]), a)), dtype=torch.int32)
        st.update(accept_len=torch.tensor(acc, dtype=torch.int32, device="cuda"), accept_path=path.cuda())
    return st


# ---- the plain forms ------------------------------------------------------------------------------
def _plain_resize(length, table, held, free, free_count, page):
    """Tables to ceil(length / page) pages: what is too much goes back to the free list first, then
    requests take from its top in their order. In place; no request exceeds what there is."""
    B, width = table.shape
    want = (length + page - 1) // page
    held64 = held.long()
    col = torch.arange(width, device=table.device)
    back = (col >= want[:, None]) & (col < held64[:, None])
    u = torch.cumsum(back.reshape(-1).long(), 0).view(B, width) - 1
    ret = back.sum()
    spot = free_count.long() + ret - 1 - u
    last = free.numel()
    padded = torch.cat([free, free.new_zeros(1)])
    padded.scatter_(0, torch.where(back, spot, torch.full_like(spot, last)).reshape(-1), table.reshape(-1))
    have = free_count.long() + ret
    take = (col >= held64[:, None]) & (col < want[:, None])
    t = torch.cumsum(take.reshape(-1).long(), 0).view(B, width) - 1
    ends = torch.cumsum((want - held64).clamp(min=0), 0)
    take &= (ends <= have)[:, None]
    page_id = padded[torch.where(take, have - 1 - t, torch.full_like(t, last)).clamp(min=0)]
    table.copy_(torch.where(take, page_id, torch.where(back, torch.full_like(table, -1), table)))
    free.copy_(padded[:last])
    held.copy_((held64 + take.sum(1) - back.sum(1)).to(torch.int32))
    free_count.copy_((have - take.sum()).to(torch.int32).view(1))


def _plain_slots(ctx, count, depth, table, page):
    node = torch.arange(depth.shape[1], device=table.device)
    t = ctx[:, None] + node
    p = table.long().gather(1, (t // page).clamp(max=table.shape[1] - 1))
    live = node < count[:, None]
    none = torch.full_like(t, -1)
    return torch.where(live, p * page + t % page, none), torch.where(live, ctx[:, None] + depth, none)


def _plain_append(k_new, v_new, slot, k, v):
    page = k.shape[1]
    b, i = torch.nonzero(slot >= 0, as_tuple=True)
    s = slot[b, i]
    k[s // page, s % page] = k_new[b, i]
    v[s // page, s % page] = v_new[b, i]


def _plain_attend(q, k, v, table, ctx, count, mask):
    B, n, hq, d = q.shape
    page, hkv = k.shape[1], k.shape[2]
    T = table.shape[1] * page
    keys = k[table.long().clamp(min=0)].reshape(B, T, hkv, d).permute(0, 2, 1, 3).float()
    vals = v[table.long().clamp(min=0)].reshape(B, T, hkv, d).permute(0, 2, 1, 3).float()
    j = torch.arange(T, device=q.device) - ctx[:, None]                     # node of each cache position
    i = torch.arange(n, device=q.device)
    seen = (j[:, None, :] <= i[:, None]) & (j[:, None, :] < count[:, None, None])
    if mask is not None:
        at = j.clamp(0, n - 1)
        word = mask.gather(2, (at // 32)[:, None, :].expand(B, n, T))
        seen &= (j[:, None, :] < 0) | (((word >> (at % 32)[:, None, :].int()) & 1) != 0)
    seen &= (i < count[:, None])[:, :, None]
    vals = vals * (j < count[:, None])[:, None, :, None]
    g = hq // hkv
    rows = q.float().view(B, n, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * g, d)
    s = torch.matmul(rows, keys.transpose(2, 3)).view(B, hkv, n, g, T) * d ** -0.5
    s = torch.where(seen[:, None, :, None, :], s, torch.full((), -float("inf"), device=q.device))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -float("inf"), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    del s
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, hkv, n * g, T), vals).view(B, hkv, n, g, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = m + torch.log(l)
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, hq, d).to(q.dtype), lse.permute(0, 2, 1, 3, 4).reshape(B, n, hq)


def _plain_commit(k, v, table, ctx, accept_len, accept_path):
    page = k.shape[2]
    step = torch.arange(accept_path.shape[1], device=k.device)
    b, i = torch.nonzero(step < accept_len[:, None], as_tuple=True)
    src, dst = ctx[b] + accept_path[b, i], ctx[b] + 1 + i
    sp, dp = table[b, src // page].long(), table[b, dst // page].long()
    k[:, dp, dst % page] = k[:, sp, src % page]
    v[:, dp, dst % page] = v[:, sp, src % page]
    return ctx + 1 + accept_len


def run(st):
    op = st["op"]
    if own:
        import speculative_decoding_draft_07_b200 as pct
        if op == "pages":
            pct.kv_pages_resize(st["ctx"], st["table"], st["held"], st["free"], st["free_count"], st["page"], count=st["count"])
            slot, pos, _ = pct.kv_tree_slots(st["ctx"], st["count"], st["table"], st["n"], st["page"], st["total"], depth=st["depths"])
            pct.kv_pages_resize(st["kept"], st["table"], st["held"], st["free"], st["free_count"], st["page"])
            return dict(slot=slot, pos=pos, table=st["table"], held=st["held"], free=st["free"], free_count=st["free_count"])
        if op == "append":
            pct.kv_append(st["k_new"], st["v_new"], st["slot"], st["k"], st["v"])
            return dict(k=st["k"], v=st["v"])
        if op == "attend":
            r = pct.tree_attention(st["q"], st["k"], st["v"], st["table"], st["ctx"], st["count"], mask=st["mask"])
            return dict(out=r.out, lse=r.lse)
        new_len, _ = pct.kv_commit(st["k"], st["v"], st["table"], st["ctx"], st["count"], st["accept_len"], st["accept_path"])
        return dict(k=st["k"], v=st["v"], new_len=new_len)
    if op == "pages":
        _plain_resize(st["ctx"] + st["count"], st["table"], st["held"], st["free"], st["free_count"], st["page"])
        slot, pos = _plain_slots(st["ctx"], st["count"], st["depths"], st["table"], st["page"])
        _plain_resize(st["kept"], st["table"], st["held"], st["free"], st["free_count"], st["page"])
        return dict(slot=slot, pos=pos, table=st["table"], held=st["held"], free=st["free"], free_count=st["free_count"])
    if op == "append":
        _plain_append(st["k_new"], st["v_new"], st["slot"], st["k"], st["v"])
        return dict(k=st["k"], v=st["v"])
    if op == "attend":
        out, lse = _plain_attend(st["q"], st["k"], st["v"], st["table"], st["ctx"], st["count"], st["mask"])
        return dict(out=out, lse=lse)
    new_len = _plain_commit(st["k"], st["v"], st["table"], st["ctx"], st["accept_len"], st["accept_path"])
    return dict(k=st["k"], v=st["v"], new_len=new_len)


# ---- what a pass cannot do without ----------------------------------------------------------------
def work(case):
    op, B, n, page = case["op"], case["batch"], case["n"], case["page"]
    ctx, count = _sizes(case)
    if op == "pages":
        moved = sum(_pages(c + m, page) - _pages(c + 1 + a, page) for c, m, a in zip(ctx, count, _paths(case)))
        # a moved page is an entry read and one written each way; slots and positions 8 bytes each, the depth 4
        return dict(bytes=20 * B * n + 4 * sum(_pages(c + m, page) - c // page for c, m in zip(ctx, count)) + 24 * moved + 36 * B, flops=0)
    e = 2 if case["dtype"] == "bf16" else 4
    row = case["hkv"] * case["d"] * e
    if op == "append":
        return dict(bytes=4 * row * sum(count) + 8 * B * n, flops=0)
    if op == "commit":
        acc = _paths(case)
        return dict(bytes=4 * row * case["layers"] * sum(acc) + 4 * sum(acc) + 28 * B, flops=0)
    hq, d = case["hq"], case["d"]
    tokens = sum(ctx) + sum(count)
    nbytes = 2 * row * tokens + sum(count) * hq * d * e + B * n * hq * (d * e + 4) + 4 * sum(_pages(c + m, page) for c, m in zip(ctx, count)) + 12 * B
    pairs = sum(c * m + (m * (m + 1) // 2 if not case["tree"] else m) for c, m in zip(ctx, count))
    if case["tree"]:
        nbytes += B * n * _pages(n, 32) * 4
    return dict(bytes=nbytes, flops=4 * d * hq * pairs)


# ---- the definitions in 64 bits -------------------------------------------------------------------
def exact(case, seed):
    """Request by request from the definitions, in 64 bits where something is computed."""
    st = prepare(case, seed)
    op, page = case["op"], case["page"]
    if op == "pages":
        return None
    ctx, count = st["ctx"].tolist(), st["count"].tolist()
    if op == "append":
        k, v, slot = st["k"].clone(), st["v"].clone(), st["slot"]
        kf, vf = k.reshape((-1,) + tuple(k.shape[2:])), v.reshape((-1,) + tuple(v.shape[2:]))
        for b in range(case["batch"]):
            kf.index_copy_(0, slot[b, : count[b]], st["k_new"][b, : count[b]])
            vf.index_copy_(0, slot[b, : count[b]], st["v_new"][b, : count[b]])
        return dict(k=kf.view_as(k), v=vf.view_as(v))
    if op == "commit":
        k, v = st["k"].clone(), st["v"].clone()
        alen = st["accept_len"].tolist()
        for b in range(case["batch"]):
            tab = st["table"][b].tolist()
            for i, node in enumerate(st["accept_path"][b, : alen[b]].tolist()):
                s, t = ctx[b] + node, ctx[b] + 1 + i
                k[:, tab[t // page], t % page] = st["k"][:, tab[s // page], s % page]
                v[:, tab[t // page], t % page] = st["v"][:, tab[s // page], s % page]
        return dict(k=k, v=v, new_len=None)
    B, n, hq, hkv, d = case["batch"], case["n"], case["hq"], case["hkv"], case["d"]
    out = torch.zeros((B, n, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, n, hq), -float("inf"), dtype=torch.float64, device="cuda")
    for b in range(B):
        c, m = ctx[b], count[b]
        used = st["table"][b, : _pages(c + m, page)].long()
        K = st["k"].index_select(0, used).flatten(0, 1)[: c + m].double()
        V = st["v"].index_select(0, used).flatten(0, 1)[: c + m].double()
        see = torch.ones((m, c + m), dtype=torch.bool, device="cuda")
        nodes = torch.arange(m, device="cuda")
        if st["mask"] is None:
            see[:, c:] = nodes[None, :] <= nodes[:, None]
        else:
            see[:, c:] = ((st["mask"][b, :m, nodes // 32].long() >> (nodes % 32)) & 1).bool() & (nodes[None, :] <= nodes[:, None])
        for h in range(hq):
            kh = h // (hq // hkv)
            a = (st["q"][b, :m, h].double() @ K[:, kh].T) / d ** 0.5
            a = a.masked_fill(~see, -float("inf"))
            w = torch.logsumexp(a, dim=1)
            out[b, :m, h] = torch.exp(a - w[:, None]) @ V[:, kh]
            lse[b, :m, h] = w
    return dict(out=out, lse=lse)
