"""Outputs that overlap inputs or each other are refused before any launch (on the host, no GPU):
blocks of one call read lengths and tables at different times and have to read the same."""
import ctypes

import pytest
import torch

import speculative_decoding_draft_07_b200 as pct

B, N, HQ, WIDTH, DEPTH = 8, 40, 8, 16, 5
DESC = pct.KvCacheDesc(64, 16, WIDTH, 4, 64, pct.PCT_BF16, 16 * 256, 256, 64)
STRIDE = (ctypes.c_int64 * 3)(N * HQ * 64, HQ * 64, 64)
# (bytes, is an output); each lies 256 MB from the next
SPANS = {
    "kv_pages_resize": dict(ctx_len=(8 * B, 0), count=(4 * B, 0), table=(4 * B * WIDTH, 1), held=(4 * B, 1),
                            free=(4 * 64, 1), free_count=(4, 1), status=(4 * B, 1)),
    "kv_tree_slots": dict(ctx_len=(8 * B, 0), count=(4 * B, 0), depth=(4 * B * N, 0), table=(4 * B * WIDTH, 0),
                          slot=(8 * B * N, 1), pos=(8 * B * N, 1), status=(4 * B, 1)),
    "kv_append": dict(slot=(8 * B * N, 0), status=(4 * B, 1)),
    "tree_attention": dict(table=(4 * B * WIDTH, 0), ctx_len=(8 * B, 0), count=(4 * B, 0), mask=(4 * B * N * 2, 0),
                           out=(2 * B * N * HQ * 64, 1), lse=(4 * B * N * HQ, 1), status=(4 * B, 1),
                           workspace=(None, 1)),     # what the call asks for
    "kv_commit": dict(table=(4 * B * WIDTH, 0), ctx_len=(8 * B, 0), count=(4 * B, 0), accept_len=(4 * B, 0),
                      path=(4 * B * DEPTH, 0), new_len=(8 * B, 1), status=(4 * B, 1)),
}


def _workspace():
    return pct.lib().tree_attention_workspace(ctypes.byref(DESC), B, N, HQ)


def _call(name, at):
    L, d = pct.lib(), ctypes.byref(DESC)
    p = {k: ctypes.c_void_p(x) for k, x in at.items()}
    far = [ctypes.c_void_p((64 + i) << 28) for i in range(4)]
    if name == "kv_pages_resize":
        return L.kv_pages_resize(B, 16, WIDTH, 64, *(p[k] for k in SPANS[name]), None)
    if name == "kv_tree_slots":
        return L.kv_tree_slots(B, N, 16, WIDTH, 64, *(p[k] for k in SPANS[name]), None)
    if name == "kv_append":
        return L.kv_append(d, B, N, far[0], far[1], STRIDE, p["slot"], far[2], far[3], p["status"], None)
    if name == "tree_attention":
        return L.tree_attention(d, B, N, HQ, 0.1, far[0], STRIDE, far[1], far[2], p["table"], p["ctx_len"], p["count"],
                                p["mask"], p["out"], p["lse"], p["status"], p["workspace"], _workspace(), None)
    return L.kv_commit(d, B, 1, 0, DEPTH, far[0], far[1], p["table"], p["ctx_len"], p["count"], p["accept_len"],
                       p["path"], p["new_len"], p["status"], None)


@pytest.mark.parametrize("name", SPANS)
def test_overlapping_arrays_are_refused(name):
    spans = {k: (_workspace() if n is None else n, out) for k, (n, out) in SPANS[name].items()}
    apart = {k: (1 + i) << 28 for i, k in enumerate(spans)}
    tried = 0
    for a, (na, out) in spans.items():
        for b, (nb, _) in spans.items():
            if a == b or not out:
                continue
            first, last = apart[b] - (na - 1) // 16 * 16, apart[b] + (nb - 1) // 16 * 16
            for x in (apart[b], first, last):        # the same place; one end in the other
                assert _call(name, apart | {a: x}) == pct.PCT_EINVAL, (a, b, x - apart[b])
                tried += 1
    assert tried > 2
    if torch.cuda.is_available():                    # the next calls have nothing wrong but their pointers
        pytest.skip("calls with made-up addresses pass the checks")
    assert _call(name, apart) not in (pct.PCT_OK, pct.PCT_EINVAL)
    order = list(spans)                              # end to end without a gap is apart
    at, x = {}, 1 << 24
    for k in order:
        at[k], x = x, x + -(-spans[k][0] // 256) * 256
    assert _call(name, at) not in (pct.PCT_OK, pct.PCT_EINVAL)


BAD = [dict(batch=0), dict(batch=65536), dict(n=0), dict(n=65537), dict(hq=0), dict(hq=6), dict(hq=4 * 65),
       dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(scale=-2.4e38), dict(q=None), dict(st=None), dict(k=None), dict(v=None),
       dict(t=None), dict(c=None), dict(out=None), dict(status=None), dict(q=264), dict(k=264), dict(v=264),
       dict(out=264), dict(st=(4096, 100, 64)), dict(st=(-8, 256, 64))]


@pytest.mark.parametrize("bad", BAD, ids=lambda d: "-".join(d))
def test_attention_refusals_with_arguments_apart(bad):
    """Each refusal by itself: nothing else is wrong with the call."""
    base = dict(batch=2, n=4, hq=8, scale=0.1, st=(4096, 256, 64), out=1 << 24, status=2 << 24, q=3 << 24, k=4 << 24,
                v=5 << 24, t=6 << 24, c=7 << 24)

    def call(a):
        p = lambda x: None if x is None else ctypes.c_void_p(x)   # noqa: E731
        st = None if a["st"] is None else (ctypes.c_int64 * 3)(*a["st"])
        return pct.lib().tree_attention(ctypes.byref(DESC), a["batch"], a["n"], a["hq"], a["scale"], p(a["q"]), st,
                                        p(a["k"]), p(a["v"]), p(a["t"]), p(a["c"]), p(8 << 24), p(9 << 24), p(a["out"]),
                                        p(10 << 24), p(a["status"]), None, 0, None)
    assert call(base | bad) == pct.PCT_EINVAL
    assert call(base) in (pct.PCT_EWORKSPACE, 4)     # no workspace, or no device


STRIDES = dict(page_stride=16 * 256, slot_stride=256, head_stride=64)


@pytest.mark.parametrize("axis", ["page_stride", "slot_stride", "head_stride", "layer_stride"])
@pytest.mark.parametrize("stride", [0, 56])
def test_calls_that_write_refuse_rows_over_each_other(axis, stride):
    """An expanded cache (stride 0) or rows closer than head_dim, where the axis has several entries."""
    far = [ctypes.c_void_p((1 + i) << 28) for i in range(9)]
    layers = 3

    def calls(sizes, strides, layers, layer_stride):
        d = ctypes.byref(pct.KvCacheDesc(sizes[0], sizes[1], WIDTH, sizes[2], 64, pct.PCT_BF16, *strides))
        L = pct.lib()
        yield "append", lambda: L.kv_append(d, B, N, far[0], far[1], STRIDE, far[2], far[3], far[4], far[5], None)
        yield "commit", lambda: L.kv_commit(d, B, layers, layer_stride, DEPTH, *far, None)

    sizes = [64, 16, 4]
    strides = dict(STRIDES, layer_stride=64 * 16 * 256)
    strides[axis] = stride
    for name, call in calls(sizes, [strides[k] for k in STRIDES], layers, strides["layer_stride"]):
        if axis != "layer_stride" or name == "commit":
            assert call() == pct.PCT_EINVAL, name
    if torch.cuda.is_available():                    # the next calls have nothing wrong but their pointers
        pytest.skip("calls with made-up addresses pass the checks")
    one = {"page_stride": 0, "slot_stride": 1, "head_stride": 2}
    if axis in one:
        sizes[one[axis]] = 1
    else:
        layers = 1
    for name, call in calls(sizes, [strides[k] for k in STRIDES], layers, strides["layer_stride"]):
        assert call() not in (pct.PCT_OK, pct.PCT_EINVAL), name


def _apart(n):
    return [ctypes.c_void_p((1 + i) << 28) for i in range(n)]


CALLS = {
    "kv_append": (dict(d=DESC, batch=2, n=4, st=(4096, 256, 64), p=6),
                  [dict(batch=0), dict(batch=65536), dict(n=0), dict(n=(1 << 20) + 1), dict(st=(4096, 4, 64)), dict(st=(-8, 256, 64)),
                   dict(st=None), dict(odd=0), dict(odd=1), dict(odd=3), dict(odd=4)] + [dict(null=i) for i in range(6)]),
    "kv_commit": (dict(d=DESC, batch=2, layers=1, ls=0, depth=4, p=9),
                  [dict(batch=0), dict(batch=65536), dict(layers=0), dict(layers=65536), dict(ls=4), dict(ls=-8), dict(depth=0),
                   dict(depth=4097), dict(odd=0), dict(odd=1)] + [dict(null=i) for i in range(9)]),
    "kv_pages_resize": (dict(batch=2, page=16, width=8, n_pages=10, p=7),
                        [dict(batch=0), dict(batch=65536), dict(page=0), dict(page=65537), dict(width=0), dict(n_pages=0),
                         dict(page=65536, width=16385)] + [dict(null=i) for i in (0, 2, 3, 4, 5, 6)]),
    "kv_tree_slots": (dict(batch=2, n=4, page=16, width=8, n_pages=10, p=7),
                      [dict(batch=0), dict(batch=65536), dict(n=0), dict(n=(1 << 20) + 1), dict(page=0), dict(page=65537),
                       dict(width=0), dict(n_pages=0), dict(page=65536, width=16385)] + [dict(null=i) for i in (0, 1, 3, 4, 5, 6)]),
}


@pytest.mark.parametrize("name", CALLS)
def test_refusals_with_arguments_apart(name):
    """Each refusal of the other calls by itself: nothing else is wrong with the call."""
    base, bad = CALLS[name]
    L = pct.lib()

    def call(a):
        p = _apart(a["p"])
        if "null" in a:
            p[a["null"]] = None
        if "odd" in a:
            p[a["odd"]] = ctypes.c_void_p(p[a["odd"]].value + 8)
        if name == "kv_append":
            st = None if a["st"] is None else (ctypes.c_int64 * 3)(*a["st"])
            return L.kv_append(ctypes.byref(a["d"]), a["batch"], a["n"], p[0], p[1], st, p[2], p[3], p[4], p[5], None)
        if name == "kv_commit":
            return L.kv_commit(ctypes.byref(a["d"]), a["batch"], a["layers"], a["ls"], a["depth"], *p, None)
        if name == "kv_pages_resize":
            return L.kv_pages_resize(a["batch"], a["page"], a["width"], a["n_pages"], *p, None)
        return L.kv_tree_slots(a["batch"], a["n"], a["page"], a["width"], a["n_pages"], *p, None)

    for b in bad:
        assert call(base | b) == pct.PCT_EINVAL, b
    if torch.cuda.is_available():                    # the next call has nothing wrong but its pointers
        pytest.skip("calls with made-up addresses pass the checks")
    assert call(base) not in (pct.PCT_OK, pct.PCT_EINVAL)
