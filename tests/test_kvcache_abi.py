"""Refusals of the paged-cache calls, on the host (no GPU): bad shapes, strides,
alignments and pointers are answered before anything is launched."""
import ctypes

import pytest
import torch

import speculative_decoding_draft_07_b200 as pct

P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)


def _desc(**kw):
    base = dict(n_pages=10, page_size=16, max_pages=8, heads_kv=4, head_dim=64, dtype=pct.PCT_BF16,
                page_stride=16 * 256, slot_stride=256, head_stride=64)
    base.update(kw)
    return pct.KvCacheDesc(*base.values())


def _st(a=4096, b=256, c=64):
    return (ctypes.c_int64 * 3)(a, b, c)


BAD_DESCS = [dict(n_pages=0), dict(page_size=0), dict(page_size=65537), dict(max_pages=0),
             dict(page_size=65536, max_pages=16385), dict(heads_kv=0), dict(heads_kv=1025),
             dict(head_dim=0), dict(head_dim=12), dict(head_dim=264), dict(dtype=2), dict(dtype=-1),
             dict(page_stride=-8), dict(page_stride=4), dict(slot_stride=257), dict(head_stride=60)]


@pytest.mark.parametrize("bad", BAD_DESCS, ids=lambda d: "-".join(d))
def test_bad_cache_descriptors(bad):
    L, d = pct.lib(), _desc(**bad)
    r = ctypes.byref(d)
    assert L.tree_attention_workspace(r, 2, 4, 4) == 0
    assert L.tree_attention(r, 2, 4, 4, 0.1, P, _st(), P, P, P, P, P, None, P, P, P, P, 1 << 40, None) == pct.PCT_EINVAL
    assert L.kv_append(r, 2, 4, P, P, _st(), P, P, P, P, None) == pct.PCT_EINVAL
    assert L.kv_commit(r, 2, 1, 0, 4, P, P, P, P, P, P, P, P, P, None) == pct.PCT_EINVAL


def test_attention_arguments():
    L, d = pct.lib(), _desc()
    r = ctypes.byref(d)

    def call(batch=2, n=4, hq=8, scale=0.1, q=P, st=_st(), k=P, v=P, t=P, c=P, out=P, status=P, ws=P, wsb=1 << 40):
        return L.tree_attention(r, batch, n, hq, scale, q, st, k, v, t, c, P, P, out, P, status, ws, wsb, None)

    for bad in (dict(batch=0), dict(batch=65536), dict(n=0), dict(n=65537), dict(hq=0), dict(hq=6),
                dict(hq=4 * 65), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None),
                dict(st=None), dict(k=None), dict(v=None), dict(t=None), dict(c=None), dict(out=None),
                dict(status=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(out=ODD),
                dict(st=_st(b=100)), dict(st=_st(a=-8))):
        assert call(**bad) == pct.PCT_EINVAL, bad
    assert L.tree_attention_workspace(r, 2, 4, 6) == 0
    assert L.tree_attention_workspace(r, 2, 4, 8) > 0


def test_cache_call_arguments():
    L, d = pct.lib(), _desc()
    r = ctypes.byref(d)
    assert L.kv_append(r, 2, 4, P, P, _st(b=4), P, P, P, P, None) == pct.PCT_EINVAL
    assert L.kv_append(r, 2, 4, ODD, P, _st(), P, P, P, P, None) == pct.PCT_EINVAL
    assert L.kv_append(r, 2, 4, P, P, _st(), None, P, P, P, None) == pct.PCT_EINVAL
    assert L.kv_append(r, 2, (1 << 20) + 1, P, P, _st(), P, P, P, P, None) == pct.PCT_EINVAL
    for layers, ls, depth in ((0, 0, 4), (65536, 0, 4), (1, 4, 4), (1, -8, 4), (1, 0, 0), (1, 0, 4097)):
        assert L.kv_commit(r, 2, layers, ls, depth, P, P, P, P, P, P, P, P, P, None) == pct.PCT_EINVAL
    assert L.kv_commit(r, 2, 1, 0, 4, P, P, P, P, P, P, P, None, P, None) == pct.PCT_EINVAL
    for b, ps, mp, n in ((0, 16, 8, 10), (65536, 16, 8, 10), (2, 0, 8, 10), (2, 65537, 8, 10), (2, 16, 0, 10),
                         (2, 16, 8, 0), (2, 65536, 16385, 10)):
        assert L.kv_pages_resize(b, ps, mp, n, P, P, P, P, P, P, P, None) == pct.PCT_EINVAL
        assert L.kv_tree_slots(b, 4, ps, mp, n, P, P, P, P, P, P, P, None) == pct.PCT_EINVAL
    assert L.kv_tree_slots(2, 0, 16, 8, 10, P, P, P, P, P, P, P, None) == pct.PCT_EINVAL
    assert L.kv_tree_slots(2, 4, 16, 8, 10, P, None, P, P, P, P, P, None) == pct.PCT_EINVAL
    assert L.kv_pages_resize(2, 16, 8, 10, P, None, P, P, None, P, P, None) == pct.PCT_EINVAL


def test_binding_refuses_host_tensors_and_wrong_types():
    z = torch.zeros
    k = z((4, 16, 2, 64), dtype=torch.bfloat16)
    t, c, n = z((1, 4), dtype=torch.int32), z(1, dtype=torch.int64), z(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pct.tree_attention(z((1, 1, 2, 64), dtype=torch.bfloat16), k, k, t, c)
    with pytest.raises(ValueError, match="CUDA"):
        pct.kv_append(k[:1, :1], k[:1, :1], z((1, 1), dtype=torch.int64), k, k)
    with pytest.raises(ValueError, match="CUDA"):
        pct.kv_commit(k, k, t, c, n, n, z((1, 3), dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        pct.kv_pages_resize(c, t, n, n, n, 16)
    with pytest.raises(ValueError, match="CUDA"):
        pct.kv_tree_slots(c, n, t, 1, 16, 4)
    with pytest.raises(TypeError):
        pct.tree_attention(None, k, k, t, c)
