"""Tree attention at the ends of the number range. Elements that an extreme input does not enter
keep their bits; bounds are those of ``test_gpu_kvcache``."""
import numpy as np
import pytest
import torch

from gpu_util import f64
from test_gpu_kvcache import DEV, _case, _check, _run

pytestmark = pytest.mark.gpu

# rows a KV head: 4, 24 and 240 (fp32: each of the three row groups; bf16: both kernels)
ROWS = [(1, 8), (6, 8), (60, 8)]
FMAX = float(torch.finfo(torch.float32).max)


def _place(table, b, t, page=16):
    return int(table[b, t // page]), t % page


def _clean(g):
    r = _run(g)
    torch.cuda.synchronize()
    return r.out.clone(), r.lse.clone()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("n,hq", ROWS)
def test_infinite_values(n, hq, d, dtype):
    """A seen V of +inf or -inf makes its column so, both together NaN; other columns keep their bits."""
    c = _case(30, dtype=dtype, n=n, hq=hq, d=d, ctx=(33, 1500, 40), q_sigma=0.5)
    g, table = c[0], c[1]
    want, wl = _clean(g)
    g["v"][_place(table, 0, 17)][:, 3] = float("inf")
    g["v"][_place(table, 1, 900)][:, d - 1] = float("-inf")
    g["v"][_place(table, 2, 1)][:, 2] = float("inf")
    g["v"][_place(table, 2, 39)][:, 2] = float("-inf")
    r = _run(g)
    torch.cuda.synchronize()
    assert torch.equal(r.lse, wl)
    assert (r.out[0, ..., 3] == float("inf")).all()
    assert (r.out[1, ..., d - 1] == float("-inf")).all()
    assert torch.isnan(r.out[2, ..., 2]).all()
    for b, col in enumerate((3, d - 1, 2)):
        rest = [j for j in range(d) if j != col]
        assert torch.equal(r.out[b][..., rest], want[b][..., rest])


@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("n,hq", ROWS)
def test_values_up_to_the_largest_number(n, hq, d):
    """fp32: finite V of any size, in one token a column (its weight is at most 1)."""
    c = _case(31, dtype="f32", n=n, hq=hq, d=d, ctx=(33, 1500), q_sigma=0.5)
    g, table = c[0], c[1]
    edge = float(np.array([0x7f7ff000], np.uint32).view(np.float32)[0])
    below = float(np.array([0x7f7fefff], np.uint32).view(np.float32)[0])
    for col, (t, x) in enumerate([(17, FMAX), (3, -FMAX), (20, edge), (32, below), (0, -edge)]):
        g["v"][_place(table, 0, t)][:, col] = x
        g["v"][_place(table, 1, 40 * t)][:, col] = x
    _check(_run(g), *c)


@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("n,hq", [(6, 8), (60, 8)])
def test_the_largest_value_of_an_unseen_node(n, hq, d):
    """fp32: V of a node that no row sees may be any finite number; nothing changes."""
    g, table, ctx, counts, m = _case(32, dtype="f32", n=n, hq=hq, d=d, ctx=(33, 100), mask="random")
    m &= np.uint32(0xfffffffd)                  # bit 1 of every word off: nobody sees node 1
    g["mask"] = torch.from_numpy(m.view(np.int32)).to(DEV)
    want, wl = _clean(g)
    for b in range(2):
        g["v"][_place(table, b, ctx[b] + 1)][:, 3:5] = torch.tensor([FMAX, -FMAX], device=DEV)
    r = _run(g)
    torch.cuda.synchronize()
    assert torch.equal(r.out, want) and torch.equal(r.lse, wl)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), FMAX])
@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("n,hq", [(6, 8), (60, 8)])
def test_fp32_keys_of_unseen_nodes_do_not_enter(n, hq, d, bad):
    """As test_keys_of_unseen_nodes_do_not_enter, in fp32: no other row's result changes by a bit."""
    g, table, ctx, counts, m = _case(7, dtype="f32", n=n, hq=hq, d=d, ctx=(33, 100), mask="random")
    m &= np.uint32(0xfffffffd)
    g["mask"] = torch.from_numpy(m.view(np.int32)).to(DEV)
    want, wl = _clean(g)
    for b in range(2):
        g["k"][_place(table, b, ctx[b] + 1)] = bad
    r = _run(g)
    torch.cuda.synchronize()
    assert torch.equal(r.out, want) and torch.equal(r.lse, wl)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n,hq,d", [(1, 8, 64), (60, 2, 64), (60, 8, 128), (60, 2, 200)])
def test_scores_of_any_size(n, hq, d, sign, dtype):
    """Scores of 2^32 to 2^40, exact in every format and far apart: a row is its best token's V.

    The best weight is 1 and the others are 0, so bf16 is exact. In fp32, V = hi + lo with hi its 11
    leading bits to nearest, |lo| <= 2^-11 |v|; the product reads 11 bits of lo, cut off, which leaves
    out at most 2^-10 |lo| <= 2^-21 |v|, and the sum of the parts, the accumulator's add and the
    division are off by at most 2^-23 + 2 * 2^-24 = 2^-22 of it: together below 2^-20 |v|."""
    g, table, ctx, counts, _ = _case(33, dtype=dtype, n=n, hq=hq, hkv=1, d=d, mask=None,
                                     ctx=(150, 33, 64, 127, 128, 5, 90, 1))
    g["q"].zero_()
    g["q"][..., 0] = 2.0 ** 20
    for b in range(len(ctx)):
        for t in range(ctx[b] + counts[b]):
            g["k"][_place(table, b, t)][:, 0] = sign * ((37 * t + 11 * b) % 251 + 1) * 2.0 ** 8
    r = _run(g, scale=16.0)
    torch.cuda.synchronize()
    out, lse = f64(r.out), f64(r.lse)
    v = f64(g["v"])
    for b in range(len(ctx)):
        score = np.array([sign * ((37 * t + 11 * b) % 251 + 1) * 2.0 ** 32 for t in range(ctx[b] + counts[b])])
        for i in range(n):
            best = int(score[: ctx[b] + i + 1].argmax())
            best_v = v[_place(table, b, best)]
            off = 0 if dtype == "bf16" else 2.0 ** -20
            assert (np.abs(out[b, i] - best_v) <= off * np.abs(best_v)).all(), (b, i)
            # base-2 and back: three roundings, and log2 e and ln 2 in fp32
            assert (np.abs(lse[b, i] - score[best]) <= 2.0 ** -21 * abs(score[best])).all(), (b, i)


@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("n,hq", [(1, 8), (8, 64), (40, 32)])
def test_large_values_of_a_token_that_raises_the_maximum(n, hq, d):
    """bf16: V of 2^122 at a token whose score is e^5 times the others': no weight is above 1."""
    c = _case(34, n=n, hq=hq, hkv=8, d=d, mask=None, ctx=(300,) * 24)
    g, table, ctx = c[0], c[1], c[2]
    g["q"].zero_()
    g["q"][..., 0] = 1.0
    g["k"][..., 0] = 0.0
    for b in range(len(ctx)):
        for t in (150, 290):
            g["k"][_place(table, b, t)][:, 0] = 5.0
        g["v"][_place(table, b, 150)][:, : d // 2] = 2.0 ** 122
        g["v"][_place(table, b, 290)][:, d // 2:] = 2.0 ** 122
    _check(_run(g, scale=1.0), *c, scale=1.0)
