"""Tree attention at the ends of the number range. Elements that an extreme input does not enter
keep their bits; bounds are those of ``test_gpu_kvcache``."""
import numpy as np
import pytest
import torch

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
