"""The paged-cache binding on the host: which device a call asks about (no GPU)."""
import pytest
import torch

import speculative_decoding_draft_07_b200 as pct
from speculative_decoding_draft_07_b200 import _lib


class _Devices:
    """torch.cuda.device and the library's workspace query, which depends on the current device."""

    def __init__(self):
        self.current = 0

    def device(self, index):
        outer = self

        class Here:
            def __enter__(self):
                self.was, outer.current = outer.current, index

            def __exit__(self, *_):
                outer.current = self.was
        return Here()

    def tree_attention_workspace(self, desc, batch, n_stride, heads_q):
        return 1000 * (1 + self.current)


@pytest.fixture
def devices(monkeypatch):
    d = _Devices()
    monkeypatch.setattr(torch.cuda, "device", d.device)
    monkeypatch.setattr(_lib, "lib", lambda: d)
    for f in (_lib._attn_workspace, _lib._attn_plan):
        f.cache_clear()
    yield d
    for f in (_lib._attn_workspace, _lib._attn_plan):
        f.cache_clear()


def test_workspace_is_asked_on_the_tensors_device(devices):
    """Tensors on device 2 while device 0 is current, and the other way round."""
    q, k = torch.Size((1, 1, 4, 64)), torch.Size((4, 16, 2, 64))
    plan = lambda device: _lib._attn_plan(q, (256, 256, 64, 1), k, (2048, 128, 64, 1), torch.bfloat16, 4, device)[2]   # noqa: E731
    assert plan(2) == 3000 and devices.current == 0
    devices.current = 2
    assert plan(0) == 1000 and plan(2) == 3000 and devices.current == 2


def test_workspace_of_host_caches_is_refused():
    k = torch.zeros((4, 16, 2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        pct.tree_attention_workspace(k, k, 4, 1, 1, 4)
