"""Host side of the evicting cache's calls and of the weight sums (no GPU needed)."""
import numpy as np
import torch

from tile_routed_mixed_causal_b200 import _lib as L


def test_shape_brings_its_status_word(monkeypatch):
    """The word is there from the start: no call creates it, on whatever stream or in whatever capture
    it runs."""
    s = L.Shape([0, 130, 194], 8, 2, 128, device="cpu")
    for name in ("zeros", "empty", "full", "tensor"):
        monkeypatch.setattr(torch, name, lambda *a, **k: (_ for _ in ()).throw(AssertionError("made late")))
    word = s.status
    assert word.dtype is torch.int32 and word.shape == (1,) and int(word) == 0
    assert s.status.data_ptr() == word.data_ptr()
    assert s.cu_dev.tolist() == [0, 130, 194] and s.cu_dev.is_contiguous()
    assert np.array_equal(s.cu_host, [0, 130, 194])
    assert L.Shape([0, 64], 8, 2, 128, device=None).status is None
