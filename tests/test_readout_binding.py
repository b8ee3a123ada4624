"""What the readout operators' Python binding and size checks refuse before any device work (no GPU
needed)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")


def test_a_workspace_is_a_contiguous_tensor_of_the_operands_device():
    from cg_tensor_product_amd import readout
    here, elsewhere = torch.device("cpu"), torch.device("meta")
    good = torch.empty(4096, dtype=torch.uint8)
    assert readout._scratch(1024, good, here) == (good, good.data_ptr(), 4096)
    words = torch.empty((16, 8), dtype=torch.float64)
    assert readout._scratch(1024, words, here) == (words, words.data_ptr(), 1024)
    with pytest.raises(TypeError):  # its address would go to a kernel of another device
        readout._scratch(1024, good, elsewhere)
    with pytest.raises(TypeError):
        readout._scratch(1024, bytearray(4096), here)
    for bad in (good[:1].expand(4096), good[::2], words.t()):  # counts more or other bytes than it owns
        with pytest.raises(ValueError):
            readout._scratch(16, bad, here)


def test_group_norm_sizes_whose_joining_launch_is_too_large_are_refused():
    # every launch of a call holds fewer than 2^32 threads, the joins of (structure, group) and of the
    # channels among them: 70000 structures of 130 rows, 1024 groups
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    size = oeq.lib().oeq_group_norm_workspace_size
    assert size(9_100_000, 70_000, 1024, 1024, ctypes.byref(f), ctypes.byref(b)) == 2
    assert size(9_100_000, 70_000, 1024, 64, ctypes.byref(f), ctypes.byref(b)) == 0
    # of no structures and no rows the weights' gradients are still written, 8 channels a workgroup
    assert size(0, 0, 2**31 - 2048, (2**31 - 2048) // 2048, ctypes.byref(f), ctypes.byref(b)) == 2
