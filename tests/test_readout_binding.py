"""What the readout operators' Python binding and size checks refuse before any device work (no GPU
needed)."""
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
