"""Argument checks of the rotary positions' binding, without a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def kq():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    import quantized_decode_gemv_block_gb300 as m
    m.load_library()
    return m


@pytest.mark.parametrize("shape", [(3, 1, 5), (1, 1, 5), (3, 5, 1)])
def test_positions_of_more_than_two_dimensions_are_refused(kq, shape):
    """(axes, batch, tokens) taken as one axis would leave the pairs of the others unturned."""
    x = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="axes, tokens"):
        kq.rope(x, None, torch.zeros(shape, dtype=torch.int32), torch.zeros(32), pair_axis=torch.zeros(32, dtype=torch.uint8), stream=0)
