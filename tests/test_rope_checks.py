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


def test_given_outputs_and_gradients_do_not_go_together(kq):
    x = torch.zeros((5, 2, 64), requires_grad=True)
    pos, f = torch.zeros(5, dtype=torch.int32), torch.zeros(32)
    with pytest.raises(ValueError, match="gradient"):
        kq.rope(x, None, pos, f, q_out=torch.zeros_like(x), stream=0)
    with pytest.raises(ValueError, match="gradient"):
        kq.rope(x.detach(), x, pos, f, k_out=torch.zeros_like(x), stream=0)
