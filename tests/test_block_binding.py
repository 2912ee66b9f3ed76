"""The binding of the operators around the projections, without a GPU: what a
call's host arguments become at the C boundary."""

import numpy as np
import pytest
import torch

from int4_quantized_gemm_amd import block_ops

POS, FREQ = torch.zeros((5, 3), dtype=torch.int32), torch.ones(4)


def _axis_bytes(pair_axis):
    """What _rope_args hands to the C call as the axis of each of four pairs."""
    return block_ops._rope_args(5, 8, POS, FREQ, pair_axis, "halves", None, None, 1e-6)[8]


@pytest.mark.parametrize("axes", [
    [0, 1, 2, 2], (0, 1, 2, 2), bytes([0, 1, 2, 2]), bytearray([0, 1, 2, 2]), np.array([0, 1, 2, 2]),
    np.array([0, 1, 2, 2], dtype=np.int32), np.array([0, 1, 2, 2], dtype=np.uint8),
    np.array([0, 1, 2, 2], dtype=np.int64)[::1], torch.tensor([0, 1, 2, 2]), torch.tensor([0, 1, 2, 2], dtype=torch.int8),
    np.array([0, 9, 1, 9, 2, 9, 2, 9])[::2], range(0)], ids=lambda v: f"{type(v).__name__}{getattr(v, 'dtype', '')}")
def test_pair_axis_of_any_integer_sequence(axes):
    if isinstance(axes, range):
        assert _axis_bytes(None) == bytes(4)
        assert _axis_bytes(range(4)) == bytes([0, 1, 2, 3])
        return
    assert _axis_bytes(axes) == bytes([0, 1, 2, 2])


@pytest.mark.parametrize("axes,error", [
    (4, TypeError), (np.int64(4), TypeError), (np.array(4), TypeError), (torch.tensor(4), TypeError), (True, TypeError),
    ([0.0, 1.0, 2.0, 2.0], TypeError), (np.zeros(4), TypeError), ("0122", TypeError), (np.zeros((4, 1)), TypeError),
    ([0, 1, 2], ValueError), ([0] * 5, ValueError), (bytes(3), ValueError), ([], ValueError),
    ([0, 1, -1, 2], ValueError), ([0, 1, 256, 2], ValueError), ([0, 1, 2 ** 70, 2], ValueError),
    (np.array([0, -1, 0, 0], dtype=np.int8), ValueError), (np.zeros(1, dtype=np.int32), ValueError)])
def test_pair_axis_refusals(axes, error):
    with pytest.raises(error, match="pair_axis must"):
        _axis_bytes(axes)
