"""What the Python binding of the losses makes of tensors, on the CPU."""
import torch

import all_gather_amd as mr
from test_loss_abi import _OnDevice


def test_rows_of_batches_without_columns():
    """Every leading dimension counts, with columns and without."""
    for shape in ((2, 3, 5), (2, 3, 0), (4, 2, 3, 0), (0, 3, 0), (7, 0)):
        rows = 1
        for k in shape[:-1]:
            rows *= k
        assert mr._rows2d(_OnDevice(torch.zeros(shape)), "logits") == (rows, shape[-1], shape[-1]), shape
    assert mr._rows2d(_OnDevice(torch.zeros(0)), "logits") == (0, 0, 0)
