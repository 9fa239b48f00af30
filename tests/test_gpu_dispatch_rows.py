"""What the quantizing dispatch takes as its rows."""
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def test_rows_are_a_number_or_two():
    say("rows of the quantizing dispatch")
    x = torch.ones((4, 256), device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")[:, None]
    q, s = fp8.quant_1x128(x)
    for rows, shape in ((6, (6, 256)), ((2, 3), (2, 3, 256)), ([3, 2], (3, 2, 256)), (torch.Size((1, 4)), (1, 4, 256))):
        xq, sa = fp8.expert_dispatch_quant(x, pos, rows)
        assert xq.shape == shape and sa.shape == (2, shape[0] * shape[1] if len(shape) == 3 else shape[0])
        assert torch.equal(xq.view(-1, 256)[:4], q) and torch.equal(sa[:, :4], s)
    for rows in ((6,), (2, 3, 4), ()):          # (of three, the rows behind the first two's were never reached)
        with pytest.raises(ValueError):
            fp8.expert_dispatch_quant(x, pos, rows)
