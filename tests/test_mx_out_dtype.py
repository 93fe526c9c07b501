"""Result types that the microscaled operators do not have are refused by name (on the CPU, by tensors without memory)."""
import pytest
import torch

import xnor_popcount_gemm_gb300 as bt
from test_mx import fake  # noqa: F401


@pytest.mark.parametrize("dtype", [torch.float64, torch.int32, torch.uint8])
def test_types_that_are_none_of_theirs(fake, dtype):  # noqa: F811
    x, w = fake.t(4, 64), fake.mx(24, 64)
    for rows in (x, fake.t(40, 64), fake.mx(4, 64)):
        with pytest.raises(ValueError, match="float32 or"):
            bt.bt_mx_linear(rows, w, out_dtype=dtype)
    with pytest.raises(ValueError, match="float32 or"):
        bt.bt_mx_dequantize(w, dtype)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        bt.bt_mx_linear_backward(fake.t(40, 24), fake.t(64, 64), out_dtype=dtype)
