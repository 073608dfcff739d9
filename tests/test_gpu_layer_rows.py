"""Products of more rows than 65535 tiles hold."""
import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv
from target_common import gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [65535 * 128, 65535 * 128 + 1, 1 << 24])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_products_of_many_rows_of_any_layout(M, dtype):
    """fp32, and 16-bit rows that are not 16-byte aligned; whole numbers, so exact."""
    g = gen(M)
    N, K = 3, 3

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(dtype)
    x, w, u, b, r = whole(M, K), whole(N, K), whole(N, K), whole(N), whole(M, N)
    ops = sv.TargetOps()
    want = x.double() @ w.double().t()
    up = x.double() @ u.double().t()
    assert torch.equal(ops.linear(x, w, b, residual=r).double(), want + b.double() + r.double())
    assert torch.equal(ops.gated_linear(x, w, u, activation="none", out_dtype=torch.float32)
                       .double(), want * up)
    assert ops.status() == sv.SV_OK
    ops.close()
