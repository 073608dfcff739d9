"""Products of more tiles than run at once: what is carried from a CTA's tile to its next
one. Whole numbers, which fp32 sums hold exactly whatever their order, so every element
counts."""
import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv
from target_common import DTYPES, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    o = sv.TargetOps()
    yield o
    assert o.status() == sv.SV_OK
    o.close()


def whole(g, dt, most, *shape):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(dt)


def check(ops, x, w, u, bias, res):
    """All of linear with a residual (its own output, and in place) and gated linear."""
    want = x.double() @ w.double().t()
    other = x.double() @ u.double().t()
    got = ops.linear(x, w, bias, residual=res.float(), out_dtype=torch.float32)
    assert torch.equal(got.double(), want + bias.double() + res.double())
    place = res.clone()
    ops.linear(x, w, residual=place, out=place)
    assert torch.equal(place, (want + res.double()).to(x.dtype))
    got = ops.gated_linear(x, w, u, bias, None, activation="relu", out_dtype=torch.float32)
    assert torch.equal(got.double(), ((want + bias.double()).clamp_min(0) * other).float().double())
    got = ops.gated_linear(x, w, u, activation="none")
    assert torch.equal(got, (want * other).float().to(x.dtype))


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# (K of one block, where no cluster shares a tile; of many, where clusters do; ragged)
@pytest.mark.parametrize("N,K", [(40001, 64), (40001, 4096), (100003, 200), (30011, 1032)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_few_rows(ops, N, K, dtype):
    assert -(-N // 128) > sms()  # a tile is 128 rows of the weight, or 64 of each of two
    g = gen(N + K)
    dt = DTYPES[dtype]
    w, u, bias = whole(g, dt, 2, N, K), whole(g, dt, 1, N, K), whole(g, dt, 2, N)
    for M in (1, 5, 16, 17, 20, 32, 33, 40, 64, 65, 100, 128):
        check(ops, whole(g, dt, 1, M, K), w, u, bias, whole(g, dt, 3, M, N))


# odd strides, 16-byte aligned ones with a ragged last column, and whole columns
@pytest.mark.parametrize("M,N,K", [(3000, 4099, 136), (5000, 8190, 64), (2600, 9004, 1032),
                                   (3001, 4104, 520), (2305, 8192, 200)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_many_rows(ops, M, N, K, dtype):
    assert -(-M // 256) * -(-N // 256) > sms()  # tiles of 256 x at most 256, for half the SMs
    g = gen(M + N + K)
    dt = DTYPES[dtype]
    check(ops, whole(g, dt, 1, M, K), whole(g, dt, 2, N, K), whole(g, dt, 1, N, K),
          whole(g, dt, 2, N), whole(g, dt, 3, M, N))
