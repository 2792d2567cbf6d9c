"""The int8 product where a sum reaches the end of 32 bits: codes of -128, which the quantiser does
not make but the product accepts."""
import pytest
import torch

import latent_mixture_experts_moe_b200 as moe


@pytest.fixture(scope="module", autouse=True)
def built():
    from latent_mixture_experts_moe_b200 import build
    build.build()
    yield


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 8, 12, 40, 200, 300, 1500])
def test_lowest_codes_at_the_greatest_depth(T):
    """131072 products of (-128) (-128) are 2^31 exactly, one more than a 32-bit integer holds; every
    other sum of 8-bit codes at this depth fits. All values below are exact in float32."""
    K, N = 131072, 130
    xc = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    wc = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    wc[1::3] = 127                       # -128 * 127 * 131072 = -2^31 + 2^24
    wc[2::3, 0] = 0                      # 2^31 - 2^14
    one = torch.ones(max(T, N), device="cuda")
    lin = moe.Int8Linear(wc, one[:N].contiguous(), T_max=1)
    got = lin.matmul(xc, one[:T].contiguous(), out_dtype=torch.float32)
    assert lin.device_status() == (0, 0)
    ref = torch.full((N,), 2.0 ** 31)
    ref[1::3] = -2.0 ** 31 + 2.0 ** 24
    ref[2::3] = float(2 ** 31 - 2 ** 14)
    assert torch.equal(got.cpu(), ref.expand(T, N))
