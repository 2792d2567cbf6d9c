"""The two ways of a row's int8 scale. INT8_SCALE_RECIPROCAL gives the codes and scales of torch's
own operations on the GPU; the float32 output of a product shows a single code that differs
(1 of 8192 codes moves its row by 1e-3 of the row's norm)."""
import ctypes

import numpy as np
import pytest
import torch

import latent_mixture_experts_moe_b200 as moe


@pytest.fixture(scope="module", autouse=True)
def built():
    from latent_mixture_experts_moe_b200 import build
    build.build()
    yield


def torch_quantise(x):
    """Codes (whole numbers in float32) and scales of every row, by torch's elementary operations."""
    scale = (x.float().abs().amax(1, keepdim=True) / 127.0).clamp_min(2.0 ** -126)
    return torch.round(x.float() / scale).clamp(-127.0, 127.0), scale


def rows(T, K, dtype, seed):
    """Rows with wide channels and, as bf16 rows have them, quotients at n + 1/2: row r holds
    (n + 1/2) / 127 of its maximum for every n."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, K, device="cuda", generator=gen)
    x[:, ::max(1, K // 8)] *= 6.0
    if K >= 256:
        top = x.abs().amax(1, keepdim=True)
        x[:, 1:128] = top * (torch.arange(127, device="cuda") + 0.5) / 127
    return x.to(dtype)


SIZES = [(1, 512, 4096), (5, 1000, 2064), (8, 300, 8192), (16, 256, 272), (40, 640, 1040), (300, 512, 8192),
         (4000, 1000, 4096)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_reciprocal_equals_torch(T, N, K, dtype):
    """Codes and scales bit for bit; outputs too: sums of the products are whole numbers below 2^24
    here, exact in float32 in any order, and what follows are single float32 operations."""
    x = rows(T, K, dtype, T + K)
    codes, scales = moe.quantize_int8_rows(x, scale_rule=moe.INT8_SCALE_RECIPROCAL)
    q, s = torch_quantise(x)
    assert torch.equal(scales, s[:, 0])
    assert torch.equal(codes.float(), q)
    gen = torch.Generator(device="cuda").manual_seed(N)
    wc = torch.randint(-7, 8, (N, K), device="cuda", generator=gen).to(torch.int8)      # 127 * 7 * 8192 < 2^24
    ws = torch.rand(N, device="cuda", generator=gen) + 0.5
    lin = moe.Int8Linear(wc, ws, T_max=T, scale_rule=moe.INT8_SCALE_RECIPROCAL)
    got = lin(x, out_dtype=torch.float32)
    assert lin.device_status() == (0, 0)
    acc = (q.double() @ wc.double().T).float()
    assert torch.equal(got, acc * (s * ws))
    assert torch.equal(got, lin.matmul(codes, scales, out_dtype=torch.float32))


@pytest.mark.gpu
def test_reciprocal_by_single_operations():
    """The same on the CPU, one float32 operation at a time, zero, subnormal, largest, infinite and
    NaN rows among them; the rules differ in some rows and agree in most."""
    x = rows(600, 512, torch.float32, 1)
    x[0] = 0.0
    x[1] = 1e-39
    x[2, 7] = 3e38
    x[3, 0] = float("inf")
    x[4, 5] = float("nan")
    codes, scales = (t.cpu().numpy() for t in moe.quantize_int8_rows(x, scale_rule=moe.INT8_SCALE_RECIPROCAL))
    h = x.cpu().numpy()
    inv = np.float32(1.0) / np.float32(127.0)
    for r in range(len(h)):
        if r in (3, 4):
            assert np.isnan(scales[r]) and not codes[r].any()
            continue
        s = max(np.float32(np.abs(h[r]).max() * inv), np.float32(2.0 ** -126))
        assert scales[r] == s
        np.testing.assert_array_equal(codes[r], np.rint(h[r] / s).astype(np.int8))
    divided = moe.quantize_int8_rows(x)[1].cpu().numpy()
    differ = np.mean(divided[5:] != scales[5:])
    assert 0.0 < differ < 0.2
    assert np.all(np.abs(divided[5:] - scales[5:]) <= np.spacing(divided[5:]))


# ------------------------------------------------------------------------- refusals (no GPU)
def test_other_rules_are_refused_before_any_launch():
    w = moe.Int8Weight(1 << 20, 1 << 21)
    for rule, code in ((0, 3), (1, 3), (2, 1), (-1, 1)):            # (3: accepted, no workspace)
        assert moe.lib().muse_int8_linear_scaled(1 << 22, 1, 4, 64, 64, ctypes.byref(w), 32, 1 << 24, 1, 32, None, 0,
                                                 None, rule, None) == code
    for rule in (2, -1):
        assert moe.lib().muse_quantize_int8_rows_scaled(1 << 20, 0, 3, 32, 32, 1 << 21, 1 << 22, rule, None) == 1
    assert moe.lib().muse_quantize_int8_rows_scaled(1 << 20, 0, 0, 32, 32, 1 << 21, 1 << 22, 1, None) == 0
    with pytest.raises(ValueError):
        moe.Int8Linear(torch.zeros(32, 64, dtype=torch.int8), torch.zeros(32), T_max=4, scale_rule=2)
