"""The int8 row quantiser and the int8 product: every code, scale and output bit for bit
against the definition in integers and float32 on the CPU (the sums are exact integers; what
remains are single float32 operations in a fixed order), and the refusals (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import latent_mixture_experts_moe_b200 as moe

SCALE_MIN = np.float32(2.0 ** -126)


@pytest.fixture(scope="module", autouse=True)
def built():
    from latent_mixture_experts_moe_b200 import build
    build.build()
    yield


def ref_quantise(x: np.ndarray):
    """float32 [rows, K] -> int8 codes and float32 scales, one float32 operation at a time."""
    codes = np.zeros(x.shape, dtype=np.int8)
    scales = np.empty(x.shape[0], dtype=np.float32)
    for r, row in enumerate(x):
        if not np.all(np.isfinite(row)):
            scales[r] = np.nan
            continue
        s = max(np.float32(np.abs(row).max() / np.float32(127.0)), SCALE_MIN)
        scales[r] = s
        codes[r] = np.rint((row / s).astype(np.float32)).astype(np.int8)
    return codes, scales


def ref_product(xc, xs, wc, ws):
    """float32 outputs: the exact integer sum rounded once, times the product of the scales."""
    acc = xc.astype(np.int64) @ wc.astype(np.int64).T
    return acc.astype(np.float32) * (xs[:, None] * ws[None, :])


def to_dtype(a: np.ndarray, dtype):
    return torch.from_numpy(a).to(dtype)


def make_rows(rows, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * torch.logspace(-3, 3, rows)[:, None]
    if rows >= 6:
        x[1] = 0.0
        x[2, K // 2] = float("nan")
        x[3, 0] = float("-inf")
        x[4] = 1e-39                       # below the smallest normal float32
        x[5, K - 1] = 3e38
    return x.to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,K,pad,shift", [(1, 16, 0, 0), (7, 48, 0, 0), (9, 2064, 48, 0), (300, 144, 3, 1),
                                              (6, 8192, 0, 5), (33, 4096, 8, 0), (2500, 32, 0, 0)])
def test_quantiser_bit_exact(dtype, rows, K, pad, shift):
    """Odd row distances and starts that are aligned to nothing but the element too."""
    x = make_rows(rows, K, dtype, rows + K)
    wide = torch.zeros(rows * (K + pad) + shift, dtype=dtype, device="cuda")
    view = torch.as_strided(wide, (rows, K), (K + pad, 1), shift)
    view.copy_(x)
    codes, scales = moe.quantize_int8_rows(view)
    rc, rs = ref_quantise(x.float().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)


@pytest.mark.gpu
def test_quantiser_rounds_halves_to_even_and_spans_the_codes():
    """With a maximum of 127 the scale is 1: halves go to the even code."""
    x = torch.arange(-127, 128, dtype=torch.float32)
    x = torch.cat([x, x[:-1] + 0.5, torch.zeros(3)])
    x = x[None, :512]
    codes, scales = moe.quantize_int8_rows(x.cuda())
    assert scales.item() == 1.0
    np.testing.assert_array_equal(codes.cpu().numpy()[0], np.rint(x.numpy()[0]).astype(np.int8))


PRODUCTS = [(1, 1, 16), (1, 4096, 8192), (2, 7, 48), (5, 1000, 2064), (8, 129, 144), (9, 128, 128), (16, 300, 400),
            (17, 127, 1040), (31, 256, 4096), (33, 512, 272), (64, 8192, 4096), (65, 640, 640), (100, 4096, 1024),
            (128, 384, 2048), (129, 96, 8192), (255, 257, 80), (256, 512, 512), (257, 1000, 2064), (300, 4096, 4096),
            (777, 2048, 176), (1024, 4097, 1040), (2048, 4096, 528)]


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", PRODUCTS)
def test_product_bit_exact_and_leaves_the_rest_alone(T, N, K, out_dtype):
    rng = np.random.default_rng(T * 7 + N * 3 + K)
    xc = rng.integers(-127, 128, (T, K), dtype=np.int8)
    wc = rng.integers(-127, 128, (N, K), dtype=np.int8)
    xs = rng.uniform(1e-4, 2.0, T).astype(np.float32)
    ws = rng.uniform(1e-4, 2.0, N).astype(np.float32)
    lin = moe.Int8Linear(torch.from_numpy(wc).cuda(), torch.from_numpy(ws).cuda(), T_max=T)
    pad = (N * 3) % 11 if N % 2 else 0
    wide = torch.full((T + 1, N + pad), 7.0, dtype=out_dtype, device="cuda")
    got = lin.matmul(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), out=wide[:T, :N])
    assert lin.device_status() == (0, 0)
    ref = to_dtype(ref_product(xc, xs, wc, ws), out_dtype)
    assert torch.equal(got.cpu(), ref)
    assert bool((wide[T] == 7.0).all()) and bool((wide[:, N:] == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 8, 40, 200, 300])
def test_largest_sums_do_not_overflow(T):
    """K = 131072 codes of +-127: the largest sum that 32 bits hold."""
    K, N = 131072, 130
    xc = torch.full((T, K), 127, dtype=torch.int8, device="cuda")
    wc = torch.full((N, K), -127, dtype=torch.int8, device="cuda")
    wc[1::2] = 127
    one = torch.ones(max(T, N), device="cuda")
    lin = moe.Int8Linear(wc, one[:N].contiguous(), T_max=1)
    got = lin.matmul(xc, one[:T].contiguous(), out_dtype=torch.float32)
    ref = torch.full((N,), -float(K * 127 * 127))
    ref[1::2] *= -1
    assert torch.equal(got.cpu(), ref.expand(T, N))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,N,K,pad", [(1, 4096, 8192, 0), (3, 513, 272, 5), (6, 1000, 2064, 48), (8, 640, 8192, 8),
                                       (12, 1000, 2064, 48), (70, 256, 1040, 3), (513, 1024, 512, 0)])
def test_linear_equals_quantiser_then_product(T, N, K, pad, dtype):
    """From float rows (NaN, infinite and zero rows among them) in one call, against the reference
    and against the two calls, bit for bit; from a captured graph on new inputs too."""
    x = make_rows(T, K, dtype, T + K)
    wc, ws = moe.quantize_int8_rows(torch.randn(N, K, generator=torch.Generator().manual_seed(N)).cuda())
    wide = torch.zeros((T, K + pad), dtype=dtype, device="cuda")
    wide[:, :K] = x
    lin = moe.Int8Linear(wc, ws, T_max=T + 3)
    got = lin(wide[:, :K])
    rc, rs = ref_quantise(x.float().numpy())
    ref = to_dtype(ref_product(rc, rs, wc.cpu().numpy(), ws.cpu().numpy()), dtype)
    assert torch.equal(got.cpu().nan_to_num(nan=123.0), ref.nan_to_num(nan=123.0))
    qc, qs = moe.quantize_int8_rows(wide[:, :K])
    two = lin.matmul(qc, qs, out_dtype=dtype)
    assert torch.equal(got.view(torch.uint8), two.view(torch.uint8))
    # captured, then replayed on other inputs
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(got)
    with torch.cuda.graph(graph, stream=side):
        lin(wide[:, :K], out=out, stream=side)
    wide[:, :K] = torch.randn(T, K, device="cuda").to(dtype)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, lin(wide[:, :K]))


@pytest.mark.gpu
def test_two_holders_on_two_streams():
    """The same weights, two workspaces, products that overlap."""
    wc, ws = moe.quantize_int8_rows(torch.randn(2048, 1024, generator=torch.Generator().manual_seed(0)).cuda())
    a, b = (moe.Int8Linear(wc, ws, T_max=700) for _ in range(2))
    xa = torch.randn(700, 1024, device="cuda").bfloat16()
    xb = torch.randn(5, 1024, device="cuda").bfloat16()
    ra, rb = a(xa).clone(), b(xb).clone()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs.append((a(xa, stream=sa), b(xb, stream=sb)))
    torch.cuda.synchronize()
    assert all(torch.equal(p, ra) and torch.equal(q, rb) for p, q in outs)


@pytest.mark.gpu
def test_no_rows():
    wc, ws = moe.quantize_int8_rows(torch.randn(64, 128).cuda())
    lin = moe.Int8Linear(wc, ws, T_max=0)
    assert lin(torch.empty(0, 128, device="cuda")).shape == (0, 64)
    assert moe.quantize_int8_rows(torch.empty(0, 128, device="cuda"))[0].shape == (0, 128)


# ------------------------------------------------------------------------- refusals (no GPU)
def _weight():
    return moe.Int8Weight(1 << 20, 1 << 21)


def _matmul(x=1 << 22, xs=1 << 23, T=4, K=64, w=None, N=32, out=1 << 24, dtype=0, ldo=32, status=0, null_w=False):
    w = w or _weight()
    return moe.lib().muse_int8_matmul(x, xs, T, K, None if null_w else ctypes.byref(w), N, out, dtype, ldo, status, None)


def test_product_refuses_bad_arguments_before_any_launch():
    for bad in (dict(x=0), dict(x=(1 << 22) + 8), dict(xs=0), dict(xs=(1 << 23) + 2), dict(T=-1), dict(K=0),
                dict(K=24), dict(N=0), dict(out=0), dict(out=(1 << 24) + 2), dict(dtype=2), dict(ldo=31),
                dict(null_w=True), dict(w=moe.Int8Weight(0, 1 << 21)), dict(w=moe.Int8Weight((1 << 20) + 4, 1 << 21)),
                dict(w=moe.Int8Weight(1 << 20, 0)), dict(status=2)):
        assert _matmul(**bad) == 1, bad
    assert _matmul(K=131072 + 16) == 2
    assert _matmul(T=(1 << 24) + 1) == 2
    assert _matmul(T=0) == 0                     # nothing to do: nothing is launched
    assert _matmul(out=(1 << 24) + 2, dtype=1, K=24) == 1


def test_linear_refuses_bad_arguments_before_any_launch():
    w = _weight()
    n = ctypes.c_size_t(0)
    lib = moe.lib()
    assert lib.muse_int8_linear_workspace_size(4, 64, ctypes.byref(n)) == 0 and n.value >= 4 * 64 + 16

    def call(x=1 << 22, xd=1, T=4, K=64, ldx=64, ws=1 << 25, nb=n.value, out=1 << 24, od=1, ldo=32):
        return lib.muse_int8_linear(x, xd, T, K, ldx, ctypes.byref(w), 32, out, od, ldo, ws, nb, None, None)
    for bad in (dict(x=0), dict(x=(1 << 22) + 1), dict(xd=3), dict(ldx=63), dict(K=40), dict(out=0), dict(ldo=8)):
        assert call(**bad) == 1, bad
    assert call(ws=0) == 3 and call(ws=(1 << 25) + 64) == 3 and call(nb=n.value - 1) == 3
    assert call(T=0) == 0
    assert lib.muse_int8_linear_workspace_size(4, 24, ctypes.byref(n)) == 1
    assert lib.muse_int8_linear_workspace_size(4, 64, None) == 1


def test_quantiser_refuses_bad_arguments_before_any_launch():
    def call(src=1 << 20, dtype=0, rows=3, K=32, ld=32, codes=1 << 21, scales=1 << 22):
        return moe.lib().muse_quantize_int8_rows(src, dtype, rows, K, ld, codes, scales, None)
    for bad in (dict(src=0), dict(src=(1 << 20) + 2), dict(dtype=5), dict(rows=-1), dict(K=8), dict(K=20), dict(ld=31),
                dict(codes=0), dict(codes=(1 << 21) + 8), dict(scales=0), dict(scales=(1 << 22) + 1)):
        assert call(**bad) == 1, bad
    assert call(K=(1 << 20) + 16, ld=1 << 21) == 2
    assert call(rows=0) == 0


def test_outputs_over_inputs_are_refused():
    base, far = 1 << 22, 1 << 26

    def quantise(codes, scales, ld=64):  # float32 [3, 64]
        return moe.lib().muse_quantize_int8_rows(base, 0, 3, 64, ld, codes, scales, None)
    for at in (base, base + 2 * 4 * 64 + 3 * 64):
        assert quantise(at, far) == 1
    assert quantise(base - 3 * 64 + 16, far) == 1
    assert quantise(far, base + 764) == 1
    size = dict(K=64, N=32)
    # x codes [4, 64] at base; out float32 [4, 32]
    for out in (base, base + 252, base - 4 * 4 * 32 + 4):
        assert _matmul(x=base, out=out, **size) == 1
    assert _matmul(out=(1 << 20) + 2044, **size) == 1             # over the weights' codes
    assert _matmul(out=(1 << 21) + 124, **size) == 1              # over their scales
    assert _matmul(out=(1 << 23) + 12, **size) == 1               # over x's scales
    w, n = _weight(), ctypes.c_size_t(0)
    moe.lib().muse_int8_linear_workspace_size(4, 64, ctypes.byref(n))

    def linear(out, ldx, ldo, nb=n.value):  # bf16 in and out; nb one short: accepted arguments give 3
        return moe.lib().muse_int8_linear(base, 1, 4, 64, ldx, ctypes.byref(w), 32, out, 1, ldo, far, nb, None, None)
    assert linear(base, 64, 32) == 1 and linear(base + 2 * 64, 128, 64) == 1
    # column ranges of one buffer of 128 columns: after the inputs, one too early, wrapped into the next row
    assert linear(base + 2 * 64, 128, 128, 0) == 3 and linear(base + 2 * 96, 128, 128, 0) == 3
    assert linear(base + 2 * 63, 128, 128) == 1 and linear(base + 2 * 97, 128, 128) == 1
    assert linear(base - 2 * 32, 128, 128, 0) == 3 and linear(base - 2 * 31, 128, 128) == 1


def test_binding_refuses_wrong_tensors():
    codes, scales = torch.zeros(32, 64, dtype=torch.int8), torch.zeros(32)
    with pytest.raises(ValueError):
        moe.Int8Linear(codes.float(), scales, T_max=4)
    with pytest.raises(ValueError):
        moe.Int8Linear(codes, scales[:31], T_max=4)
    with pytest.raises(ValueError):
        moe.Int8Linear(codes.t(), scales, T_max=4)
    with pytest.raises(ValueError):
        moe.Int8Linear(codes, scales, T_max=4)           # not on a GPU
    with pytest.raises(moe.MuseError):
        moe.Int8Linear(codes[:, :24].contiguous(), scales, T_max=4)
    with pytest.raises(ValueError):
        moe.quantize_int8_rows(torch.zeros(4, 32, dtype=torch.float64))
    with pytest.raises(ValueError):
        moe.quantize_int8_rows(torch.zeros(32, 4).t())
    with pytest.raises(ValueError):
        moe.quantize_int8_rows(torch.zeros(4, 32))       # not on a GPU
