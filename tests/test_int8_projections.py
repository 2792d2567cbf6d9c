"""The block with int8 pooler and unpooler weights. The two projections are exact integers times
two scales, so what the forward writes around them is compared bit for bit: z with the product
of the quantised input rows, the output with the product of the quantised combined latent that
the forward stored."""
import ctypes

import numpy as np
import pytest
import torch

import latent_mixture_experts_moe_b200 as moe
import oracle
import workloads as W
from latent_mixture_experts_moe_b200 import ep
from parity_util import assert_close, host, oracle_block, ws_view
from test_int8 import ref_product, ref_quantise, to_dtype


@pytest.fixture(scope="module", autouse=True)
def built():
    from latent_mixture_experts_moe_b200 import build
    build.build()
    yield


def int8_weights(inp):
    """inp with W_pool and W_unpool quantised per output channel."""
    w = {n: t for n, t in inp.items() if n not in ("x", "W_pool", "W_unpool")}
    for name in ("W_pool", "W_unpool"):
        w[name + "_codes"], w[name + "_scales"] = moe.quantize_int8_rows(inp[name])
    return w


def product(rows, w, name, dtype):
    codes, scales = ref_quantise(host(rows).astype(np.float32))
    return to_dtype(ref_product(codes, scales, w[name + "_codes"].cpu().numpy(), w[name + "_scales"].cpu().numpy()), dtype)


CASES = [
    # name, T, D, L, I, E, k, dtype, experts, act
    ("one_token", 1, 512, 256, 256, 8, 2, "bf16", "bf16", "bf16"),
    ("few", 24, 640, 384, 128, 9, 3, "bf16", "bf16", "bf16"),
    ("f32", 40, 512, 256, 384, 8, 2, "f32", "bf16", "bf16"),
    ("pairs", 300, 1152, 512, 256, 16, 4, "bf16", "bf16", "bf16"),
    ("many", 5000, 1024, 512, 256, 16, 2, "bf16", "bf16", "bf16"),
    ("w4a16", 70, 768, 512, 256, 16, 4, "bf16", "nvfp4", "bf16"),
    ("w4a4", 130, 512, 512, 256, 8, 4, "bf16", "nvfp4", "nvfp4"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_projections_bit_exact_inside_the_forward(case):
    name, T, D, L, I, E, k, dtype, experts, act = case
    w = W.Workload(name, T=T, D=D, L=L, I=I, E=E, k=k, dtype=dtype, seed=3, experts=experts, act=act)
    inp = W.make_inputs(w, "cuda")
    weights = int8_weights(inp)
    modes = dict(act_format=moe.ACT_NVFP4) if act == "nvfp4" else {}
    layer = moe.LatentMoE(weights, T_max=T, k=k, eps=w.eps, **modes)
    out = layer(inp["x"])
    cfg = layer.config(T, layer.workspace)
    assert moe.last_device_status(cfg) == (0, 0)
    lay, dt = moe.workspace_layout(cfg), inp["x"].dtype
    z = ws_view(layer.workspace, lay["z"], dt, (T, L))
    c = ws_view(layer.workspace, lay["c"], dt, (T, L))
    assert torch.equal(z.cpu(), product(inp["x"], weights, "W_pool", dt))
    assert torch.equal(out.cpu(), product(c, weights, "W_unpool", dt))
    # end to end against the block with the original weights: four quantisations (x, W_pool, c,
    # W_unpool) of at most 4.5 rms / 127 / sqrt(12) = 1.0 % each, the first two through the experts
    # (factor at most 2.1): 0.0102 sqrt(2 * 2.1^2 + 2) = 3.4 %; W4A4's own 4-bit error comes on top
    if act != "nvfp4":
        rows = np.arange(0, T, max(1, T // 24))
        ref = oracle_block(w, inp, rows)
        assert_close(host(out)[rows], ref["out"], name, rel=0.05, max_abs_rms=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 200, 3840])
def test_sublayer_and_pre_norm(T):
    """With the feed-forward sublayer: the pooler reads the normalised rows, the unpooler's output
    goes through post norm and gate, its sums of squares taken before rounding."""
    w = W.Workload("sublayer", T=T, D=1152, L=256, I=128, E=8, k=2, dtype="bf16", seed=7)
    inp = W.make_inputs(w, "cuda")
    inp.update(W.sublayer_inputs(w, "cuda"))
    weights = int8_weights(inp)
    weights["pre_norm_gain"] = (torch.randn(w.L, generator=torch.Generator().manual_seed(1)) * 0.3).bfloat16().cuda()
    layer = moe.LatentMoE(weights, T_max=T, k=w.k, eps=w.eps)
    out = layer(inp["x"])
    cfg = layer.config(T, layer.workspace)
    assert moe.last_device_status(cfg) == (0, 0)
    lay = moe.workspace_layout(cfg)
    xn = ws_view(layer.workspace, lay["xn"], torch.bfloat16, (T, w.D))
    z = ws_view(layer.workspace, lay["z"], torch.bfloat16, (T, w.L))
    c = ws_view(layer.workspace, lay["c"], torch.bfloat16, (T, w.L))
    pooled = host(product(xn, weights, "W_pool", torch.bfloat16))
    zn = oracle.centred_rmsnorm(pooled, host(weights["pre_norm_gain"]), 1e-5)
    assert_close(host(z), zn, "z", rel=2.0 ** -8, max_abs_rms=2.0 ** -8 * 8)
    # f is rounded to bf16 before the scale, then the result: 2 * 2^-8 at worst
    codes, scales = ref_quantise(host(c).astype(np.float32))
    f = ref_product(codes, scales, weights["W_unpool_codes"].cpu().numpy(), weights["W_unpool_scales"].cpu().numpy()).astype(np.float64)
    fn = oracle.input_scaled_rmsnorm(f, host(inp["ffn_post_gain"]), 1e-8)
    ref = oracle.residual_gate(host(inp["x"]), fn, host(inp["residual_gate"]), 0.3, 1e-3)
    assert_close(host(out), ref, "sublayer output", rel=2.0 ** -7, max_abs_rms=2.0 ** -7 * 8)


@pytest.mark.gpu
def test_replayed_graph_static_scratch_and_expert_parallel_agree():
    w = W.Workload("agree", T=48, D=512, L=256, I=256, E=8, k=2, dtype="bf16", seed=9)
    inp = W.make_inputs(w, "cuda")
    weights = int8_weights(inp)
    layer = moe.LatentMoE(weights, T_max=w.T, k=w.k, eps=w.eps)
    x = inp["x"]
    ref = layer(x).clone()
    out = torch.empty_like(ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer(x, out=out, stream=side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    shards = []
    for r in range(2):
        part = dict(weights, **{n: weights[n][4 * r:4 * r + 4].contiguous() for n in ("W_gate", "W_up", "W_down")})
        shards.append(ep.ExpertShard(part, r, 2, T_max=w.T, k=w.k, eps=w.eps))
    outs = ep.ep_forward_one_device(shards, [x[:20].contiguous(), x[20:].contiguous()])
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(list(outs)), ref)


# ------------------------------------------------------------------------- refusals (no GPU)
def _cfg(T=64):
    c = moe.make_config(T, 1024, 512, 256, 16, 2, "bf16")
    c.proj_weights = moe.PROJ_INT8
    return c


def test_descriptions_are_checked_before_any_launch():
    cfg, lib = _cfg(), moe.lib()
    args = [ctypes.c_void_p(4096 * (i + 1)) for i in range(9)]
    good = moe.Int8Weight(1 << 20, 1 << 21)

    def call(pool=good, unpool=good):
        a = list(args)
        a[2] = ctypes.c_void_p(ctypes.addressof(pool) if pool is not None else 0)     # x, W_router, W_pool, ...
        a[7] = ctypes.c_void_p(ctypes.addressof(unpool) if unpool is not None else 0)
        order = [0, 1, 2, 3, 4, 5, 6, 7, 8]
        return lib.muse_latent_moe_forward(ctypes.byref(cfg), *[a[i] for i in order], None)
    assert call() == 3                                           # fine: no workspace
    for bad in (None, moe.Int8Weight(0, 1 << 21), moe.Int8Weight((1 << 20) + 8, 1 << 21), moe.Int8Weight(1 << 20, 0),
                moe.Int8Weight(1 << 20, (1 << 21) + 2)):
        assert call(pool=bad) == 1
        assert call(unpool=bad) == 1
    n = ctypes.c_size_t(0)
    assert lib.muse_latent_moe_few_tokens_workspace_size(ctypes.byref(_cfg(4)), ctypes.byref(n)) == 2
    cfg.proj_weights = 5
    assert lib.muse_latent_moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == 1


def test_checked_forward_takes_two_descriptors_a_projection():
    from test_capi import _call_checked, _checked_args, _desc
    cfg = _cfg()

    def args():
        a = _checked_args(cfg)
        a["W_pool"] = (moe.Tensor * 2)(_desc(3 << 45, moe.ELEM_I8, (cfg.L, cfg.D)), _desc(5 << 45, moe.ELEM_F32, (cfg.L,)))
        a["W_unpool"] = (moe.Tensor * 2)(_desc(7 << 45, moe.ELEM_I8, (cfg.D, cfg.L)), _desc(9 << 45, moe.ELEM_F32, (cfg.D,)))
        return a
    assert _call_checked(cfg, args()) == 3                       # shapes fine: no workspace
    for name in ("W_pool", "W_unpool"):
        for part in range(2):
            for change in (lambda d: d.shape.__setitem__(0, d.shape[0] + 1), lambda d: setattr(d, "elem", moe.ELEM_U8),
                           lambda d: setattr(d, "data", 0), lambda d: d.stride.__setitem__(d.ndim - 1, 2)):
                a = args()
                change(a[name][part])
                assert _call_checked(cfg, a) == 1, (name, part)
        a = args()
        a["out"].data = a[name][0].data + 4096
        assert _call_checked(cfg, a) == 1


def test_stages_name_the_quantisers():
    names = moe.stages(_cfg())
    assert len(names) == moe.launch_count(_cfg()) == 13
    assert names.index("quant_x") + 1 == names.index("pooler")
    assert names.index("quant_c") + 1 == names.index("unpooler")
    assert moe.workspace_size(_cfg()) > moe.workspace_size(moe.make_config(64, 1024, 512, 256, 16, 2, "bf16"))
