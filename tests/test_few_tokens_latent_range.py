"""Latents outside f16's range before the pre-expert norm. The norm brings them back into it, so
NVFP4 experts, which read the normalised latent as f16, see ordinary values whatever the pooler's
scale. (f16 ends at 65504; below 2^-14 it loses bits, with steps of 2^-24.)"""
import numpy as np
import pytest
import torch

import latent_mixture_experts_moe_b200 as moe
import workloads as W
from parity_util import assert_close, check_routing, host, oracle_block, oracle_on_gpu_alternatives


@pytest.fixture(scope="module", autouse=True)
def built():
    from latent_mixture_experts_moe_b200 import build
    build.build()
    yield


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32", "nvfp4"])
@pytest.mark.parametrize("T", [1, 7])
@pytest.mark.parametrize("scale", [4e4, 4e5, 1e-6], ids=["some_clipped", "most_clipped", "subnormal"])
def test_the_norm_reads_the_latent_in_full(scale, T, kind):
    """Tolerance: the block's own (1e-2), as for ordinary latents: a relative norm does not see
    the scale (its eps, 1e-30 here, is far below the smallest mean square, 1e-12)."""
    w = W.Workload("range", T=T, D=640, L=512, I=768, E=20, k=4, dtype="f32" if kind == "f32" else "bf16", seed=11,
                   experts="nvfp4" if kind == "nvfp4" else "bf16")
    inp = W.make_inputs(w, "cuda")
    inp["W_pool"] = (inp["W_pool"].float() * scale).to(inp["W_pool"].dtype)
    gen = torch.Generator(device="cuda").manual_seed(3)
    inp["pre_norm_gain"] = torch.empty(w.L, dtype=inp["x"].dtype, device="cuda").normal_(0.0, 0.3, generator=gen)
    layer = moe.LatentMoE({n: t for n, t in inp.items() if n != "x"}, T_max=T, k=w.k, eps=w.eps, pre_norm_eps=1e-30)
    idx = torch.empty((T, w.k), dtype=torch.int32, device="cuda")
    g = torch.empty((T, w.k), dtype=torch.float32, device="cuda")
    out = layer.few_tokens(inp["x"], topk_idx=idx, topk_w=g)
    assert moe.few_tokens_status(layer.config(T, layer.few_workspace)) == (0, 0)
    rows = np.arange(T)
    ref = oracle_block(w, inp, rows, pre_norm_eps=1e-30)
    gidx = idx.cpu().numpy()
    alts = check_routing(ref, gidx, g.cpu().numpy(), w.k)
    assert_close(host(out), oracle_on_gpu_alternatives(w, inp, rows, ref, gidx, alts, pre_norm_eps=1e-30), kind)
