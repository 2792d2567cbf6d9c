"""Weights that a caller replaces after the holder was made, by an entry of layer.w or under the
same tensor object: every call computes with what the holder holds then."""
import pytest
import torch

import latent_mixture_experts_moe_b200 as moe
import workloads as W


@pytest.fixture(scope="module", autouse=True)
def built():
    from latent_mixture_experts_moe_b200 import build
    build.build()
    yield


OPTIONS = ("router_bias", "pre_norm_gain", "ffn_pre_gain", "ffn_post_gain", "residual_gate")


def make(seed, experts="bf16"):
    w = W.Workload("replaced", T=6, D=256, L=256, I=256, E=8, k=2, dtype="bf16", seed=seed, experts=experts)
    inp = W.make_inputs(w, "cuda")
    inp.update(W.sublayer_inputs(w, "cuda"))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    inp["router_bias"] = torch.empty(w.E, device="cuda").normal_(0.0, 0.5, generator=gen)
    inp["pre_norm_gain"] = torch.empty(w.L, dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.3, generator=gen)
    x = inp.pop("x")
    return w, x, inp


def layer_of(w, weights):
    return moe.LatentMoE(dict(weights), T_max=w.T, k=w.k, eps=w.eps)


def both(layer, x):
    return layer.few_tokens(x).clone(), layer(x).clone()


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["entry", "storage"])
@pytest.mark.parametrize("name", ("W_router", "W_pool", "W_unpool", "gamma", "W_gate", "W_up", "W_down") + OPTIONS)
def test_a_replaced_weight_is_used(name, how):
    w, x, weights = make(1)
    other = make(2)[2][name]
    layer = layer_of(w, {n: t.clone() for n, t in weights.items()})
    before = both(layer, x)
    kept = layer.w[name]                             # (its memory lives on: the old address stays readable)
    old = kept.data
    if how == "entry":
        layer.w[name] = other
    else:
        kept.data = other.clone()
    got = both(layer, x)
    want = both(layer_of(w, dict(weights, **{name: other})), x)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not torch.equal(want[0], before[0])
    del old


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["W_gate_codes", "W_down_scales", "W_up_mscale"])
def test_a_replaced_part_of_nvfp4_experts_is_used(name):
    w, x, weights = make(3, "nvfp4")
    other = make(4, "nvfp4")[2][name]
    layer = layer_of(w, weights)
    both(layer, x)
    old, layer.w[name] = layer.w[name], other
    want = both(layer_of(w, dict(weights, **{name: other})), x)
    assert all(torch.equal(a, b) for a, b in zip(both(layer, x), want))
    del old


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["entry", "storage"])
def test_replaced_int8_projections_are_used(how):
    w, x, weights = make(5)
    for n in ("W_pool", "W_unpool"):
        weights[n + "_codes"], weights[n + "_scales"] = moe.quantize_int8_rows(weights.pop(n))
    codes, scales = moe.quantize_int8_rows(make(6)[2]["W_pool"])
    layer = layer_of(w, {n: t.clone() for n, t in weights.items()})
    layer(x)
    old = [layer.w["W_pool_codes"].data, layer.w["W_pool_scales"].data]
    if how == "entry":
        layer.w["W_pool_codes"], layer.w["W_pool_scales"] = codes, scales
    else:
        layer.w["W_pool_codes"].data, layer.w["W_pool_scales"].data = codes.clone(), scales.clone()
    want = layer_of(w, dict(weights, W_pool_codes=codes, W_pool_scales=scales))(x)
    assert torch.equal(layer(x), want)
    del old


@pytest.mark.gpu
def test_settings_are_read_at_each_call():
    w, x, weights = make(8)
    layer = layer_of(w, weights)
    both(layer, x)
    layer.modes["pre_norm_eps"] = 1.0
    layer.dims["eps"] = 0.5
    want = both(moe.LatentMoE(dict(weights), T_max=w.T, k=w.k, eps=0.5, pre_norm_eps=1.0), x)
    assert all(torch.equal(a, b) for a, b in zip(both(layer, x), want))


@pytest.mark.gpu
def test_replacements_that_do_not_fit_are_refused():
    w, x, weights = make(9)
    layer = layer_of(w, weights)
    kept = dict(layer.w)
    for name, bad in (("W_router", weights["W_router"].float()), ("gamma", weights["gamma"][:4]),
                      ("W_pool", weights["W_pool"].t())):
        layer.w[name] = bad
        with pytest.raises(moe.MuseError):
            layer.few_tokens(x)
        with pytest.raises(moe.MuseError):
            layer(x)
        layer.w[name] = kept[name]
    layer.w["gamma"] = kept["gamma"].cpu()           # (never reaches the library)
    with pytest.raises(ValueError):
        layer.few_tokens(x)
    layer.w["gamma"] = kept["gamma"]
    assert bool(torch.isfinite(layer.few_tokens(x)).all())


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused():
    """Weights, options, workspaces, inputs and outputs alike, before anything reaches the library."""
    w, x, weights = make(10)
    layer = layer_of(w, weights)
    want = both(layer, x)

    def refused(**kw):
        for call in (layer.few_tokens, layer):
            with pytest.raises(ValueError):
                call(kw.get("x", x), **{n: t for n, t in kw.items() if n != "x"})
    for name in ("W_router", "W_pool", "W_down", "gamma", "router_bias", "residual_gate"):
        kept, layer.w[name] = layer.w[name], layer.w[name].cpu()
        refused()
        layer.w[name] = kept
    refused(x=x.cpu())
    refused(out=torch.empty_like(x).cpu())
    refused(topk_idx=torch.empty(w.T, w.k, dtype=torch.int32))
    refused(topk_w=torch.empty(w.T, w.k))
    kept = layer.workspace, layer.few_workspace
    layer.workspace, layer.few_workspace = (t.cpu() for t in kept)
    refused()
    layer.workspace, layer.few_workspace = kept
    assert all(torch.equal(a, b) for a, b in zip(both(layer, x), want))


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["attribute", "storage"])
@pytest.mark.parametrize("T", [3, 40])
def test_replaced_weights_of_a_product_are_used(T, how):
    gen = torch.Generator(device="cuda").manual_seed(7)
    a, b = (moe.quantize_int8_rows(torch.randn(96, 128, device="cuda", generator=gen)) for _ in range(2))
    x = torch.randn(T, 128, device="cuda", generator=gen)
    lin = moe.Int8Linear(a[0].clone(), a[1].clone(), T_max=T)
    lin(x)
    old = [lin.codes.data, lin.scales.data]
    if how == "attribute":
        lin.codes, lin.scales = b
    else:
        lin.codes.data, lin.scales.data = b[0].clone(), b[1].clone()
    other = moe.Int8Linear(*b, T_max=T)
    assert torch.equal(lin(x), other(x))
    xc, xs = moe.quantize_int8_rows(x)
    assert torch.equal(lin.matmul(xc, xs), other.matmul(xc, xs))
    del old


@pytest.mark.gpu
def test_replacements_that_do_not_fit_a_product_are_refused():
    codes, scales = moe.quantize_int8_rows(torch.randn(64, 128, device="cuda"))
    lin = moe.Int8Linear(codes, scales, T_max=4)
    x = torch.randn(4, 128, device="cuda")
    good = lin(x)
    for bad in ((codes[:, :64], scales), (codes[:32], scales[:32]), (codes, scales[:32]), (codes.float(), scales),
                (codes, scales.cpu()), (codes.cpu(), scales)):
        lin.codes, lin.scales = bad
        with pytest.raises(ValueError):
            lin(x)
    lin.codes, lin.scales = codes, scales
    assert torch.equal(lin(x), good)
