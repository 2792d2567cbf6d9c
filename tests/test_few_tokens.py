"""The whole layer for a few tokens in one kernel, against the FP64 oracle on the same inputs.

Tolerances. Per rounding a relative error of at most eps / 2 (bf16 2^-8, f16 2^-11, float32
2^-24). bf16: z, h and c are carried to 2^-16 (two bf16 numbers), so the output's own rounding, at
most 2^-8 of every element, is what remains: 2^-8 (1 + 2^-4) with the rest (the sublayer's xn is one
bf16 number in the oracle too; test_few_tokens_precision.py holds the arithmetic closer).
NVFP4 experts: z and h in f16, c to 2^-16, out in bf16: 2^-8 + 3.1 * 2^-11 + 2^-16 = 5.5e-3 < 1e-2
at worst. float32: only sums, of K <= 8192 products, whose rounding grows like sqrt(K) 2^-24 =
5.4e-6 at most for each of the four products in a row: 2.2e-5. Largest deviations: the
block's 5e-2 of the rms (float32: 2.2e-5 * 5 rms, 5 standard deviations)."""
import ctypes
import dataclasses

import numpy as np
import pytest
import torch

import latent_mixture_experts_moe_b200 as moe
import oracle
import workloads as W
from parity_util import assert_close, check_routing, host, oracle_block, oracle_on_gpu_alternatives

RELEASED = dict(router_mode=moe.ROUTER_SIGMOID, router_logit_scale=32 ** -0.5, routed_scaling=2.5,
                norm_mode=moe.NORM_INPUT_SCALED, gamma_shared=True)
SUBLAYER_KEYS = ("ffn_pre_gain", "ffn_post_gain", "residual_gate")


@pytest.fixture(scope="module", autouse=True)
def built():
    from latent_mixture_experts_moe_b200 import build
    build.build()
    yield


def workload(name, T, D, L, I, E, k, dtype="bf16", experts=None, seed=5):
    return W.Workload(name, T=T, D=D, L=L, I=I, E=E, k=k, dtype=dtype, seed=seed,
                      experts=experts or "bf16")


def oracle_modes(modes):
    kw = {}
    if modes.get("router_mode") == moe.ROUTER_SIGMOID:
        kw.update(router_mode="sigmoid", logit_scale=modes["router_logit_scale"], routed_scaling=modes["routed_scaling"])
    if modes.get("norm_mode") == moe.NORM_INPUT_SCALED:
        kw.update(norm_mode="input_scaled")
    return kw


def make_inputs(w, modes=(), extra=()):
    """Seeded inputs; extra: optional gains and gates, a router bias, by name."""
    inp = W.make_inputs(w, "cuda")
    g = torch.Generator(device="cuda").manual_seed(w.seed + 100)
    act = inp["x"].dtype

    def normal(n, std, dtype=act):
        return torch.empty(n, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)
    for name in extra:
        inp[name] = {"router_bias": lambda: normal(w.E, 0.05, torch.float32), "pre_norm_gain": lambda: normal(w.L, 0.3),
                     "ffn_pre_gain": lambda: normal(w.D, 0.3), "ffn_post_gain": lambda: normal(w.D, 0.3),
                     "residual_gate": lambda: normal(w.D, 1.0, torch.float32)}[name]()
    if dict(modes).get("gamma_shared"):
        inp["gamma"] = inp["gamma"][0].contiguous()
    return inp


class Few:
    """One few_tokens call with its routing."""

    def __init__(self, w, inp, T=None, **modes):
        T = w.T if T is None else T
        self.layer = moe.LatentMoE({n: t for n, t in inp.items() if n != "x"}, T_max=max(T, 1), k=w.k, eps=w.eps, **modes)
        self.idx = torch.full((T, w.k), -1, dtype=torch.int32, device="cuda")
        self.g = torch.zeros((T, w.k), dtype=torch.float32, device="cuda")
        self.out = self.layer.few_tokens(inp["x"][:T].contiguous(), topk_idx=self.idx, topk_w=self.g)
        code, detail = moe.few_tokens_status(self.layer.config(T, self.layer.few_workspace))
        assert code == 0, f"device status {moe.STATUS.get(code)} detail {detail:#x}"


def check(w, inp, few, T=None, **kw):
    rows = np.arange(w.T if T is None else T)
    ref = oracle_block(w, inp, rows, **kw)
    gidx = few.idx.cpu().numpy()
    alts = check_routing(ref, gidx, few.g.cpu().numpy(), w.k)
    out = oracle_on_gpu_alternatives(w, inp, rows, ref, gidx, alts, **kw)
    if w.dtype == "f32":
        assert_close(host(few.out), out, w.name, rel=2.2e-5, max_abs_rms=1.1e-4)
    elif w.experts == "bf16":
        assert_close(host(few.out), out, w.name, rel=2.0 ** -8 * (1 + 2.0 ** -4))
    else:
        assert_close(host(few.out), out, w.name)


SHAPES = [
    # name, T, D, L, I, E, k, dtype
    ("one_expert", 1, 128, 128, 128, 1, 1, "bf16"),
    ("all_experts", 2, 256, 128, 256, 6, 6, "bf16"),
    ("top1", 3, 384, 256, 128, 9, 1, "bf16"),
    ("odd_widths", 5, 1152, 640, 896, 40, 6, "bf16"),
    ("wide_latent", 7, 256, 4608, 128, 5, 2, "bf16"),
    ("wide_inner", 4, 128, 128, 4224, 7, 3, "bf16"),
    ("wide_model", 6, 10368, 128, 128, 3, 2, "bf16"),
    ("many_experts", 8, 256, 128, 128, 1000, 8, "bf16"),
    ("many_per_token", 8, 256, 128, 256, 48, 32, "bf16"),
    ("five_on_all", 5, 384, 640, 384, 4, 4, "bf16"),
    ("eight_on_all", 8, 640, 1152, 768, 6, 6, "bf16"),
    ("mid1", 1, 2048, 1024, 1024, 64, 4, "bf16"),
    ("mid8", 8, 2048, 1024, 1024, 64, 4, "bf16"),
    ("tiny_f32", 5, 256, 128, 128, 8, 2, "f32"),
    ("odd_f32", 8, 1152, 640, 896, 24, 5, "f32"),
    ("one_f32", 1, 2048, 1024, 1024, 64, 4, "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", SHAPES, ids=[c[0] for c in SHAPES])
def test_shapes(case):
    w = workload(*case)
    inp = make_inputs(w)
    check(w, inp, Few(w, inp))


MODES = [
    ("released", dict(RELEASED), ("router_bias", "pre_norm_gain")),
    ("softmax_bias", {}, ("router_bias",)),
    ("input_scaled_per_expert", dict(norm_mode=moe.NORM_INPUT_SCALED), ()),
    ("pre_expert_norm", {}, ("pre_norm_gain",)),
    ("sublayer", {}, SUBLAYER_KEYS),
    ("released_sublayer", dict(RELEASED), ("router_bias", "pre_norm_gain") + SUBLAYER_KEYS),
    ("gate_only", {}, ("residual_gate",)),
    ("post_only", {}, ("ffn_post_gain",)),
    ("pre_only", {}, ("ffn_pre_gain",)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32", "nvfp4"])
@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("mode", MODES, ids=[m[0] for m in MODES])
def test_modes(mode, T, kind):
    name, modes, extra = mode
    w = workload(name, T, 640, 512, 768, 20, 4, "f32" if kind == "f32" else "bf16", "nvfp4" if kind == "nvfp4" else None)
    inp = make_inputs(w, modes, extra)
    check(w, inp, Few(w, inp, **modes), **oracle_modes(modes))


NVFP4 = [
    ("nvfp4_small", 1, 128, 256, 256, 4, 2),
    ("nvfp4_odd", 5, 384, 768, 1280, 24, 5),
    ("nvfp4_wide", 8, 512, 4608, 256, 6, 3),
    ("nvfp4_wide_inner", 3, 512, 256, 4352, 6, 3),
    ("nvfp4_mid", 8, 2048, 1024, 1024, 64, 4),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", NVFP4, ids=[c[0] for c in NVFP4])
def test_nvfp4_experts(case):
    w = workload(*case, experts="nvfp4")
    inp = make_inputs(w)
    check(w, inp, Few(w, inp))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32", "nvfp4"])
def test_every_token_on_the_same_experts(kind):
    """A bias that sends all eight tokens to the same experts."""
    w = workload("same", 8, 256, 256, 512, 16, 3, "f32" if kind == "f32" else "bf16", "nvfp4" if kind == "nvfp4" else None)
    inp = make_inputs(w)
    inp["router_bias"] = torch.zeros(w.E, device="cuda")
    inp["router_bias"][[2, 9, 15]] = 100.0
    few = Few(w, inp)
    assert {2, 9, 15} == set(few.idx.flatten().tolist())
    check(w, inp, few)


@pytest.mark.gpu
def test_ties_go_to_the_lower_expert():
    w = workload("ties", 4, 256, 128, 128, 70, 5)
    inp = make_inputs(w)
    inp["W_router"][1:] = inp["W_router"][:1]          # every expert scores the same
    few = Few(w, inp)
    assert few.idx.tolist() == [[0, 1, 2, 3, 4]] * 4
    assert torch.allclose(few.g, torch.full_like(few.g, 0.2), atol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32", "nvfp4"])
def test_a_token_that_is_not_finite_stays_alone(kind):
    w = workload("nan", 6, 256, 256, 256, 12, 3, "f32" if kind == "f32" else "bf16", "nvfp4" if kind == "nvfp4" else None)
    inp = make_inputs(w)
    good = Few(w, inp)
    bad = dict(inp, x=inp["x"].clone())
    bad["x"][2, 5] = float("nan")
    few = Few(w, bad)
    keep = [0, 1, 3, 4, 5]
    assert bool(torch.isnan(few.out[2]).all())
    assert torch.equal(few.idx[keep], good.idx[keep])
    assert len(set(few.idx[2].tolist())) == w.k
    tol = 2.2e-5 if kind == "f32" else 1e-2
    assert_close(host(few.out[keep]), host(good.out[keep]), "other tokens", rel=tol, max_abs_rms=5 * tol)


@pytest.mark.gpu
@pytest.mark.parametrize("experts", ["bf16", "nvfp4"])
def test_repeats_are_bitwise_identical_and_match_the_forward(experts):
    """The same call twice; a wider workspace history (more tokens first); the token-tiled forward
    of the same holder within both paths' roundings."""
    w = workload("repeat", 8, 2048, 1024, 1024, 64, 4, experts=None if experts == "bf16" else experts)
    inp = make_inputs(w)
    few = Few(w, inp)
    x1 = inp["x"][:3].contiguous()
    a = few.layer.few_tokens(x1)
    few.layer.few_tokens(inp["x"])
    few.layer.few_workspace.random_(0, 256)            # whatever the workspace holds
    b = few.layer.few_tokens(x1)
    assert torch.equal(a, b)
    assert torch.equal(few.layer.few_tokens(inp["x"]), few.out)
    full = few.layer(inp["x"])
    assert_close(host(few.out), host(full), "few against forward", rel=2e-2, max_abs_rms=1e-1)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32", "nvfp4"])
def test_captured_and_replayed_on_another_stream(kind):
    w = workload("graph", 8, 1152, 512, 768, 32, 4, "f32" if kind == "f32" else "bf16", "nvfp4" if kind == "nvfp4" else None)
    inp = make_inputs(w, {}, SUBLAYER_KEYS)
    layer = Few(w, inp).layer
    x = inp["x"][:5].contiguous()
    wide = torch.full((8, w.D), 7.0, dtype=x.dtype, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer.few_tokens(x, out=wide[:5], stream=side)
    for seed in range(3):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(wide[:5], layer.few_tokens(x))
    assert bool((wide[5:] == 7.0).all())


@pytest.mark.gpu
def test_two_holders_on_two_streams():
    """Two cooperative launches that compete for the SMs, each with its own workspace."""
    w = workload("streams", 8, 1024, 512, 512, 32, 4)
    inp = make_inputs(w)
    weights = {n: t for n, t in inp.items() if n != "x"}
    a, b = (moe.LatentMoE(weights, T_max=8, k=w.k, eps=w.eps) for _ in range(2))
    xa, xb = inp["x"], inp["x"][:2].contiguous()
    ra, rb = a.few_tokens(xa), b.few_tokens(xb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [(a.few_tokens(xa, stream=sa), b.few_tokens(xb, stream=sb)) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, ra) and torch.equal(q, rb) for p, q in outs)


@pytest.mark.gpu
def test_decode_steps_feed_one_another():
    """Several decoder layers' feed-forward sublayers in a row, one call each: the residual stream
    of one call is the next one's input; each step against the oracle on the step's own input."""
    w = workload("steps", 4, 512, 256, 384, 16, 3)
    layers = []
    for seed in range(3):
        ws = dataclasses.replace(w, seed=seed + 20)
        inp = make_inputs(ws, {}, SUBLAYER_KEYS)
        layers.append((ws, inp, moe.LatentMoE({n: t for n, t in inp.items() if n != "x"}, T_max=4, k=w.k, eps=w.eps)))
    x = layers[0][1]["x"]
    for ws, inp, layer in layers:
        inp = dict(inp, x=x)
        check(ws, inp, Few(ws, inp))
        x = layer.few_tokens(x)


# ------------------------------------------------------------------------- refusals (no GPU)
def _cfg(T=4, dtype="bf16", **kw):
    return moe.make_config(T, 1024, 512, 256, 16, 2, dtype, **kw)


def test_unsupported_configurations_are_refused():
    n = ctypes.c_size_t(0)
    size = moe.lib().muse_latent_moe_few_tokens_workspace_size
    assert size(ctypes.byref(_cfg(8)), ctypes.byref(n)) == 0 and n.value > 0
    assert size(ctypes.byref(_cfg(9)), ctypes.byref(n)) == 2
    assert size(ctypes.byref(_cfg(0)), ctypes.byref(n)) == 1
    assert size(ctypes.byref(_cfg()), None) == 1
    assert size(None, ctypes.byref(n)) == 1
    c = _cfg(act_format=moe.ACT_NVFP4)
    c.expert_weights = moe.EXPERTS_NVFP4
    assert size(ctypes.byref(c), ctypes.byref(n)) == 2
    c = moe.make_config(4, 1024, 384, 256, 16, 2)
    c.expert_weights = moe.EXPERTS_NVFP4
    assert size(ctypes.byref(c), ctypes.byref(n)) == 2
    c = _cfg(dtype="f32")
    c.expert_weights = moe.EXPERTS_NVFP4
    assert size(ctypes.byref(c), ctypes.byref(n)) == 2


def test_workspace_grows_with_tokens_and_options():
    a, b = moe.few_tokens_workspace_size(_cfg(1)), moe.few_tokens_workspace_size(_cfg(8))
    c = _cfg(8)
    c.ffn_pre_gain = c.ffn_post_gain = 4096
    assert a < b < moe.few_tokens_workspace_size(c)


def test_null_misaligned_and_missing_workspace_are_refused_before_any_launch():
    cfg = _cfg()
    lib = moe.lib()
    args = [ctypes.c_void_p(4096 * (i + 1)) for i in range(9)]
    for bad in range(9):
        for v in (0, 4096 * (bad + 1) + 8):
            a = list(args)
            a[bad] = ctypes.c_void_p(v)
            assert lib.muse_latent_moe_few_tokens(ctypes.byref(cfg), *a, None) == 1
    assert lib.muse_latent_moe_few_tokens(ctypes.byref(cfg), *args, None) == 3
    need = moe.few_tokens_workspace_size(cfg)
    for ws, nb in ((1 << 20, need - 1), ((1 << 20) + 128, need)):
        cfg.workspace, cfg.workspace_bytes = ws, nb
        assert lib.muse_latent_moe_few_tokens(ctypes.byref(cfg), *args, None) == 3
    assert lib.muse_latent_moe_few_tokens(None, *args, None) == 1
    cfg.pre_norm_gain = 4098
    assert lib.muse_latent_moe_few_tokens(ctypes.byref(cfg), *args, None) == 1
    assert lib.muse_latent_moe_few_tokens_status(ctypes.byref(_cfg()), None, None) == 3


def test_checked_form_refuses_shapes_and_overlap():
    from test_capi import _checked_args
    cfg = _cfg()
    order = ("x", "W_router", "W_pool", "W_gate", "W_up", "W_down", "gamma", "W_unpool", "out")

    def call(args):
        ptrs = [ctypes.cast(args[n], ctypes.POINTER(moe.Tensor)) if isinstance(args[n], ctypes.Array)
                else ctypes.pointer(args[n]) for n in order]
        return moe.lib().muse_latent_moe_few_tokens_checked(ctypes.byref(cfg), *ptrs, None)
    assert call(_checked_args(cfg)) == 3               # shapes fine: no workspace
    for n in order:
        args = _checked_args(cfg)
        d = args[n][0] if isinstance(args[n], ctypes.Array) else args[n]
        d.shape[0] += 1
        assert call(args) == 1, n
    args = _checked_args(cfg)
    args["out"].data = args["x"].data
    assert call(args) == 1


@pytest.mark.gpu
def test_holder_refuses_routing_outputs_it_cannot_write():
    """Wrong shape, type or layout (the kernel writes [T, k] values one after the other)."""
    w = workload("routing_outputs", 4, 256, 128, 128, 8, 2)
    inp = make_inputs(w)
    layer = moe.LatentMoE({n: t for n, t in inp.items() if n != "x"}, T_max=4, k=w.k, eps=w.eps)
    i32 = dict(dtype=torch.int32, device="cuda")
    for idx in (torch.zeros(4, 3, **i32), torch.zeros(4, 2, dtype=torch.int64, device="cuda"),
                torch.zeros(2, 4, **i32).t(), torch.zeros(1, 2, **i32).expand(4, 2),
                torch.zeros(4, 2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            layer.few_tokens(inp["x"], topk_idx=idx)
    with pytest.raises(ValueError):
        layer.few_tokens(inp["x"], topk_w=torch.zeros(1, 1, device="cuda").expand(4, 2))
