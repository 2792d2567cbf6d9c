"""Outputs that a call makes for another stream than the current one: memory that was freed on the
current stream, where work that still writes it is pending, must not be theirs."""
import pytest
import torch

import latent_mixture_experts_moe_b200 as moe
import workloads as W
from latent_mixture_experts_moe_b200 import ep


@pytest.fixture(scope="module", autouse=True)
def built():
    from latent_mixture_experts_moe_b200 import build
    build.build()
    yield


def calls():
    """name -> (call of a stream, its output tensors)"""
    w = W.Workload("streams", T=8, D=1024, L=256, I=256, E=8, k=2, dtype="bf16", seed=2)
    inp = W.make_inputs(w, "cuda")
    x = inp.pop("x")
    layer = moe.LatentMoE(inp, T_max=8, k=w.k, eps=w.eps)
    wc, ws = moe.quantize_int8_rows(torch.randn(512, 1024, device="cuda"))
    lin = moe.Int8Linear(wc, ws, T_max=8)
    xc, xs = moe.quantize_int8_rows(x)
    shard = ep.ExpertShard(inp, 0, 1, T_max=8, k=w.k, eps=w.eps)
    z, e, _ = shard.dispatch(x)
    y, ss = shard.experts(z, e)
    torch.cuda.synchronize()
    return {"few_tokens": lambda s: (layer.few_tokens(x, stream=s),),
            "forward": lambda s: (layer(x, stream=s),),
            "linear": lambda s: (lin(x, stream=s),),
            "matmul": lambda s: (lin.matmul(xc, xs, stream=s),),
            "quantise": lambda s: moe.quantize_int8_rows(x, stream=s),
            "ep_experts": lambda s: shard.experts(z, e, stream=s),
            "ep_combine": lambda s: (shard.combine(x, y, ss, stream=s),)}


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", ["few_tokens", "forward", "linear", "matmul", "quantise", "ep_experts", "ep_combine"])
def test_output_memory_belongs_to_the_stream_of_the_call(name, handle):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, freed while the current stream has yet to write them
    held = [torch.empty_like(t) for t in want for _ in range(8)]
    torch.cuda._sleep(40_000_000)                     # about 20 ms
    for t in held:
        t.fill_(7)
    blocks = {t.data_ptr() for t in held}
    del held, t
    got = call(side.cuda_stream if handle else side)
    assert not blocks & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.gpu
def test_default_stream_by_its_handle():
    call = calls()["linear"]
    want = call(None)[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(0)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
