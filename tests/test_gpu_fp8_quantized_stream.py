"""Fp8LayerWeights.quantized on a stream other than the current one: the tensors that it allocates
may lie in memory that work queued on the current stream still reads."""
import pytest
import torch

import mtfm_synth as syn
from gpu_helpers import bf16_tensor, f32_tensor

pytestmark = pytest.mark.gpu


def layer(d=512):
    import hybrid_masked_attention_b200 as M
    w, = syn.stack_weights(syn.PAIR_HEADS, d, 7, kinds=("T",), std=0.05, std_o=0.01, random_norms=True)
    return M.LayerWeights(w.kind, f32_tensor(w.rms_w), bf16_tensor(w.w_in), bf16_tensor(w.w_kv), bf16_tensor(w.w_o),
                          f32_tensor(w.gamma), f32_tensor(w.beta))


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
               for p, q in ((a.w_in, b.w_in), (a.w_kv, b.w_kv), (a.w_o, b.w_o)) for x, y in zip(p, q))


@pytest.mark.parametrize("raw", [False, True])
def test_memory_that_the_current_stream_still_reads(raw, cuda_ok):
    import hybrid_masked_attention_b200 as M
    w = layer()
    want = M.Fp8LayerWeights.quantized(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # a block of the size of w_in's bytes and one of its scales', each read by work that starts late
    held = [torch.full(t.shape, 7, dtype=torch.uint8, device="cuda") for t in (want.w_in[0], want.w_kv[0], want.w_o[0])]
    small = torch.full((4096,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)              # about 0.1 s on the current stream
    seen = [t + 0 for t in held]
    del held, small
    got = M.Fp8LayerWeights.quantized(w, stream=side.cuda_stream if raw else side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in seen)
    assert same(got, want)


def test_outputs_freed_before_the_quantiser_ran(cuda_ok):
    """Tensors dropped while the side stream has yet to write them are not handed out meanwhile."""
    import hybrid_masked_attention_b200 as M
    w = layer()
    M.Fp8LayerWeights.quantized(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = M.Fp8LayerWeights.quantized(w, stream=side)
    shapes = [t.shape for p in (got.w_in, got.w_kv, got.w_o) for t in p]
    del got
    fresh = [torch.full(s, 9, dtype=torch.uint8, device="cuda") for s in shapes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((t == 9).all()) for t in fresh)


def test_weights_written_on_the_current_stream(cuda_ok):
    """The quantiser reads weights that the current stream has yet to write."""
    import hybrid_masked_attention_b200 as M
    w = layer()
    want = M.Fp8LayerWeights.quantized(w)
    value = w.w_in.clone()
    w.w_in.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    w.w_in.copy_(value)
    got = M.Fp8LayerWeights.quantized(w, stream=side)
    torch.cuda.synchronize()
    assert same(got, want)


def test_quantized_in_a_capture(cuda_ok):
    """On the capture's own stream and without one, replayed on new weights."""
    import hybrid_masked_attention_b200 as M
    w = layer()
    M.Fp8LayerWeights.quantized(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = M.Fp8LayerWeights.quantized(w)
        b = M.Fp8LayerWeights.quantized(w, stream=torch.cuda.current_stream())
    w.w_in.mul_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    want = M.Fp8LayerWeights.quantized(w)
    assert same(a, want) and same(b, want)
