"""Captured forwards of a layer: later calls on the layer leave their replays alone, and
they leave the layer's own calls alone."""
import dataclasses

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_ffn_forward_b200 import block, moe, synth  # noqa: E402

MX = dataclasses.replace(synth.TINY, name="MXFP4 layer", hidden=512, inter=256, n_experts=24, top_k=4, n_shared=2, gating=1,
                         seed=61, router_std=1 / 512 ** 0.5, quants=(moe.MOE_MXFP4,) * 3)
Q4 = dataclasses.replace(synth.TINY, seed=5, n_shared=1)


@pytest.fixture(params=["forward", "forward_mx"])
def layer(request):
    """(a new layer, its forward, activations of T tokens)."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from routed_expert_ffn_forward_b200 import build
    from routed_expert_ffn_forward_b200.layer import layer_from_config
    build.build()
    moe.moe_set_cache_bytes(moe.SIZE_MAX)
    cfg = MX if request.param == "forward_mx" else Q4
    L = layer_from_config(cfg)
    if request.param == "forward_mx":
        L.mx_experts_from_host()

    def x(T, seed=0):
        v = synth.activations(dataclasses.replace(cfg, seed=seed), tokens=T)
        return torch.from_numpy(np.ascontiguousarray(v).view(np.int16)).view(torch.bfloat16).cuda()

    yield L, getattr(L, request.param), x
    block.check()
    moe.moe_check(L.handle)
    L.destroy()


@pytest.mark.parametrize("T", [1, 8])
def test_a_captured_forward_and_larger_batches(layer, T):
    L, forward, x = layer
    xs = [x(T, seed) for seed in range(3)]
    want = [forward(v) for v in xs]
    buf = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(buf)
    moe.moe_check(L.handle)                          # behind a capture
    graph.replay()
    moe.moe_check(L.handle)
    assert torch.equal(out, want[0])
    big = x(100, 7)                                  # new scratch, twice
    wide = [forward(big), forward(x(300, 7))]
    assert torch.equal(forward(xs[1]), want[1])
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
    for i in (1, 2, 0):
        buf.copy_(xs[i])
        graph.replay()
        assert torch.equal(out, want[i])
    assert torch.equal(forward(big), wide[0]) and all(torch.isnan(t).all() for t in junk)
    # a second graph, on the new scratch, beside the first
    buf2 = big.clone()
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        out2 = forward(buf2)
    for _ in range(3):
        graph.replay()
        graph2.replay()
    moe.moe_check(L.handle)
    assert torch.equal(out, want[0]) and torch.equal(out2, wide[0])


def test_a_first_forward_in_a_capture_is_refused(layer):
    """It would allocate scratch: refused before it does, and what was captured beside it is sound."""
    L, forward, x = layer
    small, big = x(8), x(100)
    want = forward(small)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(moe.MoEError) as e:
            forward(big)
        out = forward(small)
    assert e.value.status == moe.MOE_ERR_NOT_READY
    graph.replay()
    assert torch.equal(out, want)
    wide = forward(big)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(big)
    graph.replay()
    assert torch.equal(out, wide)


def test_other_mx_experts_wait_for_the_last_forward(layer):
    """The old images are the caller's again when the call returns."""
    L, forward, x = layer
    if forward.__name__ != "forward_mx":
        pytest.skip("MXFP4 experts")
    v = x(8)
    want, old = forward(v), L.mx
    new = tuple(w._replace(image=w.image.clone()) for w in old)
    torch.cuda.synchronize()
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(0.3e9 * 1.9))
        out = forward(v)
        done.record()
    L.set_mx_experts(*new)
    assert done.query()
    for w in old:
        w.image.zero_()
    assert torch.equal(out, want) and torch.equal(forward(v), want)
