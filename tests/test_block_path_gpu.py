"""The operators together, as a block uses them: the norm before, the layer's
router and experts (its own kernels, or MXFP4 products), the balance loss of
its routing, the norm after with gate and residual."""
import dataclasses

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_ffn_forward_b200 import block, moe, synth  # noqa: E402
from tests import block_ref, mx_ref  # noqa: E402

MX = (moe.MOE_MXFP4,) * 3
LAYER = dataclasses.replace(synth.TINY, name="MXFP4 layer", hidden=512, inter=256, n_experts=24, top_k=4, n_shared=2,
                            gating=1, seed=61, router_std=1 / 512 ** 0.5, quants=MX)


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from routed_expert_ffn_forward_b200 import build
    from routed_expert_ffn_forward_b200.layer import layer_from_config
    build.build()
    moe.moe_set_cache_bytes(moe.SIZE_MAX)
    L = layer_from_config(LAYER)
    L.mx_experts_from_host()
    yield L
    block.check()
    moe.moe_check(L.handle)
    L.destroy()


def activations(T, seed=0):
    x = synth.activations(dataclasses.replace(LAYER, seed=seed), tokens=T)
    return torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda()


def chain(L, x):
    """forward_mx from the operators alone, on the layer's routing."""
    T, kS = x.shape[0], L.k + L.S
    ids, w = L.routing(T)
    shared = torch.arange(L.E, L.E + L.S, device="cuda", dtype=torch.int32).expand(T, L.S)
    flat = torch.cat([ids, shared], 1).reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=L.E + L.S)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    index = (order // kS).int()
    gate_up, down = L.mx
    h = block.mx_product(block.mx_quantize(x), gate_up, offsets, index)
    y = block.mx_product(block.mx_quantize(h), down, offsets, out_dtype=torch.float32)
    rows = torch.empty_like(y)
    rows[order] = y
    rows = rows.view(T, kS, L.H)
    acc = torch.zeros((T, L.H), device="cuda", dtype=torch.float64)
    for j in range(kS):
        acc += rows[:, j].double() * (w[:, j:j + 1].double() if j < L.k else 1.0)
    return h, offsets, index, y, acc, rows.double().abs().sum(1)


@pytest.mark.parametrize("T", [1, 3, 16, 70, 300, 1100])
def test_forward_mx_is_the_operators_in_a_row(layer, T):
    L = layer
    x = activations(T, T)
    out = L.forward_mx(x)
    h, offsets, index, y, acc, mag = chain(L, x)
    # the combine rounds kS products and sums in fp32, and the output once
    tol = (L.k + L.S) * 2.0 ** -23 * mag
    err = (out.double() - acc).abs()
    assert bool((err <= tol + 2.0 ** -8 * (acc.abs() + tol) + 1e-30).all())
    assert torch.equal(out, L.forward_mx(x))
    # y against the definition from the codes of x's rows and of h
    wv = mx_ref.unpack(*(t.cpu().numpy() for t in L_codes(L)[1]), L.I)
    hq = mx_ref.quantize(h.double().cpu().numpy())[2]
    off = offsets.cpu().numpy()
    for e in np.unique(np.linspace(0, L.E + L.S - 1, 5).astype(int)):
        a = hq[off[e]:off[e + 1]]
        want, m = a @ wv[e].T, np.abs(a) @ np.abs(wv[e]).T
        got = y[off[e]:off[e + 1]].double().cpu().numpy()
        assert (np.abs(got - want) <= L.I * 2.0 ** -23 * m + 1e-30).all()


def L_codes(L):
    """(gate_up, down) codes and scales of the layer's experts, from its pinned store."""
    gu, d = [], []
    for e in range(L.E + L.S):
        g, u, dn = (torch.from_numpy(v) for v in L.expert_views(e))
        gu.append(torch.cat([g, u]))
        d.append(dn)
    a, b = block.mx_from_blocks(torch.stack(gu), L.H), block.mx_from_blocks(torch.stack(d), L.I)
    return (a.codes, a.scales), (b.codes, b.scales)


def test_forward_mx_routing_is_the_layers(layer):
    L = layer
    x = activations(40, 5)
    L.forward_mx(x)
    ids, w = L.routing(40)
    logits = L.logits(40)
    want = torch.topk(logits, L.k, 1)
    assert torch.equal(ids.long().sort(1).values, want.indices.sort(1).values)
    p = torch.sigmoid(torch.gather(logits, 1, ids.long()).double())
    assert torch.allclose(w.double(), p / p.sum(1, keepdim=True), rtol=1e-5, atol=0)


def test_forward_mx_in_a_graph_and_on_a_side_stream(layer):
    L = layer
    x = activations(64, 1)
    want = L.forward_mx(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = L.forward_mx(x)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = L.forward_mx(x)
    x.copy_(activations(64, 2))
    fresh = L.forward_mx(x)
    graph.replay()
    assert torch.equal(out, fresh) and not torch.equal(fresh, want)


def test_forward_mx_refusals(layer):
    L = layer
    with pytest.raises(moe.MoEError) as e:
        moe.moe_forward_mx(L.handle, 16, 24, 4, None)
    assert e.value.status == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        L.set_mx_experts(L.mx[1], L.mx[0])
    for image in (L.mx[0].image[:-34816], L.mx[0].image.cpu()):
        with pytest.raises(ValueError):
            L.set_mx_experts(L.mx[0]._replace(image=image), L.mx[1])
    with pytest.raises(ValueError):
        L.forward_mx(torch.zeros((L.H, 4), device="cuda", dtype=torch.bfloat16).t())
    x = torch.zeros((4, L.H), device="cuda", dtype=torch.bfloat16)
    for out in (x[:3].clone(), x.float(), x.cpu(), torch.zeros((4, 2 * L.H), device="cuda", dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(ValueError):
            L.forward_mx(x, out=out)
    from routed_expert_ffn_forward_b200.layer import MoELayer
    M = MoELayer(256, 128, 4, 2, 0)
    try:
        M.set_router(np.zeros((4, 256), np.float32), None, 0)
        with pytest.raises(moe.MoEError) as e:
            M.forward_mx(torch.zeros((2, 256), device="cuda", dtype=torch.bfloat16))
        assert e.value.status == moe.MOE_ERR_NOT_READY
        with pytest.raises(ValueError):
            M.mx_experts_from_host()
    finally:
        M.destroy()
    M = MoELayer(256, 128, 4, 2, 0)
    try:
        M.set_router(np.zeros((4, 256), np.float32), None, 0)
        moe.moe_set_mx_experts(M.handle, L.mx[0].image.data_ptr(), L.mx[1].image.data_ptr())
        M.set_expert_parallel(0, 2)
        with pytest.raises(moe.MoEError) as e:
            M.forward_mx(torch.zeros((2, 256), device="cuda", dtype=torch.bfloat16))
        assert e.value.status == moe.MOE_ERR_UNSUPPORTED
    finally:
        M.destroy()
    assert L.forward_mx(torch.empty((0, L.H), device="cuda", dtype=torch.bfloat16)).shape == (0, L.H)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 37])
def test_block_and_balance_loss(layer, T, mx):
    L = layer
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    h, gate = (2 * r(T, L.H)).bfloat16(), torch.sigmoid(r(T, 1)).bfloat16()
    pre, post, nxt = (1 + 0.1 * r(3, L.H)).bfloat16()
    new, x_next = L.forward_block(h, pre, post, gate, 0.5, nxt, mx=mx)
    # the parts, one by one
    x = block.block_norm(h, pre=pre)[1]
    y = L.forward_mx(x) if mx else L.forward(x)
    a, b = block.block_norm(h, y, post, gate, 0.5, nxt)
    assert torch.equal(new, a) and torch.equal(x_next, b)
    f = lambda t: t.double().cpu()
    o, n = block_ref.block_norm(f(h), f(y), f(post), f(gate), 0.5, f(nxt), 1e-6)
    assert bool(((f(new) - o).abs() <= 2.0 ** -8 * 1.01 * o.abs() + 1e-5).all())
    assert bool(((f(x_next) - n).abs() <= 2.0 ** -8 * 1.01 * n.abs() + 1e-5).all())
    # without post: ones
    ones = L.forward_block(h, pre, None, gate, 0.5, None, mx=mx)
    assert ones[1] is None and torch.equal(ones[0], block.block_norm(h, y, torch.ones_like(pre), gate, 0.5)[0])
    # the loss of this routing
    loss, counts, d_logits = L.balance_loss(T, 0.01)
    logits, ids = L.logits(T), L.routing(T)[0]
    leaf = logits.double().cpu().requires_grad_()
    want, c = block_ref.balance_loss(leaf, ids.cpu(), 0.01, True)
    dw = torch.autograd.grad(want, leaf)[0]
    assert torch.equal(counts.cpu(), c) and int(counts.sum()) == T * L.k
    assert moe.moe_last_tokens(L.handle) == T
    with pytest.raises(ValueError):
        L.balance_loss(T + 1, 0.01)
    nothing = L.balance_loss(0, 0.01)
    assert float(nothing[0]) == 0 and int(nothing[1].sum()) == 0 and nothing[2].shape == (0, L.E)
    assert abs(float(loss) - float(want)) <= 1e-5 * float(want)
    assert bool(((f(d_logits) - dw).abs() <= 4e-5 * dw.abs().max()).all())
    with pytest.raises(ValueError):
        L.forward_block(h.float(), pre)


def test_train_step_captured(layer):
    """The router's and the norms' gradients through autograd, eager and in a graph,
    and through the functions without autograd while an eager graph is alive."""
    L = layer
    T = 24
    x = activations(T, 9)
    L.forward(x)
    logits, ids = L.logits(T).requires_grad_(), L.routing(T)[0]
    h = torch.randn((T, L.H), device="cuda").bfloat16().requires_grad_()
    w = torch.ones(L.H, device="cuda").requires_grad_()
    y = x.float().mul(0.3).bfloat16().requires_grad_()
    d = torch.full((T, L.H), 0.01, device="cuda", dtype=torch.bfloat16)

    def step():
        loss, _ = block.balance_loss(logits, ids, 0.01, L.gating)
        out, nxt = block.block_norm(h, y, w, None, 0.5, w)
        return torch.autograd.grad([loss, out, nxt], [logits, h, y, w], [torch.ones_like(loss), d, d])

    def plain():
        with torch.no_grad():
            loss, _, slope = block.balance_loss_forward(logits, ids, 0.01, L.gating)
            _, _, saved = block.block_norm_forward(h, y, w, None, 0.5, w)
            d_h, d_y, d_post, _, d_pre = block.block_norm_backward(d, d, h, y, w, None, 0.5, w, saved)
            return block.balance_loss_backward(torch.ones_like(loss), slope, logits, L.gating), d_h, d_y, d_post + d_pre

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    alive = block.block_norm(h, y, w, None, 0.5, w)      # an eager graph of the same leaves
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        got = plain()
    graph2.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert alive[0].shape == h.shape
