"""The block norms and the balance loss on the GPU against float64 references.

Tolerances count roundings in steps of 2^-24 of the magnitudes that enter: a
row's sum of squares goes through at most 32 additions per thread and 10 levels
of shuffles (42), the other factors of an output through fewer than 20
operations each, so an fp32 result with at most four such factors is within
STEPS = 250 of the sum of its terms' magnitudes; a column sum over rows adds
one step per row.  Rounding to the output's type adds half a step of it."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_ffn_forward_b200 import block, moe  # noqa: E402
from tests import block_ref as ref  # noqa: E402

U = 2.0 ** -24
STEPS = 250
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -140}   # half a subnormal step


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from routed_expert_ffn_forward_b200 import build
    build.build()
    yield
    block.check()


def close(got, want, steps):
    """|got - want| <= steps (absolute, fp32 part) + half a step of got's type."""
    g, w, s = got.double().cpu(), want.double().cpu(), steps.double().cpu()
    assert g.shape == w.shape
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    ok = ~torch.isnan(w)
    err, bound = (g - w).abs(), s + HALF[got.dtype] * (w.abs() + s) + TINY[got.dtype]
    assert bool((err <= bound)[ok].all()), float((err / bound)[ok].max())


def norm_inputs(rows, cols, dtype, weights, gate, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    h, y = (2 * r(rows, cols)).to(dtype), (0.5 * r(rows, cols)).to(dtype)
    post, pre = (1 + 0.2 * r(cols)).to(weights), (1 + 0.2 * r(cols)).to(weights)
    gates = dict(none=None, token=r(rows, 1).to(dtype), feature=r(cols).to(weights), full=r(rows, cols).to(dtype))
    return h, y, post, gates[gate], pre, r(rows, cols).to(dtype), r(rows, cols).to(dtype)


def magnitudes(h, y, post, gate, scale, pre, d_out, d_next, eps):
    """Sums of the terms' magnitudes of every output and gradient."""
    a = lambda t: None if t is None else t.double().cpu().abs()
    H, Y, W, G, P, DO, DN = map(a, (h, y, post, gate, pre, d_out, d_next))
    m = {}
    zero = torch.zeros_like(H)
    O, o = H, h.double().cpu()
    if y is not None:
        ry = 1 / torch.sqrt((Y * Y).mean(1, keepdim=True) + eps)
        NY = Y * ry
        SG = abs(scale) * (1.0 if G is None else G)
        O = H + SG * NY * W
        o, _ = ref.block_norm(o, y.double().cpu(), post.double().cpu(), None if gate is None else gate.double().cpu(), scale, None, eps)
        m["out"] = O
    D = zero if DO is None else DO
    if pre is not None:
        ro = 1 / torch.sqrt((o * o).mean(1, keepdim=True) + eps)
        rel = torch.sqrt((O * O).mean(1, keepdim=True)) * ro      # how out's errors enter its rms
        NO = O * ro * (1 + rel)
        m["next"] = NO * P
        if DN is not None:
            A = DN * P
            D = D + ro * (1 + rel) * (A + NO * (A * NO).mean(1, keepdim=True))
            m["d_pre"] = (DN * NO).sum(0)
    m["d_h"] = D
    if y is not None:
        DZ = SG * D
        B = DZ * W
        m["d_y"] = ry * (B + NY * (B * NY).mean(1, keepdim=True))
        m["d_post"] = (DZ * NY).sum(0)
        if gate is not None:
            g = abs(scale) * NY * W * D
            m["d_gate"] = g if gate.shape == h.shape else g.sum(0) if gate.dim() == 1 else g.sum(1, keepdim=True)
    return m


def check_norm(h, y, post, gate, scale, pre, d_out, d_next, eps=1e-6):
    out, nxt, saved = block.block_norm_forward(h, y, post, gate, scale, pre, eps)
    d = block.block_norm_backward(d_out if y is not None else None, d_next if pre is not None else None, h, y, post, gate,
                                  scale, pre, saved, eps)
    leaf = [None if t is None else t.double().cpu().requires_grad_() for t in (h, y, post, gate, pre)]
    H, Y, W, G, P = leaf
    o, n = ref.block_norm(H, Y, W, G, scale, P, eps)
    outs = [(t, v) for t, v in ((o, d_out), (n, d_next)) if t is not None and v is not None]
    m = magnitudes(h, y, post, gate, scale, pre, d_out if y is not None else None, d_next, eps)
    if out is not None:
        close(out, o.detach(), STEPS * U * m["out"])
    if nxt is not None:
        close(nxt, n.detach(), STEPS * U * m["next"])
    if not outs:
        return
    live = [t for t in leaf if t is not None]
    grads = torch.autograd.grad([t for t, _ in outs], live, [v.double().cpu() for _, v in outs], allow_unused=True)
    grads = iter(grads)
    for name, t, got in zip(("d_h", "d_y", "d_post", "d_gate", "d_pre"), leaf, d):
        if t is None:
            assert got is None
            continue
        want = next(grads)
        if want is None:
            assert (got == 0).all()
            continue
        rows = h.shape[0] if want.dim() == 1 else 0
        close(got, want, (STEPS + rows) * U * m[name])


NORMS = [(340, 2), (320, 1034), (310, 6010), (350, 1), (400, 7), (333, 9), (310, 250), (320, 2047), (300, 4567), (1, 7168), (5, 256), (3, 17), (33, 1003), (2, 1), (7, 8), (600, 512), (500, 1032), (300, 7168), (4, 16384), (3, 16383), (150, 8200), (2, 4104)]


@pytest.mark.parametrize("dtype,weights", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                           (torch.float16, torch.float16), (torch.float16, torch.float32),
                                           (torch.float32, torch.float32)])
@pytest.mark.parametrize("rows,cols", NORMS)
def test_block_norm(dtype, weights, rows, cols):
    for i, gate in enumerate(("none", "token", "feature", "full")):
        h, y, post, g, pre, d_out, d_next = norm_inputs(rows, cols, dtype, weights, gate, rows + cols + i)
        check_norm(h, y, post, g, 0.7, pre, d_out, d_next)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(3, 768), (40, 515)])
def test_block_norm_parts(dtype, rows, cols):
    h, y, post, g, pre, d_out, d_next = norm_inputs(rows, cols, dtype, dtype, "feature", 5)
    check_norm(h, None, None, None, 1.0, pre, None, d_next)            # before the first block
    check_norm(h, y, post, g, 1.3, None, d_out, None)                  # behind the last block
    check_norm(h, y, post, None, -0.5, pre, d_out, None)               # one output's gradient alone
    check_norm(h, y, post, g, 0.0, pre, None, d_next)


def test_block_norm_rows_of_zeros_infinities_and_nan():
    h, y, post, g, pre, d_out, d_next = norm_inputs(6, 640, torch.float32, torch.float32, "full", 9)
    h[0], y[0], y[1] = 0, 0, 0
    good = [0, 1, 3, 5]
    h[2, 7], y[4, 9] = float("nan"), float("inf")
    out, nxt, saved = block.block_norm_forward(h, y, post, g, 1.0, pre)
    for t in (out, nxt):
        assert torch.isfinite(t[good]).all()
    assert torch.isnan(nxt[2]).all() and torch.isnan(out[4, 9]) and (out[4, :9] == h[4, :9]).all()
    sub = lambda t: t[good].contiguous()
    check_norm(sub(h), sub(y), post, sub(g), 1.0, pre, sub(d_out), sub(d_next))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_block_norm_strided_rows(dtype):
    big = [t for t in norm_inputs(9, 600, dtype, dtype, "full", 11)]
    post, pre = big[2][:512].contiguous(), big[4][:512].contiguous()
    for first in (0, 3):
        cut = lambda t: t[:, first:first + 512]
        check_norm(cut(big[0]), cut(big[1]), post, cut(big[3]), 0.9, pre, cut(big[5]), cut(big[6]))
        check_norm(cut(big[0])[::2], cut(big[1])[::2], post, cut(big[3])[::2, :1], 0.9, pre, cut(big[5])[::2], cut(big[6])[::2])
    h, y = big[0].t()[:512], big[1].t()[:512]       # columns that are not contiguous
    check_norm(h, y, torch.ones(9, device="cuda", dtype=dtype), None, 1.0, torch.ones(9, device="cuda", dtype=dtype),
               big[5].t()[:512], big[6].t()[:512])
    shared = big[0][:, :512]                        # y and h the same tensor, gradients apart
    check_norm(shared, shared, post, None, 1.0, pre, big[5][:, :512], big[6][:, :512])


def test_block_norm_without_rows():
    h, y, post, g, pre, d_out, d_next = (t[:0] if t.dim() == 2 else t for t in norm_inputs(2, 64, torch.bfloat16, torch.float32, "feature", 1))
    out, nxt, saved = block.block_norm_forward(h, y, post, g, 1.0, pre)
    assert out.shape == nxt.shape == (0, 64)
    d = block.block_norm_backward(d_out, d_next, h, y, post, g, 1.0, pre, saved)
    assert d[0].shape == d[1].shape == (0, 64) and all((t == 0).all() and t.shape == (64,) for t in d[2:])


def test_block_norm_same_bits_side_stream_and_graph():
    h, y, post, g, pre, d_out, d_next = norm_inputs(700, 1024, torch.bfloat16, torch.float32, "feature", 3)

    def step():
        out, nxt, saved = block.block_norm_forward(h, y, post, g, 0.8, pre)
        return [out, nxt, *block.block_norm_backward(d_out, d_next, h, y, post, g, 0.8, pre, saved)]

    want = step()
    assert all(torch.equal(a, b) for a, b in zip(want, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    graphs, outs = [], []
    for _ in range(2):                              # two graphs, each with its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    keep = h.clone()
    for i in range(2):
        h.copy_(keep + i)
        fresh = step()
        for graph in graphs:
            graph.replay()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(fresh, o))


def test_block_norm_autograd():
    h, y, post, g, pre, d_out, d_next = norm_inputs(20, 384, torch.float32, torch.float32, "token", 21)
    leaves = [t.requires_grad_() for t in (h, y, post, g, pre)]
    out, nxt = block.block_norm(h, y, post, g, 0.6, pre)
    got = torch.autograd.grad([out, nxt], leaves, [d_out, d_next])
    saved = block.block_norm_forward(h, y, post, g, 0.6, pre)[2]
    want = block.block_norm_backward(d_out, d_next, h, y, post, g, 0.6, pre, saved)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out, nxt = block.block_norm(h, y, post, g, 0.6, pre)
    only = torch.autograd.grad(out, [h, pre], d_out, allow_unused=True)
    assert torch.equal(only[0], d_out) and (only[1] is None or (only[1] == 0).all())
    _, nxt = block.block_norm(h, pre=pre)
    torch.autograd.grad(nxt, [h, pre], d_next)


# ---------------------------------------------------------------- balance
def router(tokens, experts, top_k, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = scale * torch.randn((tokens, experts), generator=g, device="cuda") - torch.arange(experts, device="cuda") / experts
    ids = torch.topk(logits, top_k, 1).indices.int() if tokens else torch.empty((0, top_k), dtype=torch.int32, device="cuda")
    return logits, ids


def check_balance(logits, ids, sigmoid, offsets=None, mask=None, coef=0.02, up=1.7):
    gating = moe.MOE_GATE_SIGMOID_RENORM if sigmoid else moe.MOE_GATE_SOFTMAX_TOPK
    loss, counts, slope = block.balance_loss_forward(logits, ids, coef, gating, offsets, mask)
    leaf = logits.double().cpu().requires_grad_()
    off = None if offsets is None else offsets.cpu()
    mk = None if mask is None else mask.cpu()
    want, c = ref.balance_loss(leaf, ids.cpu(), coef, sigmoid, off, mk)
    assert torch.equal(counts.cpu(), c)
    # a probability: 42 steps of its sum, 20 of the rest, and the exponential's 2 + 1.2 |l - max| steps of 2^-23
    spread = float(leaf.detach()[torch.isfinite(leaf.detach())].abs().max()) * 2 if leaf.numel() else 0.0
    steps = STEPS + 3 * spread
    # a run's tokens per warp, its 16 warps, the runs: fewer than 400 additions
    close(loss, want.detach(), (steps + 400) * U * want.detach().abs())
    d = block.balance_loss_backward(torch.tensor(up, device="cuda"), slope, logits, gating, offsets, mask)
    if not want.requires_grad or not len(logits):
        assert (d == 0).all()
        return
    dw = torch.autograd.grad(want, leaf, torch.tensor(up, dtype=torch.float64))[0]
    dw = torch.where(torch.isnan(dw), torch.zeros_like(dw), dw)      # autograd of rows without a finite logit
    p = ref.probabilities(leaf.detach(), sigmoid)
    if mk is not None:
        p[~mk] = 0.0                                # exactly zeros there
    seqs = len(counts)
    bounds = torch.tensor([0, len(logits)]) if off is None else off.long().clamp(0, len(logits))
    a = torch.zeros_like(dw)
    for s in range(seqs):
        a[bounds[s]:bounds[s + 1]] = up * slope[s].double().cpu()
    close(d, dw, steps * U * p * (a + (p * a).sum(1, keepdim=True)))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 16, 2), (1, 1, 1), (64, 256, 8), (128, 1024, 8), (129, 40, 5), (33, 33, 4),
                                                   (700, 256, 8), (2000, 100, 1), (300, 1000, 32), (257, 512, 6)])
def test_balance_one_sequence(sigmoid, tokens, experts, top_k):
    logits, ids = router(tokens, experts, top_k, tokens + experts)
    check_balance(logits, ids, sigmoid)
    mask = torch.arange(tokens, device="cuda") % 3 != 1
    logits[~mask] = float("nan")                    # a masked token's logits are not looked at
    check_balance(logits, ids, sigmoid, mask=mask)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_packed_sequences(sigmoid):
    logits, ids = router(500, 64, 4, 8)
    for offsets in ([0, 500], [0, 0, 1, 2, 2, 34, 290, 500, 500], [7, 20, 20, 480], [100, 100], list(range(0, 501, 5))):
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        check_balance(logits, ids, sigmoid, off)
        mask = (torch.arange(500, device="cuda") > 40) & (torch.arange(500, device="cuda") % 7 > 0)
        check_balance(logits, ids, sigmoid, off, mask)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_offsets_outside_the_tokens(sigmoid):
    logits, ids = router(90, 16, 2, 12)
    check_balance(logits, ids, sigmoid, torch.tensor([-3, 40, 1000], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_masked_experts_and_empty_rows(sigmoid):
    for tokens in (20, 300):
        logits, ids = router(tokens, 48, 4, 15)
        logits[:, 30:] = float("-inf")              # experts that are switched off
        logits[3] = float("-inf")                   # a token without any
        logits[5] = torch.finfo(torch.float32).min
        logits[6] -= 200.0                          # every sigmoid underflows
        logits[7] += 100.0
        ids[4, 1:], ids[8, 0], ids[9] = -1, 48, 2 ** 31 - 1    # picks that are no expert
        check_balance(logits, ids, sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_nothing_counts(sigmoid):
    for tokens in (0, 5, 200):
        logits, ids = router(tokens, 8, 2, 4)
        mask = torch.zeros(tokens, dtype=torch.bool, device="cuda")
        check_balance(logits, ids, sigmoid, mask=mask)
        check_balance(logits, ids, sigmoid, torch.tensor([0, 0, tokens], dtype=torch.int32, device="cuda"), mask)
    logits, ids = router(0, 8, 2, 4)
    check_balance(logits, ids, sigmoid)


def test_balance_strided_logits_graph_and_autograd():
    base, _ = router(300, 80, 4, 30)
    logits = base[:, 5:69]
    ids = torch.topk(logits, 4, 1).indices.int()
    check_balance(logits, ids, False)
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    x = logits.contiguous().requires_grad_()
    loss, counts = block.balance_loss(x, ids, 0.01, moe.MOE_GATE_SOFTMAX_TOPK, off)
    (3.0 * loss).backward()
    l2, c2, slope = block.balance_loss_forward(x.detach(), ids, 0.01, moe.MOE_GATE_SOFTMAX_TOPK, off)
    d = block.balance_loss_backward(torch.tensor(3.0, device="cuda"), slope, x.detach(), moe.MOE_GATE_SOFTMAX_TOPK, off)
    assert torch.equal(loss.detach(), l2) and torch.equal(counts, c2) and torch.equal(x.grad, d)
    y = x.detach().clone()
    up = torch.tensor(3.0, device="cuda")

    def step():
        l, c, s = block.balance_loss_forward(y, ids, 0.01, moe.MOE_GATE_SOFTMAX_TOPK, off)
        return l, c, block.balance_loss_backward(up, s, y, moe.MOE_GATE_SOFTMAX_TOPK, off)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        y.mul_(1.3)
        want = step()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
