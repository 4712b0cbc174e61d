"""Quantisation, norms and balance loss over sizes at which their loops go round: more
chunks than the GPU takes at a time, more rows for a CTA than its ring has stages,
several tokens for a warp of the gradient.  The references are those of the small
cases, in 64 bits; the norms' are evaluated on the GPU."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_ffn_forward_b200 import block  # noqa: E402
from tests import block_ref as ref  # noqa: E402
from tests.test_block_gpu import HALF, STEPS, TINY, U, check_balance, norm_inputs, router  # noqa: E402
from tests.test_mx_gpu import check_rows  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from routed_expert_ffn_forward_b200 import build
    build.build()
    yield
    block.check()


# ---------------------------------------------------------------- quantisation
# 18944 chunks of 256 fill the GPU (then a half warp takes two), 37888 go round
@pytest.mark.parametrize("dtype,rows,cols", [(torch.bfloat16, 1500, 7169), (torch.float32, 20000, 257), (torch.float16, 6000, 2048),
                                             (torch.bfloat16, 40001, 40)])
def test_quantize_many_chunks(dtype, rows, cols):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x = (x * torch.exp(2 * torch.randn((rows, 1), generator=g, device="cuda"))).to(dtype)
    r, v = block.mx_quantize(x, values=True)
    plain = block.mx_quantize(x)
    assert torch.equal(r.codes, plain.codes) and torch.equal(r.scales, plain.scales)
    for lo in range(0, rows, 2000):
        cut = slice(lo, lo + 2000)
        check_rows(block.MXRows(r.codes[cut], r.scales[cut], cols), x[cut], v[cut])


# ---------------------------------------------------------------- norms
def close(got, want, steps):
    """|got - want| <= steps (absolute, the fp32 part) + half a step of got's type."""
    err = (got.double() - want).abs()
    bound = steps + HALF[got.dtype] * (want.abs() + steps) + TINY[got.dtype]
    assert bool((err <= bound).all()), float((err / bound).max())


def check_norm(h, y, post, gate, scale, pre, d_out, d_next, eps=1e-6):
    """As test_block_gpu.check_norm, with STEPS of 2^-24 of the terms' magnitudes and one
    more for each row of a column sum."""
    out, nxt, saved = block.block_norm_forward(h, y, post, gate, scale, pre, eps)
    got = block.block_norm_backward(d_out, d_next, h, y, post, gate, scale, pre, saved, eps)
    again = block.block_norm_backward(d_out, d_next, h, y, post, gate, scale, pre, saved, eps)
    assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)
    leaf = [None if t is None else t.double().requires_grad_() for t in (h, y, post, gate, pre)]
    o, n = ref.block_norm(*leaf[:4], scale, leaf[4], eps)
    live = [t for t in leaf if t is not None]
    want = iter(torch.autograd.grad([o, n], live, [d_out.double(), d_next.double()]))
    H, Y, W, G, P = (None if t is None else t.detach().abs() for t in leaf)
    DO, DN, o, n = d_out.double().abs(), d_next.double().abs(), o.detach(), n.detach()
    rms = lambda v: torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    ry, ro = 1 / rms(Y), 1 / rms(o)
    SG = abs(scale) * (1.0 if G is None else G)
    O = H + SG * Y * ry * W
    rel = 1 + torch.sqrt((O * O).mean(1, keepdim=True)) * ro       # how out's errors enter its rms
    NO, A = O * ro * rel, DN * P
    D = DO + ro * rel * (A + NO * (A * NO).mean(1, keepdim=True))
    B, NY = SG * D * W, Y * ry
    mags = dict(d_h=D, d_y=ry * (B + NY * (B * NY).mean(1, keepdim=True)), d_post=(SG * D * NY).sum(0), d_pre=(DN * NO).sum(0))
    if G is not None:
        g = abs(scale) * NY * W * D
        mags["d_gate"] = g if G.shape == H.shape else g.sum(0) if G.dim() == 1 else g.sum(1, keepdim=True)
    close(out, o, STEPS * U * O)
    close(nxt, n, STEPS * U * NO * P)
    for name, t in zip(("d_h", "d_y", "d_post", "d_gate", "d_pre"), got):
        if t is None:
            assert name == "d_gate" and gate is None
            continue
        close(t, next(want), (STEPS + (h.shape[0] if t.dim() == 1 else 0)) * U * mags[name])


BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("rows,cols,dtype,weights,gate", [
    # aligned: one and two vectors a thread, one and two teams of threads, up to eight CTAs an SM
    (1600, 7168, BF, FP, "feature"), (1600, 7168, BF, BF, "full"), (1500, 4104, FP, FP, "token"), (12000, 512, HF, FP, "none"),
    # pairs, and single 32-bit values
    (9000, 1002, BF, BF, "token"), (1500, 7166, HF, HF, "feature"), (9000, 1003, FP, FP, "full"), (20000, 34, BF, FP, "none"),
    # shifted words
    (9001, 1001, BF, FP, "feature"), (9001, 1001, HF, HF, "full"), (1501, 7167, BF, BF, "token"), (20001, 33, HF, FP, "none"),
    # one CTA a row
    (700, 16384, BF, BF, "full"), (601, 16383, FP, FP, "none"),
])
def test_norms_of_many_rows(rows, cols, dtype, weights, gate):
    h, y, post, g, pre, d_out, d_next = norm_inputs(rows, cols, dtype, weights, gate, rows + cols)
    check_norm(h, y, post, g, 0.7, pre, d_out, d_next)


# ---------------------------------------------------------------- balance loss
# from 9473 tokens on a warp of the gradient, and a run of the forward, has more than in the small cases
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k", [(20001, 256, 8), (20001, 257, 8), (11000, 600, 6), (33000, 60, 4)])
def test_balance_many_tokens(sigmoid, tokens, experts, top_k):
    logits, ids = router(tokens, experts, top_k, tokens + experts)
    check_balance(logits, ids, sigmoid)
    # sequences of no token, of one, shorter and longer than a run, with tokens before and behind them, some masked
    offsets = torch.tensor([5, 5, 6, 40, 41, 41, 1000, 1500, 9000, 9001, tokens - 700, tokens - 3], dtype=torch.int32, device="cuda")
    t = torch.arange(tokens, device="cuda")
    mask = (t % 7 > 0) & ((t < 1000) | (t >= 1500))
    logits[~mask] = float("nan")
    check_balance(logits, ids, sigmoid, offsets, mask)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("experts,scale,shift", [(8, 1.0, 0.0), (8, 15.0, 0.0), (1000, 3.0, 0.0), (256, 6.0, -40.0), (64, 4.0, 30.0)])
def test_balance_probabilities_one_by_one(sigmoid, experts, scale, shift):
    """One token that picked one expert: the loss is coef * experts times that expert's probability.  The documented
    bound, and 6 steps for the factors."""
    g = torch.Generator(device="cuda").manual_seed(experts)
    logits = torch.randn((60, experts), generator=g, device="cuda") * scale + shift
    pick = torch.randint(0, experts, (60, 1), generator=g, device="cuda", dtype=torch.int32)
    got = torch.stack([block.balance_loss_forward(l[None], i[None], 1.0, 1 if sigmoid else 0)[0] for l, i in zip(logits, pick)])
    l = logits.double()
    want = ref.probabilities(l, sigmoid).gather(1, pick.long())[:, 0] * experts
    top, mine = l.max(1).values, l.gather(1, pick.long())[:, 0]
    units = (-mine).clamp(min=0) + (-top).clamp(min=0) if sigmoid else top - mine
    bound = (86 + 4 * units) * U * want + experts * 1.2e-38 / (torch.sigmoid(l).sum(1) if sigmoid else 1.0)
    assert bool(((got.double() - want).abs() <= bound).all()), float(((got.double() - want).abs() / bound).max())


# ---------------------------------------------------------------- first calls
FIRST_CALLS_CAPTURED = """
import torch
from routed_expert_ffn_forward_b200 import block
g = torch.Generator(device="cuda").manual_seed(5)
r = lambda *s: torch.randn(s, generator=g, device="cuda")
h, y, w, d = r(400, 1024), r(400, 1024), r(1024), r(400, 1024)
logits = r(200, 1024)
ids = torch.topk(logits, 4, 1).indices.int()
up = torch.ones((), device="cuda")
def step():
    out, nxt, saved = block.block_norm_forward(h, y, w, None, 0.5, w)
    grads = [t for t in block.block_norm_backward(d, d, h, y, w, None, 0.5, w, saved) if t is not None]
    loss, counts, slope = block.balance_loss_forward(logits, ids, 0.01, 0)
    return [out, nxt, *grads, loss, counts, block.balance_loss_backward(up, slope, logits, 0), block.mx_quantize(h).codes]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
block.check()
print("same")
"""


def test_first_calls_of_a_process_are_captured():
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], capture_output=True, text=True, timeout=300,
                          cwd=Path(__file__).resolve().parents[1])
    assert done.returncode == 0 and done.stdout.strip() == "same", done.stdout + done.stderr
