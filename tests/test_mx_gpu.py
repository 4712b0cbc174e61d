"""MXFP4 rows and grouped products on the GPU against float64 references.

Codes and scales are exact.  Products: every term is exact in fp32 (two E2M1
values under powers of two), so an output differs from the float64 one by the
roundings of a sum of K terms, at most K steps of 2^-23 (the tensor core may
truncate) of the sum of magnitudes, and by the output's rounding, half a step
of its type."""
import numpy as np
import pytest

from tests import mx_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from routed_expert_ffn_forward_b200 import build
    build.build()
    yield
    from routed_expert_ffn_forward_b200 import block
    block.check()


from routed_expert_ffn_forward_b200 import block  # noqa: E402

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def f64(t):
    return t.double().cpu().numpy()


def check_rows(rows, x, values=None):
    code, scale, val = mx_ref.quantize(f64(x))
    nb = scale.shape[1]
    got = rows.codes.cpu().numpy().reshape(x.shape[0], -1, 16)
    both = np.concatenate([got & 15, got >> 4], -1)
    s = rows.scales.cpu().numpy()
    np.testing.assert_array_equal(s[:, :nb], scale)
    fine = np.broadcast_to((scale != 255)[..., None], code.shape)
    np.testing.assert_array_equal(both[:, :nb][fine], code[fine])
    assert (got[:, nb:] == 0).all() and (s[:, nb:] != 255).all()
    if values is not None:
        np.testing.assert_array_equal(f64(values), val)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 256), (7, 257), (4, 1000), (65, 7168), (1, 16384)])
def test_quantize(dtype, rows, cols):
    g = torch.Generator(device="cuda").manual_seed(rows * 1000 + cols)
    x = torch.randn((rows, cols), generator=g, device="cuda") * torch.exp(3 * torch.randn((rows, 1), generator=g, device="cuda"))
    x = x.to(dtype)
    r, v = block.mx_quantize(x, values=True)
    check_rows(r, x, v)
    r2 = block.mx_quantize(x)
    assert torch.equal(r.codes, r2.codes) and torch.equal(r.scales, r2.scales)


def test_quantize_every_bf16_magnitude_and_ties():
    # every positive bf16 number as a run's largest, with the eighths of it below
    bits = torch.arange(0, 0x7F80, 7, dtype=torch.int32)
    top = bits.to(torch.int16).view(torch.bfloat16).float()
    f = torch.arange(32).float() / 31
    f[::2] *= -1
    x = (top[:, None] * f).cuda()
    check_rows(*(lambda r: (r[0], x, r[1]))(block.mx_quantize(x, values=True)))
    # all ties of the levels, at several scales
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.0, 7.99, 0.0, -0.0, -0.25, -5.0, 4.0, 6.0] * 2)
    x = (ties[None] * torch.exp2(torch.arange(-130, 120).float())[:, None]).cuda()
    r, v = block.mx_quantize(x, values=True)
    check_rows(r, x, v)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantize_infinities_and_nan_stay_in_their_run(dtype):
    x = torch.randn((6, 96), device="cuda").to(dtype)
    x[0, 5], x[1, 40], x[2, 95], x[3, 32:64] = float("inf"), float("nan"), float("-inf"), 0.0
    x[4] = 0.0
    r, v = block.mx_quantize(x, values=True)
    check_rows(r, x, v)
    assert torch.isnan(v[0, :32]).all() and torch.isfinite(v[0, 32:]).all() and (v[4] == 0).all()


def test_quantize_strided_and_offset_rows():
    base = torch.randn((9, 300), device="cuda").bfloat16()
    for x in (base[:, :256], base[::2, 3:200], base[:, 1:2], base.t()[:, :5], base[2:3]):
        r, v = block.mx_quantize(x, values=True)
        check_rows(r, x, v)


def test_blocks_round_trip():
    for cols in (32, 40, 256, 288, 1000):
        x = torch.randn((3, cols), device="cuda")
        r = block.mx_quantize(x)
        b = block.mx_blocks(r)
        assert b.shape == (3, 17 * -(-cols // 32))
        back = block.mx_from_blocks(b, cols)
        assert torch.equal(back.codes, r.codes)
        nb = -(-cols // 32)
        assert torch.equal(back.scales[:, :nb], r.scales[:, :nb])


def weights(n_mats, rows, cols, g):
    nb = -(-cols // 32)
    codes = torch.randint(0, 256, (n_mats, rows, nb, 16), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(121, 127, (n_mats, rows, nb), generator=g, device="cuda", dtype=torch.uint8)
    return block.mx_rows(codes, scales, cols)


def reference(x, w, paired, offsets, index):
    """(float64 outputs by row, bound of the fp32 sums' errors), NaN rows where no group is."""
    xv = mx_ref.unpack(x.codes.cpu().numpy(), x.scales.cpu().numpy(), x.cols)
    wv = mx_ref.unpack(w.codes.cpu().numpy(), w.scales.cpu().numpy(), w.cols)
    n_rows = len(xv) if index is None else len(index)
    ix = np.arange(n_rows) if index is None else index.cpu().numpy()
    inside = (ix >= 0) & (ix < len(xv))
    sel = np.where(inside[:, None], xv[np.clip(ix, 0, len(xv) - 1)], 0.0)
    off = np.array([0, n_rows]) if offsets is None else offsets.cpu().numpy()
    feats = wv.shape[1] // 2 if paired else wv.shape[1]
    out, tol = np.full((n_rows, feats), np.nan), np.zeros((n_rows, feats))
    for e in range(len(off) - 1):
        a = sel[off[e]:off[e + 1]]
        y = a @ wv[e].T
        d = x.cols * 2.0 ** -23 * (np.abs(a) @ np.abs(wv[e]).T)
        if paired:
            g, u, dg, du = y[:, :feats], y[:, feats:], d[:, :feats], d[:, feats:]
            sig = 1 / (1 + np.exp(-g))
            h = g * sig * u
            # |silu'| <= 1.1; the fast exp is off by (2 + 1.16 |g|) steps of 2^-23, the divide by 2
            t = 1.1 * dg * np.abs(u) + np.abs(g * sig) * du + 1.1 * dg * du + (5 + 1.2 * np.abs(g)) * 2.0 ** -23 * np.abs(h)
            out[off[e]:off[e + 1]], tol[off[e]:off[e + 1]] = h, t
        else:
            out[off[e]:off[e + 1]], tol[off[e]:off[e + 1]] = y, d
    return out, tol


def check_product(got, want, tol, rows=slice(None)):
    w, t = want[rows], tol[rows]
    live = ~np.isnan(w).any(1)
    o = f64(got)[rows]
    err = np.abs(o - w)[live]
    bound = (t + HALF[got.dtype] * (np.abs(w) + t) + 1e-37)[live]
    assert (err <= bound).all(), (err / bound).max()


PRODUCTS = [
    # n_mats, counts (or None: one dense group), rows, cols, paired
    (1, None, 256, 256, False),
    (1, None, 64, 32, False),
    (1, None, 6, 1, True),
    (1, None, 1, 300, False),
    (1, None, 700, 1111, False),
    (1, None, 514, 2048, True),
    (4, [1, 0, 3, 1], 512, 512, False),
    (8, [0, 1, 2, 64, 65, 15, 16, 17], 300, 640, True),
    (3, [0, 0, 0], 256, 256, False),
    (5, [300, 0, 7, 241, 240], 333, 288, False),
    (5, [1, 480, 0, 481, 40], 258, 544, True),
    (40, None, 256, 256, False),
    # many rows: CTA pairs, an odd number of row tiles, tiles of 240 and of a few rows
    (3, [500, 0, 700], 700, 320, False),
    (4, [1, 1100, 240, 17], 1290, 288, True),
    (6, [0, 241, 112, 113, 480, 128], 513, 1500, False),
    (2, [900, 300], 200, 256, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_mats,counts,rows,cols,paired", PRODUCTS)
def test_product(dtype, n_mats, counts, rows, cols, paired):
    g = torch.Generator(device="cuda").manual_seed(rows + cols + n_mats)
    if counts is None:
        counts = [97] if n_mats == 1 else torch.randint(0, 4, (n_mats,), generator=torch.Generator().manual_seed(1)).tolist()
    n_rows, n_x = sum(counts), max(1, sum(counts) // 3 + 1)
    x = block.mx_quantize(torch.randn((n_x, cols), generator=g, device="cuda").bfloat16())
    w = weights(n_mats, rows, cols, g)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    index = torch.randint(0, n_x, (n_rows,), generator=g, device="cuda", dtype=torch.int32)
    out = block.mx_product(x, block.mx_pack(w, paired), off, index, out_dtype=dtype)
    assert out.shape == (n_rows, rows // 2 if paired else rows) and out.dtype == dtype
    check_product(out, *reference(x, w, paired, off, index))


@pytest.mark.parametrize("n", [1, 2, 8, 9, 16, 33, 64, 65, 240, 241, 1024, 1025, 1500])
@pytest.mark.parametrize("paired", [False, True])
def test_dense_product_of_every_batch_size(n, paired):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = block.mx_quantize(torch.randn((n, 2048 + 96), generator=g, device="cuda"))
    w = weights(1, 384, 2048 + 96, g)
    p = block.mx_pack(w, paired)
    out = block.mx_product(x, p)
    check_product(out, *reference(x, w, paired, None, None))
    assert torch.equal(out, block.mx_product(x, p))


def test_rows_of_no_group_and_index_outside():
    g = torch.Generator(device="cuda").manual_seed(3)
    for n_rows in (20, 1300):
        x = block.mx_quantize(torch.randn((8, 320), generator=g, device="cuda"))
        w = weights(2, 130, 320, g)
        off = torch.tensor([3, 9, n_rows - 4], dtype=torch.int32, device="cuda")
        index = torch.randint(0, 8, (n_rows,), generator=g, device="cuda", dtype=torch.int32)
        index[4], index[10], index[11] = -1, 8, 2 ** 31 - 1
        out = torch.full((n_rows, 130), 7.0, device="cuda")
        block.mx_product(x, block.mx_pack(w), off, index, out=out)
        want, tol = reference(x, w, False, off, index)
        check_product(out, want, tol)
        assert (out[:3] == 7).all() and (out[-4:] == 7).all() and (out[[4, 10, 11]] == 0).all()


def test_offsets_outside_the_rows_are_taken_into_them():
    g = torch.Generator(device="cuda").manual_seed(4)
    x = block.mx_quantize(torch.randn((12, 256), generator=g, device="cuda"))
    w = weights(2, 256, 256, g)
    out = torch.full((12, 256), 7.0, device="cuda")
    off = torch.tensor([-5, 4, 1000], dtype=torch.int32, device="cuda")
    block.mx_product(x, block.mx_pack(w), off, out=out)
    check_product(out, *reference(x, w, False, torch.tensor([0, 4, 12]), None))


def test_output_rows_with_a_stride_and_odd_features():
    g = torch.Generator(device="cuda").manual_seed(5)
    x = block.mx_quantize(torch.randn((70, 512), generator=g, device="cuda"))
    w = weights(1, 131, 512, g)
    for dtype, width, first in ((torch.bfloat16, 200, 0), (torch.bfloat16, 201, 1), (torch.float32, 133, 2)):
        base = torch.full((70, width), 7.0, dtype=dtype, device="cuda")
        view = base[:, first:first + 131]
        block.mx_product(x, block.mx_pack(w), out=view)
        check_product(view, *reference(x, w, False, None, None))
        assert (base[:, first + 131:] == 7).all() and (base[:, :first] == 7).all()


def test_nan_rows_stay_in_their_row():
    g = torch.Generator(device="cuda").manual_seed(6)
    xf = torch.randn((20, 256), generator=g, device="cuda")
    xf[7, 3] = float("nan")
    x = block.mx_quantize(xf)
    out = block.mx_product(x, block.mx_pack(weights(1, 256, 256, g)), out_dtype=torch.float32)
    assert torch.isnan(out[7]).all() and torch.isfinite(out[:7]).all() and torch.isfinite(out[8:]).all()


def test_product_on_a_side_stream_and_in_a_graph():
    g = torch.Generator(device="cuda").manual_seed(7)
    w = weights(4, 512, 512, g)
    p = block.mx_pack(w)
    xs = [torch.randn((50, 512), generator=g, device="cuda") for _ in range(3)]
    off = torch.tensor([0, 10, 11, 40, 50], dtype=torch.int32, device="cuda")
    want = [block.mx_product(block.mx_quantize(x), p, off) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [block.mx_product(block.mx_quantize(x), p, off) for x in xs]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.mx_product(block.mx_quantize(x), p, off)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        graph.replay()
        assert torch.equal(out, want[i])


FIRST_CALL_CAPTURED = """
import torch
from routed_expert_ffn_forward_b200 import block
g = torch.Generator(device="cuda").manual_seed(5)
x = block.mx_quantize(torch.randn(1, 7168, device="cuda", generator=g))
w = block.mx_pack(block.mx_quantize(torch.randn(512, 7168, device="cuda", generator=g)))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = block.mx_product(x, w, out_dtype=torch.float32)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(got, block.mx_product(x, w, out_dtype=torch.float32))
block.check()
print("same")
"""


def test_first_product_of_a_process_is_captured():
    """What the split of K asks of the device once, it may ask during a capture."""
    import subprocess
    import sys
    from pathlib import Path
    done = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], capture_output=True, text=True, timeout=300,
                          cwd=Path(__file__).resolve().parents[1])
    assert done.returncode == 0 and done.stdout.strip() == "same", done.stdout + done.stderr
