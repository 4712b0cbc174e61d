"""Products in which every CTA (or pair of CTAs) takes several units, so that the
ring of stages, the accumulators' slots and the order of the units go on from one
unit to the next; the references and bounds of test_mx_gpu.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_ffn_forward_b200 import block  # noqa: E402
from tests import mx_ref  # noqa: E402
from tests.test_mx_gpu import check_product, reference, weights  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from routed_expert_ffn_forward_b200 import build
    build.build()
    yield
    block.check()


def grouped(counts, rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_rows = sum(counts)
    x = block.mx_quantize(torch.randn((n_rows // 3 + 1, cols), generator=g, device="cuda").bfloat16())
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    index = torch.randint(0, n_rows // 3 + 1, (n_rows,), generator=g, device="cuda", dtype=torch.int32)
    return x, weights(len(counts), rows, cols, g), off, index


def mixed_counts(n, seed):
    """Groups of no row, of less than half an accumulator (112), just above it (113..128), of one tile, of several."""
    pick = np.random.default_rng(seed).choice([0, 1, 17, 60, 112, 113, 120, 128, 129, 200, 240, 241, 352, 480, 700], n)
    return [int(c) for c in pick]


# pairs: 9 row tiles are 5 pairs of tiles, of 54 tiles of rows and more: 270 units and more for 74 pairs;
# one CTA each: 38 tiles of rows and more, of 9 row tiles: 342 units and more for 148
CASES = [("pairs", mixed_counts(40, 1), 2050, 544), ("pairs", mixed_counts(44, 2), 2306, 200),
         # accumulators that take both slots and one slot in turn, with one step each
         ("pairs", [240, 112, 240, 16, 112] * 12, 1026, 96),
         ("single", [25] * 36 + [64, 36, 0], 2050, 544), ("single", [65, 16, 1, 300, 0, 128] + [7] * 30, 2306, 1500)]


@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form,counts,rows,cols", CASES)
def test_many_units(form, counts, rows, cols, dtype, paired):
    assert (sum(counts) > 1024) == (form == "pairs")
    tiles = sum(-(-c // (240 if form == "pairs" else 64)) for c in counts) * (-(-rows // 512) if form == "pairs" else -(-rows // 256))
    assert tiles > 2 * (74 if form == "pairs" else 148)
    x, w, off, index = grouped(counts, rows, cols, rows + cols)
    out = block.mx_product(x, block.mx_pack(w, paired), off, index, out_dtype=dtype)
    check_product(out, *reference(x, w, paired, off, index))


def test_products_behind_one_another_same_bits():
    """Pairs, single CTAs and clusters that split K take turns on the same processors,
    each CTA starting where another has just left."""
    forms = [grouped(counts, rows, cols, 5) for counts, rows, cols in
             ((mixed_counts(24, 3), 1026, 300), ([25] * 36, 1026, 300), ([900, 400], 512, 256), ([8], 512, 4096), ([1100], 200, 32))]
    packed = [block.mx_pack(w) for _, w, _, _ in forms]
    run = lambda i: block.mx_product(forms[i][0], packed[i], forms[i][2], forms[i][3])
    want = [run(i) for i in range(len(forms))]
    block.check()
    order = np.random.default_rng(7).integers(0, len(forms), 400)
    got = [(i, run(i)) for i in order]
    assert all(torch.equal(out, want[i]) for i, out in got)
    block.check()


@pytest.mark.parametrize("rows", [4, 100, 1100])
def test_swiglu_of_fp32_outputs_is_exact_to_fp32(rows):
    """Gates and ups that are exact in fp32 (eight E2M1 values, multiples of 2^-7 below 2^9), so that the output shows
    silu's own arithmetic in steps of 2^-24: the exponential off by at most 2, the sum by 1/2, the division by 4 and the
    product by 1/2, 7 in all (7.1 with their products).  Below -87.3 (1 + exp(-gate) above 2^126, where the division's
    range ends) 0 for less than 1.1e-36."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    cols, feats = 256, 512
    ones = torch.zeros((rows, cols), device="cuda")
    ones[:, ::32] = 1.0                                      # one value of every run
    x = block.mx_quantize(ones)
    codes = torch.randint(0, 256, (1, 2 * feats, 8, 16), generator=g, device="cuda", dtype=torch.uint8)
    codes[..., 1:] = 0
    codes[..., 0] &= 15                                      # element 0 of the run
    scales = torch.randint(127 - 6, 127 + 4, (1, 2 * feats, 8), generator=g, device="cuda", dtype=torch.uint8)
    scales[:, :, 7] = 127 + 4                                # gates up to 96 and beyond
    w = block.mx_rows(codes, scales, cols)
    out = block.mx_product(x, block.mx_pack(w, True), out_dtype=torch.float32).double()
    y = mx_ref.unpack(w.codes.cpu().numpy(), w.scales.cpu().numpy(), cols)[0][:, ::32].sum(1)
    gate, up = torch.from_numpy(y[:feats]), torch.from_numpy(y[feats:])
    assert float(gate.min()) < -80 and float(gate.max()) > 80 and bool((gate == gate.float()).all())
    want = gate / (1 + torch.exp(-gate)) * up
    err, bound = (out.cpu() - want).abs(), 7.1 * 2.0 ** -24 * want.abs() + 1.1e-36 * (gate < -87.3) * up.abs()
    assert bool((err <= bound + 2.0 ** -149).all()), float((err / (bound + 2.0 ** -149)).max())
