"""The operators around the layer without a GPU: what they refuse (before any
launch), MXFP4 row layouts, and the float64 references' own checks."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import moe_ref  # noqa: E402
from routed_expert_ffn_forward_b200 import block, build, moe  # noqa: E402
from tests import block_ref, mx_ref  # noqa: E402

P = 1 << 20   # an address that is never touched


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def refused(status, call, *args):
    with pytest.raises(moe.MoEError) as e:
        call(*args)
    assert e.value.status == status and moe.moe_last_error()


BAD, NO = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("status,args", [
    (BAD, (P, moe.MOE_F32, 31, 4, 32, P, P, None)),          # ld below cols
    (BAD, (P, moe.MOE_F32, 0, 4, 0, P, P, None)),
    (BAD, (P, moe.MOE_F32, 32, -1, 32, P, P, None)),
    (BAD, (P, moe.MOE_F32, 70000, 4, 70000, P, P, None)),
    (NO, (P, moe.MOE_Q8_0, 32, 4, 32, P, P, None)),
    (NO, (P, moe.MOE_BF16, 65536, 1 << 24, 65536, P, P, None)),
    (BAD, (None, moe.MOE_F32, 32, 4, 32, P, P, None)),
    (BAD, (P, moe.MOE_F32, 32, 4, 32, P + 8, P, None)),      # codes not aligned
    (BAD, (P, moe.MOE_F32, 32, 4, 32, P, P + 4, None)),
    (BAD, (P + 2, moe.MOE_F32, 32, 4, 32, P, P, None)),
    (BAD, (P, moe.MOE_BF16, 32, 4, 32, P, P, P + 1)),
])
def test_quantize_refusals(status, args):
    refused(status, moe.moe_mx_quantize, *args)


def test_image_bytes_and_pack_refusals():
    assert moe.moe_mx_image_bytes(1, 256, 256) == 34816
    assert moe.moe_mx_image_bytes(3, 257, 257) == 3 * 2 * 2 * 34816
    for bad in ((0, 256, 256), (1025, 256, 256), (1, 0, 256), (1, 256, 0), (1, 256, 65537), (1, (1 << 20) + 1, 256)):
        assert moe.moe_mx_image_bytes(*bad) == 0
    refused(BAD, moe.moe_mx_pack, P, P, 1, 255, 256, True, P)         # paired needs even rows
    refused(BAD, moe.moe_mx_pack, P, None, 1, 256, 256, False, P)
    refused(BAD, moe.moe_mx_pack, P, P, 1, 256, 256, False, P + 8)


@pytest.mark.parametrize("status,changes", [
    (BAD, dict(n_mats=0)), (BAD, dict(rows=0)), (BAD, dict(cols=0)), (BAD, dict(rows=255, paired=True)),
    (BAD, dict(n_rows=-1)), (BAD, dict(n_x=-1)), (BAD, dict(ld=255)), (BAD, dict(offsets=None)),
    (BAD, dict(index=None, n_rows=9)), (NO, dict(out_type=moe.MOE_F16)), (BAD, dict(codes=None)), (BAD, dict(image=None)),
    (BAD, dict(out=None)), (BAD, dict(codes=P + 4)), (BAD, dict(scales=P + 4)), (BAD, dict(image=P + 8)),
    (BAD, dict(out=P + 1)), (BAD, dict(offsets=P + 2)), (BAD, dict(index=P + 1)),
])
def test_product_refusals(status, changes):
    a = dict(codes=P, scales=P, n_x=8, image=P, n_mats=2, rows=256, cols=256, paired=False, offsets=P, index=P, n_rows=8,
             out=P, out_type=moe.MOE_BF16, ld=256)
    a.update(changes)
    refused(status, moe.moe_mx_product, *a.values())


def norm(**changes):
    a = dict(h=P, y=P, post=P, gate=P, pre=P, out=P, next=P, stats=P, ld_h=64, ld_y=64, ld_gate=64, ld_out=64, ld_next=64,
             rows=4, cols=64, type=moe.MOE_BF16, weight_type=moe.MOE_F32, gate_kind=moe.MOE_GATE_FULL, scale=1.0, eps=1e-6)
    a.update(changes)
    return moe.moe_norm_args(**a)


@pytest.mark.parametrize("status,changes", [
    (BAD, dict(rows=-1)), (BAD, dict(cols=0)), (BAD, dict(cols=16385, ld_h=16385)), (NO, dict(type=12)),
    (NO, dict(weight_type=moe.MOE_F16)), (BAD, dict(gate_kind=4)), (BAD, dict(post=None, pre=None)), (BAD, dict(post=None)),
    (BAD, dict(h=None)), (BAD, dict(y=None)), (BAD, dict(out=None)), (BAD, dict(next=None)), (BAD, dict(gate=None)),
    (BAD, dict(ld_h=63)), (BAD, dict(ld_y=63)), (BAD, dict(ld_gate=63)), (BAD, dict(ld_out=63)), (BAD, dict(ld_next=63)),
    (BAD, dict(h=P + 1)), (BAD, dict(post=P + 2)), (BAD, dict(stats=P + 2)),
    (BAD, dict(gate_kind=moe.MOE_GATE_FEATURE, gate=P + 2)),
])
def test_norm_refusals(status, changes):
    refused(status, moe.moe_block_norm, norm(**changes))


def test_norm_gradient_refusals():
    size = moe.moe_block_norm_workspace(4, 64)
    assert size > 0 and moe.moe_block_norm_workspace(4, 16385) == 0
    g = dict(d_out=P, d_next=P, d_h=P, d_y=P, d_post=P, d_gate=P, d_pre=P, ld_d_out=64, ld_d_next=64, ld_d_h=64, ld_d_y=64,
             ld_d_gate=64)
    for changes in (dict(d_h=None), dict(d_y=None), dict(d_post=None), dict(d_pre=None), dict(d_next=None), dict(d_gate=None),
                    dict(ld_d_h=1), dict(ld_d_out=1), dict(ld_d_next=1), dict(ld_d_y=1), dict(ld_d_gate=1), dict(d_h=P + 1)):
        refused(BAD, moe.moe_block_norm_grad, norm(), moe.moe_norm_grads(**{**g, **changes}), P, size)
    refused(BAD, moe.moe_block_norm_grad, norm(), moe.moe_norm_grads(**g), P, size - 1)
    refused(BAD, moe.moe_block_norm_grad, norm(), moe.moe_norm_grads(**g), P + 8, size)
    refused(BAD, moe.moe_block_norm_grad, norm(stats=None), moe.moe_norm_grads(**g), P, size)
    assert moe.lib().moe_block_norm_grad(ctypes.byref(norm()), None, P, size, None) == BAD
    assert moe.lib().moe_block_norm(None, None) == BAD


@pytest.mark.parametrize("rows", [0, 4, 3000])
def test_norm_gradient_of_an_output_that_is_not_there(rows):
    """Without pre there is no next, and a gradient of it is refused at any number
    of rows (a stage of the ring has no room for it)."""
    size = moe.moe_block_norm_workspace(rows, 64)
    g = dict(d_out=P, d_h=P, d_y=P, d_post=P, d_gate=P, ld_d_out=64, ld_d_h=64, ld_d_y=64, ld_d_gate=64)
    for ld in (0, 64):
        refused(BAD, moe.moe_block_norm_grad, norm(rows=rows, pre=None, next=None),
                moe.moe_norm_grads(d_next=P, ld_d_next=ld, **g), P, size)


def test_balance_refusals():
    size = moe.moe_balance_workspace(64, 16, 1)
    assert size > 0
    for bad in ((-1, 16, 1), (64, 0, 1), (64, 1025, 1), (64, 16, 0), (64, 16, 65536)):
        assert moe.moe_balance_workspace(*bad) == 0
    base = dict(logits=P, ld=16, ids=P, tokens=64, experts=16, top_k=2, gating=0, offsets=None, seqs=1, mask=None, coef=0.1,
                loss=P, counts=P, slope=P, workspace=P, workspace_bytes=size)
    for changes in (dict(tokens=-1), dict(experts=0), dict(experts=1025, ld=2000), dict(top_k=0), dict(top_k=33), dict(ld=15),
                    dict(gating=2), dict(seqs=0), dict(seqs=2), dict(logits=None), dict(ids=None), dict(loss=None),
                    dict(counts=None), dict(slope=None), dict(workspace=None), dict(logits=P + 2), dict(workspace=P + 4),
                    dict(workspace_bytes=size - 1)):
        refused(BAD, moe.moe_balance_loss, *{**base, **changes}.values())
    grad = dict(d_loss=P, slope=P, logits=P, ld=16, tokens=64, experts=16, gating=0, offsets=None, seqs=1, mask=None,
                d_logits=P, ld_out=16)
    for changes in (dict(slope=None), dict(logits=None), dict(d_logits=None), dict(ld_out=15), dict(gating=5), dict(seqs=3),
                    dict(d_loss=P + 1), dict(tokens=-2), dict(experts=2000)):
        refused(BAD, moe.moe_balance_loss_grad, *{**grad, **changes}.values())


def test_cluster_barriers_are_reached_by_whole_warps():
    """The aligned cluster barrier is undefined for a warp whose lanes are apart:
    every use follows a __syncwarp() directly."""
    import os
    csrc = os.path.join(os.path.dirname(build.__file__), "csrc")
    uses = 0
    for path in build.sources():
        lines = [l.split("//")[0].strip() for l in open(path)]
        lines = [l for l in lines if l]
        for before, line in zip(lines, lines[1:]):
            if "cluster_sync()" in line:
                uses += 1
                assert before == "__syncwarp();", (os.path.relpath(path, csrc), before, line)
    assert uses >= 4


def test_dynamic_shared_memory_is_aligned_to_its_widest_access():
    """The operators access their dynamic shared memory in 16-byte words, and it says
    so: an array of floats may be placed at any multiple of four bytes behind static
    shared memory."""
    import os
    import re
    declared = []
    for name in ("balance.cu", "block_norm.cu", "mx_product.cu"):
        text = open(os.path.join(os.path.dirname(build.__file__), "csrc", name)).read()
        declared += re.findall(r"extern __shared__[^;]*;", text)
    assert len(declared) == 3 and all("__align__(16)" in d for d in declared), declared


def test_warps_that_stay_together_give_up_together():
    """The product's MMA and epilogue warps shuffle and load tensor memory as whole
    warps, so each of their bounded waits ends with one answer of the warp."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(build.__file__), "csrc", "mx_product.cu")).read()
    mma = text.index("- MMA (the whole warp")
    epilogue = text.index("- epilogue\n", mma)
    end = text.index("__syncthreads()", epilogue)
    roles = re.sub(r"//[^\n]*", "", text[mma:end])
    waits = [m.start() for m in re.finditer(r"mbar_wait", roles)]
    agreed = [i for m in re.finditer(r"warp_agrees\((.*?)\);", roles, re.S) for i in range(m.start(), m.end())]
    assert len(waits) >= 6 and set(waits) <= set(agreed)


def test_the_product_s_launcher_chooses_its_stores():
    """Every caller of the product gets the stores that its output allows: none sets
    them, or leaves them out, by itself."""
    import os
    import re
    found = {}
    for path in build.sources():
        n = len(re.findall(r"\.wide_store\s*=", open(path).read()))
        if n:
            found[os.path.basename(path)] = n
    assert found == {"mx_product.cu": 1}


def test_forward_mx_refusals_without_a_layer():
    refused(BAD, moe.moe_forward_mx, None, P, P, 4)
    refused(BAD, moe.moe_set_mx_experts, None, P, P)


def bare_layer(**attrs):
    """A MoELayer without a library layer, for checks that come before its use."""
    from routed_expert_ffn_forward_b200.layer import MoELayer
    L = MoELayer.__new__(MoELayer)
    L.E, L.S, L.H, L.I, L.k, L.handle = 4, 0, 256, 128, 2, None
    for name, value in attrs.items():
        setattr(L, name, value)
    return L


def test_forward_mx_tensor_checks():
    L, bf = bare_layer(), torch.bfloat16
    x = torch.zeros((4, 256), dtype=bf)
    meta = torch.zeros((4, 256), dtype=bf, device="meta")
    gate_up = block.MXWeights(torch.zeros(4 * 34816, dtype=torch.uint8), 4, 256, 256, True)
    down = block.MXWeights(torch.zeros(4 * 34816, dtype=torch.uint8), 4, 256, 128, False)
    for call in (
        lambda: L.forward_mx(x),                                             # not on a GPU
        lambda: L.forward_mx(meta),
        lambda: L.forward_mx(x.float()),
        lambda: L.forward_mx(x[:, :128]),
        lambda: L.set_mx_experts(gate_up, down),                             # not on a GPU
        lambda: L.set_mx_experts(gate_up._replace(paired=False), down),
        lambda: L.set_mx_experts(gate_up._replace(cols=128), down),
    ):
        with pytest.raises(ValueError):
            call()


def test_balance_loss_of_another_number_of_tokens(monkeypatch):
    """Routing and logits are copied for the last forward's tokens, whatever the
    tensors hold: another T is refused before anything is allocated."""
    assert moe.moe_last_tokens(None) == 0
    monkeypatch.setattr(moe, "moe_last_tokens", lambda handle: 8)
    for T in (7, 9, -1):
        with pytest.raises(ValueError, match="the last forward had 8"):
            bare_layer(gating=1).balance_loss(T, 0.01)


def test_tensor_checks():
    bf, f32 = torch.bfloat16, torch.float32
    x, w = torch.zeros((4, 64), dtype=bf), torch.ones(64, dtype=bf)
    u8 = torch.uint8
    rows = block.MXRows(torch.zeros((4, 128), dtype=u8), torch.zeros((4, 8), dtype=u8), 64)
    weights = block.MXWeights(torch.zeros(2 * 34816, dtype=u8), 2, 100, 64, False)
    one = weights._replace(n_mats=1)
    off = torch.zeros(3, dtype=torch.int32)
    logits, ids = torch.zeros((4, 16)), torch.zeros((4, 2), dtype=torch.int32)
    for call in (
        lambda: block.mx_quantize(x),                                        # not on a GPU
        lambda: block.mx_quantize(x.double()),
        lambda: block.mx_quantize(x[0]),
        lambda: block.mx_pack(rows),
        lambda: block.mx_pack(rows._replace(cols=300)),
        lambda: block.mx_pack(rows._replace(codes=rows.codes[:3], scales=rows.scales[:3]), paired=True),
        lambda: block.mx_rows(torch.zeros((3, 2, 16), dtype=u8), torch.zeros((3, 3), dtype=u8), 64),
        lambda: block.mx_rows(torch.zeros((3, 2, 16)), torch.zeros((3, 2)), 64),
        lambda: block.mx_from_blocks(torch.zeros((3, 33), dtype=u8), 64),
        lambda: block.mx_product(rows, weights),                             # offsets missing
        lambda: block.mx_product(rows, weights, off.long()),
        lambda: block.mx_product(rows, weights, off[:2]),
        lambda: block.mx_product(rows, weights, off, torch.zeros(4)),
        lambda: block.mx_product(rows, weights, off, out_dtype=torch.float16),
        lambda: block.mx_product(rows._replace(cols=65), weights, off),
        lambda: block.mx_product(rows, weights._replace(rows=300), off),     # an image of other weights
        lambda: block.mx_product(rows, one, out=torch.zeros((4, 99), dtype=bf)),
        lambda: block.mx_product(rows, one, out=torch.zeros((100, 4), dtype=bf).t()),
        lambda: block.mx_product(rows, one),                                 # not on a GPU
        lambda: block.block_norm_forward(x, None, None, None, 1.0, None),
        lambda: block.block_norm_forward(x, x, None, None, 1.0, w),
        lambda: block.block_norm_forward(x, None, w, None, 1.0, w),
        lambda: block.block_norm_forward(x, None, None, x, 1.0, w),
        lambda: block.block_norm_forward(x, x.float(), w, None, 1.0, w),
        lambda: block.block_norm_forward(x, x[:3], w, None, 1.0, w),
        lambda: block.block_norm_forward(x, x, w.half(), None, 1.0, None),
        lambda: block.block_norm_forward(x, x, w, None, 1.0, w.float()),
        lambda: block.block_norm_forward(x, x, w, torch.zeros((2, 64), dtype=bf), 1.0, None),
        lambda: block.block_norm_forward(x, x, w, x.float(), 1.0, None),
        lambda: block.block_norm_forward(x, x, w.float(), w, 1.0, None),
        lambda: block.block_norm_forward(x.double(), None, None, None, 1.0, w.double()),
        lambda: block.block_norm_forward(x, x, w, None, 1.0, w),             # not on a GPU
        lambda: block.block_norm_backward(x, None, x, None, None, None, 1.0, w, torch.zeros((4, 2))),
        lambda: block.block_norm_backward(None, x, x, x, w, None, 1.0, None, torch.zeros((4, 2))),
        lambda: block.block_norm_backward(None, x, x, None, None, None, 1.0, w, torch.zeros((3, 2))),
        lambda: block.block_norm_backward(None, x.float(), x, None, None, None, 1.0, w, torch.zeros((4, 2))),
        lambda: block.balance_loss_forward(logits.half(), ids, 0.1, 0),
        lambda: block.balance_loss_forward(logits, ids.long(), 0.1, 0),
        lambda: block.balance_loss_forward(logits, ids[:3], 0.1, 0),
        lambda: block.balance_loss_forward(logits, ids[0], 0.1, 0),
        lambda: block.balance_loss_forward(logits, ids, 0.1, 2),
        lambda: block.balance_loss_forward(logits, ids, 0.1, 0, torch.zeros(1, dtype=torch.int32)),
        lambda: block.balance_loss_forward(logits, ids, 0.1, 0, torch.zeros(3)),
        lambda: block.balance_loss_forward(logits, ids, 0.1, 0, None, torch.zeros(4)),
        lambda: block.balance_loss_forward(logits, ids, 0.1, 0),             # not on a GPU
        lambda: block.balance_loss_backward(None, torch.zeros((2, 16)), logits, 0),
        lambda: block.balance_loss_backward(torch.zeros(1), torch.zeros((1, 16)), logits, 0),
    ):
        with pytest.raises(ValueError):
            call()


def test_rows_from_gguf_blocks_hold_the_oracle_s_values():
    g = np.random.default_rng(3)
    for cols in (32, 64, 256, 288, 1024):
        raw = g.integers(0, 256, size=(5, cols // 32 * 17), dtype=np.uint8)
        raw[:, ::17] = g.integers(100, 150, size=(5, cols // 32))
        rows = block.mx_from_blocks(torch.from_numpy(raw), cols)
        assert rows.codes.shape == (5, 128 * -(-cols // 256)) and rows.scales.shape == (5, 8 * -(-cols // 256))
        got = mx_ref.unpack(rows.codes.numpy(), rows.scales.numpy(), cols)
        np.testing.assert_array_equal(got, moe_ref.mxfp4_dequant(raw))
        assert torch.equal(block.mx_blocks(rows), torch.from_numpy(raw))


def test_rows_clear_what_lies_behind_the_last_column():
    codes = torch.full((2, 2, 16), 0x77, dtype=torch.uint8)
    scales = torch.full((2, 2), 127, dtype=torch.uint8)
    for cols in (33, 40, 47, 48, 49, 63):
        rows = block.mx_rows(codes, scales, cols)
        v = mx_ref.unpack(rows.codes.numpy(), rows.scales.numpy(), 256)
        assert (v[:, :cols] == 6).all() and (v[:, cols:] == 0).all()
    assert (codes == 0x77).all()


def test_reference_quantisation_is_the_nearest_value():
    g = np.random.default_rng(5)
    x = g.standard_normal((20, 96)) * np.exp2(g.integers(-140, 100, size=(20, 1)).astype(float))
    code, scale, value = mx_ref.quantize(x)
    v = np.abs(np.pad(x, ((0, 0), (0, 0)))).reshape(20, 3, 32)
    top = v.max(-1)
    s = np.exp2(scale.astype(float) - 127)
    assert ((top / s < 8) & ((top / s >= 4) | (scale == 0))).all()
    err = np.abs(value - x).reshape(20, 3, 32)
    nearest = np.abs(v[..., None] - mx_ref.LEVELS * s[..., None, None]).min(-1)
    np.testing.assert_array_equal(err, nearest)
    # ties to the even code, saturation at 6
    t = np.zeros((1, 32))
    t[0, :9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -2.5]
    np.testing.assert_array_equal(mx_ref.quantize(t)[2][0, :9], [0, 1, 1, 2, 2, 4, 4, 6, -2])


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).requires_grad_()
    h, y, post, gate, pre = r(3, 5), r(3, 5), r(5), r(3, 1), r(5)
    assert torch.autograd.gradcheck(lambda *a: block_ref.block_norm(a[0], a[1], a[2], a[3], 0.7, a[4], 1e-6), (h, y, post, gate, pre))
    logits = r(7, 6)
    ids = torch.topk(logits.detach(), 2, 1).indices
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 1], dtype=torch.bool)
    for sigmoid in (False, True):
        f = lambda l: block_ref.balance_loss(l, ids, 0.3, sigmoid, torch.tensor([0, 3, 3, 6]), mask)[0]
        assert torch.autograd.gradcheck(f, (logits,))
