"""Operators around the routed experts, on torch tensors.

What a model puts before, after and beside ``moe_forward``: MXFP4 rows and
grouped products over them, the block's norms with its gate and residual, the
router's balance loss.  The arithmetic runs in libmoe.so (include/moe.h,
"Operators around the layer"); this module checks tensors, allocates outputs
and passes pointers.  Every call runs on the current stream of its tensors'
device, does not wait for the GPU and can be captured in a CUDA graph.

Tensors that do not fit raise ValueError, refused calls of the library
``moe.MoEError``.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import moe

TYPES = {torch.float32: moe.MOE_F32, torch.float16: moe.MOE_F16, torch.bfloat16: moe.MOE_BF16}
MX_CHUNK = 256   # columns per chunk of an MXFP4 row (128 code bytes, 8 scale bytes)


def _launch(device: torch.device, call, *args) -> None:
    """call(*args, stream) on the device's current stream."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, not on {device}")
    if device.index == torch.cuda.current_device():
        call(*args, torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(device):
            call(*args, torch.cuda.current_stream().cuda_stream)


def _type(t: torch.Tensor, name: str) -> int:
    if t.dtype not in TYPES:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    return TYPES[t.dtype]


def _matrix(t: torch.Tensor, name: str) -> torch.Tensor:
    """t as rows of contiguous elements (any row stride; copied if it has none)."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, not {t.dim()}")
    if (t.stride(1) == 1 or t.shape[1] == 1) and (t.stride(0) >= t.shape[1] or t.shape[0] <= 1):
        return t
    return t.contiguous()


def _ld(t: torch.Tensor) -> int:
    return max(t.stride(0), t.shape[1]) if t.shape[0] > 1 else t.shape[1]


def _like(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape, device: torch.device) -> int:
    """Pointer of an optional contiguous tensor of this type, shape and device (None: 0)."""
    if t is None:
        return 0
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on {device}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


# ---------------------------------------------------------------- MXFP4
class MXRows(NamedTuple):
    """Rows in MXFP4: codes uint8 [..., 128 kc] and scales uint8 [..., 8 kc] of
    ``cols`` values in kc = ceil(cols / 256) chunks (runs of 32, GGUF order)."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int


class MXWeights(NamedTuple):
    """Packed weights of ``mx_product``: n_mats matrices [rows, cols]."""
    image: torch.Tensor
    n_mats: int
    rows: int
    cols: int
    paired: bool


def mx_quantize(x: torch.Tensor, values: bool = False):
    """x [rows, cols] (float32, float16 or bfloat16) in MXFP4.  With ``values``
    returns (rows, what they stand for as bfloat16 [rows, cols])."""
    kind = _type(x, "x")
    x = _matrix(x, "x")
    rows, cols = x.shape
    kc = -(-cols // MX_CHUNK)
    codes = torch.empty((rows, 128 * kc), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, 8 * kc), dtype=torch.uint8, device=x.device)
    v = torch.empty((rows, cols), dtype=torch.bfloat16, device=x.device) if values else None
    _launch(x.device, moe.moe_mx_quantize, x.data_ptr(), kind, _ld(x), rows, cols, codes.data_ptr(), scales.data_ptr(),
            v.data_ptr() if values else None)
    out = MXRows(codes, scales, cols)
    return (out, v) if values else out


def mx_rows(codes: torch.Tensor, scales: torch.Tensor, cols: int) -> MXRows:
    """Rows from the fields of GGUF MXFP4 blocks: codes uint8 [..., n_blocks, 16]
    and E8M0 scales uint8 [..., n_blocks] of ceil(cols / 32) blocks a row."""
    nb = -(-cols // 32)
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise ValueError("codes and scales must be uint8")
    if cols < 1 or codes.shape != scales.shape + (16,) or scales.shape[-1] != nb:
        raise ValueError(f"{cols} columns need codes [..., {nb}, 16] and scales [..., {nb}], "
                         f"not {tuple(codes.shape)} and {tuple(scales.shape)}")
    if cols % 32:   # values behind the last column are not part of the row
        codes = codes.clone()
        live = cols % 32
        j = torch.arange(16, device=codes.device)
        keep = torch.where(j < live, 0x0F, 0) + torch.where(j + 16 < live, 0xF0, 0)
        codes[..., -1, :] &= keep.to(torch.uint8)
    pad = -nb % 8
    if pad:
        codes = torch.nn.functional.pad(codes, (0, 0, 0, pad))
        scales = torch.nn.functional.pad(scales, (0, pad), value=127)
    return MXRows(codes.flatten(-2).contiguous(), scales.contiguous(), cols)


def mx_blocks(rows: MXRows) -> torch.Tensor:
    """The rows as GGUF MXFP4 blocks, uint8 [..., 17 * ceil(cols / 32)]: what a
    layer's host store holds for MXFP4 weights."""
    nb = -(-rows.cols // 32)
    codes = rows.codes.unflatten(-1, (-1, 16))[..., :nb, :]
    return torch.cat([rows.scales[..., :nb, None], codes], -1).flatten(-2)


def mx_from_blocks(blocks: torch.Tensor, cols: int) -> MXRows:
    """Rows from GGUF MXFP4 blocks, uint8 [..., 17 * ceil(cols / 32)]."""
    if blocks.dtype != torch.uint8 or blocks.shape[-1] != 17 * -(-cols // 32):
        raise ValueError(f"{cols} columns are uint8 [..., {17 * -(-cols // 32)}], not {blocks.dtype} {tuple(blocks.shape)}")
    b = blocks.unflatten(-1, (-1, 17))
    return mx_rows(b[..., 1:], b[..., 0], cols)


def mx_pack(rows: MXRows, paired: bool = False) -> MXWeights:
    """Weights laid out once for ``mx_product``: rows [n_mats, n, ...] or [n, ...].
    ``paired``: the first n/2 rows are gate rows, the rest up rows, and the
    product returns silu(gate) * up."""
    codes, scales, cols = rows
    if codes.dim() == 2:
        codes, scales = codes.unsqueeze(0), scales.unsqueeze(0)
    kc = -(-cols // MX_CHUNK)
    if codes.dim() != 3 or codes.shape[2] != 128 * kc:
        raise ValueError(f"codes of {cols} columns must be [n_mats, rows, {128 * kc}], not {tuple(codes.shape)}")
    n_mats, n, _ = codes.shape
    c = _like(codes, "codes", torch.uint8, (n_mats, n, 128 * kc), codes.device)
    s = _like(scales, "scales", torch.uint8, (n_mats, n, 8 * kc), codes.device)
    size = moe.moe_mx_image_bytes(n_mats, n, cols)
    if size == 0 or (paired and n % 2):
        raise ValueError(f"{n_mats} matrices of {n} x {cols} (1..1024 of 1..2^20 x 1..65536, an even n if paired)")
    image = torch.empty(size, dtype=torch.uint8, device=codes.device)
    _launch(codes.device, moe.moe_mx_pack, c, s, n_mats, n, cols, paired, image.data_ptr())
    return MXWeights(image, n_mats, n, cols, paired)


def mx_product(x: MXRows, weights: MXWeights, offsets: Optional[torch.Tensor] = None,
               index: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[r] = weights[g] x[index[r]] for the rows offsets[g] <= r < offsets[g + 1]
    of each group g, in fp32 sums, rounded once to out_dtype (bfloat16 or
    float32); silu(gate) * up of it for paired weights.

    offsets: int32 [n_mats + 1], not decreasing (None for one matrix: all rows).
    index: int32 [n_rows] (None: row r of x); an entry that is no row of x gives
    a row of zeros.  out: [n_rows, features] to write into (any row stride);
    rows of no group are left as they were (in a tensor allocated here:
    undefined)."""
    codes, scales, cols = x
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"the output is bfloat16 or float32, not {out_dtype}")
    if cols != weights.cols or codes.dim() != 2:
        raise ValueError(f"rows of {cols} columns against weights of {weights.cols}")
    dev, n_x = codes.device, codes.shape[0]
    kc = -(-cols // MX_CHUNK)
    n_rows = n_x if index is None else index.shape[0]
    feats = weights.rows // 2 if weights.paired else weights.rows
    if offsets is None and weights.n_mats != 1:
        raise ValueError(f"{weights.n_mats} matrices need offsets")
    c = _like(codes, "codes", torch.uint8, (n_x, 128 * kc), dev)
    s = _like(scales, "scales", torch.uint8, (n_x, 8 * kc), dev)
    w = _like(weights.image, "the weights' image", torch.uint8, weights.image.shape, dev)
    off = _like(offsets, "offsets", torch.int32, (weights.n_mats + 1,), dev)
    ix = _like(index, "index", torch.int32, (n_rows,), dev)
    if out is None:
        out = torch.empty((n_rows, feats), dtype=out_dtype, device=dev)
    elif tuple(out.shape) != (n_rows, feats) or out.device != dev or _matrix(out, "out") is not out:
        raise ValueError(f"out must be [{n_rows}, {feats}] with contiguous rows on {dev}")
    _launch(dev, moe.moe_mx_product, c, s, n_x, w, weights.n_mats, weights.rows, cols, weights.paired, off, ix, n_rows,
            out.data_ptr(), TYPES[out_dtype], _ld(out))
    return out


def mx_check() -> None:
    """Wait for the current GPU and raise MoEError if a product on it gave up on
    a bounded wait."""
    moe.moe_mx_check()


# ---------------------------------------------------------------- the block's norms
def _gate_kind(gate: Optional[torch.Tensor], h: torch.Tensor) -> int:
    if gate is None:
        return moe.MOE_GATE_NONE
    if gate.shape == h.shape:
        return moe.MOE_GATE_FULL
    if gate.shape == h.shape[:1] + (1,):
        return moe.MOE_GATE_TOKEN
    if gate.shape == h.shape[1:]:
        return moe.MOE_GATE_FEATURE
    raise ValueError(f"the gate must be {tuple(h.shape)}, {(h.shape[0], 1)} or {(h.shape[1],)}, not {tuple(gate.shape)}")


def _norm_args(h, y, post, gate, scale, pre, eps):
    """(arguments without outputs, the tensors they point into)."""
    kind = _type(h, "h")
    h = _matrix(h, "h")
    weights = post if post is not None else pre
    if weights is None:
        raise ValueError("neither post nor pre weights")
    if (y is None) != (post is None) or (gate is not None and y is None):
        raise ValueError("y and post weights come together, and a gate with them")
    if weights.dtype not in (h.dtype, torch.float32):
        raise ValueError(f"weights must be {h.dtype} or float32, not {weights.dtype}")
    rows, cols = h.shape
    a = moe.moe_norm_args(h=h.data_ptr(), ld_h=_ld(h), rows=rows, cols=cols, type=kind, weight_type=TYPES[weights.dtype],
                          scale=scale, eps=eps)
    a.pre = _like(pre, "pre", weights.dtype, (cols,), h.device)
    if y is not None:
        if y.shape != h.shape or y.dtype != h.dtype or y.device != h.device:
            raise ValueError(f"y must be {h.dtype} {tuple(h.shape)} on {h.device}, not {y.dtype} {tuple(y.shape)} on {y.device}")
        y = _matrix(y, "y")
        a.y, a.ld_y = y.data_ptr(), _ld(y)
        a.post = _like(post, "post", weights.dtype, (cols,), h.device)
        a.gate_kind = _gate_kind(gate, h)
        if gate is not None:
            want = weights.dtype if a.gate_kind == moe.MOE_GATE_FEATURE else h.dtype
            if gate.dtype != want or gate.device != h.device:
                raise ValueError(f"this gate must be {want} on {h.device}, not {gate.dtype} on {gate.device}")
            gate = gate.contiguous() if gate.dim() == 1 else _matrix(gate, "gate")
            a.gate, a.ld_gate = gate.data_ptr(), _ld(gate) if gate.dim() == 2 else cols
    return a, (h, y, gate)


def block_norm_forward(h: torch.Tensor, y: Optional[torch.Tensor], post: Optional[torch.Tensor],
                       gate: Optional[torch.Tensor], scale: float, pre: Optional[torch.Tensor], eps: float = 1e-6):
    """out = h + scale * gate * rmsnorm(y) * post and next = rmsnorm(out) * pre in
    one pass (rmsnorm(v) = v / sqrt(mean(v^2) + eps)); see ``block_norm``.
    Returns (out, next, saved): out is None without y, next without pre; saved
    (1/rms of both norms) is for ``block_norm_backward``."""
    a, keep = _norm_args(h, y, post, gate, scale, pre, eps)
    h = keep[0]
    new = lambda: torch.empty(h.shape, dtype=h.dtype, device=h.device)
    out, nxt = None if y is None else new(), None if pre is None else new()
    saved = torch.empty((h.shape[0], 2), dtype=torch.float32, device=h.device)
    a.stats, a.ld_out, a.ld_next = saved.data_ptr(), a.cols, a.cols
    if out is not None:
        a.out = out.data_ptr()
    if nxt is not None:
        a.next = nxt.data_ptr()
    _launch(h.device, moe.moe_block_norm, a)
    return out, nxt, saved


def block_norm_backward(d_out: Optional[torch.Tensor], d_next: Optional[torch.Tensor], h: torch.Tensor,
                        y: Optional[torch.Tensor], post: Optional[torch.Tensor], gate: Optional[torch.Tensor],
                        scale: float, pre: Optional[torch.Tensor], saved: torch.Tensor, eps: float = 1e-6):
    """Gradients (d_h, d_y, d_post, d_gate, d_pre) of ``block_norm_forward`` with
    the same arguments, None for what was not given.  d_out or d_next None:
    zeros."""
    d_pre = None
    if d_next is None and pre is not None:   # nothing comes through the second norm
        d_pre, pre_used = torch.zeros_like(pre), None
        if y is None:
            return torch.zeros_like(h), None, None, None, d_pre
    else:
        pre_used = pre
    a, keep = _norm_args(h, y, post, gate, scale, pre_used, eps)
    h, y, gate = keep
    a.stats = _like(saved, "saved", torch.float32, (a.rows, 2), h.device)
    g = moe.moe_norm_grads()
    held = []
    for name, t in (("d_out", d_out), ("d_next", d_next)):
        if t is None:
            continue
        if (name == "d_next" and pre is None) or (name == "d_out" and y is None):
            raise ValueError(f"{name} without its output")
        if t.shape != h.shape or t.dtype != h.dtype or t.device != h.device:
            raise ValueError(f"{name} must be {h.dtype} {tuple(h.shape)} on {h.device}, "
                             f"not {t.dtype} {tuple(t.shape)} on {t.device}")
        t = _matrix(t, name)
        held.append(t)
        setattr(g, name, t.data_ptr())
        setattr(g, "ld_" + name, _ld(t))
    new = lambda t: torch.empty(t.shape, dtype=t.dtype, device=t.device)
    d_h = new(h)
    g.d_h, g.ld_d_h = d_h.data_ptr(), a.cols
    d_y = d_post = d_gate = None
    if y is not None:
        d_y, d_post = new(y), new(post)
        g.d_y, g.ld_d_y, g.d_post = d_y.data_ptr(), a.cols, d_post.data_ptr()
        if gate is not None:
            d_gate = new(gate)
            g.d_gate, g.ld_d_gate = d_gate.data_ptr(), d_gate.shape[-1]
    if pre_used is not None:
        d_pre = new(pre)
        g.d_pre = d_pre.data_ptr()
    size = moe.moe_block_norm_workspace(a.rows, a.cols)
    work = torch.empty(size, dtype=torch.uint8, device=h.device)
    _launch(h.device, moe.moe_block_norm_grad, a, g, work.data_ptr(), size)
    return d_h, d_y, d_post, d_gate, d_pre


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, y, post, gate, scale, pre, eps):
        out, nxt, saved = block_norm_forward(h, y, post, gate, scale, pre, eps)
        ctx.save_for_backward(h, y, post, gate, pre, saved)
        ctx.scale, ctx.eps = scale, eps
        ctx.set_materialize_grads(False)
        return out, nxt

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out, d_next):
        h, y, post, gate, pre, saved = ctx.saved_tensors
        d_h, d_y, d_post, d_gate, d_pre = block_norm_backward(d_out, d_next, h, y, post, gate, ctx.scale, pre, saved,
                                                              ctx.eps)
        return d_h, d_y, d_post, d_gate, None, d_pre, None


def block_norm(h: torch.Tensor, y: Optional[torch.Tensor] = None, post: Optional[torch.Tensor] = None,
               gate: Optional[torch.Tensor] = None, scale: float = 1.0, pre: Optional[torch.Tensor] = None,
               eps: float = 1e-6):
    """The norms around a block with its gate and residual, differentiable:

        out  = h + scale * gate * rmsnorm(y) * post
        next = rmsnorm(out) * pre

    h, y: [rows, cols], float32, float16 or bfloat16, any row stride.  post, pre:
    [cols] of that type or float32 (both the same).  gate: [rows, cols] or
    [rows, 1] of h's type, [cols] of the weights' type, or None.  Without y, out
    is None and next = rmsnorm(h) * pre; without pre, next is None.  Returns
    (out, next)."""
    return _BlockNorm.apply(h, y, post, gate, scale, pre, eps)


# ---------------------------------------------------------------- the balance loss
def _balance_args(logits, gating, offsets, mask):
    if logits.dtype != torch.float32:
        raise ValueError(f"logits must be float32, not {logits.dtype}")
    logits = _matrix(logits, "logits")
    dev, tokens = logits.device, logits.shape[0]
    if gating not in (moe.MOE_GATE_SOFTMAX_TOPK, moe.MOE_GATE_SIGMOID_RENORM):
        raise ValueError(f"gating={gating}")
    if offsets is not None and (offsets.dim() != 1 or len(offsets) < 2):
        raise ValueError("offsets must hold at least two tokens' places")
    seqs = 1 if offsets is None else len(offsets) - 1
    off = _like(offsets, "offsets", torch.int32, (seqs + 1,), dev)
    m = _like(mask, "mask", torch.bool, (tokens,), dev)
    return logits, seqs, off, m


def balance_loss_forward(logits: torch.Tensor, ids: torch.Tensor, coef: float, gating: int,
                         offsets: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None):
    """The balance loss of a router (see ``balance_loss``): (loss float32 [],
    counts int32 [seqs, experts], slope float32 [seqs, experts] for
    ``balance_loss_backward``)."""
    logits, seqs, off, m = _balance_args(logits, gating, offsets, mask)
    dev = logits.device
    tokens, experts = logits.shape
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top_k]")
    top_k = ids.shape[1]
    i = _like(ids, "ids", torch.int32, (tokens, top_k), dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    counts = torch.empty((seqs, experts), dtype=torch.int32, device=dev)
    slope = torch.empty((seqs, experts), dtype=torch.float32, device=dev)
    size = moe.moe_balance_workspace(tokens, experts, seqs)
    work = torch.empty(size, dtype=torch.uint8, device=dev)
    _launch(dev, moe.moe_balance_loss, logits.data_ptr(), _ld(logits), i, tokens, experts, top_k, gating, off, seqs, m,
            coef, loss.data_ptr(), counts.data_ptr(), slope.data_ptr(), work.data_ptr(), size)
    return loss, counts, slope


def balance_loss_backward(d_loss: Optional[torch.Tensor], slope: torch.Tensor, logits: torch.Tensor, gating: int,
                          offsets: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the logits, float32 [tokens, experts], times d_loss (float32 [],
    None: 1); zeros for tokens of no sequence and masked ones."""
    logits, seqs, off, m = _balance_args(logits, gating, offsets, mask)
    dev = logits.device
    tokens, experts = logits.shape
    s = _like(slope, "slope", torch.float32, (seqs, experts), dev)
    d = _like(d_loss, "d_loss", torch.float32, (), dev)
    out = torch.empty((tokens, experts), dtype=torch.float32, device=dev)
    _launch(dev, moe.moe_balance_loss_grad, d, s, logits.data_ptr(), _ld(logits), tokens, experts, gating, off, seqs, m,
            out.data_ptr(), experts)
    return out


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, coef, gating, offsets, mask):
        loss, counts, slope = balance_loss_forward(logits, ids, coef, gating, offsets, mask)
        ctx.save_for_backward(logits, slope, offsets, mask)
        ctx.gating = gating
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_loss, _):
        logits, slope, offsets, mask = ctx.saved_tensors
        return balance_loss_backward(d_loss, slope, logits, ctx.gating, offsets, mask), None, None, None, None, None


def balance_loss(logits: torch.Tensor, ids: torch.Tensor, coef: float, gating: int,
                 offsets: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None):
    """Load-balance loss of the router and per-expert counts, differentiable in
    the logits: (loss float32 [], counts int32 [seqs, experts]).

    logits: float32 [tokens, experts] (``MoELayer.logits``).  ids: int32 [tokens,
    top_k] (``MoELayer.routing``).  gating: MOE_GATE_SOFTMAX_TOPK or
    MOE_GATE_SIGMOID_RENORM, the probabilities' form.  offsets: int32 [seqs + 1],
    packed sequences (None: one of all tokens); the loss is the mean over those
    with tokens.  mask: bool [tokens], False for tokens that do not count."""
    return _BalanceLoss.apply(logits, ids, coef, gating, offsets, mask)
