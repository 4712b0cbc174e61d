"""Operators around the routed experts, on torch tensors.

What a model puts before, after and beside ``moe_forward``: MXFP4 rows and
grouped products over them, the block's norms with its gate and residual, the
router's balance loss.  The arithmetic runs in libmoe.so (include/moe.h,
"Operators around the layer"); this module checks tensors, allocates outputs
and passes pointers.  Every call runs on the current stream of its tensors'
device, does not wait for the GPU and can be captured in a CUDA graph.

Tensors that do not fit raise ValueError, refused calls of the library
``moe.MoEError``.

``block_norm`` and ``balance_loss`` are differentiable (once); the *_forward and
*_backward functions below them are the same operators without autograd.  A
backward pass through autograd can be captured in a CUDA graph as long as no
eager graph of the same leaves is alive (torch's rule for every operator: the
leaves' nodes keep the eager graph's stream, and the capture fails); the
*_forward and *_backward functions can always be captured.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import moe

TYPES = {torch.float32: moe.MOE_F32, torch.float16: moe.MOE_F16, torch.bfloat16: moe.MOE_BF16}
MX_CHUNK = 256   # columns per chunk of an MXFP4 row (128 code bytes, 8 scale bytes)
MX_BLOCK = 34816  # bytes of 256 weight rows x 256 columns in a packed image


# A call on a few tokens takes the GPU two or three microseconds, less than the
# host's work around it, so that work is kept short: shapes and dtypes are read
# once, outputs come from empty_strided and empty_like (1.5 and 1.3 us, against
# 2.4 for torch.empty with a dtype and device), and the stream's handle is asked
# for without building a Stream object.
_raw_stream = torch._C._cuda_getCurrentRawStream
_empty = torch.empty_strided
_U8, _F32, _BF16, _I32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


def _launch(device: torch.device, call, *args) -> None:
    """call(*args, stream) on the device's current stream."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, not on {device}")
    index = device.index
    if index == torch.cuda.current_device():
        call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            call(*args, _raw_stream(index))


def _type(dtype: torch.dtype, name: str) -> int:
    kind = TYPES.get(dtype)
    if kind is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, not {dtype}")
    return kind


def _rows(t: torch.Tensor, name: str):
    """(t with contiguous elements in its rows, its row stride): any row stride
    stays as it is, other layouts are copied."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, not {t.dim()}")
    rows, cols = t.shape
    if t.is_contiguous():
        return t, cols
    ld, one = t.stride()
    if (one == 1 or cols == 1) and (ld >= cols or rows <= 1):
        return t, ld if rows > 1 else cols
    return t.contiguous(), cols


def _like(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple, device: torch.device) -> int:
    """Pointer of an optional contiguous tensor of this type, shape and device (None: 0)."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
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
    kind = _type(x.dtype, "x")
    x, ld = _rows(x, "x")
    rows, cols = x.shape
    kc = -(-cols // MX_CHUNK)
    dev = x.device
    codes = _empty((rows, 128 * kc), (128 * kc, 1), dtype=_U8, device=dev)
    scales = _empty((rows, 8 * kc), (8 * kc, 1), dtype=_U8, device=dev)
    if not values:
        _launch(dev, moe.moe_mx_quantize, x.data_ptr(), kind, ld, rows, cols, codes.data_ptr(), scales.data_ptr(), None)
        return MXRows(codes, scales, cols)
    v = _empty((rows, cols), (cols, 1), dtype=_BF16, device=dev)
    _launch(dev, moe.moe_mx_quantize, x.data_ptr(), kind, ld, rows, cols, codes.data_ptr(), scales.data_ptr(),
            v.data_ptr())
    return MXRows(codes, scales, cols), v


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
    w = weights.image.data_ptr()
    if weights.image.device != dev or weights.image.numel() != weights.n_mats * -(-weights.rows // 256) * kc * MX_BLOCK:
        raise ValueError(f"the weights' image is {weights.image.numel()} bytes on {weights.image.device}, "
                         f"not that of {weights.n_mats} matrices {weights.rows} x {cols} on {dev}")
    off = _like(offsets, "offsets", torch.int32, (weights.n_mats + 1,), dev)
    ix = _like(index, "index", torch.int32, (n_rows,), dev)
    if out is None:
        out, ld = _empty((n_rows, feats), (feats, 1), dtype=out_dtype, device=dev), feats
    else:
        rows, ld = _rows(out, "out")
        if out.shape != (n_rows, feats) or out.device != dev or rows is not out:
            raise ValueError(f"out must be [{n_rows}, {feats}] with contiguous rows on {dev}")
    _launch(dev, moe.moe_mx_product, c, s, n_x, w, weights.n_mats, weights.rows, cols, weights.paired, off, ix, n_rows,
            out.data_ptr(), TYPES[out_dtype], ld)
    return out


def check() -> None:
    """Wait for the current GPU and raise MoEError if one of these operators'
    kernels on it gave up on a bounded wait since the last check."""
    moe.moe_block_check()


# ---------------------------------------------------------------- the block's norms
def _norm_args(h, y, post, gate, scale, pre, eps):
    """(arguments without outputs, the tensors h, y and gate that they point into)."""
    dtype, dev, shape = h.dtype, h.device, h.shape
    kind = _type(dtype, "h")
    h, ld = _rows(h, "h")
    weights = post if post is not None else pre
    if weights is None:
        raise ValueError("neither post nor pre weights")
    if (y is None) != (post is None) or (gate is not None and y is None):
        raise ValueError("y and post weights come together, and a gate with them")
    wtype = weights.dtype
    if wtype != dtype and wtype != torch.float32:
        raise ValueError(f"weights must be {dtype} or float32, not {wtype}")
    rows, cols = shape
    yp = gp = post_p = pre_p = ld_y = ld_g = gate_kind = 0
    if pre is not None:
        pre_p = _like(pre, "pre", wtype, (cols,), dev)
    if y is not None:
        if y.shape != shape or y.dtype != dtype or y.device != dev:
            raise ValueError(f"y must be {dtype} {tuple(shape)} on {dev}, not {y.dtype} {tuple(y.shape)} on {y.device}")
        y, ld_y = _rows(y, "y")
        yp = y.data_ptr()
        post_p = _like(post, "post", wtype, (cols,), dev)
        if gate is not None:
            want = dtype
            if gate.shape == shape:
                gate_kind = moe.MOE_GATE_FULL
            elif gate.shape == (rows, 1):
                gate_kind = moe.MOE_GATE_TOKEN
            elif gate.shape == (cols,):
                gate_kind, want = moe.MOE_GATE_FEATURE, wtype
            else:
                raise ValueError(f"the gate must be {tuple(shape)}, {(rows, 1)} or {(cols,)}, not {tuple(gate.shape)}")
            if gate.dtype != want or gate.device != dev:
                raise ValueError(f"this gate must be {want} on {dev}, not {gate.dtype} on {gate.device}")
            if gate_kind == moe.MOE_GATE_FEATURE:
                gate = gate.contiguous()
            else:
                gate, ld_g = _rows(gate, "gate")
            gp = gate.data_ptr()
    # in the order of moe_norm_args; out, next and stats are the caller's
    a = moe.moe_norm_args(h.data_ptr(), yp, post_p, gp, pre_p, 0, 0, 0, ld, ld_y, ld_g, cols, cols, rows, cols, kind,
                          TYPES[wtype], gate_kind, scale, eps)
    return a, h, y, gate


def _new(t: torch.Tensor) -> torch.Tensor:
    """An uninitialised contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def block_norm_forward(h: torch.Tensor, y: Optional[torch.Tensor], post: Optional[torch.Tensor],
                       gate: Optional[torch.Tensor], scale: float, pre: Optional[torch.Tensor], eps: float = 1e-6):
    """out = h + scale * gate * rmsnorm(y) * post and next = rmsnorm(out) * pre in
    one pass (rmsnorm(v) = v / sqrt(mean(v^2) + eps)); see ``block_norm``.
    Returns (out, next, saved): out is None without y, next without pre; saved
    (1/rms of both norms) is for ``block_norm_backward``."""
    a, h, y, gate = _norm_args(h, y, post, gate, scale, pre, eps)
    out = nxt = None
    dev = h.device
    saved = _empty((h.shape[0], 2), (2, 1), dtype=_F32, device=dev)
    a.stats = saved.data_ptr()
    if y is not None:
        out = _new(h)
        a.out = out.data_ptr()
    if pre is not None:
        nxt = _new(h)
        a.next = nxt.data_ptr()
    _launch(dev, moe.moe_block_norm, a)
    return out, nxt, saved


def _norm_grad(t: torch.Tensor, name: str, h: torch.Tensor):
    """(rows of an output's gradient, pointer, row stride)."""
    if t.shape != h.shape or t.dtype != h.dtype or t.device != h.device:
        raise ValueError(f"{name} must be {h.dtype} {tuple(h.shape)} on {h.device}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    t, ld = _rows(t, name)
    return t, t.data_ptr(), ld


def block_norm_backward(d_out: Optional[torch.Tensor], d_next: Optional[torch.Tensor], h: torch.Tensor,
                        y: Optional[torch.Tensor], post: Optional[torch.Tensor], gate: Optional[torch.Tensor],
                        scale: float, pre: Optional[torch.Tensor], saved: torch.Tensor, eps: float = 1e-6):
    """Gradients (d_h, d_y, d_post, d_gate, d_pre) of ``block_norm_forward`` with
    the same arguments, None for what was not given.  d_out or d_next None:
    zeros."""
    if (d_next is not None and pre is None) or (d_out is not None and y is None):
        raise ValueError("a gradient without its output")
    d_pre = None
    if d_next is None and pre is not None:   # nothing comes through the second norm
        d_pre, pre = torch.zeros_like(pre), None
        if y is None:
            return torch.zeros_like(h), None, None, None, d_pre
    a, h, y, gate = _norm_args(h, y, post, gate, scale, pre, eps)
    rows, cols = a.rows, a.cols
    a.stats = _like(saved, "saved", torch.float32, (rows, 2), h.device)
    d_h = _new(h)
    g = moe.moe_norm_grads(d_h=d_h.data_ptr(), ld_d_h=cols)
    d_y = d_post = d_gate = None
    if d_out is not None:
        d_out, g.d_out, g.ld_d_out = _norm_grad(d_out, "d_out", h)
    if pre is not None:
        d_next, g.d_next, g.ld_d_next = _norm_grad(d_next, "d_next", h)
        d_pre = _new(pre)
        g.d_pre = d_pre.data_ptr()
    if y is not None:
        d_y, d_post = _new(y), _new(post)
        g.d_y, g.ld_d_y, g.d_post = d_y.data_ptr(), cols, d_post.data_ptr()
        if gate is not None:
            d_gate = _new(gate)
            g.d_gate, g.ld_d_gate = d_gate.data_ptr(), d_gate.shape[-1]
    size = moe.moe_block_norm_workspace(rows, cols)
    work = _empty((size,), (1,), dtype=_U8, device=h.device)
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
    """(logits' rows, their stride, tokens, experts, sequences, pointers of offsets and mask)."""
    if logits.dtype != torch.float32:
        raise ValueError(f"logits must be float32, not {logits.dtype}")
    logits, ld = _rows(logits, "logits")
    tokens, experts = logits.shape
    if gating != moe.MOE_GATE_SOFTMAX_TOPK and gating != moe.MOE_GATE_SIGMOID_RENORM:
        raise ValueError(f"gating={gating}")
    seqs, off, m = 1, 0, 0
    if offsets is not None:
        if offsets.dim() != 1 or len(offsets) < 2:
            raise ValueError("offsets must be [seqs + 1]")
        seqs = len(offsets) - 1
        off = _like(offsets, "offsets", torch.int32, (seqs + 1,), logits.device)
    if mask is not None:
        m = _like(mask, "mask", torch.bool, (tokens,), logits.device)
    return logits, ld, tokens, experts, seqs, off, m


def balance_loss_forward(logits: torch.Tensor, ids: torch.Tensor, coef: float, gating: int,
                         offsets: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None):
    """The balance loss of a router (see ``balance_loss``): (loss float32 [],
    counts int32 [seqs, experts], slope float32 [seqs, experts] for
    ``balance_loss_backward``)."""
    logits, ld, tokens, experts, seqs, off, m = _balance_args(logits, gating, offsets, mask)
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top_k]")
    top_k = ids.shape[1]
    i = _like(ids, "ids", torch.int32, (tokens, top_k), logits.device)
    dev = logits.device
    loss = _empty((), (), dtype=_F32, device=dev)
    counts = _empty((seqs, experts), (experts, 1), dtype=_I32, device=dev)
    slope = _empty((seqs, experts), (experts, 1), dtype=_F32, device=dev)
    size = moe.moe_balance_workspace(tokens, experts, seqs)
    work = _empty((size,), (1,), dtype=_U8, device=dev)
    _launch(dev, moe.moe_balance_loss, logits.data_ptr(), ld, i, tokens, experts, top_k, gating, off, seqs, m,
            coef, loss.data_ptr(), counts.data_ptr(), slope.data_ptr(), work.data_ptr(), size)
    return loss, counts, slope


def balance_loss_backward(d_loss: Optional[torch.Tensor], slope: torch.Tensor, logits: torch.Tensor, gating: int,
                          offsets: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the logits, float32 [tokens, experts], times d_loss (float32 [],
    None: 1); zeros for tokens of no sequence and masked ones."""
    logits, ld, tokens, experts, seqs, off, m = _balance_args(logits, gating, offsets, mask)
    s = _like(slope, "slope", torch.float32, (seqs, experts), logits.device)
    d = _like(d_loss, "d_loss", torch.float32, (), logits.device)
    out = _new(logits)
    _launch(logits.device, moe.moe_balance_loss_grad, d, s, logits.data_ptr(), ld, tokens, experts, gating, off, seqs, m,
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
