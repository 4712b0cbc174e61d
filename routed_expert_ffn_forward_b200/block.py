"""Operators around the routed experts, on torch tensors.

What a model puts before, after and beside ``moe_forward``: MXFP4 rows and
grouped products over them.  The arithmetic runs in libmoe.so (include/moe.h,
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
