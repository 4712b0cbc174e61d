"""Plain float64 references of the MXFP4 operators (numpy, from the OCP
microscaling definition), written apart from the kernels."""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x float64 [R, C] -> (codes uint8 [R, nb, 32] one per value, scale bytes
    uint8 [R, nb], values float64 [R, C]), nb = ceil(C / 32)."""
    R, C = x.shape
    nb = -(-C // 32)
    v = np.zeros((R, nb * 32))
    v[:, :C] = x
    v = v.reshape(R, nb, 32)
    top = np.abs(v).max(-1)
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(top)
        e = np.where((top > 0) & ~bad, np.frexp(np.where(bad, 1.0, top))[1] - 1 - 2, -127)
        e = np.maximum(e, -127)
        a = np.abs(np.where(bad[..., None], 0.0, v)) * np.exp2(-e.astype(np.float64))[..., None]
    # nearest level, a tie to the even code
    dist = np.abs(a[..., None] - LEVELS)
    best = dist.min(-1, keepdims=True)
    cand = dist == best
    even = cand & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), cand.argmax(-1))
    value = LEVELS[code] * np.exp2(e.astype(np.float64))[..., None]
    neg = np.signbit(v)
    value = np.where(neg, -value, value)
    value[bad] = np.nan
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    return (code + 8 * neg).astype(np.uint8), scale, value.reshape(R, -1)[:, :C]


def unpack(codes, scales, cols):
    """uint8 codes [..., 128 kc] and scales [..., 8 kc] -> float64 [..., cols]."""
    b = codes.reshape(codes.shape[:-1] + (-1, 16))
    c = np.concatenate([b & 15, b >> 4], -1)
    v = np.concatenate([LEVELS, -LEVELS])[c] * np.exp2(scales.astype(np.float64) - 127)[..., None]
    v[np.broadcast_to((scales == 255)[..., None], v.shape)] = np.nan
    return v.reshape(codes.shape[:-1] + (-1,))[..., :cols]
