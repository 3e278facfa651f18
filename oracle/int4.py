"""int4 weights with one scale, and optionally a zero point, per group along K.

Landing page "grouped-nf4-gemm", "Owns": the int4 GEMV of a decode step's
dense projections and its packer.  The page gives neither rounding rule nor
layout; the reading here is the NF4 packer's: nearest level in exact
arithmetic, ties to the lower code, the first element in the high nibble.
"""

import numpy as np

from .nf4 import ref_round_bf16


def ref_int4_pack(w, group, zero_points=False, scale_dtype="bf16"):
    """``w [N, K]`` fp32 -> (packed uint8 [N, K/2], scales fp32 values
    [N, K/group], zeros uint8 or None).

    Symmetric: s = fl32(max|w| / 7), z = 8.  With zero points: s =
    fl32(fl32(hi / 15) + fl32(lo / 15)) for hi = max(w, 0), lo = max(-w, 0);
    z counts the j in 0..14 with lo > (j + 1/2) s.  s is then rounded to its
    stored type.  A code counts the j with w > (j + 1/2 - z) s (products exact
    in fp64).  s == 0 stores z (0 with zero points) everywhere."""
    w = np.asarray(w, dtype=np.float32)
    N, K = w.shape
    assert K % group == 0
    b = w.reshape(N, K // group, group)
    if zero_points:
        hi = np.maximum(b.max(axis=2), np.float32(0))
        lo = np.maximum((-b).max(axis=2), np.float32(0))
        s = hi / np.float32(15) + lo / np.float32(15)
    else:
        s = np.abs(b).max(axis=2) / np.float32(7)
    assert s.dtype == np.float32
    if scale_dtype == "bf16":
        s = np.asarray(ref_round_bf16(s), dtype=np.float32)
    sd = s.astype(np.float64)
    mids = np.arange(15, dtype=np.float64) + 0.5
    if zero_points:
        z = (lo.astype(np.float64)[..., None] > mids * sd[..., None]).sum(axis=2)
        z = np.where(sd == 0, 0, z)
    else:
        z = np.full(s.shape, 8, dtype=np.int64)
    thr = (mids - z[..., None]) * sd[..., None]                      # [N, K/group, 15]
    codes = (b.astype(np.float64)[..., None] > thr[:, :, None, :]).sum(axis=3)
    codes = np.where((sd == 0)[..., None], z[..., None], codes).reshape(N, K)
    packed = ((codes[:, 0::2] << 4) | codes[:, 1::2]).astype(np.uint8)
    return packed, s, z.astype(np.uint8) if zero_points else None


def ref_int4_unpack(packed, scales, zeros=None):
    """(code - z) * s in fp64, [N, K]."""
    packed = np.asarray(packed, dtype=np.uint8)
    N, half = packed.shape
    codes = np.empty((N, 2 * half), dtype=np.float64)
    codes[:, 0::2] = packed >> 4
    codes[:, 1::2] = packed & 15
    scales = np.asarray(scales, dtype=np.float64)
    group = 2 * half // scales.shape[1]
    z = 8.0 if zeros is None else np.repeat(np.asarray(zeros, dtype=np.float64), group, axis=1)
    return (codes - z) * np.repeat(scales, group, axis=1)


def ref_int4_linear(x, packed, scales, zeros=None, bias=None):
    """``x [M, K] @ W^T + bias`` in fp64, unrounded."""
    y = np.asarray(x, dtype=np.float64) @ ref_int4_unpack(packed, scales, zeros).T
    return y if bias is None else y + np.asarray(bias, dtype=np.float64)
