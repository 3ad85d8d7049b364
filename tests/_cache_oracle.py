"""fp64 restatement of the cache operators for their tests (numpy; tables from the oracle)."""
import math

import numpy as np

import oracle as O

EPS = 1e-8


def rotation(d, h, seed=0, permute=True):
    """R as a dense matrix: z = R x, z_i = sum_j H[i, j] sign[j] / sqrt(h) x[perm[j]]."""
    perm, sign = O.build_rpbh(d, seed) if permute else O.build_block_rht(d, seed)
    H = np.kron(np.eye(d // h), O.hadamard(h)) / math.sqrt(h)
    R = np.zeros((d, d))
    R[:, perm] = H * sign
    return R


def quantize(x, R, bits):
    """codes, norms and the unit values u of rows x [..., d]."""
    z = x @ R.T
    norm = np.sqrt((z * z).sum(-1))
    u = z / (norm + EPS)[..., None] * math.sqrt(x.shape[-1])
    _, t = O.codebook(bits)
    return np.searchsorted(t, u, side="right"), norm, u


def values(codes, norms, R, bits):
    c, _ = O.codebook(bits)
    return c[codes] @ R * (norms / math.sqrt(R.shape[0]))[..., None]


def unpack(packed, bits):
    """LSB-first codes of [..., bytes]."""
    b = np.unpackbits(packed, axis=-1, bitorder="little")
    b = b.reshape(*b.shape[:-1], -1, bits).astype(np.int64)
    return (b << np.arange(bits)).sum(-1)


def pack(codes, bits):
    b = (codes[..., None] >> np.arange(bits)) & 1
    b = b.reshape(*codes.shape[:-1], -1).astype(np.uint8)
    return np.packbits(b, axis=-1, bitorder="little")


def attend(q, k, v, see, scale):
    """q [n, d], k, v [S, d], see [n, S] -> (o [n, d], sum p |v|, score bound scale |q| max|k|)."""
    o = np.zeros_like(q)
    weight = np.zeros(len(q))
    for i in range(len(q)):
        if not see[i].any():
            continue
        kk, vv = k[see[i]], v[see[i]]
        x = scale * (kk @ q[i])
        p = np.exp(x - x.max())
        p /= p.sum()
        o[i] = p @ vv
        weight[i] = p @ np.linalg.norm(vv, axis=-1)
    return o, weight


def rope(x, pos, freq, amp, rot, layout, inverse=False):
    """x [T, heads, d] -> rotated, in fp64."""
    y = x.astype(np.float64).copy()
    ang = pos[:, None].astype(np.float64) * freq
    c, s = amp * np.cos(ang)[:, None], amp * np.sin(ang)[:, None]
    s = -s if inverse else s
    i = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (
        slice(0, rot, 2), slice(1, rot, 2))
    a, b = y[..., i[0]].copy(), y[..., i[1]].copy()
    y[..., i[0]], y[..., i[1]] = a * c - b * s, a * s + b * c
    return y
