"""float64 definitions of the 4-bit products that read every weight, of the
gated pair and of the block norm, and the byte layout of their packed blob.

Plain definitions, written from the formulas; nothing here follows the order
or the tiling of the device code.
"""
from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def q4_dequantize(q, s, z, group):
    """w^[n][k] = s[n][k//group] * (q[n][k] - z[n][k//group]); z None: 8."""
    q = np.asarray(q).astype(np.float64)
    of = np.arange(q.shape[1]) // group
    zk = 8.0 if z is None else np.asarray(z).astype(np.float64)[:, of]
    return np.asarray(s, dtype=np.float64)[:, of] * (q - zk)


def q4_product(x, q, s, z, group, bias=None):
    """y[m][n] = sum_k w^[n][k] x[m][k] + bias[n]."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        y = x @ q4_dequantize(q, s, z, group).T
    return y if bias is None else y + np.asarray(bias, dtype=np.float64)[None, :]


def q4_scale(x, q, s, z, group, offset=0.0):
    """Error scale of a product: sum_k |s| |q - z| |x|, or, with an offset,
    sum_k |s| (q + z + 2 offset) |x|."""
    q = np.asarray(q).astype(np.float64)
    of = np.arange(q.shape[1]) // group
    zk = np.full_like(q, 8.0) if z is None else np.asarray(z).astype(np.float64)[:, of]
    a = np.abs(q - zk) if offset == 0.0 else q + zk + 2 * offset
    return np.abs(np.asarray(x, dtype=np.float64)) @ (np.abs(np.asarray(s, dtype=np.float64))[:, of] * a).T


def gate_function(v, act):
    v = np.asarray(v, dtype=np.float64)
    if act == "silu":
        with np.errstate(over="ignore"):
            return v / (1.0 + np.exp(-v))
    if act == "gelu":
        return 0.5 * v * _erfc(-v / math.sqrt(2.0))   # 1 + erf(t), which cancels in 64 bits too
    return np.where(v < 0, 0.0, v)


def norm(v, weight=None, bias=None, center=False, plus_one=False, eps=0.0):
    """(v - c) / sqrt(mean((v - c)^2) + eps) * weight + bias, row by row."""
    v = np.asarray(v, dtype=np.float64)
    if center:
        v = v - v.mean(axis=-1, keepdims=True)
    out = v / np.sqrt((v * v).mean(axis=-1, keepdims=True) + eps)
    if weight is not None:
        out = out * (np.asarray(weight, dtype=np.float64) + (1.0 if plus_one else 0.0))
    return out if bias is None else out + np.asarray(bias, dtype=np.float64)


def block_norm(residual, y=None, gate=None, scale=1.0, post=False, post_weight=None, post_bias=None, weight=None,
               bias=None, center=False, plus_one=False, eps=0.0):
    """(r, x): r = residual + scale * gate * (y or its norm), x = norm(r)."""
    r = np.asarray(residual, dtype=np.float64)
    if y is not None:
        u = norm(y, post_weight, post_bias, center, plus_one, eps) if post else np.asarray(y, dtype=np.float64)
        if gate is not None:
            u = u * np.asarray(gate, dtype=np.float64)
        r = r + scale * u
    return r, norm(r, weight, bias, center, plus_one, eps)


# ---------------------------------------------------------------------------
# the packed blob
# ---------------------------------------------------------------------------
GATED, ZEROS, BF16_SCALES = 1, 2, 4


def q4_header_fields(N, K, group, flags):
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    cells = -(-N // 16) * (2 if flags & GATED else 1) * -(-K // 128)
    P = 128 // group
    h = {"N": N, "K": K, "group": group, "flags": flags, "w_off": 256, "w_bytes": cells * 1024}
    h["s_off"], h["s_bytes"] = 256 + h["w_bytes"], cells * 32 * P
    h["z_off"], h["z_bytes"] = up(h["s_off"] + h["s_bytes"]), cells * 8 * P if flags & ZEROS else 0
    h["total_bytes"] = up(h["z_off"] + h["z_bytes"])
    return h


def q4_pack_spec(parts, group, bf16_scales=False):
    """The blob of one part or of a gate and an up part, each (q uint8
    [N][K], scale bits uint16, zero-points uint8 or None), by the formula."""
    (N, K), zeros = parts[0][0].shape, parts[0][2] is not None
    flags = (GATED if len(parts) == 2 else 0) | (ZEROS if zeros else 0) | (BF16_SCALES if bf16_scales else 0)
    h = q4_header_fields(N, K, group, flags)
    blob = np.zeros(h["total_bytes"], dtype=np.uint8)
    blob[:4] = np.frombuffer(b"SGQ1", dtype=np.uint8)
    for at, v, t in ((4, 1, "<u4"), (8, N, "<i4"), (12, K, "<i4"), (16, group, "<i4"), (20, flags, "<u4"),
                     (24, h["w_off"], "<u8"), (32, h["w_bytes"], "<u8"), (40, h["s_off"], "<u8"),
                     (48, h["s_bytes"], "<u8"), (56, h["z_off"], "<u8"), (64, h["z_bytes"], "<u8"),
                     (72, h["total_bytes"], "<u8")):
        b = np.array([v], dtype=t).view(np.uint8)
        blob[at:at + len(b)] = b
    B, P, n_parts = -(-K // 128), 128 // group, len(parts)
    for p, (q, s, z) in enumerate(parts):
        for n in range(N):
            t, r = divmod(n, 16)
            for k in range(K):
                b, kk = divmod(k, 128)
                j, kk = divmod(kk, 32)
                c, i = divmod(kk, 8)
                cell = (t * n_parts + p) * B + b
                nibble = (i >> 1) + 4 * (i & 1)
                at = h["w_off"] + cell * 1024 + (16 * c + r) * 16 + 4 * j + nibble // 2
                blob[at] |= int(q[n, k]) << (4 * (nibble % 2))
            for g in range(s.shape[1]):
                b, i = divmod(g, P)
                at = (((t * n_parts + p) * B + b) * 16 + r) * P + i
                blob[h["s_off"] + 2 * at] = int(s[n, g]) & 255
                blob[h["s_off"] + 2 * at + 1] = int(s[n, g]) >> 8
                if zeros:
                    blob[h["z_off"] + at // 2] |= int(z[n, g]) << (4 * (at % 2))
    return blob
