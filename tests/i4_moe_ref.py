"""Plain implementations, on the host and in 64 bits where values are computed, of the I4
products and codec and of the expert layer's sort, gather and combine.  They share no code
with the library."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# half the spacing of numbers over the smaller of them: what one rounding may cost
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
# ... and absolute, where binary16 runs out of exponents
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}


def matrix(rng, n, k, group, kind, zeros, pad_c=0, pad_s=0, exact=False):
    """Codes, scales and zero points as host tensors.  What lies beyond K (pad bytes of codes,
    scales and zero points after the last group) holds NaN and 255."""
    groups = k // group
    ldc = -(-(k // 2) // 16) * 16 + pad_c
    lds = -(-groups // 4) * 4 + pad_s
    codes = np.full((n, ldc), 0xFF, np.uint8)
    codes[:, : k // 2] = rng.integers(0, 256, (n, k // 2))
    scale = torch.full((n, lds), float("nan")).to(TORCH[kind])
    if exact:
        s = 2.0 ** rng.integers(-2, 3, (n, groups))
    else:
        s = rng.uniform(0.01, 0.1, (n, groups)) * rng.choice([-1.0, 1.0], (n, groups), p=[0.1, 0.9])
    scale[:, :groups] = torch.from_numpy(s).to(TORCH[kind])
    zero = None
    if zeros:
        zero = np.full((n, lds), 255, np.uint8)
        zero[:, :groups] = rng.integers(0, 16, (n, groups))
        zero = torch.from_numpy(zero)
    return torch.from_numpy(codes), scale, zero


def dense(codes, scale, zero, k, group):
    """(code - zero) * scale, code and zero, each (N, K) in 64 bits."""
    c = codes.numpy()[:, : k // 2]
    code = np.empty((c.shape[0], k))
    code[:, 0::2] = c & 15
    code[:, 1::2] = c >> 4
    s = np.repeat(scale[:, : k // group].double().numpy(), group, 1)
    z = np.full_like(s, 8.0) if zero is None else np.repeat(
        (zero.numpy()[:, : k // group] & 15).astype(float), group, 1)
    return (code - z) * s, code, s, z


def product(x, codes, scale, zero, k, group, kind):
    """The exact product and a bound on the kernel's distance from it: binary32 sums of
    x * (16 + code) and x * (16 + zero) within a group (group terms, and one more per
    group and per part that joins; 2^-23 per step covers any rounding of the matrix cores),
    then one rounding to the type."""
    w, code, s, z = dense(codes, scale, zero, k, group)
    x = x[:, :k].double().numpy()
    y = x @ w.T
    spread = np.abs(x) @ (np.abs(s) * (32 + code + z)).T
    steps = group + k // group + 16
    bound = spread * steps * 2.0 ** -23
    return y, bound + (np.abs(y) + bound) * HALF[kind] + TINY[kind]


def rne(v, kind):
    """Binary32 (or exact 64-bit) values rounded once to the type."""
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(TORCH[kind])


def quant(x, group, kind):
    """Codes (bytes) and scales of bf16 / binary16 rows, by the definition."""
    v = x.float().numpy()
    g = v.reshape(v.shape[0], -1, group)
    amax = np.abs(g).max(2)
    scale = torch.from_numpy((amax / np.float32(7)).astype(np.float32)).to(TORCH[kind])
    s = scale.float().numpy()[:, :, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, np.rint((g / s).astype(np.float32)), 0)
    c = (np.clip(q, -7, 7) + 8).astype(np.uint8).reshape(v.shape[0], -1)
    return c[:, 0::2] | (c[:, 1::2] << 4), scale


def sort(ids, experts):
    """off, src, pos of the stable sort, slot by slot."""
    flat = [int(e) if 0 <= e < experts else experts for e in ids.reshape(-1).tolist()]
    src = sorted(range(len(flat)), key=flat.__getitem__)     # stable
    pos = [0] * len(flat)
    for row, slot in enumerate(src):
        pos[slot] = row
    off = [0] * (experts + 1)
    counts = np.bincount(flat, minlength=experts + 1) if flat else np.zeros(experts + 1, int)
    off[1:] = np.cumsum(counts[:-1]).tolist()
    return (np.array(off, np.int32), np.array(src, np.int32), np.array(pos, np.int32))


def combine32(rows, pos, kept, weight, topk):
    """The weighted sum in binary32 in the defined order, before its rounding."""
    t = len(pos) // topk
    acc = np.zeros((t, rows.shape[1]), np.float32)
    r = rows.float().numpy()
    p = pos.reshape(t, topk)
    for j in range(topk):
        on = p[:, j] < kept
        part = r[p[on, j]]
        if weight is not None:
            part = (weight.reshape(t, topk)[on, j, None] * part).astype(np.float32)
        acc[on] = acc[on] + part
    return acc
