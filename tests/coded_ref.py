"""Plain 64-bit forms of a cache of 8 or 4 bits, for the tests: tables of what the
codes stand for and the nearest of them, sharing nothing with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)])
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALES = np.array([m * 2.0 ** -17 for m in range(8)] + [(8 + m) * 2.0 ** (e - 18) for e in range(1, 31) for m in range(8)])
MOST_SCALE = 10240.0
FP16_HALF_STEP = torch.finfo(torch.float16).eps / 2  # 2^-11


def scale_bytes(bits, D):
    return 1 if bits == 8 else D // 16


def nearest(x, grid):
    """Index of the nearest grid value of each x >= 0, halves to the even index, the last above it."""
    x = np.minimum(x, grid[-1])
    up = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    below, above = x - grid[up - 1], grid[up] - x
    return np.where((below < above) | ((below == above) & (up % 2 == 1)), up - 1, up)


def quantise(x, bits):
    """(codes uint8 [..., D bits / 8], scales uint8 [..., n]) of values [..., D] (a tensor, as float64)."""
    y = x.detach().cpu().double().numpy()
    if bits == 8:
        top = np.abs(y).max(-1, keepdims=True)
        c = np.full(top.shape, 79)
        for p in range(79, 175):  # the least that fits
            c = np.where((c == p) & ~(top <= 448.0 * 2.0 ** (p - 127)), p + 1, c)
        with np.errstate(invalid="ignore"):
            z = y / 2.0 ** (c - 127.0)
            code = nearest(np.abs(np.nan_to_num(z, nan=0.0, posinf=1e9, neginf=-1e9)), E4M3) | (np.signbit(z) << 7)
        return code.astype(np.uint8), np.where(np.isfinite(top), c, 255).astype(np.uint8)
    blocks = y.reshape(*y.shape[:-1], -1, 16)
    top = np.abs(blocks).max(-1, keepdims=True)
    fine = np.isfinite(top)
    byte = nearest(np.minimum(np.where(fine, top, 0.0) / 6.0, MOST_SCALE), SCALES)
    s = SCALES[byte]
    z = np.divide(np.where(fine, blocks, 0.0), s, out=np.zeros_like(blocks), where=s > 0)
    code = (nearest(np.abs(z), E2M1) | (np.signbit(blocks) << 3)).reshape(y.shape)
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8), np.where(fine, byte, 255)[..., 0].astype(np.uint8)


def values(codes, scales, bits):
    """float64 tensor [..., D] on the CPU of what codes and scales (tensors or arrays) stand for."""
    c, s = (np.asarray(t.cpu() if isinstance(t, torch.Tensor) else t) for t in (codes, scales))
    if bits == 8:
        one = np.append(E4M3, np.nan)
        by = np.where(s == 255, np.nan, 2.0 ** (np.clip(s.astype(float), 79, 175) - 127))
        return torch.from_numpy(np.where(c > 127, -1.0, 1.0) * one[c & 127] * by)
    both = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1)
    by = np.append(SCALES, [np.inf] + [np.nan] * 7)[np.minimum(s, 255)]
    with np.errstate(invalid="ignore"):
        return torch.from_numpy(np.where(both > 7, -1.0, 1.0) * E2M1[both & 7] * np.repeat(by, 16, -1))


def decode(q, k, v, table, lens, scale):
    """(out [B, H, D], lse [H, B], bound on |out error|, bound on |lse error|) in float64,
    over the values k, v [pages, page, Hkv, D] (float64, CPU).

    Bounds, as paged_ref.decode's but for the weights: a score is a sum of D products of
    exact operands in fp32, off by at most 2 D 2^-24 scale sum |q k| in any order of
    additions; exponentials and the running rescale add 2^-17 relative; a sum of n weights
    or weighted values adds 2 n 2^-24.  So far delta; it moves the output by at most
    2 delta sum p |v|, lse by delta.  A weight enters the product with V as one fp16 number:
    1 + m / 1024 times a power of two, m whole, so steps are 2^-10 of the power and half of
    one is at most 2^-11 of the weight (finfo.eps / 2); or half the smallest, 2^-25, where the largest
    weight (8 bits: times its row's power of two) is 2^15: 2^-40 of the largest, times codes
    of at most 448, of which a row's largest is above 224."""
    B, H, D = q.shape
    page, hk = k.shape[1], k.shape[2]
    q, table, lens = q.detach().cpu().double(), table.cpu().numpy(), lens.cpu().numpy()
    out = torch.zeros((B, H, D), dtype=torch.float64)
    lse = torch.full((H, B), -math.inf, dtype=torch.float64)
    off, off_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        n = int(lens[b])
        if n <= 0 or n > table.shape[1] * page:
            continue
        t = np.arange(n)
        p = table[b, t // page].astype(np.int64)
        live = (p >= 0) & (p < k.shape[0])
        if not live.any():
            continue
        at = torch.from_numpy(p[live]), torch.from_numpy((t % page)[live])
        kb, vb = k[at], v[at]
        for h in range(H):
            g = h // (H // hk)
            s = scale * (kb[:, g] @ q[b, h])
            w = torch.softmax(s, 0)
            out[b, h] = w @ vb[:, g]
            lse[h, b] = torch.logsumexp(s, 0)
            size = float((abs(scale) * (kb[:, g].abs() @ q[b, h].abs())).max())
            delta = 2 * D * 2.0 ** -24 * size + 2.0 ** -17 + 2 * n * 2.0 ** -24
            mass = w @ vb[:, g].abs()
            off[b, h] = (2 * delta + FP16_HALF_STEP) * mass + n * 2.0 ** -39 * vb[:, g].abs().amax()
            off_lse[h, b] = delta + 2.0 ** -23 * abs(float(lse[h, b]))
    step = torch.finfo(torch.bfloat16).eps / 2
    return out, lse, off * (1 + step) + step * out.abs(), off_lse
