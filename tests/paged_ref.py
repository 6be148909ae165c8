"""Plain 64-bit forms of the rotary and paged-cache operators, for the tests:
one request, row and page at a time, sharing nothing with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

NO_PAGES, BAD_LENGTH, BAD_PAGE = 1, 2, 4


def rotate(x, positions, inv_freq, axis, interleaved=False, inverse=False):
    """float64 [rows, heads, D]; positions [rows, axes] or [rows]."""
    y = x.detach().cpu().double().clone()
    half = len(inv_freq)
    pos = positions.detach().cpu().double()
    if pos.dim() == 1:
        pos = pos[:, None].expand(-1, int(max(axis)) + 1)
    for i in range(half):
        phi = pos[:, int(axis[i])] * float(inv_freq[i])
        c, s = torch.cos(phi)[:, None], torch.sin(phi)[:, None] * (-1.0 if inverse else 1.0)
        u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = y[:, :, u].clone(), y[:, :, w].clone()
        y[:, :, u], y[:, :, w] = a * c - b * s, b * c + a * s
    return y


def rotate_bound(x, ref, half, interleaved, dtype):
    """Allowed |error| of the fp32 rotation of x, rounded to dtype.

    The angle in half turns is rounded to fp32 (at most 2^-25, times pi is
    9.4e-8) after a truncation of 2^-31; sine and cosine, the two products and
    the sum add at most 2^-24 each of |a| + |b|: below 2^-21 (|a| + |b|) in all.
    Rounding to the type is half a step."""
    m = x.detach().cpu().double().abs().clone()
    if interleaved:
        s = m[:, :, 0:2 * half:2] + m[:, :, 1:2 * half:2]
        m[:, :, 0:2 * half:2], m[:, :, 1:2 * half:2] = s, s
    else:
        s = m[:, :, :half] + m[:, :, half:2 * half]
        m[:, :, :half], m[:, :, half:2 * half] = s, s
    m[:, :, 2 * half:] = 0  # copied
    inner = 2.0 ** -21 * m
    if dtype == torch.float32:
        return inner
    step = torch.finfo(dtype).eps / 2
    return inner * (1 + step) + torch.where(m > 0, step * ref.abs(), 0.0)


def tables(lens, delta, table, free_list, n_free, rows, page, num_pages):
    """numpy int64 in, copies out: (lens, n_free, slots, positions, offsets, table, free_list, status)."""
    lens, delta = lens.astype(np.int64), delta.astype(np.int64)
    table, free = table.copy(), free_list.copy()
    B, width = table.shape
    capacity = width * page
    pages = lambda n: -(-int(n) // page)  # noqa: E731
    status, served, offsets, at = 0, [], [0], 0
    for b in range(B):
        at += max(int(delta[b]), 0)
        offsets.append(min(at, 2**31 - 1))
        after = lens[b] + delta[b]
        ok = 0 <= lens[b] <= capacity and 0 <= after <= capacity and (delta[b] <= 0 or at <= rows)
        if not ok:
            status |= BAD_LENGTH
        served.append(ok)
    freed = [table[b, i] for b in range(B) if served[b]
             for i in range(pages(lens[b] + delta[b]), pages(lens[b]))]
    top = int(n_free) + len(freed)
    if n_free < 0 or top > num_pages:
        status |= BAD_PAGE
        served, freed, top, taken = [False] * B, [], int(n_free), 0
    else:
        free[n_free:top] = freed
        taken = wanted = 0
        for b in range(B):
            need = pages(lens[b] + delta[b]) - pages(lens[b]) if served[b] else 0
            if need <= 0:
                continue
            if wanted + need > top:
                served[b], status = False, status | NO_PAGES
            else:
                for i in range(need):
                    table[b, pages(lens[b]) + i] = free[top - 1 - wanted - i]
                taken = wanted + need
            wanted += need
    slots, positions = np.full(rows, -1, np.int64), np.zeros(rows, np.int64)
    for b in range(B):
        for r in range(offsets[b], min(offsets[b + 1], rows)):
            t = lens[b] + r - offsets[b]
            positions[r] = t
            if served[b]:
                p = table[b, t // page]
                if 0 <= p < num_pages:
                    slots[r] = p * page + t % page
                else:
                    status |= BAD_PAGE
    lens_out = np.where(served, lens + delta, lens)
    return lens_out, top - taken, slots, positions, np.array(offsets), table, free, status


def decode(q, k_pages, v_pages, table, lens, scale):
    """(out [B, H, D], lse [H, B], bound on |out error|, bound on |lse error|) in float64.

    Bounds: a score is a sum of D products in fp32, off by at most
    2 D 2^-24 scale sum |q k| in any order of additions; exponentials, the
    running rescale and a weight held in 16 bits or more add 2^-15 relative; a sum
    of n weights or weighted values adds 2 n 2^-24.  The weights' relative error
    delta moves the output by at most 2 delta sum p |v|, lse by delta."""
    B, H, D = q.shape
    page, hk = k_pages.shape[1], k_pages.shape[2]
    num_pages = k_pages.shape[0]
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
        live = (p >= 0) & (p < num_pages)
        idx = torch.from_numpy(p[live] * 1).to(k_pages.device), torch.from_numpy((t % page)[live]).to(k_pages.device)
        if not live.any():
            continue
        k, v = k_pages[idx].cpu().double(), v_pages[idx].cpu().double()
        for h in range(H):
            g = h // (H // hk)
            s = scale * (k[:, g] @ q[b, h])
            w = torch.softmax(s, 0)
            out[b, h] = w @ v[:, g]
            lse[h, b] = torch.logsumexp(s, 0)
            size = float((abs(scale) * (k[:, g].abs() @ q[b, h].abs())).max())
            delta = 2 * D * 2.0 ** -24 * size + 2.0 ** -15 + 2 * n * 2.0 ** -24
            off[b, h] = 2 * delta * (w @ v[:, g].abs())
            off_lse[h, b] = delta + 2.0 ** -23 * abs(float(lse[h, b]))
    step = torch.finfo(torch.bfloat16).eps / 2
    return out, lse, off * (1 + step) + step * out.abs(), off_lse
