"""Plain forms of the rotation and of a cache in 8 bits, for their tests: element by element from the
definitions, in 64 bits but where a step is fp32 by definition."""

import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def rotated(x, angles, positions, interleaved):
    """x [T, H, d] turned by the rows `positions` of angles [positions, dim]: the products and sums rounded to
    32 bits each, as numpy does; [T, H, d] float32."""
    x = x.float().cpu().numpy().copy()
    table = angles.cpu().numpy()[np.asarray(positions)]
    half = table.shape[1] // 2
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c, s = table[:, None, j], table[:, None, half + j]
        x1, x2 = x[:, :, a].copy(), x[:, :, b].copy()
        x[:, :, a] = x1 * c - x2 * s
        x[:, :, b] = x2 * c + x1 * s
    return torch.from_numpy(x)


def least(most, scale):
    """The least i with most <= 448 scale 2^i, by exact fractions of Python's integers."""
    from fractions import Fraction
    m, s = Fraction(float(most)), Fraction(float(scale)) * 448
    i = math.floor(math.log2(most)) - math.floor(math.log2(scale)) - 12
    while m > s * Fraction(2) ** i:
        i += 1
    return i


def append(x, values, scales, table, start, lens, rows=None):
    """Rows x [T, H, d] (float32) into values [n_pages, H, page, d] e4m3 and scales [n_pages, H, blocks] (CPU tensors,
    changed in place), sequence after sequence, block after block, head after head."""
    page, per = values.shape[2], scales.shape[2]
    block = page // per
    at = 0
    for b, n in enumerate(lens):
        i = 0
        while i < n:
            pos = int(start[b]) + i
            step = min(n - i, block - pos % block)
            p, r = int(table[b][pos // page]), pos % page
            w, kept = r // block, r % block
            of = list(range(at + i, at + i + step))
            new = x[[int(rows[j]) for j in of] if rows is not None else of]  # [step, H, d]
            for h in range(values.shape[1]):
                y = new[:, h]
                fine = torch.isfinite(y)
                most = float(torch.where(fine, y.abs(), 0.0).max())
                old = float(scales[p, h, w])
                if kept and math.isfinite(old) and old >= 2.0 ** -126:
                    k = max(0, least(most, old)) if most > 0 else 0
                    now = old * 2.0 ** k
                    if k:
                        was = values[p, h, r - kept: r].double()
                        values[p, h, r - kept: r] = (was * 2.0 ** -k).float().to(E4M3)
                else:
                    now = 2.0 ** max(-118, least(most, 1.0)) if most > 0 else 2.0 ** -118
                scales[p, h, w] = now
                inv = np.float32(1.0) / np.float32(now)
                z = torch.from_numpy(y.numpy() * inv)
                values[p, h, r: r + step] = torch.where(fine, z, float("nan")).to(E4M3)
            i += step
        at += n


def dequantised(values, scales):
    """[n_pages, H, page, d] float64."""
    return (values.double().unflatten(2, (scales.shape[2], -1)) * scales.double()[..., None, None]).flatten(2, 3)


def quantised(x, blocks):
    """A cache [n_pages, H, page, d] float32 as e4m3 values and scales, each block near the type's range."""
    y = x.unflatten(2, (blocks, -1))
    scale = torch.exp2(torch.ceil(torch.log2(y.abs().amax((-2, -1)).clamp(min=1e-30) / 440.0)))
    return (y / scale[..., None, None]).flatten(2, 3).to(E4M3), scale
