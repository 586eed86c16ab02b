"""MXFP4 and the experts' product in 64 bits (numpy / torch on the host), for the operator tests."""

import numpy as np
import torch

GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def quantize(x: np.ndarray):
    """(codes [rows, C/2], scales [rows, C/32]) of float64 rows, by exhaustive search over scales and codes."""
    rows, c = x.shape
    b = x.astype(np.float64).reshape(-1, 32)
    bad = ~np.isfinite(b).all(axis=1)
    b = np.where(bad[:, None], 0.0, b)
    top = np.abs(b).max(axis=1)
    fits = 6.0 * np.exp2(np.arange(-127, 128))[None, :] >= top[:, None]
    byte = fits.argmax(axis=1)                                  # the smallest that fits
    a = np.abs(b) / np.exp2(byte - 127.0)[:, None]
    dist = np.abs(a[:, :, None] - GRID[None, None, :8])
    near = dist == dist.min(axis=2, keepdims=True)              # one code, or two at a tie
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=2), even.argmax(axis=2), near.argmax(axis=2))
    code = code + 8 * np.signbit(b)
    code[bad] = 0
    byte[bad] = 255
    code = code.reshape(rows, -1, 2).astype(np.uint8)
    return code[:, :, 0] | (code[:, :, 1] << 4), byte.reshape(rows, -1).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    v = np.stack((GRID[codes & 15], GRID[codes >> 4]), axis=-1).reshape(codes.shape[0], -1)
    s = np.exp2(scales.astype(np.float64) - 127)
    s[scales == 255] = np.nan
    return v * np.repeat(s, 32, axis=1)


def values_t(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """values() on the tensors' device, float64, any leading dimensions."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=codes.device)
    v = torch.stack((grid[(codes & 15).long()], grid[(codes >> 4).long()]), dim=-1).flatten(-2)
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.nan, s)
    return v * s.repeat_interleave(32, dim=-1)


def spans(offset, cap, rows):
    """[r0, r1) of every expert from its prefix sums (padded if cap > 0)."""
    off = [int(v) for v in offset]
    if cap:
        return [(e * cap, e * cap + min(cap, off[e + 1] - off[e])) for e in range(len(off) - 1)]
    return [(off[e], off[e + 1]) for e in range(len(off) - 1)]


def product(a, sa, w, sw, where):
    """(y, s): y[r] = a[r] @ w[e].T in float64 and s the same sum of absolute products; NaN in rows of no expert."""
    y = torch.full((a.shape[0], w.shape[1]), torch.nan, dtype=torch.float64, device=a.device)
    s = y.clone()
    for e, (r0, r1) in enumerate(where):
        if r1 > r0:
            va, vw = values_t(a[r0:r1], sa[r0:r1]), values_t(w[e], sw[e])
            y[r0:r1] = va @ vw.T
            s[r0:r1] = va.abs() @ vw.abs().T
    return y, s


def codes_like(rows, c, gen, device, lo=120, hi=127):
    """Random codes, and scale bytes in [lo, hi]."""
    codes = torch.randint(0, 256, (rows, c // 2), dtype=torch.uint8, generator=gen, device=device)
    scales = torch.randint(lo, hi + 1, (rows, c // 32), dtype=torch.int32, generator=gen, device=device).to(torch.uint8)
    return codes, scales
