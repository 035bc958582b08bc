"""fp64 definitions of the quantized linear layer's operators, for the tests: decoded operands, nearest grid
values by distance, scales by distance.  Plain and slow; shares no code with the library."""
from __future__ import annotations

import numpy as np
import torch

GROUP = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:-1])
QMAX = {"nvfp4": 6.0, "mxfp4": 6.0, "mxfp8": 448.0}


def nearest_index(v: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the grid entry nearest to v >= 0, a tie to the even index (even mantissa), clipped at the top."""
    hi = np.clip(np.searchsorted(grid, v, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = v - grid[lo], grid[hi] - v
    return np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))


def block_values(fmt: str, scales: np.ndarray) -> np.ndarray:
    if fmt == "nvfp4":
        v = E4M3[np.minimum(scales & 0x7F, 126)]
        return np.where((scales & 0x7F) == 0x7F, np.nan, v)
    return np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))


def code_values(fmt: str, codes: np.ndarray) -> np.ndarray:
    if fmt == "mxfp8":
        v = E4M3[np.minimum(codes & 0x7F, 126)]
        v = np.where((codes & 0x7F) == 0x7F, np.nan, v)
        return np.where(codes & 0x80, -v, v)
    c = np.stack([codes & 15, codes >> 4], axis=2).reshape(codes.shape[0], -1)
    return np.where(c & 8, -E2M1[c & 7], E2M1[c & 7])


def decode(t: dict, fmt: str) -> np.ndarray:
    """a q (without the tensor scale) in fp64."""
    q = code_values(fmt, t["codes"].cpu().numpy())
    a = block_values(fmt, t["block_scales"].cpu().numpy())
    return (q.reshape(q.shape[0], a.shape[1], -1) * a[:, :, None]).reshape(q.shape)


def tensor_scale(t: dict, fmt: str) -> float:
    return float(t["tensor_scale"].cpu()[0]) if fmt == "nvfp4" else 1.0


def matmul(x: dict, w: dict, fmt: str):
    """(Y, sum of magnitudes) in fp64."""
    xv, wv = decode(x, fmt), decode(w, fmt)
    s = tensor_scale(x, fmt) * tensor_scale(w, fmt)
    return (xv @ wv.T) * s, (np.abs(xv) @ np.abs(wv).T) * abs(s)


def quantize(x: np.ndarray, fmt: str) -> dict:
    """Codes (bytes as stored), block scale bytes and the tensor scale of fp64 values x [rows, cols].  A group
    with a value that is not finite in fp32 has the NaN scale and zero codes and no share in the tensor scale."""
    rows, cols = x.shape
    g = x.reshape(rows, cols // GROUP[fmt], GROUP[fmt])
    fine = np.abs(g) <= float(np.finfo(np.float32).max)
    mag = np.where(fine, np.abs(g), 0.0)
    bad = ~fine.all(axis=2)
    top = mag.max(axis=2)
    sT = np.float32(1.0)
    if fmt == "nvfp4":
        if mag.max() > 0:
            sT = max(np.float32(mag.max() / 2688.0), np.float32(2.0 ** -149))
        idx = np.maximum(nearest_index(np.minimum(top / 6.0 / float(sT), 448.0), E4M3), 1)
        idx = np.where(top == 0, 0x38, idx)
        a = E4M3[idx] * float(sT)
        stored = np.where(bad, 0x7F, idx).astype(np.uint8)
    else:
        ratio = np.clip(top / QMAX[fmt], 2.0 ** -126, 2.0 ** 126)
        k = np.floor(np.log2(ratio)).astype(np.int64)
        k -= (np.ldexp(1.0, k) > ratio)
        k += (ratio >= 1.5 * np.ldexp(1.0, k))
        k = np.where(top == 0, 0, np.clip(k, -126, 126))
        a = np.ldexp(1.0, k)
        stored = np.where(bad, 255, k + 127).astype(np.uint8)
    grid = E4M3 if fmt == "mxfp8" else E2M1
    idx = nearest_index(np.minimum(mag / a[:, :, None], QMAX[fmt]), grid)
    neg = (g < 0) & (idx > 0)
    idx = np.where(bad[:, :, None], 0, idx + neg * (0x80 if fmt == "mxfp8" else 8)).reshape(rows, cols).astype(np.uint8)
    codes = idx if fmt == "mxfp8" else (idx[:, 0::2] | (idx[:, 1::2] << 4)).astype(np.uint8)
    return {"codes": codes, "block_scales": stored, "tensor_scale": sT}


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def norm(x: torch.Tensor, residual, weight, b, eps: float):
    """(h in x's type, x' in fp64): the sum rounded to the type, then the norm of what was stored."""
    h = x.cpu() if residual is None else (x.cpu().to(torch.float64) + residual.cpu().to(torch.float64)).to(x.dtype)
    v = f64(h)
    one = np.ones(x.shape[1])
    with np.errstate(all="ignore"):
        ms = (v * v).sum(axis=1, keepdims=True) / x.shape[1]
        r = np.where(np.isfinite(ms), 1.0 / np.sqrt(ms + np.float64(np.float32(eps))), np.nan)
        return h, v * ((one if weight is None else f64(weight)) * (one if b is None else f64(b))) * r


def glu(gate: torch.Tensor, up: torch.Tensor, b) -> np.ndarray:
    g, u = f64(gate), f64(up)
    with np.errstate(all="ignore"):
        return g / (1.0 + np.exp(-g)) * (u * (np.ones(g.shape[1]) if b is None else f64(b)))


def random_quantized(rows: int, cols: int, fmt: str, seed: int, spread: float = 1.0) -> dict:
    """A quantized matrix with every code and a wide range of scales (CPU tensors)."""
    rng = np.random.default_rng(seed)
    nb = cols // GROUP[fmt]
    if fmt == "mxfp8":
        codes = rng.integers(0, 256, (rows, cols), dtype=np.uint8)
        codes = np.where((codes & 0x7F) == 0x7F, codes & 0x80, codes)
    else:
        codes = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    if fmt == "nvfp4":
        scales = rng.integers(1, 0x7F, (rows, nb), dtype=np.uint8)
    else:
        scales = np.clip(np.rint(rng.normal(120, 3 * spread, (rows, nb))), 1, 250).astype(np.uint8)
    return {"codes": torch.from_numpy(codes), "block_scales": torch.from_numpy(scales),
            "tensor_scale": torch.tensor([float(rng.uniform(0.5, 2.0)) * 2.0 ** -6], dtype=torch.float32)}


def to(t: dict, device) -> dict:
    return {k: v.to(device) for k, v in t.items()}
