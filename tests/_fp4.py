"""Plain 64-bit references of the row and 4-bit floating point operators, in numpy."""
from __future__ import annotations

import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# halfway points between neighbouring magnitudes and whether the upper one has the even code
HALFWAY = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
UPPER_EVEN = np.array([False, True, False, True, False, True, False])


def quantize(x: np.ndarray):
    """x [rows, K] -> codes [rows, K] (0..15), scale bytes [rows, K / 32], from the definition."""
    b = np.asarray(x, np.float64).reshape(x.shape[0], -1, 32)
    finite = np.isfinite(b).all(-1)
    m = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0)).max(-1), 0)
    exponent = np.frexp(m)[1] - 1
    byte = np.where(m == 0, 0, np.maximum(exponent - 2 + 127, 0))
    v = np.where(finite[..., None], np.where(np.isfinite(b), b, 0) / np.exp2(byte - 127.0)[..., None], 0.0)
    a = np.abs(v)[..., None]
    code = ((a > HALFWAY) | ((a == HALFWAY) & UPPER_EVEN)).sum(-1)
    code = code + 8 * (np.signbit(v) & finite[..., None])
    return code.reshape(x.shape).astype(np.uint8), np.where(finite, byte, 255).astype(np.uint8)


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    code = np.stack((q & 15, q >> 4), -1).reshape(q.shape[:-1] + (-1,))
    v = np.where(code >= 8, -1.0, 1.0) * LEVELS[code & 7]
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return v * np.repeat(scale, 32, axis=-1)


def dev(a: np.ndarray, dtype=None) -> torch.Tensor:
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def wide(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def rounded(a: np.ndarray, dtype) -> np.ndarray:
    """64-bit values rounded once to a torch type."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).double().numpy()


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def floor_of(dtype) -> float:
    """Half the smallest step of a type, for results below its normal numbers."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def slot_rows(sorted_ids: np.ndarray, rows: int, n: int) -> np.ndarray:
    out = np.full(n, -1, np.int32)
    for p, s in enumerate(sorted_ids[:rows]):
        if s < n:
            out[s] = p
    return out


def routing(rng, T, topk, E, G):
    """Distinct experts of [0, G) for each token; those from E on are not resident."""
    if T == 0:
        return np.zeros((0, topk), np.int32)
    return np.argsort(rng.random((T, G)), axis=1)[:, :topk].astype(np.int32)
