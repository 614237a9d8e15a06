"""Plain fp64 reference of the FP4 copies (numpy, no library code), for the GPU tests."""
import numpy as np

import oracle

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def padded(k: int) -> int:
    return -(-k // 256) * 256


def nearest_even(v: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the nearest entry of the ascending table for v >= 0, ties to the even index."""
    mid = (table[1:] + table[:-1]) / 2
    lo = np.searchsorted(mid, v, side="left")
    hi = np.searchsorted(mid, v, side="right")
    return np.where(lo % 2 == 0, lo, hi)


E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def quantize(w: np.ndarray):
    """w [V, H] fp64 values of a finite BF16 matrix -> (codes [V, Hp] uint8, block scale codes
    [V, Hp/16] uint8, row scales [V] fp32), from the definition: one rounding per real quotient."""
    V, H = w.shape
    p = np.zeros((V, padded(H)))
    p[:, :H] = w
    sign = np.zeros((V, padded(H)), np.uint8)
    sign[:, :H] = np.where(np.signbit(w), 8, 0)
    rs = (np.float32(np.abs(p).max(1)) / np.float32(2688.0)).astype(np.float32)
    r = rs.astype(np.float64)[:, None]
    amax = np.abs(p).reshape(V, -1, 16).max(2)
    sc = nearest_even(np.divide(amax, 6.0 * r, out=np.zeros_like(amax), where=r > 0), E4M3).astype(np.uint8)
    d = np.repeat(E4M3[sc] * r, 16, axis=1)
    c = nearest_even(np.divide(np.abs(p), d, out=np.zeros_like(p), where=d > 0), E2M1).astype(np.uint8) | sign
    return np.where(d > 0, c, 0).astype(np.uint8), sc, rs


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q: np.ndarray) -> np.ndarray:
    c = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    c[:, 0::2] = q & 15
    c[:, 1::2] = q >> 4
    return c


def values(q: np.ndarray, bs: np.ndarray, rs: np.ndarray, H: int) -> np.ndarray:
    """fp64 values [V, H] of a packed copy."""
    c = unpack(q)
    v = np.where(c > 7, -E2M1[c & 7], E2M1[c & 7]) * np.repeat(E4M3[bs], 16, axis=1)
    return (v * rs.astype(np.float64)[:, None])[:, :H]


def norm(x_bits: np.ndarray, w_bits: np.ndarray, eps: float) -> np.ndarray:
    """BF16 rms_norm_vanilla rows as fp64 values (the rounding of the fp64 expression)."""
    x, w = oracle.bf16_to_f64(x_bits), oracle.bf16_to_f64(w_bits)
    y = x * w / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    return oracle.bf16_to_f64(oracle.f64_to_bf16(y))
