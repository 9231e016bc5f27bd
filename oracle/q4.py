"""Plain numpy 4-bit group quantization, its packed layout and its products in
fp64 (the definitions in include/externd.h, written out entry by entry)."""
import numpy as np


def _bf16(x):
    """Nearest bfloat16 (ties to even) of a float32 array, as float32; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float32)
    bits = x.view(np.uint32).astype(np.uint64)
    out = ((bits + 0x7FFF + ((bits >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000)).astype(np.uint32)
    return np.where(np.isnan(x), np.float32(np.nan), out.view(np.float32)).astype(np.float32)


def quantize(W, group, symmetric):
    """(codes uint8 (rows, cols), scales float32 (rows, groups), minima float32 or None)."""
    W = np.asarray(W, dtype=np.float32)
    rows, cols = W.shape
    ng = -(-cols // group)
    codes = np.zeros((rows, cols), dtype=np.uint8)
    scales = np.zeros((rows, ng), dtype=np.float32)
    mins = None if symmetric else np.zeros((rows, ng), dtype=np.float32)
    with np.errstate(all="ignore"):
        for j in range(ng):
            w = W[:, j * group:(j + 1) * group]
            bad = ~np.isfinite(w).all(1)
            if symmetric:
                s = _bf16(np.abs(w).max(1) / np.float32(7))
                m = np.zeros_like(s)
                lo, hi, zero = -8, 7, 8
            else:
                s = _bf16((w.max(1) - w.min(1)) / np.float32(15))
                m = _bf16(w.min(1))
                lo, hi, zero = 0, 15, 0
            bad |= ~np.isfinite(s) | ~np.isfinite(m)
            s, m = np.where(bad, np.float32(np.nan), s), np.where(bad, np.float32(np.nan), m)
            on = s > 0
            t = np.rint((w - m[:, None]) / np.where(on, s, np.float32(1))[:, None])
            t = np.clip(np.where(on[:, None], t, 0), lo, hi)
            codes[:, j * group:(j + 1) * group] = t + (8 if symmetric else 0)
            scales[:, j] = s
            if mins is not None:
                mins[:, j] = m
    return codes, scales, mins


def values(codes, scales, mins, group):
    """fp64 values of codes."""
    cols = codes.shape[1]
    spread = lambda t: np.repeat(t.astype(np.float64), group, axis=1)[:, :cols]
    if mins is None:
        return (codes.astype(np.float64) - 8) * spread(scales)
    return codes.astype(np.float64) * spread(scales) + spread(mins)


def pack_codes(codes):
    """The packed words, one code at a time."""
    rows, cols = codes.shape
    tiles, chunks = -(-rows // 16), -(-cols // 128)
    words = np.zeros((tiles, chunks, 64, 4), dtype=np.uint32)
    for row in range(rows):
        for col in range(cols):
            k = col % 128
            i, p, j = k // 32, k % 32 // 8, k % 8
            shift = 4 * (j // 2) + 16 * (j % 2)
            words[row // 16, col // 128, row % 16 + 16 * p, i] |= np.uint32(int(codes[row, col]) << shift)
    return words


def pack_table(table, cols, group):
    """A (rows, groups) table in the packed order, zero in the padding."""
    rows = table.shape[0]
    tiles, chunks, per = -(-rows // 16), -(-cols // 128), 128 // group
    out = np.zeros((tiles, chunks, 16, per), dtype=table.dtype)
    for row in range(rows):
        for g in range(table.shape[1]):
            out[row // 16, g // per, row % 16, g % per] = table[row, g]
    return out
