"""The 8-bit append by its definition in fp32, codes as bytes: a rounding to e4m3 by
table and the pool's state after an append, one block, head and row at a time; no
code of the library and no conversion of torch's.
"""

import numpy as np

# the 127 values of the codes 0 .. 126; code + 128 is the value's negative, 127 and 255 NaN
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                 for c in range(127)])


def code_of(x):
    """fp32 array -> e4m3 codes: nearest, ties to the even code, saturating, NaN 0x7F."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    up, down = E4M3[hi] - a, a - E4M3[hi - 1]
    c = np.where(up < down, hi, np.where(up > down, hi - 1, hi - hi % 2))
    return np.where(np.isnan(x), 0x7F, c + 128 * np.signbit(x)).astype(np.uint8)


def value_of(codes):
    c = codes.astype(np.int64)
    v = np.where(c & 128, -1.0, 1.0) * E4M3[np.minimum(c & 127, 126)]
    return np.where((c & 127) == 127, np.nan, v).astype(np.float32)


def append_bytes(codes, scales, rows, slots):
    """The pool after an append, by its definition in fp32: codes uint8 [nb, 2, H, 16, D],
    scales fp32 [nb, H, 2], rows fp32 [n, 2, H, D].  A block's old scale counts when it
    holds rows below the first new one; one that is not positive and finite counts as
    zero, and the rows it holds with it."""
    codes, scales = codes.copy(), scales.copy()
    f = np.float32
    for b in sorted({s // 16 for s in slots if 0 <= s < 16 * len(codes)}):
        toks = [t for t, s in enumerate(slots) if s >= 0 and s // 16 == b]
        first = min(slots[t] % 16 for t in toks)
        for kv in range(2):
            for h in range(codes.shape[2]):
                size = np.abs(rows[toks, kv, h])
                amax = f(size[np.isfinite(size)].max(initial=0.0))
                old = scales[b, h, kv] if first else f(0)
                if not (old > 0 and np.isfinite(old)):
                    old = f(0)
                s = old
                if old == 0 or f(448) * old < amax:
                    s = f(2.0 ** -64)
                    while f(448) * s < amax:
                        s = s * f(2)
                    held = codes[b, kv, h, :first]
                    codes[b, kv, h, :first] = code_of(value_of(held) * f(old / s))
                scales[b, h, kv] = s
                for t in toks:
                    codes[b, kv, h, slots[t] % 16] = code_of(rows[t, kv, h] / s)
    return codes, scales
