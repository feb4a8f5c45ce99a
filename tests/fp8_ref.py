"""Plain 64-bit forms of the rotating append, the 8-bit pool and attention over it.

Written from the definitions with numpy, one token, block and row at a time; no
code of the library.  `e4m3` values are decoded through torch's CPU conversion.
"""

from __future__ import annotations

import numpy as np
import torch

BLOCK = 16
E4M3_MAX = 448.0


def bf16(x) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def f64(t) -> np.ndarray:
    return t.detach().cpu().to(torch.float32).to(torch.float64).numpy()


def decode(pool) -> np.ndarray:
    """e4m3 tensor -> float64 values (NaN codes stay NaN)."""
    return pool.detach().cpu().view(torch.float8_e4m3fn).to(torch.float32).to(torch.float64).numpy()


def encode(x) -> torch.Tensor:
    """float64 -> e4m3, nearest even, saturating (a float64 with few bits is exact in fp32)."""
    x32 = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).clamp(-E4M3_MAX, E4M3_MAX)
    return x32.to(torch.float8_e4m3fn)


def table(max_pos: int, rot: int, base=10000.0) -> np.ndarray:
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    a = np.arange(max_pos, dtype=np.float64)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def rotate(x, positions, cos_sin, interleaved, dtype=np.float64):
    """x [n, H, D] rotated (float64, or float32 with every operation rounded), and
    the size |a c| + |b s| that bounds the rounding of each element."""
    x = np.asarray(x, dtype=dtype)
    rot = cos_sin.shape[1]
    h = rot // 2
    c = cos_sin[positions, :h].astype(dtype)[:, None]
    s = cos_sin[positions, h:].astype(dtype)[:, None]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    y, size = x.copy(), np.abs(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    size[..., ia] = np.abs(a * c) + np.abs(b * s)
    size[..., ib] = np.abs(b * c) + np.abs(a * s)
    return y, size


def pow2_scale(amax: float) -> float:
    """Smallest power of two s >= 2^-64 with amax <= 448 s, by trial."""
    s = 2.0 ** -64
    while amax > E4M3_MAX * s:
        s *= 2.0
    return s


def append_fp8(codes, scales, rows, slots):
    """Reference state of an 8-bit pool after an append.

    codes: float64 [nb, 2, Hkv, 16, D] (values before scaling); scales float64
    [nb, Hkv, 2]; rows [n, 2, Hkv, D]: the new K and V rows; slots [n].
    Returns (exact new codes before rounding, new scales, rounded [nb, 2, Hkv, 16]
    bool: rows whose codes were rounded by this step)."""
    codes, scales = codes.copy(), scales.copy()
    rounded = np.zeros(codes.shape[:4], dtype=bool)
    nslots = codes.shape[0] * BLOCK
    for b in sorted({s // BLOCK for s in slots if 0 <= s < nslots}):
        toks = [t for t, s in enumerate(slots) if s >= 0 and s // BLOCK == b]
        first = min(slots[t] % BLOCK for t in toks)
        for kv in range(2):
            for h in range(codes.shape[2]):
                new = rows[toks, kv, h]
                size = np.abs(new)
                amax = float(size[np.isfinite(size)].max(initial=0.0))
                old = scales[b, h, kv]
                if first > 0 and E4M3_MAX * old >= amax:
                    s = old
                else:
                    s = pow2_scale(amax)
                    if first > 0:
                        codes[b, kv, h, :first] *= old / s
                        rounded[b, kv, h, :first] = True
                scales[b, h, kv] = s
                for t in toks:
                    codes[b, kv, h, slots[t] % BLOCK] = rows[t, kv, h] / s
                    rounded[b, kv, h, slots[t] % BLOCK] = True
    return codes, scales, rounded


def attention(q, cu, ctx, tables, values, scale):
    """out [total_q, Hq, D] float64; also, for the error bounds, per element
    sum_p w_p |v_p| and per row max_p sum_d |q_d k_pd| |scale|.

    values: float64 [nb, 2, Hkv, 16, D], the values the pool stands for."""
    q = np.asarray(q, dtype=np.float64)
    total, hq, d = q.shape
    hkv = values.shape[2]
    out, wabs = np.zeros_like(q), np.zeros_like(q)
    mag = np.zeros((total, hq, 1))
    for s in range(len(ctx)):
        n = int(cu[s + 1] - cu[s])
        if n == 0:
            continue
        c = int(ctx[s])
        ids = tables[s][:-(-c // BLOCK)]
        kv = values[ids].transpose(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, :c]
        seen = np.arange(c)[None] <= (c - n + np.arange(n))[:, None]
        for h in range(hq):
            qi = q[cu[s]:cu[s + 1], h]
            k, v = kv[0, h * hkv // hq], kv[1, h * hkv // hq]
            x = np.where(seen, qi @ k.T * scale, -np.inf)
            w = np.exp(x - x.max(axis=1, keepdims=True))
            w /= w.sum(axis=1, keepdims=True)
            out[cu[s]:cu[s + 1], h] = w @ v
            wabs[cu[s]:cu[s + 1], h] = w @ np.abs(v)
            m = np.where(seen, np.abs(qi) @ np.abs(k).T, 0.0)
            mag[cu[s]:cu[s + 1], h, 0] = m.max(axis=1) * abs(scale)
    return out, wabs, mag
