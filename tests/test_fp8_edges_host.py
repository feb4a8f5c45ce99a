"""CPU tests of the 8-bit pool at its edges."""

import numpy as np
import torch

from fp8_bytes import E4M3, code_of, value_of


def test_rounding_of_its_own_agrees_with_torch():
    """(The reference above against another implementation: every code's value, ties.)"""
    all_codes = np.arange(256, dtype=np.uint8)
    v = torch.from_numpy(all_codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.nan_to_num(v, nan=-1), np.nan_to_num(value_of(all_codes), nan=-1))
    rng = np.random.default_rng(0)
    x = np.concatenate([(E4M3[1:] + E4M3[:-1]) / 2, np.exp2(rng.uniform(-14, 9, 20000))]).astype(np.float32)
    x = np.concatenate([x, -x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(1e9))])
    x = np.clip(x, -448, 448)
    assert np.array_equal(code_of(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
