"""The number formats of the FP8 pools' attention, as include/sml.h states them, on the CPU."""
import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def e4m3(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(E4M3).float().numpy()


def test_two_e4m3_terms_of_a_bf16_query():
    """q = s (hi + lo) for every bf16 magnitude up to 448 s, s = 1: exact from 2^-2 s on, within 2^-10 s
    below (half of E4M3's smallest step), and not exact everywhere below."""
    bits = np.arange(1, 0x43E1, dtype=np.uint32) << 16          # 0x43E0 is 448
    q = bits.view(np.float32)
    assert q[-1] == 448.0
    hi = e4m3(q)
    off = np.abs(q - hi - e4m3(q - hi))
    assert (off[q >= 0.25] == 0).all()
    assert off.max() <= 2.0 ** -10
    inexact = q[(off > 0) & (q >= 2.0 ** -6)]
    assert len(inexact) == 392 and inexact.max() == 0.2490234375
