"""Angles of the rotation at every int32 position against decimal arithmetic: off by at most 3e-7 rad."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import sparse_attention_prefill_tcgen05_gb300 as K

getcontext().prec = 60


def _pi():
    def arctan_of_inverse(n):
        term = total = Decimal(1) / n
        k = 1
        while abs(term) > Decimal(10) ** -58:
            term = -term / (n * n)
            k += 2
            total += term / k
        return total
    return 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))


TURN = 2 * _pi()
POSITIONS = [0, 1, -1, 77, 4095, 487935, -487936, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2]


@pytest.mark.gpu
@pytest.mark.parametrize("rot,base,factor", [(64, 10000.0, 1.0), (128, 10000.0, 1.0), (96, 500000.0, 1.0),
                                             (64, 1e6, 4.0), (48, 2.0, 1.0)])
def test_angles_at_any_position(rot, base, factor):
    n = len(POSITIONS)
    pos = torch.tensor(POSITIONS, dtype=torch.int32, device="cuda")
    x = torch.zeros((n, 1, rot), device="cuda")
    x[:, :, :rot // 2] = 1.0                             # the turned pairs are (cos, sin)
    out = K.indexer_rope(K.indexer_rope_create(rot, rot, base=base, factor=factor), x, pos)
    out = out[:, 0].double().cpu().numpy()
    off = 0.0
    for i in range(rot // 2):
        f = Decimal(base) ** (Decimal(-2 * i) / rot) / Decimal(factor)
        for t, p in enumerate(POSITIONS):
            a = float((p * f) % TURN)
            # the angle the pair stands at, from the wanted one
            c, s = out[t, i], out[t, i + rot // 2]
            off = max(off, abs(np.arctan2(s * np.cos(a) - c * np.sin(a), c * np.cos(a) + s * np.sin(a))))
    # the angle's 3e-7, and 1.5e-7 of the sine and cosine (each once: they are across the angle)
    assert off <= 3e-7 + 1.5e-7 * 2 ** 0.5, off
