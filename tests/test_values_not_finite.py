"""Values that are not finite under causal attention (indexer_causal_attention): an infinity or NaN in
column d of a value is one in column d of the outputs of the rows that see its key, as the sum
of the formula has it, and changes nothing else: not other columns, not other rows, whichever form a
call takes and wherever the key lies in it.

Weights of randn scores over these few keys are far from 0, so the kind of a column is that of the sum of the
values; the other columns have to be bit for bit those of a call with zeros in the places.
"""
import math

import numpy as np
import pytest
import torch

from tests.test_causal_attention import Batch
from tests.test_causal_tiles import KINDS

# requests, Hq, Hkv, window, sinks, page, in tiles
BATCHES = {
    "tiles": ([(300, 300)], 2, 2, 0, 0, 16, 1),
    "tiles, cut": ([(260, 1500), (3, 3)], 8, 1, 0, 0, 48, 1),
    "tiles, cut, packed": ([(900, 1500), (301, 700)], 16, 4, 0, 0, 0, 1),
    "tiles, long": ([(4000, 4000)], 16, 4, 0, 0, 64, 1),          # runs of more than 16 tiles of an item
    "tiles, window": ([(500, 900)], 4, 2, 60, 3, 1, 1),
    "rows": ([(2, 900), (1, 40)], 4, 2, 0, 0, 16, 0),
    "rows, window": ([(50, 300)], 4, 2, 60, 3, 16, 0),
    "rows, split": ([(2, 9000)], 8, 2, 0, 0, 64, 0),
}


def plant(b, rng, n=16):
    """Places (key, key/value head, column) of values of request 0, and what goes there: keys at both ends,
    around a tile's border and anywhere; column 9 gets infinities of either sign."""
    L = int(b.cu_k[1])
    keys = [0, 1, 127, 128, L - 1, L - 2, L // 2, *rng.integers(0, L, n)]
    places = {}
    for i, j in enumerate(keys):
        kind = math.nan if b.kv == "fp8" else (math.inf, -math.inf, math.nan)[i % 3]
        places[min(int(j), L - 1), int(rng.integers(b.Hkv)), int(rng.integers(b.D))] = kind
    if b.kv != "fp8":
        places[L // 3, 0, 9], places[L - L // 20 - 1, 0, 9] = math.inf, -math.inf
    return places


def values(b, places, mark):
    v = b.v.clone()
    for (j, g, d), x in places.items():
        at = int(b.slot_of(0, np.array([j]))[0])
        v[at, g, d] = (0x7F if mark else 0) if b.kv == "fp8" else (x if mark else 0.0)
    return v


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("name", list(BATCHES))
def test_columns_of_rows_that_see_them(name, dt, kv, D):
    requests, Hq, Hkv, window, sinks, page, tiles = BATCHES[name]
    rng = np.random.default_rng(41)
    b = Batch(requests, Hq, Hkv, D, window, sinks, dt, kv, page, seed=41)
    if name == "tiles":
        b.lens[rng.integers(0, b.T, 20)] = 0                      # padding: every tile has blind rows
    places = plant(b, rng)
    b.v = values(b, places, False)
    clean, lse = b.run()
    assert b.attn.info()["tiles"] == tiles
    b.check(clean, lse, rows=sorted({0, 1, b.T - 1, *rng.integers(0, b.T, 30)}))
    b.v = values(b, places, True)
    wide = torch.full((b.T, Hq, D + 3), 7.0, dtype=b.dt, device="cuda")
    got, got_lse = b.run(out=wide[:, :, :D]) if name in ("tiles", "rows") else b.run()
    assert torch.equal(got_lse, lse)
    want = torch.zeros(b.T, Hq, D, dtype=torch.float64)
    G = Hq // Hkv
    n = torch.from_numpy(np.clip(b.lens, 0, b.L))
    for (j, g, d), x in places.items():
        see = (j < n) & ((j >= n - window) | (j < sinks) | (window == 0)) & torch.from_numpy(b.req == 0)
        want[see, g * G:(g + 1) * G, d] += x
    off = ~torch.isfinite(want)
    assert off.any() and not off.all(-1).any()
    got, clean = got.cpu(), clean.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)].double(), want[torch.isinf(want)])
    assert torch.equal(got[~off], clean[~off])
    assert torch.all(wide[:, :, D:] == 7)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,kv", KINDS)
def test_every_value_of_the_last_keys(dt, kv):
    """Whole vectors that are not finite, in keys that some rows see."""
    b = Batch([(300, 500)], 4, 2, 64, dt=dt, kv=kv, page=16, seed=42)
    at = torch.from_numpy(b.slot_of(0, np.arange(400, 500)))
    b.v[at] = 0
    clean, lse = b.run()
    assert b.attn.info()["tiles"] == 1
    b.v[at] = 0xFF if kv == "fp8" else math.inf
    got, got_lse = b.run()
    sees = torch.from_numpy(b.lens > 400).cuda()
    assert torch.equal(got[~sees], clean[~sees]) and torch.equal(got_lse, lse)
    assert torch.all(torch.isnan(got[sees]) if kv == "fp8" else got[sees] == math.inf)
