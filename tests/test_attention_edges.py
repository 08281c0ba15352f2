"""Attention over the selected keys where its softmax is tested hardest: tiles without a key before,
between and after others, heads and value vectors of very different sizes, long lists; against the
formula in 64 bits.

Tolerance, from the operations, per row, head and element.  A score is a product of D terms summed
in fp32 (over e4m3 caches, of a query in e4m3 terms whose rest is below 2^-20 of its head's largest
element): off by at most
    ds = scale (D 2^-24 sum_i |q_i k_i| + 2^-20 max|q| sum_i |k_i|).
A weight is then off by a relative 2 max(ds) + 2^-20 (exponential, sum) and rounded to u_p: 2^-8 where
the queries are bf16, 2^-11 where they are fp16.  The product with v is summed in fp32, 16 keys a
step: 2^-23 a step.  fp16 weights end at 2^-24, 2^-31 of the row's largest: each is off by half of that
as well.  The output is rounded once, to u_o.  Nothing else: no term stands for weights that are lost.
"""
import numpy as np
import pytest
import torch

from sparse_attention_prefill_tcgen05_gb300 import _lib as K
from tests.test_attention import Batch, reference, selected

pytestmark = pytest.mark.gpu

MODES = [("bf16", "same"), ("fp16", "same"), ("bf16", "fp8"), ("fp16", "fp8")]
TILE = 128


def expect(b, scale=None, keys=None):
    """The formula's output and log-sum-exp of a batch, and the tolerance of each."""
    if keys is None:
        keys = selected(b.sel, b.count, b.lens, b.L, b.block)
    kf, vf = b.values()
    out, lse, ds, wabs, vabs, pmax = reference(b.q.double().numpy(), kf, vf, keys, b.slot_of, b.Hkv,
                                               b.D ** -0.5 if scale is None else scale)
    listed = b.nsel * b.block
    floor = 2.0 ** -32 * pmax[..., None] * vabs if (b.dt, b.kv) == (torch.float16, "same") else 0.0
    tol = (b.u + 2 * ds[..., None] + 2.0 ** -20 + listed / 16 * 2.0 ** -23) * wabs + floor + b.u * np.abs(out)
    tol_lse = ds + 2.0 ** -20 * (1 + np.abs(lse)) + listed / TILE * 2.0 ** -24
    return out, lse, tol, tol_lse


def hold(b, got, lse, want):
    out, want_lse, tol, tol_lse = want
    # a subnormal of the output's type is half its least step off
    step = 2.0 ** -25 if b.dt == torch.float16 else 2.0 ** -134
    g, z, none = got.double().cpu().numpy(), lse.double().cpu().numpy(), np.isneginf(want_lse)
    assert np.all(np.isfinite(g))
    off = np.abs(g - out) - (tol + step)
    assert np.all(off <= 0), (float(off.max()), np.argwhere(off > 0)[:8].tolist())
    assert np.array_equal(np.isneginf(z), none)
    assert np.all(np.abs(z - want_lse)[~none] <= tol_lse[~none])
    assert np.all(g[none] == 0)


def check(b, scale=None, keys=None, **kw):
    out, lse = b.run(scale, **kw)
    hold(b, out, lse, expect(b, scale, keys))
    return out, lse


# ------------------------------------------------------------ tiles that hold no key


# which of a row's eight tiles hold no key
EMPTY = [(0,), (0, 1), (0, 1, 2), (0, 1, 2, 3, 4), (2, 3, 4, 5), (1, 3, 5, 7), (0, 2, 4, 6), (5, 6, 7),
         (0, 1, 3, 4, 6, 7), (0, 2, 3, 5, 6, 7), ()]


def empty_tiles(b, tiles=8):
    """Row t loses tiles EMPTY[t % ...], to entries below zero and past its keys in turn."""
    per = TILE // b.block
    past = 2 ** 31 - 1
    for t in range(b.T):
        for n in EMPTY[t % len(EMPTY)]:
            b.sel[t, n * per:(n + 1) * per] = (-1, past, int(b.lens[t]) // b.block + 1)[(t + n) % 3]


@pytest.mark.parametrize("rows", [11, 170])               # split over blocks; whole
@pytest.mark.parametrize("D,group,Hkv", [(64, 5, 2), (128, 16, 1), (64, 32, 1), (128, 64, 1)])
@pytest.mark.parametrize("block", [1, 64, 128])
@pytest.mark.parametrize("dt,kv", MODES)
def test_tiles_without_a_key(dt, kv, block, D, group, Hkv, rows):
    keys = 1024 + 128 + rows
    b = Batch(((rows, keys),), group * Hkv, Hkv, D, 1024 // block, block, dt, kv, 16, seed=group + block,
              spread=3.0)
    empty_tiles(b)
    check(b)


@pytest.mark.parametrize("dt,kv", MODES)
def test_unmapped_pages_before_mapped_ones(dt, kv):
    b = Batch(((12, 2048),), 32, 1, 128, 16, 128, dt, kv, 64, seed=21, spread=3.0)
    b.sel = torch.arange(16, dtype=torch.int32).repeat(12, 1)
    b.table[0, :10] = -1                                   # the first five tiles
    b.table[0, 16:20] = b.slots // 64 + 5                  # two tiles in the middle
    check(b)


@pytest.mark.parametrize("rows", [11, 170])
@pytest.mark.parametrize("group", [8, 32, 64])
@pytest.mark.parametrize("dt,kv", MODES)
def test_scores_far_below_zero_next_to_tiles_without_a_key(dt, kv, group, rows):
    """A tile without a key has no maximum: not 0 either, beside which exp(-150) is nothing."""
    b = Batch(((rows, 1024),), group, 1, 64, 1024, 1, dt, kv, 0, seed=group, lens=[1024] * rows)
    g = torch.Generator().manual_seed(22)
    b.q = torch.full((rows, group, 64), 5.0).to(b.dt)
    if kv == "fp8":
        b.k = (-240.0 - 8 * torch.rand((1024, 1, 64), generator=g)).to(torch.float8_e4m3fn).view(torch.uint8)
        b.ks = (0.0155 + 0.0002 * torch.rand((1024, 1), generator=g))
    else:
        b.k = (-3.7 - 0.1 * torch.rand((1024, 1, 64), generator=g)).to(b.dt)
    empty_tiles(b)
    out, lse = check(b)
    assert bool((lse[:, 0] < -130).all())


@pytest.mark.parametrize("rows", [10, 170])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_keys_of_no_weight_before_others(dt, rows):
    """Scores of -inf in a row's first tiles, for every head or for some: the others keep theirs."""
    b = Batch(((rows, 1024),), 32, 1, 64, 1024, 1, dt, "same", 0, seed=23, spread=2.0, lens=[1024] * rows)
    b.sel = torch.arange(1024, dtype=torch.int32).repeat(rows, 1)
    b.q[:, :, 0], b.q[:, ::2, 1], b.q[:, 1::2, 1] = 1.0, 1.0, 0.0
    dead = torch.arange(1024) < 300
    b.k[dead, :, 0] = -float("inf")
    keys = [list(range(300, 1024))] * rows
    finite = b.k.clone()
    got, lse = b.run()
    b.k[dead] = 0
    hold(b, got, lse, expect(b, keys=keys))
    # only heads whose first element is not zero
    b.k = finite
    b.k[dead, :, 0] = 0.0
    b.q[:, ::2, 0], b.q[:, 1::2, 0] = 1.0, 0.0
    want, some = expect(b), expect(b, keys=keys)
    b.k[dead, :, 0] = torch.finfo(b.dt).min
    got, lse = b.run()
    for a, c in zip(want, some):
        a[:, ::2] = c[:, ::2]
    hold(b, got, lse, want)

# ---------------------------------------------------- weights over e4m3 caches


@pytest.mark.parametrize("rows", [3, 160])
@pytest.mark.parametrize("nats", [5.0, 8.0, 12.0])
@pytest.mark.parametrize("size", [1.0, 1e-4])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_a_value_of_zeros_far_above_the_rest(dt, size, nats, rows):
    """The key of the largest score has a value of zeros, whose scale is 1 as the cache's writer
    leaves it: the output is what the rest weighs."""
    b = Batch(((rows, 600),), 8, 1, 128, 512, 1, dt, "fp8", 0, seed=24, lens=[600] * rows)
    b.q[:, :, 0] = 8.0
    b.k[:, :, 0] = 0
    b.vs *= size
    for t in range(rows):
        b.sel[t, 77] = 599                                 # (rows have it once)
        b.sel[t][torch.arange(512) != 77] = torch.randperm(599, generator=b.g)[:511].to(torch.int32)
    top = torch.zeros(128)
    top[0] = 448.0
    b.k[599, 0] = top.to(torch.float8_e4m3fn).view(torch.uint8)
    b.ks[599] = nats * 128 ** 0.5 / 8 / 448
    b.v[599], b.vs[599] = 0, 1.0
    check(b)


@pytest.mark.parametrize("n", [2048, 16384, 65536])
@pytest.mark.parametrize("dt,kv,nats", [("bf16", "fp8", 13.0), ("fp16", "fp8", 13.0), ("bf16", "same", 13.0)])
def test_one_key_far_above_a_long_list(dt, kv, nats, n):
    """Every weight but one is e^-nats of the largest; together they weigh as much as it does or more."""
    one_far_above(dt, kv, nats, n)


def one_far_above(dt, kv, nats, n, rows=2):
    b = Batch(((rows, n),), 16, 1, 64, n, 1, dt, kv, 0, seed=25, lens=[n] * rows)
    b.sel = torch.stack([torch.arange(n), torch.arange(n - 1, -1, -1)] * (rows // 2)).to(torch.int32)
    g = torch.Generator().manual_seed(26)
    b.q = torch.zeros((rows, 16, 64))
    b.q[:, :, 0] = 8.0
    b.q = b.q.to(b.dt)
    k = torch.zeros((n, 1, 64))
    k[n // 3, 0, 0] = 448.0 if kv == "fp8" else nats
    v = 100 + 300 * torch.rand((n, 1, 64), generator=g)
    v[n // 3] = 1.0
    if kv == "fp8":
        b.k, b.v = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        b.ks, b.vs = torch.full((n, 1), nats / 448), torch.full((n, 1), 0.01)
    else:
        b.k, b.v = k.to(b.dt), v.to(b.dt)
    check(b)


@pytest.mark.parametrize("D,group,Hkv,nsel,block", [(128, 32, 1, 300, 1), (64, 5, 2, 20, 8), (64, 64, 1, 7, 64),
                                                    (128, 20, 2, 129, 1), (128, 16, 1, 1, 1)])
def test_fp16_queries_over_e4m3_keep_their_eleven_bits(D, group, Hkv, nsel, block):
    check(Batch(((9, 700),), group * Hkv, Hkv, D, nsel, block, "fp16", "fp8", 16, seed=27, spread=2.0))


def test_value_scales_far_apart():
    """Scales from 2^-100 to 2^60 in one list: each value counts with its own."""
    b = Batch(((5, 512),), 16, 1, 64, 512, 1, "bf16", "fp8", 0, seed=28, lens=[512] * 5)
    b.vs = torch.exp2(torch.randint(-100, 60, (512, 1), generator=b.g).float())
    check(b)
    b.vs = torch.exp2(torch.randint(-100, -60, (512, 1), generator=b.g).float())
    check(b)


@pytest.mark.parametrize("rows", [2, 200])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [1, 5, 8, 20, 40])
def test_places_of_a_tile_without_a_head_hold_nothing_of_the_last_call(group, dt, rows):
    """The same bits after a call that has filled the shared memory with other queries, keys and
    weights, in wider groups."""
    b = Batch(((rows, 600),), group, 1, 128, 500, 1, dt, "fp8", 16, seed=30 + group)
    first, lse = check(b)
    for wide in (group, 64):
        other = Batch(((200, 600),), wide, 1, 128, 500, 1, dt, "fp8", 16, seed=31, spread=400.0)
        other.run()
        again, lse2 = b.run()
        assert torch.equal(first, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("rows", [2, 170])
def test_fp16_weights_far_below_the_largest(rows):
    """Weights of 2^-25.5 of the largest, which keep some bits in fp16 relative to 2^7 of it."""
    one_far_above("fp16", "same", 17.7, 2048, rows)


@pytest.mark.parametrize("dt,far", [("bf16", 1e30), ("bf16", 1e-30), ("fp16", 2.0 ** 14), ("fp16", 2.0 ** -12)])
def test_heads_of_very_different_sizes(dt, far):
    """A head's queries are held relative to its own largest element, not to its neighbours'."""
    b = Batch(((6, 400),), 20, 1, 128, 300, 1, dt, "fp8", 16, seed=29)
    b.q[:, 3] *= far
    b.q[:, 11] /= far if dt == "bf16" else 1.0
    if dt == "fp16" and far > 1:
        b.q[:, 4:] *= 2.0 ** -12
    check(b, scale=1.0)


@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_and_small_values_under_large_scores(sign, kv):
    """Scores of +-60 in base 2 over values of 1e25 or 1e-30: the output is as large as the values."""
    b = Batch(((4, 600),), 16, 1, 64, 400, 1, "bf16", kv, 0, seed=30, lens=[600] * 4)
    b.q = torch.full((4, 16, 64), sign * 1.0).to(b.dt)
    one = 60 * np.log(2) / 8                              # the score, over sqrt(64) and 64 products
    rnd = torch.rand((600, 1, 64), generator=b.g)
    if kv == "fp8":
        b.k = (200 - 16 * rnd).to(torch.float8_e4m3fn).view(torch.uint8)
        b.ks = torch.full((600, 1), one / 200)
        b.vs = torch.full((600, 1), 1e23 if sign > 0 else 1e-32)
    else:
        b.k = (one - 0.1 * rnd).to(b.dt)
        b.v = ((1e25 if sign > 0 else 1e-30) * (1 + rnd)).to(b.dt)
    check(b)
