"""Codes of e4m3 caches are those of the fp32 quotient x / scale, ties to the even code."""
import pytest
import torch

import sparse_attention_prefill_tcgen05_gb300 as K

pytestmark = pytest.mark.gpu


def write(x, aligned=True):
    """Codes and scales of [rows, D] in one call (rows a two-byte step off their 16 bytes take the
    kernel for any alignment)."""
    rows, D = x.shape
    if not aligned:
        wide = torch.zeros((rows, 1, D + 1), dtype=x.dtype, device="cuda")
        wide[:, 0, 1:] = x
        x = wide[:, :, 1:]
    else:
        x = x[:, None]
    codes = torch.empty((rows, 1, D), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, 1), device="cuda")
    K.indexer_cache_write(x, codes, scales)
    return codes[:, 0], scales


def quotients(x):
    """The same in torch, in fp32: amax / 448 and x / scale (by tensors: torch multiplies by the
    reciprocal of a number)."""
    x = x.float()
    amax = x.abs().amax(dim=1, keepdim=True)
    s = torch.where(amax > 0, (amax / torch.full_like(amax, 448)).clamp(min=2.0 ** -126),
                    torch.ones_like(amax))
    return (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_every_pair_of_a_largest_element_and_another(dt, aligned):
    """All mantissas of 8 bits against all, at several exponents: among them every tie."""
    m = torch.arange(128, 256, device="cuda").float()
    rows = []
    for shift in range(0, 10):
        # a row: its largest element, then the 128 mantissas (those not above it), both signs
        other = (m * 2.0 ** -shift).expand(128, 128)
        other = torch.where(other <= m[:, None], other, torch.zeros_like(other))
        rows.append(torch.cat([m[:, None], -other, other[:, :127]], dim=1))
    x = torch.cat(rows)
    for size in (1.0, 2.0 ** -10, 2.0 ** (8 if dt == torch.float16 else 60)):
        y = (x * size).to(dt)
        codes, s = write(y, aligned)
        want, want_s = quotients(y)
        assert torch.equal(s, want_s)
        assert torch.equal(codes, want)


@pytest.mark.parametrize("aligned", [True, False])
def test_many_fp32_rows(aligned):
    g = torch.Generator(device="cuda").manual_seed(0)
    for _ in range(6):
        x = torch.randn((100000, 128), generator=g, device="cuda")
        codes, s = write(x, aligned)
        want, want_s = quotients(x)
        assert torch.equal(s, want_s) and torch.equal(codes, want)


@pytest.mark.parametrize("aligned", [True, False])
def test_small_zero_and_infinite_rows(aligned):
    x = torch.zeros((6, 64), device="cuda")
    x[1] = torch.linspace(-1, 1, 64, device="cuda") * 1e-38      # the scale's floor
    x[2] = torch.linspace(-1, 1, 64, device="cuda") * 1e-44
    x[3, :4] = torch.tensor([float("inf"), -float("inf"), 1.0, 3e38], device="cuda")
    x[4, :2] = torch.tensor([float("nan"), 5.0], device="cuda")
    x[5] = torch.linspace(-1, 1, 64, device="cuda") * 3.4e38
    codes, s = write(x, aligned)
    for t in (0, 1, 2, 5):
        want, want_s = quotients(x[t:t + 1])
        assert torch.equal(codes[t:t + 1] & 0x7F, want & 0x7F) and torch.equal(s[t:t + 1], want_s)
    v = codes.view(torch.float8_e4m3fn).float()
    assert v[3, :3].tolist() == [448.0, -448.0, 0.0] and float(v[3, 3]) == 384.0
    assert v[4, :2].tolist() == [0.0, 448.0] and torch.all(v[4, 2:] == 0)
