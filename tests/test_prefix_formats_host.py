"""The number formats of the shared-prefix decode, emulated with torch's types: what its
comments state, and what the GPU tests' tolerances may count on.

A probability is an e4m3 term and an e5m2 residual.  A query row, scaled by a power of
two to a maximum in [128, 256), is e4m3 + 2^-5 e4m3, and 2^-5 e5m2 more in rows that
want a third term.
"""
import pytest
import torch


def e4m3(x):
    return x.float().clamp(-448, 448).to(torch.float8_e4m3fn).double()


def e5m2(x):
    return x.float().to(torch.float8_e5m2).double()


def query_terms(x):
    hi = e4m3(x)
    mid = e4m3((x - hi) * 32)
    return hi + mid / 32, hi + (mid + e5m2((x - hi) * 32 - mid)) / 32


@pytest.mark.parametrize("k,worst,rms", [(0, 4.25e-3, 1.35e-3), (6, 4.25e-3, 1.35e-3),
                                         (12, 4.25e-3, 1.35e-3), (13, 7.8e-3, 2.5e-3),
                                         (14, 1.5e-2, 5e-3), (17, 0.115, 0.055)])
def test_probability_pair(k, worst, rms):
    # weights 2^-k to 2^(1-k) of the row's reference; a weight 1 is fed as 2^6, through fp16
    p = (1 + torch.arange(4096, dtype=torch.float64) / 4096) * 2.0 ** (6 - k)
    p16 = p.to(torch.float16).double()
    hi = e4m3(p16)
    off = ((hi + e5m2(p16 - hi)) / p - 1).abs()
    assert float(off.max()) <= worst
    assert float(off.square().mean().sqrt()) <= rms


def scaled_bf16(e):
    """Every bf16 number of [2^e, 2^(e+1)), the values of a row scaled to below 2^8."""
    return (1 + torch.arange(128, dtype=torch.float64) / 128) * 2.0 ** e


@pytest.mark.parametrize("e", range(-30, 8))
def test_query_terms(e):
    x = scaled_bf16(e)
    two, three = query_terms(x)
    assert torch.equal(two, x) or e < -7                     # within 2^-14 of the maximum
    assert torch.equal(three, x) or e < -11                  # within 2^-18
    assert float((two - x).abs().max()) <= 2.0 ** -15        # 2^-22 of a maximum of 2^7
    assert float((three - x).abs().max()) <= 2.0 ** -19      # 2^-26
