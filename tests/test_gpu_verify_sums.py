"""Sums of kvd_verify_drafts that fp32 alone cannot hold: long rows whose small
weights do not add up exactly, and weights whose sum is above the largest fp32."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from test_gpu_verify import expect

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


def pieces(x):
    """fp32 numbers that sum to x (a multiple of 2^-100) exactly."""
    out = []
    while x > 0:
        f = np.float32(float(x))
        if Fraction(float(f)) > x:
            f = np.nextafter(f, np.float32(0))
        out.append(float(f))
        x -= Fraction(float(f))
    return out


@pytest.mark.parametrize("V", [1 << 17, 1 << 20, 1 << 22], ids=["2^17", "2^20", "2^22"])
def test_long_rows(kvd, V):
    """Half of a row is ones with many weights of 2^-25 / 3 behind them, which a
    running sum near one takes as rounding errors only; the other half sums to a
    share of 2^-40 more (row 0) or less (row 1) exactly.  With u = 1/2 the wanted
    sum is the first half's by 2^-41 of it: the token is the first of the second
    half, or the last of the first.  A sum that is right to 2^-43 decides it."""
    half, t = V // 2, np.float32(2.0 ** -25 / 3)
    first = np.full(half, t, np.float32)
    first.reshape(-1, V // 128)[:, :128] = 1.0   # one per lane and warp where a CTA has 16 warps of V / 128
    ones = int((first == 1).sum())
    total = Fraction(ones) + Fraction(float(t)) * (half - ones)
    rows = []
    for sign in (1, -1):
        want = total * (1 + sign * Fraction(1, 1 << 40))
        want = Fraction(round(want * (1 << 100)), 1 << 100)
        second = np.zeros(half, np.float32)
        second[:ones] = 1.0
        rest = pieces(want - ones)
        second[ones:ones + len(rest)] = rest
        assert sum(map(Fraction, second[ones:].tolist())) + ones == want
        rows.append(np.concatenate([first, second]))
    # the border's neighbours are heavier than what decides
    assert total / (1 << 41) < Fraction(float(t)) and total / (1 << 41) < 1
    p = torch.from_numpy(np.stack(rows)).cuda()[:, None]
    tokens, _ = kvd.verify_drafts(p, None, None, None, torch.full((2,), 0.5, device="cuda"))
    assert tokens[:, 0].tolist() == [half, half - 1]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 1000, 50257, 200000])
def test_sums_above_the_largest_fp32(kvd, V, dtype):
    """Weights need not be normalised: finite ones count whatever their sum.  A
    difference p - q may be above the largest fp32 by itself."""
    g = torch.Generator(device="cuda").manual_seed(V)
    p = torch.rand((6, 2, V), generator=g, device="cuda") * 3e38
    p = torch.where(torch.rand((6, 2, V), generator=g, device="cuda") < 0.3, 0.0, p).to(dtype)
    q = (torch.rand((6, 1, V), generator=g, device="cuda") * 3e38).to(dtype)
    q[3:] = -q[3:]
    x = torch.zeros((6, 1), dtype=torch.int32, device="cuda")
    p[:, 0, 0], q[:, 0, 0] = 0.0, 1.0             # the draft is always rejected
    u = torch.full((6, 1), 0.5, device="cuda")
    us = torch.tensor([0.0, 0.37, 0.999], device="cuda").repeat(2)
    status = kvd.status_tensor()
    tokens, acc = kvd.verify_drafts(p, q, x, u, us, dev_status=status)
    want, n = expect(p, q, x, u, us, [1] * 6)
    assert int(status.item()) == 0
    assert torch.equal(tokens.cpu(), want) and torch.equal(acc.cpu(), n)
    rows = p[:, :1].contiguous()
    tokens, _ = kvd.verify_drafts(rows, None, None, None, us, dev_status=status)
    want, _ = expect(rows, None, torch.zeros((6, 0), dtype=torch.int32), None, us, [0] * 6)
    assert int(status.item()) == 0 and torch.equal(tokens.cpu(), want)


def test_infinite_weights_are_refused(kvd):
    """One infinite weight among finite ones whose sum is above the largest fp32."""
    p = torch.full((3, 1, 5000), 1e36, device="cuda")
    p[1, 0, 4321] = float("inf")
    status = kvd.status_tensor()
    tokens, _ = kvd.verify_drafts(p, None, None, None, torch.full((3,), 0.5, device="cuda"),
                                  dev_status=status)
    assert int(status.item()) == kvd.DEV_PROBS
    assert tokens[:, 0].tolist() == [2500, -1, 2500]
