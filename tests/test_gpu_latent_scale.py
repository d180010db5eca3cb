"""Scales of the latent calls that are not ordinary positive numbers."""
import math

import pytest
import torch

import latent_ref as ref
from test_gpu_expanded import Packed

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


def attend(kvd, c, scale):
    lse = torch.empty(c.ql.shape[:3], device="cuda")
    out = kvd.attend_latent(c.ql, c.qr, c.latent, c.rope, c.table, c.seq_lens, scale,
                            seq_offset=c.seq_offset, lse=lse)
    return out, lse


def same(out, lse, nan, none):
    """NaN in the rows of `nan`, zeros and -inf in those of `none`; together all rows."""
    assert bool((nan ^ none).all())
    assert bool(torch.isnan(out[nan]).all()) and bool(torch.isnan(lse[nan]).all())
    assert bool((out[none] == 0).all()) and bool(torch.isneginf(lse[none]).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [40, 0, 2, 65], [3000, 7]], ids=["one", "short", "shared"])
def test_nan_reaches_every_query_that_sees_a_key(kvd, lens, dtype):
    """Whole sequences and ones that several workers share; queries of tokens
    that come before the sequence's first see nothing and stay zero."""
    T, H = 3, 5
    c = ref.LatentCase(lens, T, H, 128, 16, dtype, seed=len(lens))
    out, lse = attend(kvd, c, math.nan)
    n = torch.tensor(lens, device="cuda")
    sees = (n[:, None] - T + torch.arange(T, device="cuda") >= 0)[:, :, None].expand(-1, -1, H)
    same(out, lse, sees, ~sees)


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_nan_in_the_expanded_form(kvd, dtype, causal):
    """Sequences with more queries than keys, with none and with several key tiles."""
    nq, nk = [5, 3, 200, 1], [2, 0, 300, 1]
    c = Packed(nq, nk, 2, 128, 64, dtype, seed=1, causal=causal)
    c.scale = math.nan
    out, lse, bits = c.call(kvd)
    assert bits == 0
    sees = torch.cat([torch.arange(a, device="cuda") + b - a >= 0 if causal
                      else torch.full((a,), b > 0, device="cuda") for a, b in zip(nq, nk)])
    sees = sees[:, None].expand(-1, 2)
    same(out[:sum(nq)], lse[:sum(nq)], sees, ~sees)


# Products of 1e34 and more: a scale of zero still gives the mean of what a
# query sees, and one of 1e-34 ordinary scores.  The kernels' bounds hold as
# they are, with one addition at scale zero: the bf16 kernels take the
# smallest number of fp32 (2^-149) in its place, so that a score of up to 2^127
# is off by 2^-22, a weight by a factor of 1 + 2^-21, an lse by 2^-22.
HUGE = 2.0 ** 56


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-34, -1e-34], ids=["0", "-0", "+", "-"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_small_scales(kvd, dtype, scale):
    c = ref.LatentCase([300, 64, 1], 2, 4, 128, 16, dtype, seed=5)
    c.ql, c.qr = c.ql * HUGE, c.qr * HUGE
    c.latent, c.rope = c.latent * HUGE, c.rope * HUGE
    c.rows = [(x * HUGE, y * HUGE) for x, y in c.rows]
    c.scale = scale
    out, lse = attend(kvd, c, scale)
    o, z, A, d = c.reference()
    ref.check("latent", out, lse, o, z, A, d + (2.0 ** -22 if scale == 0 else 0), 300, dtype)


@pytest.mark.parametrize("scale", [0.0, 1e-34, -1e-34], ids=["0", "+", "-"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_small_scales_in_the_expanded_form(kvd, dtype, scale):
    c = Packed([130, 7], [200, 9], 2, 128, 64, dtype, seed=6)
    c.q, c.kv, c.kr = c.q * HUGE, c.kv * HUGE, c.kr * HUGE
    c.scale = scale
    out, lse, bits = c.call(kvd)
    assert bits == 0
    o, z, A, d = c.reference()
    ref.check("expanded", out[:137], lse[:137], o, z, A, d + (2.0 ** -22 if scale == 0 else 0), 200,
              dtype)
