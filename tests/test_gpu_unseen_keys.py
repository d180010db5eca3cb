"""Keys that a query does not see take no part in its result, whatever they
hold: the call is repeated with keys of a sequence made NaN or infinite (the
values stay finite).  Queries that come before such a key have to give the same
bits as before, the others have to show it."""
import math

import pytest
import torch

import latent_ref as ref
from test_gpu_expanded import Packed

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


def attend(kvd, c):
    lse = torch.empty(c.ql.shape[:3], device="cuda")
    out = kvd.attend_latent(c.ql, c.qr, c.latent, c.rope, c.table, c.seq_lens, c.scale,
                            seq_offset=c.seq_offset, lse=lse)
    return out, lse


# T, H, R, BS: tokens of one tile's end, rows of two groups, rows of many tiles, pages
# inside a tile and odd ones
@pytest.mark.parametrize("T, H, R, BS", [(4, 16, 512, 64), (3, 40, 128, 16), (150, 1, 256, 128),
                                         (5, 2, 384, 7)], ids=str)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_latent(kvd, T, H, R, BS, dtype):
    lens = [300, 65, 192, 2, 1000]
    c = ref.LatentCase(lens, T, H, R, BS, dtype, seed=T)
    clean, cl = attend(kvd, c)
    bad = [max(0, n - back) for n, back in zip(lens, (2, 1, T, 1, T // 2))]
    for b, j in enumerate(bad):
        c.rope[int(c.table[b, j // BS]), j % BS, 0, 5] = NAN
    out, lse = attend(kvd, c)
    n = torch.tensor(lens, device="cuda")
    last = n[:, None] - T + torch.arange(T, device="cuda")
    sees = (last >= torch.tensor(bad, device="cuda")[:, None])[:, :, None].expand(-1, -1, H)
    assert bool(sees.any()) and not bool(sees.all())
    assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse[~sees], cl[~sees])
    assert bool(torch.isnan(out[sees]).all()) and bool(torch.isnan(lse[sees]).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shared", [True, False], ids=["rotary", "own"])
def test_expanded_keys(kvd, dtype, shared):
    c = Packed([300, 40], [437, 20], 3, 128, 128, dtype, seed=2)
    clean, cl, _ = c.call(kvd)
    if shared:
        c.kr[255, 9] = NAN
        c.kr[437 + 15, 9] = INF
    else:
        c.kv[255, :, 9] = NAN
        c.kv[437 + 15, :, 9] = -INF
    out, lse, _ = c.call(kvd)
    i = torch.arange(out.shape[0], device="cuda")
    hit = ((i < 300) & (i + 137 >= 255)) | ((i >= 300) & (i < 340) & (i - 300 - 20 >= 15))
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], cl[~hit])
    sees_nan = hit & (i < 300)
    assert bool(torch.isnan(out[sees_nan]).all()) and bool(torch.isnan(lse[sees_nan]).all())
