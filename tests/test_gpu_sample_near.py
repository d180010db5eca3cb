"""kvd_sample and kvd_filter_probs: logits that hardly differ, beside others that do not
count."""
import math

import pytest
import torch

from test_gpu_sample import same

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [64, 4096, 4097, 50257, 128000])
@pytest.mark.parametrize("hidden", [math.nan, -math.inf])
def test_near_logits_beside_hidden_ones(kvd, V, hidden, dtype):
    """Logits within 1 of each other and many that do not count (NaN, -inf): these add nothing to
    the sum that top-p takes its share of, whatever min-p keeps."""
    R = 12
    g = torch.Generator().manual_seed(V)
    logits = -torch.rand(R, V, generator=g)
    logits[torch.rand(R, V, generator=g) < torch.tensor([0.3, 0.7, 0.9]).repeat(4)[:, None]] = hidden
    logits[:, V // 2] = 0.0
    logits = logits.to(dtype).cuda()
    u = torch.rand(R, generator=g).cuda()
    T = torch.tensor([1.0] * 6 + [0.5] * 3 + [20.0] * 3).cuda()
    p = torch.tensor([0.5, 0.5, 0.5, 0.6, 0.6, 0.6] * 2).cuda()
    m = torch.tensor([0.5, 0.5, 0.5, 0.7, 0.7, 0.7] + [0.3] * 3 + [0.97] * 3).cuda()
    same(kvd, logits, u, T=T, p=p, m=m)
    same(kvd, logits, u, T=T, p=p)
    same(kvd, logits, u, T=T, m=m)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [50256, 50257, 50260])
def test_flat_rows(kvd, V, dtype):
    """Logits that hardly differ, in rows that start at and beside whole vectors, with and without
    one at -inf or most of them: the bins follow the finite ones."""
    R = 8
    g = torch.Generator().manual_seed(V)
    logits = (torch.rand(R, V, generator=g) * 0.05).to(dtype)
    logits[R // 2:, 1234] = -math.inf
    logits[:2, 5000:] = -math.inf
    logits = logits.cuda()
    u = torch.rand(R, generator=g).cuda()
    p = torch.tensor([0.3, 0.9, 0.5, 0.99] * 2, device="cuda")
    same(kvd, logits, u, p=p)
    same(kvd, logits, u, T=p, p=p, m=torch.full((R,), 0.97, device="cuda"))
