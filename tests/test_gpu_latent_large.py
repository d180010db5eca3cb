"""The latent-cache calls on tensors of more than 2^32 bytes (2^31 elements): the
last rows are addressed right.  Only what is used is filled."""
import math

import pytest
import torch

import latent_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_append_and_attend(kvd, dtype):
    R, P, BS, H = 512, 64, 128, 4
    NB = 2 ** 31 // (R * BS) + 40                # the latent cache: above 2^31 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    latent = torch.empty(NB, BS, 1, R, dtype=dtype, device="cuda")
    rope = torch.empty(NB, BS, 1, P, dtype=dtype, device="cuda")
    n = [300, 77]
    table = torch.tensor([[NB - 1, 0, NB - 2], [NB - 3, 1, 2]], dtype=torch.int32, device="cuda")
    c = torch.randn(sum(n), R, generator=g, device="cuda").to(dtype)
    r = torch.randn(sum(n), P, generator=g, device="cuda").to(dtype)
    lens = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    status = kvd.status_tensor()
    kvd.append_latent(latent, rope, table, None, c, r, lens, zero, status)
    assert torch.equal(latent[NB - 1, :, 0], c[:BS]) and torch.equal(rope[NB - 3, :77, 0], r[300:])
    ql = torch.randn(2, 1, H, R, generator=g, device="cuda").to(dtype)
    qr = torch.randn(2, 1, H, P, generator=g, device="cuda").to(dtype)
    lse = torch.empty(2, 1, H, device="cuda")
    scale = 1 / math.sqrt(R + P)
    out = kvd.attend_latent(ql, qr, latent, rope, table, lens, scale, lse=lse, dev_status=status)
    for b, rows in ((0, slice(0, 300)), (1, slice(300, 377))):
        k = torch.cat([c[rows], r[rows]], 1).double()
        q = torch.cat([ql[b, 0], qr[b, 0]], 1).double()
        o, z, A, d = ref.attention(q, k, c[rows].double(), scale,
                                   torch.ones(H, n[b], dtype=torch.bool, device="cuda"))
        ref.check("large", out[b, 0], lse[b, 0], o, z, A, d, n[b], dtype)
    assert int(status.item()) == 0


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_expanded(kvd, dtype):
    H, Dn, Dv, P = 128, 128, 128, 64
    Nk = 2 ** 31 // (H * (Dn + Dv)) + 500        # kv: above 2^31 elements
    g = torch.Generator(device="cuda").manual_seed(2)
    kv = torch.empty(Nk, H, Dn + Dv, dtype=dtype, device="cuda")
    kr = torch.empty(Nk, P, dtype=dtype, device="cuda")
    last = 200
    kv[-last:] = torch.randn(last, H, Dn + Dv, generator=g, device="cuda").to(dtype)
    kr[-last:] = torch.randn(last, P, generator=g, device="cuda").to(dtype)
    q = torch.randn(3, H, Dn + P, generator=g, device="cuda").to(dtype)
    ql = torch.tensor([0, 0, 3], dtype=torch.int32, device="cuda")
    kl = torch.tensor([0, Nk - last, Nk], dtype=torch.int32, device="cuda")
    lse = torch.empty(3, H, device="cuda")
    out = kvd.attend_expanded(q, kv, kr, ql, kl, lse=lse)
    seen = torch.arange(last, device="cuda")[None] <= (last - 3 + torch.arange(3, device="cuda"))[:, None]
    for h in (0, 77, 127):
        rows = kv[-last:, h].double()
        o, z, A, d = ref.attention(q[:, h].double(), torch.cat([rows[:, :Dn], kr[-last:].double()], 1),
                                   rows[:, Dn:], 1 / math.sqrt(Dn + P), seen)
        ref.check("large", out[:, h], lse[:, h], o, z, A, d, last, dtype)


def test_verify(kvd):
    V = 2 ** 20 + 3
    Q = 2 ** 31 // (2 * V) + 8                   # target: above 2^31 elements
    g = torch.Generator(device="cuda").manual_seed(3)
    p = torch.zeros(Q, 2, V, dtype=BF, device="cuda")
    q = torch.zeros(Q, 1, V, dtype=BF, device="cuda")
    token = torch.randint(0, V, (Q,), generator=g, device="cuda")
    other = (token + 1 + torch.randint(0, V - 1, (Q,), generator=g, device="cuda")) % V
    b = torch.arange(Q, device="cuda")
    p[b, 0, token] = 1.0                          # the replacement of a rejected draft
    p[b, 1, other] = 1.0                          # the token behind an accepted one
    q[b, 0, other] = 1.0
    x = other.to(torch.int32)[:, None].clone()
    x[1::2] = token[1::2, None].to(torch.int32)   # drafted right every other time
    q[b[1::2], 0, token[1::2]] = 0.5
    tokens, accepted = kvd.verify_drafts(p, q, x.contiguous(), torch.full((Q, 1), 0.25, device="cuda"),
                                         torch.rand(Q, generator=g, device="cuda"))
    assert accepted.tolist() == [i % 2 for i in range(Q)]
    assert torch.equal(tokens[0::2, 0].long(), token[0::2])
    assert torch.equal(tokens[1::2, 0].long(), token[1::2])
    assert torch.equal(tokens[1::2, 1].long(), other[1::2])


def test_no_keys_at_all(kvd):
    """Nk = 0: every row is empty; an empty batch returns."""
    for dtype in (BF, F32):
        q = torch.randn(5, 2, 192, device="cuda").to(dtype)
        kv, kr = torch.empty(0, 2, 256, dtype=dtype, device="cuda"), torch.empty(0, 64, dtype=dtype, device="cuda")
        lens, none = torch.tensor([0, 5], dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
        lse = torch.zeros(5, 2, device="cuda")
        out = kvd.attend_expanded(q, kv, kr, lens, none, lse=lse)
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
        assert kvd.attend_expanded(q[:0], kv, kr, none, none).shape == (0, 2, 128)
