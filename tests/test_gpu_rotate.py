"""kvd_rotate and kvd_rotate_append_paged against the formulas in 64 bits."""
import math

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


def normal(g, *shape, s=1.0):
    return torch.randn(shape, generator=g) * s


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("D,Dr", [(64, 0), (64, 16), (64, 48), (64, 64), (128, 32), (128, 96),
                                  (128, 128)])
@pytest.mark.parametrize("N,H,norm", [(1, 1, True), (5, 3, False), (37, 40, True)])
def test_rotate(kvd, N, H, norm, D, Dr, inter, dtype):
    g = torch.Generator().manual_seed(N * D + Dr)
    x = normal(g, N, H, D, s=2.0).to(dtype).cuda()
    w = (1 + normal(g, D, s=0.2)).to(dtype).cuda() if norm else None
    pos = torch.randint(0, 200000, (N,), generator=g).to(torch.int32).cuda()
    freqs = (10000.0 ** (-2 * torch.arange(Dr // 2, dtype=torch.float64) / max(Dr, 1))).cuda()
    want, size = ref.rotate(x.double(), w, pos, freqs, inter, 1.25, 1e-5)
    keep = x.clone()
    got = kvd.rotate(x, pos, freqs, weight=w, eps=1e-5, interleaved=inter, rotary_scale=1.25)
    ref.check_rotated("rotate", got, want, size, D, dtype)
    assert torch.equal(x, keep)
    assert kvd.rotate(x, pos, freqs, weight=w, eps=1e-5, interleaved=inter, rotary_scale=1.25,
                      out=x) is x
    assert torch.equal(x, got)  # in place


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,Hq,Hkv,D,Dr,BS", [(1, 1, 1, 64, 64, 1), (3, 7, 1, 128, 64, 7),
                                              (64, 32, 8, 128, 128, 16), (129, 6, 2, 64, 32, 24),
                                              (5, 96, 16, 128, 128, 128)])
@pytest.mark.parametrize("norm", [0, 1, 2])
def test_append(kvd, N, Hq, Hkv, D, Dr, BS, norm, dtype):
    """Queries out, keys and values in their rows, every other row as it was."""
    g = torch.Generator().manual_seed(N + Hq)
    NB = -(-N // BS) + 4
    x = normal(g, N, Hq + 2 * Hkv, D).to(dtype).cuda()
    kc, vc = normal(g, NB, BS, Hkv, D).to(dtype).cuda(), normal(g, NB, BS, Hkv, D).to(dtype).cuda()
    qw = (1 + normal(g, D, s=0.2)).to(dtype).cuda() if norm else None
    kw = (1 + normal(g, D, s=0.2)).to(dtype).cuda() if norm == 2 else None
    slots = torch.randperm(NB * BS, generator=g)[:N].to(torch.int32).cuda()
    pos = torch.randint(0, 5000, (N,), generator=g).to(torch.int32).cuda()
    freqs = kvd.rotary_freqs(Dr, base=500000.0, scaling="parts", factor=4.0)
    q0, s0 = ref.rotate(x[:, :Hq].double(), qw, pos, freqs, False, 1.0, 1e-6)
    k0, s1 = ref.rotate(x[:, Hq:Hq + Hkv].double(), kw, pos, freqs, False, 1.0, 1e-6)
    wk, wv = kc.clone(), vc.clone()
    status = kvd.status_tensor()
    q = kvd.rotate_append_paged(x, kc, vc, slots, pos, freqs, q_weight=qw, k_weight=kw,
                                dev_status=status)
    assert int(status.item()) == 0
    rows = slots.long()
    ref.check_rotated("queries", q, q0, s0, D, dtype)
    ref.check_rotated("keys", kc.view(-1, Hkv, D)[rows], k0, s1, D, dtype)
    wk.view(-1, Hkv, D)[rows] = kc.view(-1, Hkv, D)[rows]
    wv.view(-1, Hkv, D)[rows] = x[:, Hq + Hkv:]
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    # the queries are those of kvd_rotate, bit for bit
    assert torch.equal(q, kvd.rotate(x[:, :Hq].contiguous(), pos, freqs, weight=qw))


def test_far_positions(kvd):
    """Positions up to 2^31 - 1 at a frequency of a radian a token: an angle in fp32
    would be off by a hundred radians.  64-bit reference: p f is off by 2^-53 of 2^31."""
    pos = torch.tensor([0, 1, 10 ** 6, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1],
                       dtype=torch.int32, device="cuda")
    x = torch.zeros(6, 1, 64, device="cuda")
    x[..., :8] = 1.0
    freqs = torch.tensor([1.0, 0.5, 0.25, 1e-3, 3.0, 7.5, -1.0, 0.0], dtype=torch.float64,
                         device="cuda")
    want, size = ref.rotate(x.double(), None, pos, freqs, False, 1.0, 0.0)
    ref.check_rotated("far", kvd.rotate(x, pos, freqs), want, size + 1, 64, F32)


def test_tokens_without_a_place(kvd):
    N, Hq, Hkv, D = 6, 2, 1, 64
    x = torch.randn(N, Hq + 2 * Hkv, D, device="cuda")
    pos = torch.tensor([-1, 3, 4, -7, 5, 6], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, -1, 0, 1, 8, -2], dtype=torch.int32, device="cuda")
    freqs = kvd.rotary_freqs(64)
    kc, vc = torch.full((2, 4, Hkv, D), 9.0, device="cuda"), torch.full((2, 4, Hkv, D), 9.0, device="cuda")
    out = torch.full((N, Hq, D), 5.0, device="cuda")
    status = kvd.status_tensor()
    kvd.rotate_append_paged(x, kc, vc, slots, pos, freqs, out=out, dev_status=status)
    assert int(status.item()) == kvd.DEV_POS_RANGE | kvd.DEV_BLOCK_RANGE
    assert bool((out[[0, 3]] == 5).all())
    want, size = ref.rotate(x[:, :Hq].double(), None, pos.clamp(min=0), freqs, False, 1.0, 0)
    live = [1, 2, 4, 5]
    ref.check_rotated("queries", out[live], want[live], size[live], D, F32)
    flat = vc.view(-1, Hkv, D)
    assert torch.equal(flat[0], x[2, Hq + Hkv:]) and bool((flat[1:] == 9).all())
    assert bool((kc.view(-1, Hkv, D)[1:] == 9).all())
    out = torch.full((N, Hq, D), 5.0, device="cuda")
    status.zero_()
    kvd.rotate(x[:, :Hq].contiguous(), pos, freqs, out=out, dev_status=status)
    assert int(status.item()) == kvd.DEV_POS_RANGE and bool((out[[0, 3]] == 5).all())
    assert kvd.rotate(x[:0, :Hq].contiguous(), pos[:0], freqs).shape == (0, Hq, D)


def test_values_are_copied_as_they_are(kvd):
    """NaN and infinities: values bit for bit, other heads and tokens not touched."""
    x = torch.randn(4, 4, 64, dtype=BF, device="cuda")
    clean = x.clone()
    x[1, 3] = math.nan
    x[2, 3, 5] = math.inf
    x[1, 0] = math.inf
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    freqs = kvd.rotary_freqs(64)
    w = torch.ones(64, dtype=BF, device="cuda")

    def go(x):
        kc, vc = torch.zeros(1, 4, 1, 64, dtype=BF, device="cuda"), torch.zeros(1, 4, 1, 64, dtype=BF, device="cuda")
        return kvd.rotate_append_paged(x, kc, vc, pos, pos, freqs, q_weight=w, k_weight=w), kc, vc
    q, k, v = go(x)
    q0, k0, v0 = go(clean)
    assert torch.equal(v.view(torch.int16)[0, :, 0], x[:, 3].view(torch.int16))
    assert torch.equal(k, k0)
    assert torch.equal(q[:, 1], q0[:, 1]) and torch.equal(q[[0, 2, 3]], q0[[0, 2, 3]])


def test_refusals(kvd):
    x = torch.randn(4, 4, 64, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    kc, vc = torch.zeros(1, 4, 1, 64, device="cuda"), torch.zeros(1, 4, 1, 64, device="cuda")
    f = kvd.rotary_freqs(64)
    with pytest.raises(TypeError):
        kvd.rotate(x.half(), pos, f)
    with pytest.raises(TypeError):
        kvd.rotate(x, pos.long(), f)
    with pytest.raises(TypeError):
        kvd.rotate(x, pos, f.float())
    with pytest.raises(ValueError):
        kvd.rotate(x.transpose(0, 1), pos, f)
    with pytest.raises(ValueError):
        kvd.rotate(x, pos[:3], f)
    with pytest.raises(ValueError):
        kvd.rotate(x, pos, f.cpu())
    with pytest.raises(TypeError):
        kvd.rotate(x, pos, f, weight=torch.ones(64, dtype=BF, device="cuda"))
    with pytest.raises(kvd.KvdError):
        kvd.rotate(x, pos, kvd.rotary_freqs(72))     # more than the head
    with pytest.raises(kvd.KvdError):
        kvd.rotate(x, pos, kvd.rotary_freqs(24))
    with pytest.raises(ValueError):
        kvd.rotate_append_paged(x[:, :2].contiguous(), kc, vc, pos, pos, f)  # no query head
    with pytest.raises(TypeError):
        kvd.rotate_append_paged(x, kc.to(BF), vc, pos, pos, f)
    with pytest.raises(ValueError):
        kvd.rotate_append_paged(x, kc, vc[:, :2].contiguous(), pos, pos, f)
    with pytest.raises(ValueError):
        kvd.rotate_append_paged(x, kc, vc, pos[:2], pos, f)
