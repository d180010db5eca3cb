"""Packed attention over keys and values expanded from latent rows
(kvd_attend_expanded) against a plain 64-bit form."""
import math

import pytest
import torch

import latent_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
P = 64


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


class Packed:
    """Packed queries and keys with two spare rows behind the last sequence,
    whose keys and values are NaN."""

    def __init__(self, nq, nk, H, Dn, Dv, dtype, seed=0, causal=True):
        g = torch.Generator().manual_seed(seed)
        self.nq, self.nk, self.H, self.Dn, self.Dv = nq, nk, H, Dn, Dv
        self.dtype, self.causal = dtype, causal
        N, M = sum(nq) + 2, sum(nk) + 2
        self.q = torch.randn(N, H, Dn + P, generator=g).to(dtype).cuda()
        self.kv = torch.randn(M, H, Dn + Dv, generator=g).to(dtype).cuda()
        self.kr = torch.randn(M, P, generator=g).to(dtype).cuda()
        self.kv[-2:] = math.nan
        self.kr[-2:] = math.inf
        cum = lambda x: torch.tensor([0] + x).cumsum(0).to(torch.int32).cuda()  # noqa: E731
        self.ql, self.kl = cum(nq), cum(nk)
        self.scale = 1.0 / math.sqrt(Dn + P)

    def call(self, kvd):
        N = self.q.shape[0]
        out = torch.full((N, self.H, self.Dv), 7.0, dtype=self.dtype, device="cuda")
        lse = torch.full((N, self.H), 7.0, device="cuda")
        status = kvd.status_tensor()
        kvd.attend_expanded(self.q, self.kv, self.kr, self.ql, self.kl, self.scale, self.causal,
                            out=out, lse=lse, dev_status=status)
        return out, lse, int(status.item())

    def reference(self):
        N = sum(self.nq)
        out = torch.zeros((N, self.H, self.Dv), dtype=torch.float64, device="cuda")
        A, lse = torch.zeros_like(out), torch.zeros((N, self.H), dtype=torch.float64, device="cuda")
        d = torch.zeros_like(lse)
        q0 = k0 = 0
        for nq, nk in zip(self.nq, self.nk):
            i, j = torch.arange(nq, device="cuda"), torch.arange(nk, device="cuda")
            seen = j[None] <= (i + nk - nq)[:, None]
            if not self.causal:
                seen = torch.ones_like(seen)
            kr = self.kr[k0:k0 + nk].double()
            for h in range(self.H):
                kv = self.kv[k0:k0 + nk, h].double()
                o, z, a, e = ref.attention(self.q[q0:q0 + nq, h].double(),
                                           torch.cat([kv[:, :self.Dn], kr], 1), kv[:, self.Dn:],
                                           self.scale, seen)
                out[q0:q0 + nq, h], lse[q0:q0 + nq, h] = o, z
                A[q0:q0 + nq, h], d[q0:q0 + nq, h] = a, e
            q0, k0 = q0 + nq, k0 + nk
        return out, lse, A, d

    def same(self, kvd, what):
        out, lse, bits = self.call(kvd)
        assert bits == 0
        n = sum(self.nq)
        assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all()), "rows behind the last"
        o, z, A, d = self.reference()
        ref.check(what, out[:n], lse[:n], o, z, A, d, max(max(self.nk), 1), self.dtype)


# nq, nk, H, Dn, Dv
SHAPES = [
    ([1], [1], 1, 128, 128),
    ([3, 0, 1, 5], [3, 7, 0, 2], 2, 128, 128),
    ([127, 128, 129], [127, 128, 129], 3, 128, 128),
    ([255, 256, 257, 1], [255, 300, 600, 513], 2, 128, 128),
    ([130, 64], [70, 64], 2, 128, 64),
    ([65, 300], [65, 450], 2, 64, 64),
    ([31, 33, 200], [95, 33, 264], 4, 64, 128),
    ([700], [1411], 5, 128, 128),
]


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(s[0])}H{s[2]}D{s[3]}.{s[4]}")
def test_shapes(kvd, shape, dtype, causal):
    Packed(*shape, dtype, seed=len(shape[0]), causal=causal).same(kvd, "shape")


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("shape", SHAPES[2:], ids=lambda s: f"{len(s[0])}x{max(s[0])}D{s[3]}.{s[4]}")
def test_more_heads_than_fit_at_once(kvd, shape, causal):
    """The same lengths with 152 heads: more CTAs than SMs."""
    nq, nk, _, Dn, Dv = shape
    Packed(nq, nk, 152, Dn, Dv, BF, seed=7, causal=causal).same(kvd, "heads")


def test_many_sequences(kvd):
    nq = [(i * 29) % 70 for i in range(300)]
    Packed(nq, [n + (n * 13) % 40 for n in nq], 2, 128, 128, BF, seed=3).same(kvd, "many")


def test_growing_scores(kvd):
    """The running maximum rises with every tile by far more than 2^8."""
    c = Packed([400, 90], [520, 90], 2, 128, 128, BF, seed=4)
    ramp = torch.linspace(0, 10, c.kv.shape[0], device="cuda")
    c.kv[:-2, :, :128] = (c.q[0, :, :128].float()[None] * ramp[:-2, None, None]).to(BF)
    c.same(kvd, "growing")


def test_neighbours_do_not_leak(kvd):
    """Keys of other sequences may be NaN without reaching this one."""
    c = Packed([100, 50, 30], [100, 50, 30], 2, 128, 128, BF, seed=5)
    clean, cl, _ = c.call(kvd)
    c.kv[100:150] = math.nan
    c.kr[100:150] = math.nan
    out, lse, _ = c.call(kvd)
    keep = torch.ones(out.shape[0], dtype=torch.bool, device="cuda")
    keep[100:150] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], cl[keep])
    assert bool(torch.isnan(out[100:150]).all())


def test_bad_lengths(kvd):
    c = Packed([40, 50, 30], [40, 50, 30], 2, 128, 128, BF, seed=6)
    good, gl, _ = c.call(kvd)
    c.kl[3] = c.kv.shape[0] + 1              # past the keys: sequence 2 has none
    out, lse, bits = c.call(kvd)
    assert bits == kvd.DEV_SEQLENS
    assert torch.equal(out[:90], good[:90])
    assert bool((out[90:120] == 0).all()) and bool(torch.isneginf(lse[90:120]).all())
    c.kl[3] = 120
    c.ql[3] = c.q.shape[0] + 9               # past the queries: sequence 2 is not computed
    out, lse, bits = c.call(kvd)
    assert bits == kvd.DEV_SEQLENS
    assert torch.equal(out[:90], good[:90]) and bool((out[90:] == 7).all())


def test_graph_and_repeat(kvd):
    c = Packed([300, 200], [300, 260], 4, 128, 128, BF, seed=7)
    want, wl, _ = c.call(kvd)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    kvd.attend_expanded(c.q, c.kv, c.kr, c.ql, c.kl, c.scale, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvd.attend_expanded(c.q, c.kv, c.kr, c.ql, c.kl, c.scale, out=out, lse=lse)
    out.fill_(7.0)
    lse.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
