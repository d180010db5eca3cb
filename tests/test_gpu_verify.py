"""Verification of drafted tokens (kvd_verify_drafts) against a sequential
64-bit form: the tokens have to be equal."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


def plain(p, q, x, u, us, m):
    """One sequence in Python floats: p [T+1, V], q [T, V] float64 on the CPU."""
    n = 0
    while n < m and u[n] * float(q[n, x[n]]) < float(p[n, x[n]]):
        n += 1
    w = p[n].clamp(min=0)
    if n < m:
        rest = (p[n] - q[n]).clamp(min=0)
        if float(rest.sum()) > 0:
            w = rest
    cum = torch.cumsum(w, 0)
    above = torch.nonzero(cum > us * float(cum[-1]))
    token = int(above[0]) if len(above) else int(torch.nonzero(w).max())
    return n, token


def expect(p, q, x, u, us, m):
    Q, T1, V = p.shape
    tokens, accepted = torch.full((Q, T1), -1, dtype=torch.int32), torch.zeros(Q, dtype=torch.int32)
    P, D = p.double().cpu(), None if q is None else q.double().cpu()
    for b in range(Q):
        n, token = plain(P[b], None if D is None else D[b], x[b].tolist() if T1 > 1 else [],
                         u[b].tolist() if T1 > 1 else [], float(us[b]), int(m[b]))
        tokens[b, :n] = x[b, :n].cpu() if n else tokens[b, :n]
        tokens[b, n] = token
        accepted[b] = n
    return tokens, accepted


def draws(Q, T, V, dtype, seed, near=0.4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lo = torch.randn((Q, T + 1, V), generator=g, device="cuda") * 2
    p = torch.softmax(lo, -1).to(dtype)
    qs = torch.softmax(lo[:, :T] + near * torch.randn((Q, T, V), generator=g, device="cuda"), -1)
    x = torch.multinomial(qs.reshape(-1, V), 1, generator=g).view(Q, T).to(torch.int32)
    u = torch.rand((Q, T), generator=g, device="cuda")
    us = torch.rand((Q,), generator=g, device="cuda")
    return p, qs.to(dtype), x, u, us


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("QTV", [(1, 1, 1), (3, 1, 2), (5, 3, 31), (40, 4, 257), (33, 7, 4099),
                                 (7, 40, 1000), (9, 2, 50257), (4, 5, 200003)],
                         ids=lambda s: "x".join(map(str, s)))
def test_random(kvd, QTV, dtype):
    Q, T, V = QTV
    p, q, x, u, us = draws(Q, T, V, dtype, seed=V + T)
    status = kvd.status_tensor()
    tokens, accepted = kvd.verify_drafts(p, q, x, u, us, dev_status=status)
    want, n = expect(p, q, x, u, us, [T] * Q)
    assert int(status.item()) == 0
    assert torch.equal(accepted.cpu(), n) and torch.equal(tokens.cpu(), want)


def test_all_counts_are_met(kvd):
    """Every number of accepted drafts from none to all occurs and is right, with
    fewer drafts than T for some sequences."""
    Q, T, V = 200, 5, 97
    p, q, x, u, us = draws(Q, T, V, F32, seed=1, near=1.0)
    m = torch.arange(Q, device="cuda", dtype=torch.int32) % (T + 1)
    tokens, accepted = kvd.verify_drafts(p, q, x, u, us, num_drafts=m)
    want, n = expect(p, q, x, u, us, m.tolist())
    assert set(n.tolist()) == set(range(T + 1))
    assert torch.equal(accepted.cpu(), n) and torch.equal(tokens.cpu(), want)


def test_no_drafts(kvd):
    p, _, _, _, us = draws(6, 0, 3001, F32, seed=2)
    tokens, accepted = kvd.verify_drafts(p, None, None, None, us)
    want, n = expect(p, None, torch.zeros(6, 0, dtype=torch.int32), None, us, [0] * 6)
    assert torch.equal(tokens.cpu(), want) and torch.equal(accepted.cpu(), n)


def test_borders(kvd):
    """Dyadic probabilities, so that every sum is exact: a sum equal to the wanted
    one does not end the search, zeros are never drawn, u = 0 gives the first
    token with weight."""
    V = 64
    p = torch.zeros(5, 1, V, device="cuda")
    p[:, 0, 10], p[:, 0, 20], p[:, 0, 63] = 0.25, 0.25, 0.5
    us = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -24], device="cuda")
    tokens, _ = kvd.verify_drafts(p, None, None, None, us)
    assert tokens[:, 0].tolist() == [10, 20, 63, 63, 63]
    # u * q(x) = p(x) rejects, a hair less accepts
    q = torch.full((2, 1, 2), 0.5, device="cuda")
    p = torch.tensor([[[0.25, 0.75], [1, 0]]] * 2, device="cuda").contiguous()
    x = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    u = torch.tensor([[0.5], [0.5 - 2.0 ** -25]], device="cuda")
    tokens, acc = kvd.verify_drafts(p, q, x, u, torch.zeros(2, device="cuda"))
    assert acc.tolist() == [0, 1] and tokens.tolist() == [[1, -1], [0, 0]]


def test_sums_need_more_than_32_bits(kvd):
    """A large first weight and many tiny ones behind it: a sum in 32 bits would
    not move. Equal rows leave nothing: the target itself decides."""
    V = 100000
    p = torch.full((3, 2, V), 2.0 ** -27, device="cuda")
    p[:, :, 0] = 1.0
    q = torch.zeros(3, 1, V, device="cuda")
    q[2] = p[2, 0]
    x = torch.ones(3, 1, dtype=torch.int32, device="cuda")
    q[:, 0, 1] = 1.0                          # the draft is always rejected
    u = torch.full((3, 1), 0.99, device="cuda")
    us = torch.tensor([0.99995, 0.9997, 0.9999], device="cuda")
    tokens, acc = kvd.verify_drafts(p, q, x, u, us)
    want, n = expect(p, q, x, u, us, [1] * 3)
    assert torch.equal(tokens.cpu(), want) and torch.equal(acc.cpu(), n)
    same = p[:, :1].clone()
    same[:, 0, 1] = p[:, 0, 1]
    u = torch.ones(3, 1, device="cuda")       # u = 1: p(x) < p(x) fails, p - q = 0 everywhere
    tokens, acc = kvd.verify_drafts(p, same, x, u, us)
    want, n = expect(p, same, x, u, us, [1] * 3)
    assert n.tolist() == [0, 0, 0] and torch.equal(tokens.cpu(), want)


def test_refused_on_the_device(kvd):
    p, q, x, u, us = draws(5, 2, 333, F32, seed=3)
    good, ga = kvd.verify_drafts(p, q, x, u, us)
    x2 = x.clone()
    x2[0, 0], x2[1, 0] = -1, 333              # outside the vocabulary: rejected
    u2 = u.clone()
    u2[:2] = 0.0
    status = kvd.status_tensor()
    tokens, acc = kvd.verify_drafts(p, q, x2, u2, us, dev_status=status)
    assert int(status.item()) == kvd.DEV_TOKEN_RANGE
    assert acc[:2].tolist() == [0, 0] and bool((tokens[:2, 0] >= 0).all())
    assert torch.equal(tokens[2:], good[2:]) and torch.equal(acc[2:], ga[2:])
    status.zero_()
    m = torch.tensor([3, -1, 2, 2, 2], dtype=torch.int32, device="cuda")
    tokens, acc = kvd.verify_drafts(p, q, x, u, us, num_drafts=m, dev_status=status)
    assert int(status.item()) == kvd.DEV_POS_RANGE
    assert tokens[:2].tolist() == [[-1] * 3] * 2 and acc[:2].tolist() == [0, 0]
    assert torch.equal(tokens[2:], good[2:])
    status.zero_()
    bad = torch.zeros(4, 1, 50, device="cuda")  # nothing; NaN; an infinite sum; negative
    bad[1], bad[2, 0, 3], bad[3] = math.nan, math.inf, -1.0
    tokens, acc = kvd.verify_drafts(bad, None, None, None, us[:4].contiguous(), dev_status=status)
    assert int(status.item()) == kvd.DEV_PROBS and tokens[:, 0].tolist() == [-1] * 4
    one = torch.full((1, 1, 50), math.nan, device="cuda")
    one[0, 0, 17] = 0.5                       # NaN counts as zero
    assert kvd.verify_drafts(one, None, None, None, us[:1].contiguous())[0].tolist() == [[17]]


def test_graph(kvd):
    p, q, x, u, us = draws(8, 3, 5000, BF, seed=4)
    tokens, acc = torch.empty(8, 4, dtype=torch.int32).cuda(), torch.empty(8, dtype=torch.int32).cuda()
    kvd.verify_drafts(p, q, x, u, us, tokens=tokens, accepted=acc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvd.verify_drafts(p, q, x, u, us, tokens=tokens, accepted=acc)
    for k in range(3):
        u.copy_(torch.rand_like(u))
        us.copy_(torch.rand_like(us))
        graph.replay()
        torch.cuda.synchronize()
        want, n = expect(p, q, x, u, us, [3] * 8)
        assert torch.equal(tokens.cpu(), want) and torch.equal(acc.cpu(), n)
