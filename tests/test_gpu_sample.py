"""kvd_sample and kvd_filter_probs against 64-bit forms: the same tokens, the same
tokens kept, probabilities within a rounding."""
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


def settings(R, g, use="kpmt"):
    """Settings of every kind, row by row."""
    r = lambda lo, hi: torch.rand(R, generator=g) * (hi - lo) + lo  # noqa: E731
    at = torch.arange(R)
    T = torch.where(at % 7 == 3, torch.zeros(R), torch.where(at % 11 == 5, torch.full((R,), 30.0), r(0.3, 2.0)))
    k = torch.where(at % 3 == 0, torch.zeros(R), torch.exp(r(0, 8.0))).to(torch.int32)
    p = torch.where(at % 4 == 1, torch.ones(R), r(0.05, 1.0))
    m = torch.where(at % 2 == 0, torch.zeros(R), r(0, 0.3))
    return (T.cuda() if "t" in use else None, k.cuda() if "k" in use else None,
            p.cuda() if "p" in use else None, m.cuda() if "m" in use else None)


def expect(logits, T, k, p, m):
    """The weights that stay [R, V], float64."""
    rows = []
    for r in range(logits.shape[0]):
        x = logits[r].double()
        x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
        if float(x.max()) == -math.inf:  # nothing to draw: refused
            rows.append(torch.zeros_like(x))
            continue
        rows.append(ref.kept_weights(x, 1.0 if T is None else float(T[r]),
                                     0 if k is None else int(k[r]), 1.0 if p is None else float(p[r]),
                                     0.0 if m is None else float(m[r])))
    return torch.stack(rows)


def same(kvd, logits, u, T=None, k=None, p=None, m=None, probs=(BF, F32)):
    w = expect(logits, T, k, p, m)
    status = kvd.status_tensor()
    tokens = kvd.sample(logits, u, temperature=T, top_k=k, top_p=p, min_p=m, dev_status=status)
    some = (w.sum(1) > 0).tolist()
    want = [ref.draw(w[r], float(u[r])) if some[r] else -1 for r in range(w.shape[0])]
    assert tokens.tolist() == want
    q = w / w.sum(1, keepdim=True).clamp(min=0.5)
    for dt in probs:
        got = kvd.filter_probs(logits, temperature=T, top_k=k, top_p=p, min_p=m, dev_status=status,
                               out=torch.full(logits.shape, 3.0, dtype=dt, device="cuda"))
        g = got.double()
        assert torch.equal(g > 0, q.to(dt) > 0) or \
            float((g - q).abs()[(g > 0) != (q.to(dt) > 0)].max()) < 2.0 ** -125
        # w (rounded to fp32), the factor and their product: a rounding each; below 2^-125
        # of the largest a weight may lose its last places
        tol = q * (ref.U[dt] + 3 * 2.0 ** -24) + 2.0 ** -126
        assert float(((g - q).abs() / tol).max()) <= 1.0
    assert int(status.item()) == (0 if all(some) else kvd.DEV_PROBS)
    return tokens


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,V", [(1, 1), (5, 2), (14, 31), (40, 257), (25, 1000), (30, 4099),
                                 (12, 50257), (6, 128000), (3, 262144)])
def test_random(kvd, R, V, dtype):
    g = torch.Generator().manual_seed(V)
    logits = (torch.randn(R, V, generator=g) * 3).to(dtype).cuda()
    u = torch.rand(R, generator=g).cuda()
    same(kvd, logits, u, *settings(R, g))


@pytest.mark.parametrize("use", ["", "t", "tk", "tp", "tm", "kp", "pm", "km"])
def test_each_filter(kvd, use):
    R, V = 24, 3001
    g = torch.Generator().manual_seed(len(use))
    logits = (torch.randn(R, V, generator=g) * 4).cuda()
    same(kvd, logits, torch.rand(R, generator=g).cuda(), *settings(R, g, use))


def test_borders(kvd):
    """Equal logits weigh exactly alike, so every border is exact: a running sum equal to
    the wanted one does not end the search."""
    V = 8
    u = torch.tensor([i / 8 for i in range(8)] + [1 - 2.0 ** -24], device="cuda")
    logits = torch.full((9, V), 1.5, device="cuda")
    assert same(kvd, logits, u).tolist() == list(range(8)) + [7]
    p = torch.tensor([0.0, 0.125, 0.25, 0.5, 0.75, 1.0, 2.0, -1.0, 0.25 + 2.0 ** -24], device="cuda")
    kept = (kvd.filter_probs(logits, top_p=p) > 0).sum(1).tolist()
    assert kept == [1, 1, 2, 4, 6, 8, 8, 1, 3]
    k = torch.tensor([0, 1, 3, 7, 8, 9, -1, 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    probs = kvd.filter_probs(logits, top_k=k)
    assert (probs > 0).sum(1).tolist() == [8, 1, 3, 7, 8, 8, 8, 2, 8]
    for r, n in enumerate([8, 1, 3, 7, 8, 8, 8, 2, 8]):  # ties go to the lowest index
        assert bool((probs[r, :n] > 0).all())
    m = torch.tensor([0.0, 1.0, 2.0, 0.5, -1.0, 1.0, 0, 0, 0], device="cuda")
    assert (kvd.filter_probs(logits, min_p=m) > 0).sum(1).tolist() == [8] * 9
    # half weights: exp(-ln 2) is below 0.5 or not by the last place; a hair on either side
    two = torch.tensor([[0.0, -0.6931], [0.0, -0.6932]], device="cuda")
    half = torch.full((2,), 0.5, device="cuda")
    assert (kvd.filter_probs(two, min_p=half) > 0).sum(1).tolist() == [2, 1]


def test_ties_across_the_row(kvd):
    """Few distinct values, so that every cut falls among equal logits far apart."""
    R, V = 40, 20011
    g = torch.Generator().manual_seed(5)
    logits = torch.randint(0, 6, (R, V), generator=g).float().cuda()
    k = torch.randint(1, V, (R,), generator=g).to(torch.int32).cuda()
    p = (torch.rand(R, generator=g) * 0.9 + 0.05).cuda()
    u = torch.rand(R, generator=g).cuda()
    same(kvd, logits, u, k=k)
    same(kvd, logits, u, p=p)
    same(kvd, logits, u, T=torch.full((R,), 0.7, device="cuda"), k=k, p=p)
    logits = torch.where(torch.rand(R, V, generator=g).cuda() < 0.5, -0.0, 0.0)  # signed zeros tie
    same(kvd, logits, u, k=k, p=p)


def test_all_equal_and_steep(kvd):
    V = 100003
    u = torch.rand(6, generator=torch.Generator().manual_seed(1)).cuda()
    p = torch.tensor([0.1, 0.37, 0.5, 0.9, 0.999, 1.0], device="cuda")
    same(kvd, torch.full((6, V), -3.25, device="cuda"), u, p=p)
    steep = torch.linspace(0, -400, V, device="cuda").repeat(6, 1)
    same(kvd, steep, u, p=p)
    same(kvd, steep.flip(1).contiguous(), u, p=p, T=torch.full((6,), 1e-3, device="cuda"))
    # one large weight and many that a sum in 32 bits would lose
    tail = torch.full((6, V), -17.0, device="cuda")
    tail[:, 777] = 0.0
    u = torch.tensor([0.0, 0.005, 0.01, 0.99, 0.9961, 0.9999], device="cuda")
    same(kvd, tail, u)
    same(kvd, tail, u, p=torch.full((6,), 0.9975, device="cuda"))


@pytest.mark.parametrize("shift,T", [(100.0, 0.01), (-3000.0, 0.7), (2.0 ** 20, 30.0)])
def test_logits_far_from_zero(kvd, shift, T):
    """The largest logit over the temperature up to 4 * 10^4: the differences count, taken
    before anything is rounded (the logits lie on fp32's grid there)."""
    R, V = 12, 7001
    g = torch.Generator().manual_seed(11)
    logits = (torch.randn(R, V, generator=g) * 3 * T + shift).cuda()
    u = torch.rand(R, generator=g).cuda()
    _, k, p, m = settings(R, g)
    temp = torch.full((R,), T, device="cuda")
    same(kvd, logits, u, T=temp)
    same(kvd, logits, u, T=temp, p=p)
    same(kvd, logits, u, T=temp, k=k, p=p, m=m)


def test_infinities_and_nan(kvd):
    V = 5000
    g = torch.Generator().manual_seed(9)
    logits = torch.randn(8, V, generator=g).cuda()
    logits[0, ::2] = -math.inf
    logits[1, 1::3] = math.nan
    logits[2] = -math.inf
    logits[2, 4321] = -5.0
    logits[3, [7, 4000]] = math.inf      # share the weight alike
    logits[4, 17:] = -math.inf           # fewer than k
    logits[5] = torch.finfo(F32).min
    logits[6, :10] = torch.finfo(F32).max
    logits[7, 3] = torch.finfo(F32).min
    u = torch.tensor([0.3, 0.9, 0.5, 0.5, 0.99, 0.5, 0.5, 0.2], device="cuda")
    k = torch.full((8,), 50, dtype=torch.int32, device="cuda")
    p = torch.full((8,), 0.95, device="cuda")
    tokens = same(kvd, logits, u, k=k, p=p)
    assert tokens[2] == 4321 and tokens[3] == 4000
    same(kvd, logits, u)
    same(kvd, logits, u, T=torch.full((8,), 1e-30, device="cuda"), p=p)
    same(kvd, logits, u, T=torch.full((8,), 1e30, device="cuda"), k=k)
    same(kvd, logits.to(BF), u, k=k, p=p)


@pytest.mark.parametrize("V", [3, 9000])
def test_refused_rows(kvd, V):
    """Rows without a logit above -inf, and parameters out of range: -1 and zeros; the
    rows beside them are served."""
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(9, V, generator=g).cuda()
    ones, u = torch.ones(9, device="cuda"), torch.full((9,), 0.5, device="cuda")
    good = kvd.sample(logits, u)
    for name, row, value in [("T", 1, -1.0), ("T", 2, math.nan), ("T", 3, math.inf),
                             ("p", 4, math.nan), ("m", 5, math.nan), ("u", 6, 1.0),
                             ("u", 7, -0.1), ("u", 8, math.nan)]:
        a = {"T": ones.clone(), "p": ones.clone(), "m": 0 * ones, "u": u.clone()}
        a[name][row] = value
        status = kvd.status_tensor()
        t = kvd.sample(logits, a["u"], temperature=a["T"], top_p=a["p"], min_p=a["m"], dev_status=status)
        want = good.clone()
        want[row] = -1
        assert torch.equal(t, want) and int(status.item()) == kvd.DEV_PARAM
        if name != "u":
            status.zero_()
            q = kvd.filter_probs(logits, temperature=a["T"], top_p=a["p"], min_p=a["m"], dev_status=status)
            assert int(status.item()) == kvd.DEV_PARAM
            assert bool((q[row] == 0).all()) and bool((q.sum(1)[[r for r in range(9) if r != row]] > 0.99).all())
    logits[0] = -math.inf
    logits[4] = math.nan
    status = kvd.status_tensor()
    t = kvd.sample(logits, u, dev_status=status)
    assert int(status.item()) == kvd.DEV_PROBS and t[[0, 4]].tolist() == [-1, -1]
    assert torch.equal(t[[1, 2, 3, 5, 6, 7, 8]], good[[1, 2, 3, 5, 6, 7, 8]])
    status.zero_()
    q = kvd.filter_probs(logits, dev_status=status)
    assert int(status.item()) == kvd.DEV_PROBS and bool((q[[0, 4]] == 0).all())


def test_unaligned_rows_and_guards(kvd):
    """Rows that start at odd addresses; what lies beside the outputs stays."""
    for dtype in (BF, F32):
        g = torch.Generator().manual_seed(4)
        R, V = 7, 4999
        flat = torch.full((R * V + 3,), 99.0, dtype=dtype, device="cuda")
        logits = flat[1:1 + R * V].view(R, V)
        logits.copy_(torch.randn(R, V, generator=g) * 3)
        u = torch.rand(R, generator=g).cuda()
        T, k, p, m = settings(R, g)
        same(kvd, logits, u, T, k, p, m)
        buf = torch.full((R * V + 2,), 8.0, dtype=dtype, device="cuda")
        kvd.filter_probs(logits, T, k, p, m, out=buf[1:1 + R * V].view(R, V))
        assert float(buf[0]) == 8.0 and float(buf[-1]) == 8.0
        tok = torch.full((R + 2,), 5, dtype=torch.int32, device="cuda")
        kvd.sample(logits, u, T, k, p, m, tokens=tok[1:-1])
        assert tok[[0, -1]].tolist() == [5, 5]


def test_the_draws_follow_the_distribution(kvd):
    """Every multiple of 1/4096 as u: each token as often as its probability says, to
    within one draw at either end of its interval."""
    V, n = 50, 4096
    g = torch.Generator().manual_seed(8)
    row = torch.randn(1, V, generator=g).cuda() * 2
    u = (torch.arange(n, device="cuda") / n).float()
    tokens = kvd.sample(row.repeat(n, 1), u, top_k=torch.full((n,), 20, dtype=torch.int32, device="cuda"))
    q = kvd.filter_probs(row, top_k=torch.tensor([20], dtype=torch.int32, device="cuda"))[0]
    counts = torch.bincount(tokens.long(), minlength=V)
    assert float((counts - n * q).abs().max()) <= 1.0 and int((counts > 0).sum()) <= 20


def test_graph_and_same_result_each_time(kvd):
    R, V = 33, 32000
    g = torch.Generator().manual_seed(2)
    a, b = ((torch.randn(R, V, generator=g) * 3).cuda() for _ in range(2))
    u = torch.rand(R, generator=g).cuda()
    T, k, p, m = settings(R, g)
    static = a.clone()
    want = [(kvd.sample(x, u, T, k, p, m), kvd.filter_probs(x, T, k, p, m)) for x in (a, b)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens = kvd.sample(static, u, T, k, p, m)
        probs = kvd.filter_probs(static, T, k, p, m)
    for x, (t, q) in zip((b, a, b), (want[1], want[0], want[1])):
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tokens, t) and torch.equal(probs, q)


def test_refusals(kvd):
    l, u = torch.zeros(3, 8, device="cuda"), torch.zeros(3, device="cuda")
    with pytest.raises(TypeError):
        kvd.sample(l.half(), u)
    with pytest.raises(ValueError):
        kvd.sample(l, u[:2])
    with pytest.raises(TypeError):
        kvd.sample(l, u.double())
    with pytest.raises(ValueError):
        kvd.sample(l[0], u)
    with pytest.raises(ValueError):
        kvd.sample(l.t().contiguous().t(), u)
    with pytest.raises(TypeError):
        kvd.sample(l, u, top_k=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        kvd.filter_probs(l, temperature=u[:1])
    with pytest.raises(TypeError):
        kvd.filter_probs(l, out=torch.zeros(3, 8, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        kvd.filter_probs(l, out=torch.zeros(3, 9, device="cuda"))
    assert kvd.sample(l[:0], u[:0]).shape == (0,)
