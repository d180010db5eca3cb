"""The serving-step calls at the ends of their ranges: caches past 2^31 elements, the
longest rows, several streams and host threads at once, graphs that share a workspace,
padded batches."""
import math
import threading

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,Hkv", [(BF, 8), (F32, 4)], ids=["bf16", "f32"])
def test_caches_past_32_bits(kvd, dtype, Hkv):
    """The same step in a small cache and, page by page, behind element 2^31 of a large one:
    the same to the bit."""
    BS, D, Q, P = 16, 128, 5, 150
    g = torch.Generator().manual_seed(4)
    own = [20, 0, 1, 16, 33]
    NB_small, NB = 40, (2 ** 31 + 2 ** 28) // (BS * Hkv * D)
    lowest = 2 ** 31 // (BS * Hkv * D)
    pages = torch.randperm(NB_small, generator=g)
    far = lowest + 1 + torch.randperm(NB - lowest - 1, generator=g)[:NB_small]
    # page i of the small cache is page far[i] of the large one; the first 10 are the prefix's
    pre = pages[:-(-P // BS)][None]
    table, at = torch.zeros(Q, 3, dtype=torch.int64), 10
    for b, n in enumerate(own):
        for j in range(-(-n // BS)):
            table[b, j] = pages[at]
            at += 1
    ends = [sum(own[:j]) for j in range(Q + 1)]
    rows = [(b, t) for b, n in enumerate(own) for t in range(n)]
    slots = torch.tensor([int(table[b, t // BS]) * BS + t % BS for b, t in rows] +
                         [int(pre[0, t // BS]) * BS + t % BS for t in range(P)])
    pos = i32([P + t for _, t in rows] + list(range(P)))
    qkv = torch.randn(len(slots), 2 * Hkv + 2 * Hkv, D, generator=g).to(dtype).cuda()
    freqs = kvd.rotary_freqs(D).cuda()
    query = torch.randn(Q, 2 * Hkv, D, generator=g).to(dtype).cuda()
    results = []
    for big in (False, True):
        move = (lambda p: far[p]) if big else (lambda p: p)
        shape = (NB if big else NB_small, BS, Hkv, D)
        kc, vc = (torch.empty(shape, dtype=dtype, device="cuda") for _ in range(2))
        where = (move(slots // BS) * BS + slots % BS).to(torch.int32).cuda()
        status = kvd.status_tensor()
        q = kvd.rotate_append_paged(qkv, kc, vc, where, pos, freqs, dev_status=status)
        lse = torch.empty(Q, 2 * Hkv, device="cuda")
        out = kvd.attend_paged_prefix(query, kc, vc, move(pre).to(torch.int32).cuda(), i32([P]),
                                      i32([0, Q]), move(table).to(torch.int32).cuda(), i32(ends),
                                      lse=lse, dev_status=status)
        assert int(status.item()) == 0
        flat = kc.view(-1, Hkv, D), vc.view(-1, Hkv, D)
        results.append((q, out, lse, flat[0][where.long()], flat[1][where.long()]))
        del kc, vc, flat
    torch.cuda.empty_cache()
    for x, y in zip(*results):
        assert torch.equal(x, y)
    assert torch.equal(results[1][4], qkv[:, 3 * Hkv:])  # the values as they were


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_the_longest_rows(kvd, dtype):
    """2^20 logits: steep and flat, top-k within and past one CTA's list, each filter."""
    V = 2 ** 20
    g = torch.Generator().manual_seed(9)
    logits = torch.randn(7, V, generator=g) * 3
    logits[1] *= 0.01
    logits[2] = 1.0
    logits = logits.to(dtype).cuda()
    T = torch.tensor([1.0, 1.0, 1.0, 0.5, 1.3, 1.0, 0.7], device="cuda")
    k = i32([0, 0, 700000, 5000, 0, 2048, V])
    p = torch.tensor([0.9, 0.5, 0.3, 1.0, 1.0, 0.95, 0.99], device="cuda")
    m = torch.tensor([0.0, 0.0, 0.0, 0.0, 1e-4, 0.02, 0.0], device="cuda")
    u = torch.rand(7, generator=g).cuda()
    status = kvd.status_tensor()
    tokens = kvd.sample(logits, u, temperature=T, top_k=k, top_p=p, min_p=m, dev_status=status)
    probs = kvd.filter_probs(logits, temperature=T, top_k=k, top_p=p, min_p=m, dev_status=status)
    assert int(status.item()) == 0
    for r in range(7):
        w = ref.kept_weights(logits[r].double(), float(T[r]), int(k[r]), float(p[r]), float(m[r]))
        assert int(tokens[r]) == ref.draw(w, float(u[r]))
        q = w / w.sum()
        got = probs[r].double()
        assert torch.equal(got > 0, q.to(probs.dtype) > 0)
        tol = q * (ref.U[probs.dtype] + 3 * 2.0 ** -24) + 2.0 ** -126  # as for shorter rows
        assert float(((got - q).abs() / tol).max()) <= 1.0


class Step:
    """One decode step of Q sequences behind one prefix, from page plan to token."""

    def __init__(self, kvd, seed, Q=6, P=100, BS=16, Hq=8, Hkv=2, D=128, V=3001):
        g = torch.Generator().manual_seed(seed)
        self.kvd, self.BS, self.Q = kvd, BS, Q
        cols, NB = 4, 4 * Q + 10
        order = torch.randperm(NB, generator=g).to(torch.int32).cuda()
        self.pre = order[:-(-P // BS)][None].contiguous()
        self.free = torch.cat([order[-(-P // BS):], torch.zeros(-(-P // BS), dtype=torch.int32, device="cuda")])
        self.count = i32([NB - (-(-P // BS))])
        self.table, self.held = torch.full((Q, cols), -1, dtype=torch.int32, device="cuda"), i32([0] * Q)
        self.kept, self.new = i32([0] * Q), i32(list(range(Q + 1)))
        self.plens, self.groups = i32([P]), i32([0, Q])
        self.base = i32([P] * Q)
        self.qkv = torch.randn(Q, Hq + 2 * Hkv, D, generator=g).to(BF).cuda()
        self.kc = torch.randn(NB, BS, Hkv, D, generator=g).to(BF).cuda()
        self.vc = torch.randn(NB, BS, Hkv, D, generator=g).to(BF).cuda()
        # logits without a matrix product, whose sums may depend on the stream
        self.pick = torch.randint(Hq * D, (V,), generator=g).cuda()
        self.head = (torch.randn(V, generator=g) * 5).cuda()
        self.u = torch.rand(Q, generator=g).cuda()
        self.k, self.p = i32([40] * Q), torch.full((Q,), 0.9, device="cuda")
        self.freqs = kvd.rotary_freqs(D).cuda()
        self.workspace = kvd.workspace(kvd.attend_paged_prefix_workspace_bytes(
            Q, 1, Hq, Hkv, BS, self.pre.shape[1], cols, D, BF))

    def run(self, workspace=None):
        kvd = self.kvd
        lens, slots, pos = kvd.plan_pages(self.table, self.held, self.free, self.count, self.kept,
                                          self.new, self.BS, self.Q, pos_base=self.base)
        q = kvd.rotate_append_paged(self.qkv, self.kc, self.vc, slots, pos, self.freqs)
        out = kvd.attend_paged_prefix(q, self.kc, self.vc, self.pre, self.plens, self.groups,
                                      self.table, lens,
                                      workspace=self.workspace if workspace is None else workspace)
        logits = out.flatten(1)[:, self.pick].float() * self.head
        tokens = kvd.sample(logits, self.u, top_k=self.k, top_p=self.p)
        self.kept.copy_(lens[1:] - lens[:-1])
        return out, tokens


def trail(kvd, seed, steps=12):
    s = Step(kvd, seed)
    return [tuple(x.clone() for x in s.run()) for _ in range(steps)]


def agree(a, b):
    return all(torch.equal(x, y) for s, t in zip(a, b) for x, y in zip(s, t))


def test_streams_at_once(kvd):
    want = [trail(kvd, seed) for seed in range(3)]
    torch.cuda.synchronize()
    steps = [Step(kvd, seed) for seed in range(3)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    got = [[], [], []]
    for _ in range(12):
        for i, s in enumerate(steps):
            with torch.cuda.stream(streams[i]):
                got[i].append(s.run())
    torch.cuda.synchronize()
    assert all(agree(a, b) for a, b in zip(want, got))


def test_host_threads_at_once(kvd):
    want = [trail(kvd, seed) for seed in range(4)]
    torch.cuda.synchronize()
    steps, got, errors = [Step(kvd, seed) for seed in range(4)], [[] for _ in range(4)], []
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(12):
                    got[i].append(steps[i].run())
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (told to the test's thread)
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    assert all(agree(a, b) for a, b in zip(want, got))


def test_graphs_share_a_workspace(kvd):
    """Two captured steps of different requests with one workspace, replayed in turn."""
    want = [trail(kvd, seed, 9) for seed in (1, 2)]
    warm = Step(kvd, 7)
    warm.run()
    steps = [Step(kvd, seed) for seed in (1, 2)]
    shared = torch.full_like(warm.workspace, 170)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(s.run(shared))
        graphs.append(graph)
    got = [[], []]
    for _ in range(9):
        for i, graph in enumerate(graphs):
            graph.replay()
            got[i].append(tuple(x.clone() for x in outs[i]))
    torch.cuda.synchronize()
    assert all(agree(a, b) for a, b in zip(want, got))


def test_padded_batch(kvd):
    """A step of fixed size with fewer tokens and sequences in it: what lies behind is left
    as it was, and the rest is as without it."""
    Q, N, BS, Hkv, D = 8, 24, 16, 2, 64
    g = torch.Generator().manual_seed(3)
    live, counts = 5, [3, 0, 7, 1, 2]
    ends = [sum(counts[:min(j, live)]) for j in range(Q + 1)]
    qkv = torch.randn(N, 8 + 2 * Hkv, D, generator=g).to(BF).cuda()
    freqs = kvd.rotary_freqs(D).cuda()
    results = []
    for n, size in ((live, ends[live]), (Q, N)):
        NB = 20
        kc, vc = (torch.full((NB, BS, Hkv, D), 5.0, dtype=BF, device="cuda") for _ in range(2))
        table, held = torch.zeros(n, 2, dtype=torch.int32, device="cuda"), i32([0] * n)
        status = kvd.status_tensor()
        lens, slots, pos = kvd.plan_pages(table, held, i32(list(range(NB))), i32([NB]), i32([0] * n),
                                          i32(ends[:n + 1]), BS, size, dev_status=status)
        q = torch.full((size, 8, D), 9.0, dtype=BF, device="cuda")
        kvd.rotate_append_paged(qkv[:size].contiguous(), kc, vc, slots, pos, freqs, out=q,
                                dev_status=status)
        one = torch.randn(Q, 8, D, generator=torch.Generator().manual_seed(8)).to(BF).cuda()[:n]
        lse = torch.empty(n, 8, device="cuda")
        out = kvd.attend_paged_prefix(one.contiguous(), kc, vc, i32([[0, 1]]), i32([0]), i32([0, 2]),
                                      table, lens, lse=lse, dev_status=status)
        assert int(status.item()) == 0
        results.append((lens, slots, pos, q, out, lse, kc, vc))
    a, b = results
    assert b[0].tolist() == a[0].tolist() + [ends[live]] * (Q - live)
    for i, m in ((1, ends[live]), (2, ends[live]), (3, ends[live]), (4, live), (5, live)):
        assert torch.equal(a[i], b[i][:m])
    assert (b[1][ends[live]:] == -1).all() and (b[2][ends[live]:] == -1).all()
    assert (b[3][ends[live]:] == 9.0).all()
    assert (b[4][live:] == 0).all() and (b[5][live:] == -math.inf).all()
    assert torch.equal(a[6], b[6]) and torch.equal(a[7], b[7])


@pytest.mark.parametrize("V", [37, 5000])
@pytest.mark.parametrize("T", [1e-45, 1e-38, 3e-20, 1e20, 1e30])
def test_far_temperatures(kvd, T, V):
    """A division that overflows keeps the largest logits alone; one that vanishes all finite
    ones alike."""
    g = torch.Generator().manual_seed(V)
    logits = torch.randn(6, V, generator=g) * 5
    logits[1, 3] = logits[1, 20] = 40.0
    logits[2, ::2] = -math.inf
    logits[3] = 0.0
    logits[4] *= 1e-30
    logits = logits.cuda()
    t = torch.full((6,), T, device="cuda")
    k, p = i32([0, 0, 0, 0, 0, 9]), torch.tensor([1.0, 1.0, 0.7, 1.0, 0.6, 0.8], device="cuda")
    u = torch.rand(6, generator=g).cuda()
    status = kvd.status_tensor()
    tokens = kvd.sample(logits, u, temperature=t, top_k=k, top_p=p, dev_status=status)
    probs = kvd.filter_probs(logits, temperature=t, top_k=k, top_p=p, dev_status=status)
    assert int(status.item()) == 0
    for r in range(6):
        w = ref.kept_weights(logits[r].double(), float(t[r]), int(k[r]), float(p[r]), 0.0)
        assert int(tokens[r]) == ref.draw(w, float(u[r]))
        q = w / w.sum()
        got = probs[r].double()
        tol = q * (ref.U[F32] + 3 * 2.0 ** -24) + 2.0 ** -126  # as for other rows
        assert float(((got - q).abs() / tol).max()) <= 1.0


@pytest.mark.parametrize("D", [64, 128])
def test_many_short_pieces_give_the_same_each_time(kvd, D):
    """Workers that go from piece to piece: groups of a few sequences behind prefixes of
    one to a few hundred tokens, again and again, the same to the bit and as in 64 bits."""
    import latent_ref as lref
    from test_gpu_prefix import Case
    sizes = [8, 8, 8, 7, 7, 7, 60, 1, 1, 33]
    pre = [700, 500, 390, 1, 1, 20, 260, 17, 1, 129]
    c = Case(sizes, pre, [3 + i % 20 for i in range(sum(sizes))], 16, 4, D, 16, BF, seed=5)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    want = kvd.attend_paged_prefix(*c.args(), lse=lse)
    lref.check("first", want, lse, *c.reference(), max(pre) + 23, BF)
    outs = [kvd.attend_paged_prefix(*c.args()) for _ in range(300)]
    assert all(torch.equal(want, x) for x in outs)
