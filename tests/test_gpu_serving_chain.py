"""The serving step's operators together: pages planned, projections rotated into
them, attention behind shared prefixes, tokens drawn; the caches and tables are
followed step by step in plain 64-bit forms."""
import math

import pytest
import torch

import latent_ref as lref
import serving_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HQ, HKV, D, BS, V = 8, 2, 64, 16, 997


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_serving_loop(kvd, dtype):
    """Two groups behind prefixes and one request alone: prompts of unequal lengths, then
    steps, drafted tokens of which some are rejected, a request that ends and one that
    takes its place.  The oracle's cache holds what the kernels left in the planned rows
    (checked against the rotation), so that each step is checked by itself."""
    g = torch.Generator().manual_seed(3)
    Q, cols, F = 5, 12, 80
    dev = "cuda"
    kc = torch.full((F, BS, HKV, D), math.nan, dtype=dtype, device=dev)
    vc = torch.full((F, BS, HKV, D), math.inf, dtype=dtype, device=dev)
    table = torch.full((Q, cols), -1, dtype=torch.int32, device=dev)
    held, count = ints([0] * Q), ints([F - 12])
    free = torch.randperm(F, generator=g).to(torch.int32).cuda()
    spare = free[F - 12:].clone()          # pages of the prefixes
    freqs = kvd.rotary_freqs(D, scaling="linear", factor=2.0)
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2))
    head = torch.randn(HQ * D, V, generator=g).cuda() * 0.3
    status = kvd.status_tensor()

    def project(n):
        return torch.randn(n, HQ + 2 * HKV, D, generator=g).to(dtype).cuda()

    # the prefixes: rotated and appended once, by hand-made slots
    pre = [70, 37]
    ptable = torch.stack([spare[:6], spare[6:12]]).contiguous()
    plens, glens = ints(pre), ints([0, 2, 4])   # sequences 0 1 | 2 3, and 4 alone
    for i, n in enumerate(pre):
        t = torch.arange(n, device=dev)
        slots = (ptable[i].long()[t // BS] * BS + t % BS).to(torch.int32)
        kvd.rotate_append_paged(project(n), kc, vc, slots, t.to(torch.int32), freqs, q_weight=qw,
                                k_weight=kw, dev_status=status)
    base = ints([70, 70, 37, 37, 0])

    def step(kept, n):
        """n new tokens of every sequence, the last one's query attends."""
        new = [0]
        for x in n:
            new.append(new[-1] + x)
        lens, slots, pos = kvd.plan_pages(table, held, free, count, ints(kept), ints(new), BS,
                                          new[-1], pos_base=base, dev_status=status)
        total = [k + x for k, x in zip(kept, n)]
        assert (lens[1:] - lens[:-1]).tolist() == total
        x = project(new[-1])
        q = kvd.rotate_append_paged(x, kc, vc, slots, pos, freqs, q_weight=qw, k_weight=kw,
                                    dev_status=status)
        q0, s0 = ref.rotate(x[:, :HQ].double(), qw, pos, freqs, False, 1.0, 1e-6)
        k0, s1 = ref.rotate(x[:, HQ:HQ + HKV].double(), kw, pos, freqs, False, 1.0, 1e-6)
        ref.check_rotated("queries", q, q0, s0, D, dtype)
        ref.check_rotated("keys", kc.view(-1, HKV, D)[slots.long()], k0, s1, D, dtype)
        assert torch.equal(vc.view(-1, HKV, D)[slots.long()], x[:, HQ + HKV:])
        some = [q for q in range(Q) if n[q]]
        last = torch.tensor([new[q + 1] - 1 for q in some], device=dev)
        qs = torch.zeros(Q, HQ, D, dtype=dtype, device=dev)
        qs[some] = q[last]
        lse = torch.empty(Q, HQ, device=dev)
        out = kvd.attend_paged_prefix(qs, kc, vc, ptable, plens, glens, table, lens, lse=lse,
                                      dev_status=status)
        want = torch.zeros(Q, HQ, D, dtype=torch.float64, device=dev)
        A, d = torch.zeros_like(want), torch.zeros(Q, HQ, dtype=torch.float64, device=dev)
        z = torch.full_like(d, -math.inf)
        for b in range(Q):
            rows = []
            for tab, m in ([(ptable[b // 2], pre[b // 2])] if b < 4 else []) + [(table[b], total[b])]:
                t = torch.arange(m, device=dev)
                rows.append(tab.long()[t // BS] * BS + t % BS)
            rows = torch.cat(rows)
            k, v = (c.view(-1, HKV, D)[rows].double() for c in (kc, vc))
            for h in range(HKV):
                hs = slice(4 * h, 4 * h + 4)
                seen = torch.ones((4, len(rows)), dtype=torch.bool, device=dev)
                want[b, hs], z[b, hs], A[b, hs], d[b, hs] = lref.attention(
                    qs[b, hs].double(), k[:, h], v[:, h], 1 / math.sqrt(D), seen)
        lref.check("attention", out, lse, want, z, A, d, 300, dtype)
        assert int(status.item()) == 0
        return out, total

    def tokens_of(out):
        logits = out.float().reshape(Q, -1) @ head
        u = torch.rand(Q, generator=g).cuda()
        k, p = ints([40] * Q), torch.full((Q,), 0.9, device=dev)
        got = kvd.sample(logits, u, top_k=k, top_p=p, dev_status=status)
        for b in range(Q):
            w = ref.kept_weights(logits[b].double(), 1.0, 40, float(p[b]), 0.0)
            assert int(got[b]) == ref.draw(w, float(u[b]))
        # one way to draw: the filtered distribution through the verification without drafts
        probs = kvd.filter_probs(logits, top_k=k, top_p=p)
        again, _ = kvd.verify_drafts(probs[:, None].contiguous(), None, None, None, u)
        assert (again[:, 0] == got).float().mean() > 0.5
        assert bool((probs.gather(1, again.long()) > 0).all())
        return got

    out, lens = step([0] * Q, [1, 33, 16, 17, 100])        # prompts
    tokens_of(out)
    for i in range(20):                                    # steps across page borders
        out, lens = step(lens, [1] * Q)
    tokens_of(out)
    kept = lens
    out, _ = step(kept, [4] * Q)                           # three drafts and the newest token
    kept = [k + 1 + (b % 4) for b, k in enumerate(kept)]   # some of them rejected
    out, lens = step(kept, [4] * Q)
    lens[1], lens[4] = 0, 0                                # two requests end, one begins
    out, lens = step(lens, [1, 50, 1, 1, 0])
    assert held.tolist() == [-(-n // BS) for n in lens]
    owned = [p for b in range(Q) for p in table[b, :held[b]].tolist()] + free[:int(count)].tolist()
    assert sorted(owned + spare.tolist()) == list(range(F))


def test_drafted_step_under_filters(kvd):
    """Target and draft distributions under the same settings, drafts drawn from the
    filtered draft: tokens that the filters drop are never accepted or drawn."""
    Qs, T = 30, 3
    g = torch.Generator().manual_seed(5)
    logits = (torch.randn(Qs, T + 1, V, generator=g) * 3).cuda()
    near = logits[:, :T] + 0.3 * torch.randn(Qs, T, V, generator=g).cuda()
    k = torch.randint(1, 60, (Qs,), generator=g).to(torch.int32).cuda()
    p = (torch.rand(Qs, generator=g) * 0.5 + 0.5).cuda()
    temp = (torch.rand(Qs, generator=g) + 0.4).cuda()

    def rows(x, n):
        return x[:, None].expand(Qs, n).reshape(-1).contiguous()
    target = kvd.filter_probs(logits.view(-1, V), rows(temp, T + 1), rows(k, T + 1), rows(p, T + 1))
    draft = kvd.filter_probs(near.reshape(-1, V), rows(temp, T), rows(k, T), rows(p, T))
    u = torch.rand(Qs * T, generator=g).cuda()
    drafts = kvd.sample(near.reshape(-1, V), u, rows(temp, T), rows(k, T), rows(p, T))
    assert bool((draft.gather(1, drafts.long()[:, None]) > 0).all())
    target, draft = target.view(Qs, T + 1, V), draft.view(Qs, T, V)
    tokens, accepted = kvd.verify_drafts(target, draft, drafts.view(Qs, T),
                                         torch.rand(Qs, T, generator=g).cuda(),
                                         torch.rand(Qs, generator=g).cuda())
    assert set(accepted.tolist()) >= {0, T}
    for b in range(Qs):
        for i in range(int(accepted[b]) + 1):
            assert float(target[b, i, int(tokens[b, i])]) > 0


def test_captured_step(kvd):
    """One decode step in a graph, replayed: the tables move on by themselves and each
    replay equals the same calls made one by one on a copy of the state."""
    Q, cols, F = 6, 10, 70
    g = torch.Generator().manual_seed(6)
    freqs = kvd.rotary_freqs(D)

    def fresh():
        gen = torch.Generator().manual_seed(7)
        return dict(table=torch.full((Q, cols), -1, dtype=torch.int32, device="cuda"),
                    held=ints([0] * Q), count=ints([F]),
                    free=torch.randperm(F, generator=gen).to(torch.int32).cuda(),
                    kept=ints([0] * Q), kc=torch.zeros(F, BS, HKV, D, dtype=BF, device="cuda"),
                    vc=torch.zeros(F, BS, HKV, D, dtype=BF, device="cuda"))
    new = ints(list(range(Q + 1)))
    none = (torch.zeros(1, 1, dtype=torch.int32, device="cuda"), ints([0]), ints([0, 0]))
    x = torch.zeros(Q, HQ + 2 * HKV, D, dtype=BF, device="cuda")
    u = torch.zeros(Q, device="cuda")
    need = kvd.attend_paged_prefix_workspace_bytes(Q, 1, HQ, HKV, BS, 1, cols, D)
    head = torch.randn(HQ * D, V, generator=g).cuda()

    def step(s, ws):
        lens, slots, pos = kvd.plan_pages(s["table"], s["held"], s["free"], s["count"], s["kept"],
                                          new, BS, Q)
        q = kvd.rotate_append_paged(x, s["kc"], s["vc"], slots, pos, freqs)
        out = kvd.attend_paged_prefix(q, s["kc"], s["vc"], *none, s["table"], lens, workspace=ws)
        tokens = kvd.sample(out.float().view(Q, -1) @ head, u)
        s["kept"].copy_(lens[1:] - lens[:-1])
        return out, tokens, slots
    a, b = fresh(), fresh()
    ws = [kvd.workspace(need) for _ in range(2)]
    step(fresh(), ws[0])  # the matrix product's own set-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a, ws[0])
    for i in range(2 * BS + 3):
        x.copy_(torch.randn(x.shape, generator=g))
        u.copy_(torch.rand(Q, generator=g))
        graph.replay()
        want = step(b, ws[1])
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert torch.equal(a["kc"], b["kc"]) and torch.equal(a["table"], b["table"])
    assert a["held"].tolist() == [3] * Q
