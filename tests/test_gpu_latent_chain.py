"""The latent-cache calls together, as a serving loop makes them: prompts into
the paged cache, gathered and expanded for their own attention, then drafted
steps (append, absorbed attention, verification) whose rejected tokens are
overwritten by the next step."""
import math

import pytest
import torch

import latent_ref as ref

pytestmark = pytest.mark.gpu

R, P, DN, DV, H, BS = 128, 64, 64, 128, 4, 16


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


class Model:
    """Projections of one attention layer, fp32."""

    def __init__(self, g):
        n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.uk, self.uv = n(H, DN, R) / math.sqrt(R), n(H, DV, R) / math.sqrt(R)
        self.scale = 1.0 / math.sqrt(DN + P)
        self.n = n

    def tokens(self, N):
        """Latent row, rotary key row and per-head queries of N tokens."""
        return self.n(N, R), self.n(N, P), self.n(N, H, DN), self.n(N, H, P)


def cum(x):
    return torch.tensor([0] + list(x), device="cuda").cumsum(0).to(torch.int32)


def truth(m, rows, ropes, qn, qr, sees):
    """One query in 64 bits: rows [n, R], ropes [n, P], qn [H, DN], qr [H, P]."""
    c, r = rows[:sees].double(), ropes[:sees].double()
    k = torch.einsum("hdr,nr->hnd", m.uk.double(), c)
    s = m.scale * (torch.einsum("hd,hnd->hn", qn.double(), k) + qr.double() @ r.T)
    w = torch.softmax(s, -1)
    return torch.einsum("hdr,hr->hd", m.uv.double(), w @ c)


# Every stage is fp32 sums of at most 192 terms: each is off by at most 192 * 2^-24
# of its terms' magnitudes, weights by twice that times the scores' magnitude (below
# 64 here), and a projection of 128 terms follows: below 2^-9 of the magnitudes that
# are summed at the end, which a row of unit variance keeps below 8.
TOL = 2.0 ** -9 * 8


def test_serving_loop(kvd):
    g = torch.Generator(device="cuda").manual_seed(5)
    m = Model(g)
    prompts, T, V = [37, 1, 120], 3, 211
    Q = len(prompts)
    cols = 16
    table = torch.randperm(Q * cols, generator=g, device="cuda").view(Q, cols).to(torch.int32)
    latent = torch.full((Q * cols, BS, 1, R), math.nan, device="cuda")
    rope = torch.full((Q * cols, BS, 1, P), math.nan, device="cuda")
    status = kvd.status_tensor()

    # prompts: append, gather, expand, attend
    c, r, qn, qr = m.tokens(sum(prompts))
    lens = cum(prompts)
    kvd.append_latent(latent, rope, table, None, c, r, lens, torch.zeros(Q, dtype=torch.int32,
                                                                         device="cuda"), status)
    gc, gr = kvd.gather_paged(latent, rope, table, lens, dev_status=status)
    assert torch.equal(gc[:, 0], c) and torch.equal(gr[:, 0], r)
    kv = torch.cat([torch.einsum("hdr,nr->nhd", m.uk, gc[:, 0]),
                    torch.einsum("hdr,nr->nhd", m.uv, gc[:, 0])], -1).contiguous()
    out = kvd.attend_expanded(torch.cat([qn, qr], -1).contiguous(), kv, gr[:, 0].contiguous(),
                              lens, lens, m.scale, dev_status=status)
    ends = lens.tolist()
    rows = [c[ends[b]:ends[b + 1]] for b in range(Q)]
    ropes = [r[ends[b]:ends[b + 1]] for b in range(Q)]
    for b in range(Q):
        for i in (0, prompts[b] // 2, prompts[b] - 1):
            want = truth(m, rows[b], ropes[b], qn[ends[b] + i], qr[ends[b] + i], i + 1)
            assert float((out[ends[b] + i].double() - want).abs().max()) <= TOL

    # drafted steps: T + 1 tokens each, then only the accepted ones stay
    have = list(prompts)
    for step in range(4):
        c, r, qn, qr = m.tokens(Q * (T + 1))
        kvd.append_latent(latent, rope, table, None, c, r, cum([T + 1] * Q),
                          torch.tensor(have, dtype=torch.int32, device="cuda"), status)
        full = cum([n + T + 1 for n in have])
        ql = torch.einsum("hdr,nhd->nhr", m.uk, qn).reshape(Q, T + 1, H, R).contiguous()
        out = kvd.attend_latent(ql, qr.reshape(Q, T + 1, H, P).contiguous(), latent, rope, table,
                                full, m.scale, dev_status=status)
        up = torch.einsum("hdr,qthr->qthd", m.uv, out)
        p = torch.softmax(3 * torch.randn(Q, T + 1, V, generator=g, device="cuda"), -1)
        d = torch.softmax(p[:, :T].log() + 0.5 * torch.randn(Q, T, V, generator=g, device="cuda"), -1)
        x = torch.multinomial(d.reshape(-1, V), 1, generator=g).view(Q, T).to(torch.int32)
        u, us = torch.rand(Q, T, generator=g, device="cuda"), torch.rand(Q, generator=g, device="cuda")
        tokens, accepted = kvd.verify_drafts(p, d, x, u, us, dev_status=status)
        for b in range(Q):
            mine = slice(b * (T + 1), (b + 1) * (T + 1))
            rows[b] = torch.cat([rows[b][:have[b]], c[mine]])
            ropes[b] = torch.cat([ropes[b][:have[b]], r[mine]])
            for t in range(T + 1):
                want = truth(m, rows[b], ropes[b], qn[b * (T + 1) + t], qr[b * (T + 1) + t],
                             have[b] + t + 1)
                assert float((up[b, t].double() - want).abs().max()) <= TOL, (step, b, t)
            n = int(accepted[b])
            assert tokens[b, :n].tolist() == x[b, :n].tolist() and tokens[b, n + 1:].tolist() == [-1] * (T - n)
            have[b] += n + 1
    assert int(status.item()) == 0


def test_absorbed_and_expanded_forms_agree_in_bf16(kvd):
    """Both tensor-core paths over the same cache, each against the 64-bit values
    of its own bf16 inputs."""
    g = torch.Generator(device="cuda").manual_seed(6)
    bf, n, T = torch.bfloat16, 333, 5
    m = Model(g)
    c, r, qn, qr = (x.to(bf) for x in m.tokens(n))
    cols = -(-n // BS)
    latent, rope = torch.zeros(cols, BS, 1, R, dtype=bf).cuda(), torch.zeros(cols, BS, 1, P, dtype=bf).cuda()
    table = torch.randperm(cols, generator=g, device="cuda").view(1, cols).to(torch.int32)
    kvd.append_latent(latent, rope, table, None, c, r, cum([n]),
                      torch.zeros(1, dtype=torch.int32, device="cuda"))
    kv = torch.cat([torch.einsum("hdr,nr->nhd", m.uk, c.float()),
                    torch.einsum("hdr,nr->nhd", m.uv, c.float())], -1).to(bf).contiguous()
    q = torch.cat([qn, qr], -1)[-T:].contiguous()
    lse = torch.empty(T, H, device="cuda")
    out = kvd.attend_expanded(q, kv, r, cum([T]), cum([n]), m.scale, lse=lse)
    ql = torch.einsum("hdr,nhd->nhr", m.uk, qn[-T:].float()).to(bf).view(1, T, H, R).contiguous()
    zl = torch.empty(1, T, H, device="cuda")
    ol = kvd.attend_latent(ql, qr[-T:].reshape(1, T, H, P).contiguous(), latent, rope, table,
                           cum([n]), m.scale, lse=zl)
    t = torch.arange(T, device="cuda")
    seen = torch.arange(n, device="cuda")[None] <= (n - T + t)[:, None]
    for h in range(H):
        kh = torch.cat([kv[:, h, :DN], r], 1).double()
        o, z, A, d = ref.attention(q[:, h].double(), kh, kv[:, h, DN:].double(), m.scale, seen)
        ref.check("expanded", out[:, h], lse[:, h], o, z, A, d, n, bf)
        qh = torch.cat([ql[0, :, h], qr[-T:, h]], 1).double()
        o, z, A, d = ref.attention(qh, torch.cat([c, r], 1).double(), c.double(), m.scale, seen)
        ref.check("absorbed", ol[0, :, h], zl[0, :, h], o, z, A, d, n, bf)
    up = torch.einsum("hdr,thr->thd", m.uv, ol[0].float())
    # the forms round different things to bf16 (keys and values here, queries and
    # outputs there): four roundings of 2^-8 of terms whose root sum square is the
    # output's scale
    assert float((up - out.float()).norm() / up.norm()) <= 4 * 2.0 ** -8
