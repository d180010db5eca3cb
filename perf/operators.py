"""Cases of the latent-attention and drafted-decoding operators, with their plain forms.

A serving program with a latent key-value cache keeps one row a token, shared by
all heads: R latent values (keys and values at once) and P rotary key values.
It calls, in this order,

  append     new rows of every sequence into the paged latent cache
  expanded   attention of a prompt (or a chunk of one) over per-head keys and
             values that were expanded from the latent rows: packed sequences,
             causal, the last query of a sequence sees all its keys
  latent     attention of the newest T tokens of every sequence straight over
             the paged latent rows (queries already multiplied into the latent
             space), each token seeing the tokens up to itself
  verify     drafted tokens accepted or replaced by the target's probabilities,
             from given random numbers

Lengths are spread over [lo, hi] by a fixed rule of the case, so that the work
is a function of the case alone; everything else comes from the seed.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one user's decode step: a single sequence, a sixteenth of the heads, latency only
        {"name": "latent_one", "op": "latent", "Q": 1, "T": 1, "H": 16, "R": 512, "BS": 128,
         "lo": 1000, "hi": 1000, "dtype": "bf16"},
        # a served batch of unequal lengths: the cache's bandwidth
        {"name": "latent_batch", "op": "latent", "Q": 64, "T": 1, "H": 16, "R": 512, "BS": 128,
         "lo": 512, "hi": 8192, "dtype": "bf16"},
        # scoring three drafted tokens and the newest one over long caches: 128 rows a sequence
        {"name": "latent_drafts", "op": "latent", "Q": 16, "T": 4, "H": 32, "R": 512, "BS": 64,
         "lo": 1001, "hi": 16384, "dtype": "bf16"},
        # an fp32 check run of a small model
        {"name": "latent_f32", "op": "latent", "Q": 3, "T": 2, "H": 8, "R": 256, "BS": 32,
         "lo": 1, "hi": 2001, "dtype": "f32"},
        # short prompts of a chat turn, ragged
        {"name": "expanded_short", "op": "expanded", "Q": 5, "H": 16, "Dn": 128, "Dv": 128,
         "lo": 17, "hi": 301, "past": 0, "dtype": "bf16"},
        # whole prompts: compute bound
        {"name": "expanded_prompts", "op": "expanded", "Q": 4, "H": 32, "Dn": 128, "Dv": 128,
         "lo": 1024, "hi": 4096, "past": 0, "dtype": "bf16"},
        # a chunk of a prompt behind tokens that are in the cache already, fp32
        {"name": "expanded_chunk_f32", "op": "expanded", "Q": 2, "H": 4, "Dn": 64, "Dv": 64,
         "lo": 100, "hi": 391, "past": 301, "dtype": "f32"},
        # one user's drafted step
        {"name": "verify_one", "op": "verify", "Q": 1, "T": 3, "V": 32000, "dtype": "f32"},
        # a served batch with a large vocabulary
        {"name": "verify_batch", "op": "verify", "Q": 64, "T": 4, "V": 128000, "dtype": "f32"},
        # bf16 probabilities, rows of odd length
        {"name": "verify_bf16", "op": "verify", "Q": 128, "T": 7, "V": 50257, "dtype": "bf16"},
        # the decode step's append
        {"name": "append_step", "op": "append", "Q": 64, "R": 512, "BS": 128, "lo": 1, "hi": 1,
         "dtype": "bf16"},
        # whole prompts into the cache, small pages
        {"name": "append_prompts", "op": "append", "Q": 8, "R": 512, "BS": 16, "lo": 1024,
         "hi": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["latent", "latent", "expanded", "verify", "append"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "latent":
        H, T, R = _log(rng, 1, 128), _log(rng, 1, 8), rng.choice([128, 256, 384, 512, 512])
        BS = rng.choice([16, 32, 48, 64, 128])
        rows = T * H
        Q = _log(rng, 1, 64)
        top = min(16384, 262144 // Q, (16 * 16384 * 128) // (2 * Q * rows))
        if dtype == "f32":
            top = min(top, 2 ** 22 // (Q * rows))
        top = max(top, 8)
        hi = _log(rng, 8, top)
        return {"op": op, "Q": Q, "T": T, "H": H, "R": R, "BS": BS, "lo": rng.randint(1, hi),
                "hi": hi, "dtype": dtype}
    if op == "expanded":
        Dn, Dv = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64)])
        H, Q = _log(rng, 1, 32), _log(rng, 1, 8)
        most = 8 * 4 * 4096 ** 2 if dtype == "bf16" else 2 ** 24
        hi = _log(rng, 4, min(4096, max(4, int(math.sqrt(most / (H * Q))))))
        past = rng.choice([0, 0, _log(rng, 1, 1024)])
        if (hi + past) * hi * H * Q > most:
            past = 0
        return {"op": op, "Q": Q, "H": H, "Dn": Dn, "Dv": Dv, "lo": rng.randint(1, hi), "hi": hi,
                "past": past, "dtype": dtype}
    if op == "verify":
        Q, T = _log(rng, 1, 96), rng.randint(1, 7)
        V = _log(rng, 1000, min(200000, 64 * 5 * 128000 // (Q * (T + 1))))
        return {"op": op, "Q": Q, "T": T, "V": V, "dtype": dtype}
    hi = _log(rng, 1, 4096)
    return {"op": op, "Q": _log(rng, 1, 16384 // max(hi, 128)), "R": rng.choice([128, 256, 384, 512]),
            "BS": rng.choice([16, 32, 48, 64, 128]), "lo": rng.randint(1, hi), "hi": hi,
            "dtype": dtype}


_P = 64  # rotary key values of a token


def _lens(case):
    """Q lengths over [lo, hi]: the first is hi, the others spread by a fixed multiplicative rule."""
    lo, hi = case["lo"], case["hi"]
    return [hi - (i * 2654435761 >> 7) % (hi - lo + 1) if i else hi for i in range(case["Q"])]


def _pages(lens, BS, g, dev):
    """Random pages for sequences of these lengths: (block_tables, number of pages)."""
    cols = max(-(-n // BS) for n in lens)
    total = sum(-(-n // BS) for n in lens)
    NB = total + 3
    order = torch.randperm(NB, generator=g, device=dev).to(torch.int32)
    need = torch.tensor([-(-n // BS) for n in lens], device=dev)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(cols, device=dev)
    at = first[:, None] + col[None, :]
    table = torch.where(col[None, :] < need[:, None], order[at.clamp(max=NB - 1)].long(), 0)
    return table.to(torch.int32).contiguous(), NB


def _cumsum(lens, dev):
    return torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 17)

    def normal(*shape, s=1.0, dt=torch.float32):
        return (torch.randn(shape, generator=g, device=dev) * s).to(dt)

    op, Q = case["op"], case["Q"]
    dt = _DT[case["dtype"]]
    st = {"case": case}
    if op == "latent":
        T, H, R, BS = case["T"], case["H"], case["R"], case["BS"]
        lens = [max(n, T) for n in _lens(case)]
        st["table"], NB = _pages(lens, BS, g, dev)
        st["latent"] = normal(NB, BS, 1, R, dt=dt)
        st["rope"] = normal(NB, BS, 1, _P, dt=dt)
        st["ql"] = normal(Q, T, H, R, dt=dt)
        st["qr"] = normal(Q, T, H, _P, dt=dt)
        st["lens"] = _cumsum(lens, dev)
        st["longest"] = max(lens)
        st["scale"] = 1.0 / math.sqrt(R + _P)
        if own:  # the workspace that a serving program allocates once and keeps
            from decode_attention_kv_gb300 import kvd
            st["workspace"] = kvd.workspace(
                kvd.attend_latent_workspace_bytes(Q, T, H, BS, st["table"].shape[1], R, _P, dt))
    elif op == "expanded":
        H, Dn, Dv = case["H"], case["Dn"], case["Dv"]
        ql = _lens(case)
        kl = [n + case["past"] for n in ql]
        st["q"] = normal(sum(ql), H, Dn + _P, dt=dt)
        st["kv"] = normal(sum(kl), H, Dn + Dv, dt=dt)
        st["kr"] = normal(sum(kl), _P, dt=dt)
        st["qlens"], st["klens"] = _cumsum(ql, dev), _cumsum(kl, dev)
        st["scale"] = 1.0 / math.sqrt(Dn + _P)
        st["most"] = (max(ql), max(kl))
        # which sequence every packed query belongs to, and its place there
        st["seq"] = torch.repeat_interleave(torch.arange(Q, device=dev),
                                            torch.tensor(ql, device=dev))
        st["at"] = torch.arange(sum(ql), device=dev) - st["qlens"].long()[st["seq"]]
    elif op == "verify":
        T, V = case["T"], case["V"]
        logits = normal(Q, T + 1, V, s=3.0)
        st["target"] = torch.softmax(logits, -1).to(dt)
        # the draft model is nearly right: three drafts in four or so are accepted
        draft = torch.softmax(logits[:, :T] + normal(Q, T, V, s=0.3), -1)
        st["draft"] = draft.to(dt)
        noise = torch.rand((Q, T, V), generator=g, device=dev).clamp_(min=1e-20)
        st["tokens"] = (draft.log() - (-noise.log()).log()).argmax(-1).to(torch.int32)
        st["u"] = torch.rand((Q, T), generator=g, device=dev)
        st["us"] = torch.rand((Q,), generator=g, device=dev)
    else:
        R, BS = case["R"], case["BS"]
        new = _lens(case)
        pos = torch.randint(0, 300, (Q,), generator=g, device=dev).to(torch.int32)
        # pages for the longest a sequence may come to be
        st["table"], NB = _pages([n + 299 for n in new], BS, g, dev)
        st["pos"] = pos
        st["latent"] = normal(NB, BS, 1, R, dt=dt)
        st["rope"] = normal(NB, BS, 1, _P, dt=dt)
        st["cn"] = normal(sum(new), R, dt=dt)
        st["rn"] = normal(sum(new), _P, dt=dt)
        st["new"] = _cumsum(new, dev)
        st["seq"] = torch.repeat_interleave(torch.arange(Q, device=dev),
                                            torch.tensor(new, device=dev))
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _own(op, st)
    if op == "latent":
        return _latent(st)
    if op == "expanded":
        return _expanded(st)
    if op == "verify":
        return _verify(st)
    return _append(st)


def _own(op, st):
    from decode_attention_kv_gb300 import kvd
    if op == "latent":
        Q, T, H, _ = st["ql"].shape
        lse = torch.empty((Q, T, H), dtype=torch.float32, device="cuda")
        out = kvd.attend_latent(st["ql"], st["qr"], st["latent"], st["rope"], st["table"],
                                st["lens"], st["scale"], lse=lse, workspace=st["workspace"])
        return {"out": out, "lse": lse}
    if op == "expanded":
        N, H, _ = st["q"].shape
        lse = torch.empty((N, H), dtype=torch.float32, device="cuda")
        out = kvd.attend_expanded(st["q"], st["kv"], st["kr"], st["qlens"], st["klens"],
                                  st["scale"], lse=lse)
        return {"out": out, "lse": lse}
    if op == "verify":
        tokens, accepted = kvd.verify_drafts(st["target"], st["draft"], st["tokens"], st["u"],
                                             st["us"])
        return {"tokens": tokens, "accepted": accepted}
    kvd.append_latent(st["latent"], st["rope"], st["table"], None, st["cn"], st["rn"], st["new"],
                      st["pos"])
    return {"latent": st["latent"], "rope": st["rope"]}


def _softmax_sums(s, seen):
    """Weights of a masked softmax and their log-sum-exp; a row that sees nothing gets zeros and -inf."""
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - top.masked_fill(top == -math.inf, 0.0))
    total = e.sum(-1, keepdim=True)
    lse = (torch.log(total) + top).squeeze(-1)
    return e / total.clamp(min=1e-38), lse


def _latent(st):
    dt = st["ql"].dtype
    Q, T, H, R = st["ql"].shape
    BS = st["latent"].shape[1]
    dev = st["ql"].device
    t = torch.arange(st["longest"], device=dev)
    rows = st["table"].long()[:, t // BS] * BS + t % BS                    # [Q, L]
    c = st["latent"].reshape(-1, R)[rows].float()                          # [Q, L, R]
    r = st["rope"].reshape(-1, _P)[rows].float()
    s = st["ql"].float().reshape(Q, T * H, R) @ c.transpose(1, 2)
    s = (s + st["qr"].float().reshape(Q, T * H, _P) @ r.transpose(1, 2)) * st["scale"]
    n = (st["lens"][1:] - st["lens"][:-1]).long()
    last = n[:, None] - T + torch.arange(T, device=dev)                    # newest token seen
    seen = (t <= last[:, :, None]).repeat_interleave(H, 1)                 # [Q, T*H, L]
    w, lse = _softmax_sums(s, seen)
    out = w @ c.masked_fill((t >= n[:, None])[:, :, None], 0.0)
    return {"out": out.reshape(Q, T, H, R).to(dt), "lse": lse.reshape(Q, T, H)}


def _expanded(st):
    dt = st["q"].dtype
    Lq, Lk = st["most"]
    N, H, Dqk = st["q"].shape
    Dn = Dqk - _P
    dev = st["q"].device
    q0, k0 = st["qlens"].long()[:-1], st["klens"].long()[:-1]
    nq, nk = st["qlens"].long()[1:] - q0, st["klens"].long()[1:] - k0
    i, j = torch.arange(Lq, device=dev), torch.arange(Lk, device=dev)
    qi = (q0[:, None] + i).clamp(max=N - 1)
    kj = (k0[:, None] + j).clamp(max=st["kv"].shape[0] - 1)
    q = st["q"][qi].float().transpose(1, 2)                                # [Q, H, Lq, D]
    kv = st["kv"][kj].float().transpose(1, 2)                              # [Q, H, Lk, Dn+Dv]
    kr = st["kr"][kj].float()[:, None]                                     # [Q, 1, Lk, P]
    s = q[..., :Dn] @ kv[..., :Dn].transpose(2, 3) + q[..., Dn:] @ kr.transpose(2, 3)
    s *= st["scale"]
    seen = j <= i[:, None] + (nk - nq)[:, None, None]                      # [Q, Lq, Lk]
    w, lse = _softmax_sums(s, seen[:, None])
    out = w @ kv[..., Dn:]                                                 # [Q, H, Lq, Dv]
    seq, at = st["seq"], st["at"]
    return {"out": out[seq, :, at].to(dt).contiguous(), "lse": lse[seq, :, at].contiguous()}


def _verify(st):
    p, q, x = st["target"], st["draft"], st["tokens"].long()
    Q, T, V = q.shape
    b = torch.arange(Q, device=p.device)
    px = p[:, :T].gather(2, x[..., None])[..., 0].double()
    qx = q.gather(2, x[..., None])[..., 0].double()
    ok = st["u"].double() * qx < px
    n = ok.long().cumprod(1).sum(1)                                        # accepted drafts
    w = p[b, n].double()
    rest = (w - q[b, n.clamp(max=T - 1)].double()).clamp(min=0.0)
    rest = torch.where((rest.sum(1) > 0)[:, None], rest, w)                # nothing left: the target itself
    w = torch.where((n < T)[:, None], rest, w)
    cum = w.cumsum(1)
    hit = cum > st["us"].double()[:, None] * cum[:, -1:]
    token = hit.long().argmax(1)
    at = torch.arange(T + 1, device=p.device)
    drafts = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(at < n[:, None], drafts, torch.where(at == n[:, None], token[:, None], -1))
    return {"tokens": tokens.to(torch.int32), "accepted": n.to(torch.int32)}


def _append(st):
    BS = st["latent"].shape[1]
    seq = st["seq"]
    t = torch.arange(seq.numel(), device=seq.device) - st["new"].long()[seq] + st["pos"].long()[seq]
    rows = st["table"].long()[seq, t // BS] * BS + t % BS
    st["latent"].view(-1, st["latent"].shape[-1])[rows] = st["cn"]
    st["rope"].view(-1, _P)[rows] = st["rn"]
    return {"latent": st["latent"], "rope": st["rope"]}


# ------------------------------------------------------------------ the work

def work(case):
    es, op, Q = _ES[case["dtype"]], case["op"], case["Q"]
    if op == "latent":
        T, H, R = case["T"], case["H"], case["R"]
        lens = [max(n, T) for n in _lens(case)]
        seen = sum(T * n - T * (T - 1) // 2 for n in lens)
        io = Q * T * H * ((2 * R + _P) * es + 4)
        return {"bytes": sum(lens) * (R + _P) * es + io, "flops": 2 * H * seen * (2 * R + _P)}
    if op == "expanded":
        H, Dn, Dv, past = case["H"], case["Dn"], case["Dv"], case["past"]
        ql = _lens(case)
        seen = sum(n * past + n * (n + 1) // 2 for n in ql)
        nq, nk = sum(ql), sum(ql) + Q * past
        nbytes = (nq * H * (Dn + _P + Dv) + nk * (H * (Dn + Dv) + _P)) * es + nq * H * 4
        return {"bytes": nbytes, "flops": 2 * H * seen * (Dn + _P + Dv)}
    if op == "verify":
        # one row of each distribution a sequence decides the replaced token
        return {"bytes": Q * (2 * case["V"] * es + case["T"] * (2 * es + 8) + 4 * case["T"] + 12),
                "flops": 4 * Q * case["V"]}
    n = sum(_lens(case))
    return {"bytes": 2 * n * (case["R"] + _P) * es, "flops": 0}


# ------------------------------------------------------------------ 64 bits, by the definitions

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "latent":
        Q, T, H, R = st["ql"].shape
        BS = st["latent"].shape[1]
        ends = st["lens"].tolist()
        out = torch.empty((Q, T, H, R), dtype=torch.float64, device="cuda")
        lse = torch.empty((Q, T, H), dtype=torch.float64, device="cuda")
        for b in range(Q):
            n = ends[b + 1] - ends[b]
            pages = st["table"][b, : -(-n // BS)].long()
            c = st["latent"][pages].reshape(-1, R)[:n].double()
            k = torch.cat([c, st["rope"][pages].reshape(-1, _P)[:n].double()], 1)
            for t in range(T):
                m = n - T + 1 + t
                qt = torch.cat([st["ql"][b, t], st["qr"][b, t]], 1).double()
                s = st["scale"] * (qt @ k[:m].T)
                lse[b, t] = torch.logsumexp(s, 1)
                out[b, t] = torch.exp(s - lse[b, t][:, None]) @ c[:m]
        return {"out": out, "lse": lse}
    if op == "expanded":
        N, H, D = st["q"].shape
        Dn, Dv = case["Dn"], case["Dv"]
        qe, ke = st["qlens"].tolist(), st["klens"].tolist()
        out = torch.empty((N, H, Dv), dtype=torch.float64, device="cuda")
        lse = torch.empty((N, H), dtype=torch.float64, device="cuda")
        for b in range(case["Q"]):
            nq, nk = qe[b + 1] - qe[b], ke[b + 1] - ke[b]
            kr = st["kr"][ke[b]:ke[b + 1]].double()
            hide = torch.ones((nq, nk), dtype=torch.bool, device="cuda").triu(nk - nq + 1)
            for h in range(H):
                kv = st["kv"][ke[b]:ke[b + 1], h].double()
                q = st["q"][qe[b]:qe[b + 1], h].double()
                s = st["scale"] * (q @ torch.cat([kv[:, :Dn], kr], 1).T)
                s[hide] = -math.inf
                z = torch.logsumexp(s, 1)
                lse[qe[b]:qe[b + 1], h] = z
                out[qe[b]:qe[b + 1], h] = torch.exp(s - z[:, None]) @ kv[:, Dn:]
        return {"out": out, "lse": lse}
    if op == "verify":
        Q, T, V = st["draft"].shape
        x, u, us = st["tokens"].tolist(), st["u"].tolist(), st["us"].tolist()
        tokens = torch.full((Q, T + 1), -1, dtype=torch.int32)
        accepted = torch.zeros(Q, dtype=torch.int32)
        for b in range(Q):
            p, q = st["target"][b].double().cpu(), st["draft"][b].double().cpu()
            n = 0
            while n < T and u[b][n] * float(q[n, x[b][n]]) < float(p[n, x[b][n]]):
                tokens[b, n] = x[b][n]
                n += 1
            w = p[n]
            if n < T:
                rest = torch.relu(p[n] - q[n])
                w = rest if float(rest.sum()) > 0 else w
            cum = torch.cumsum(w, 0)
            at = int(torch.searchsorted(cum, us[b] * float(cum[-1]), right=True))
            tokens[b, n] = min(at, int(torch.nonzero(w).max()))
            accepted[b] = n
        return {"tokens": tokens, "accepted": accepted}
    BS = case["BS"]
    c, r = st["latent"].double(), st["rope"].double()
    ends, pos = st["new"].tolist(), st["pos"].tolist()
    for b in range(case["Q"]):
        n = ends[b + 1] - ends[b]
        t = torch.arange(pos[b], pos[b] + n, device="cuda")
        page, slot = st["table"][b].long()[t // BS], t % BS
        c[page, slot, 0] = st["cn"][ends[b]:ends[b + 1]].double()
        r[page, slot, 0] = st["rn"][ends[b]:ends[b + 1]].double()
    return {"latent": c, "rope": r}
