"""Cases of a serving step's operators around the paged cache, with their plain forms.

A program that serves many requests from a paged key-value cache makes these
calls in every step:

  plan    pages for the step's new tokens taken from the free list (or given back
          to it), block tables, slots and positions on the GPU, from the requests'
          lengths alone
  rotate  the fused projection's queries and keys normed a head and rotated by
          position, queries into a tensor, keys and values into their slots
  prefix  one query token a sequence over a prefix that a group of sequences
          shares, kept once, and over the sequence's own pages
  sample  a token a row from logits: temperature, top-k, top-p, min-p, from given
          random numbers
  probs   the same filters as probabilities, which drafted decoding compares

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
        # a decode step of a served batch: a token each, a page now and then
        {"name": "plan_step", "op": "plan", "Q": 64, "BS": 16, "klo": 512, "khi": 8192,
         "lo": 1, "hi": 1, "short": False},
        # many new requests at once, small pages, more than the pool holds
        {"name": "plan_prompts", "op": "plan", "Q": 1024, "BS": 16, "klo": 0, "khi": 0,
         "lo": 1, "hi": 127, "short": True},
        # a decode step's projections
        {"name": "rotate_step", "op": "rotate", "N": 64, "Hq": 32, "Hkv": 8, "D": 128, "Dr": 128,
         "half": True, "norm": True, "far": 8192, "BS": 128, "dtype": "bf16"},
        # prompts: the memory's bandwidth
        {"name": "rotate_prompts", "op": "rotate", "N": 8192, "Hq": 32, "Hkv": 8, "D": 128,
         "Dr": 128, "half": True, "norm": True, "far": 32768, "BS": 128, "dtype": "bf16"},
        # a small model's check run: part of the head, interleaved pairs, far positions
        {"name": "rotate_f32", "op": "rotate", "N": 1001, "Hq": 8, "Hkv": 2, "D": 64, "Dr": 32,
         "half": False, "norm": False, "far": 1000000, "BS": 16, "dtype": "f32"},
        # a few users behind one system prompt: latency
        {"name": "prefix_few", "op": "prefix", "Q": 4, "G": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "BS": 16, "P": 1000, "lo": 1, "hi": 64, "dtype": "bf16"},
        # a served batch behind one long prompt, own turns of unequal lengths
        {"name": "prefix_batch", "op": "prefix", "Q": 64, "G": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "BS": 128, "P": 16384, "lo": 64, "hi": 1024, "dtype": "bf16"},
        # an fp32 check run of a small model, two prompts in one batch
        {"name": "prefix_f32", "op": "prefix", "Q": 9, "G": 2, "Hq": 8, "Hkv": 2, "D": 64,
         "BS": 32, "P": 515, "lo": 1, "hi": 200, "dtype": "f32"},
        # one user's token
        {"name": "sample_one", "op": "sample", "R": 1, "V": 32000, "use": "kpm", "dtype": "f32"},
        # a served batch with a large vocabulary, every row with settings of its own
        {"name": "sample_batch", "op": "sample", "R": 64, "V": 128000, "use": "kpm",
         "dtype": "f32"},
        # the target's rows of one drafted step
        {"name": "probs_drafts", "op": "probs", "R": 4, "V": 32000, "use": "p", "dtype": "f32"},
        # drafted steps of a batch in bf16: logits with many ties, rows of odd length
        {"name": "probs_batch", "op": "probs", "R": 96, "V": 50257, "use": "kpm",
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rotate", "rotate", "prefix", "prefix", "prefix", "sample", "sample",
                     "probs"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "plan":
        Q = _log(rng, 1, 1024)
        hi = _log(rng, 1, 131072 // Q)
        khi = rng.choice([0, _log(rng, 1, 8192)])
        return {"op": op, "Q": Q, "BS": rng.choice([1, 16, 24, 64, 128]), "klo": khi // 3,
                "khi": khi, "lo": rng.randint(0, hi), "hi": hi, "short": rng.random() < 0.3}
    if op == "rotate":
        Hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4])
        D = rng.choice([64, 128])
        N = _log(rng, 1, min(8192, 8192 * 48 * 128 * 2 // ((g + 2) * Hkv * D * _ES[dtype])))
        return {"op": op, "N": N, "Hq": Hkv * g, "Hkv": Hkv,
                "D": D, "Dr": rng.choice([16, D // 2, D]), "half": rng.random() < 0.6,
                "norm": rng.random() < 0.6, "far": _log(rng, 16, 1000000),
                "BS": rng.choice([16, 24, 64, 128]), "dtype": dtype}
    if op == "prefix":
        Hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        D = rng.choice([64, 128])
        Q = _log(rng, 1, 64)
        most = 64 * 32 * 16384 if dtype == "bf16" else 64 * 4 * 1024
        top = max(32, min(16384, most // (Q * Hkv * g)))
        P = _log(rng, 16, top)
        hi = _log(rng, 1, min(768, max(2, top // 8)))
        return {"op": op, "Q": Q, "G": rng.randint(1, min(4, Q)), "Hq": Hkv * g, "Hkv": Hkv,
                "D": D, "BS": rng.choice([16, 24, 32, 64, 128]), "P": P,
                "lo": rng.randint(0, hi), "hi": hi, "dtype": dtype}
    R = _log(rng, 1, 64)
    return {"op": op, "R": R, "V": _log(rng, 1000, min(200000, 64 * 128000 // R)),
            "use": rng.choice(["", "k", "p", "m", "kp", "kpm"]), "dtype": dtype}


def _lens(n, lo, hi):
    """n lengths over [lo, hi]: the first is hi, the others spread by a fixed multiplicative rule."""
    return [hi - (i * 2654435761 >> 7) % (hi - lo + 1) if i else hi for i in range(n)]


def _groups(case):
    """Sequences of each group, as even as they come."""
    Q, G = case["Q"], case["G"]
    return [Q // G + (i < Q % G) for i in range(G)]


def _prefix_lens(case):
    return [max(1, case["P"] * (4 - i) // 4) for i in range(case["G"])]


def _pages(lens, BS, g, dev, spare=3):
    """Random pages for lists of these lengths: (block_tables, number of pages)."""
    cols = max(1, max(-(-n // BS) for n in lens))
    total = sum(-(-n // BS) for n in lens)
    NB = total + spare
    order = torch.randperm(NB, generator=g, device=dev).to(torch.int32)
    need = torch.tensor([-(-n // BS) for n in lens], device=dev)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(cols, device=dev)
    at = first[:, None] + col[None, :]
    table = torch.where(col[None, :] < need[:, None], order[at.clamp(max=NB - 1)].long(), 0)
    return table.to(torch.int32).contiguous(), NB


def _i32(x, dev):
    return torch.tensor(x, device=dev, dtype=torch.int32)


def _cumsum(lens, dev):
    return torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 29)

    def normal(*shape, s=1.0, dt=torch.float32):
        return (torch.randn(shape, generator=g, device=dev) * s).to(dt)

    def uniform(n, lo, hi):
        return torch.rand((n,), generator=g, device=dev) * (hi - lo) + lo

    op = case["op"]
    st = {"case": case}
    if op == "plan":
        Q, BS = case["Q"], case["BS"]
        kept, new = _lens(Q, case["klo"], case["khi"]), _lens(Q, case["lo"], case["hi"])
        held = [-(-k // BS) for k in kept]
        need = [-(-(k + n) // BS) for k, n in zip(kept, new)]
        grow = sum(need) - sum(held)
        cols = max(need) + 2
        F = sum(held) + (grow * 3 // 4 if case["short"] else grow + 5)
        order = torch.randperm(F, generator=g, device=dev).to(torch.int32)
        st["table"] = torch.full((Q, cols), -1, dtype=torch.int32, device=dev)
        have = torch.arange(cols, device=dev) < torch.tensor(held, device=dev)[:, None]
        st["table"][have] = order[:sum(held)]
        st["held"] = _i32(held, dev)
        st["free"] = torch.zeros(F, dtype=torch.int32, device=dev)
        st["free"][:F - sum(held)] = order[sum(held):]
        st["count"] = _i32([F - sum(held)], dev)
        st["kept"], st["new"] = _i32(kept, dev), _cumsum(new, dev)
        st["none"] = torch.zeros(Q + 1, dtype=torch.int32, device=dev)
        st["base"] = torch.randint(0, 1000, (Q,), generator=g, device=dev).to(torch.int32)
        st["N"] = sum(new)
        return st
    if op == "rotate":
        dt = _DT[case["dtype"]]
        N, Hq, Hkv, D, Dr, BS = (case[k] for k in ("N", "Hq", "Hkv", "D", "Dr", "BS"))
        NB = -(-N // BS) + 3
        st["qkv"] = normal(N, Hq + 2 * Hkv, D, dt=dt)
        st["kc"] = normal(NB, BS, Hkv, D, dt=dt)
        st["vc"] = normal(NB, BS, Hkv, D, dt=dt)
        st["wq"] = (1 + normal(D, s=0.1)).to(dt) if case["norm"] else None
        st["wk"] = (1 + normal(D, s=0.1)).to(dt) if case["norm"] else None
        i = torch.arange(Dr // 2, device=dev, dtype=torch.float64)
        st["freqs"] = 500000.0 ** (-2.0 * i / Dr) / 4.0          # positions brought closer by 4
        st["stretch"] = 0.1 * math.log(4.0) + 1.0
        st["pos"] = torch.randint(0, case["far"], (N,), generator=g, device=dev).to(torch.int32)
        st["slots"] = torch.randperm(NB * BS, generator=g, device=dev)[:N].to(torch.int32)
        return st
    if op == "prefix":
        dt = _DT[case["dtype"]]
        Q, G, Hq, Hkv, D, BS = (case[k] for k in ("Q", "G", "Hq", "Hkv", "D", "BS"))
        own_lens, pre = _lens(Q, case["lo"], case["hi"]), _prefix_lens(case)
        both, NB = _pages(pre + own_lens, BS, g, dev)
        pc, oc = max(-(-n // BS) for n in pre), max(1, max(-(-n // BS) for n in own_lens))
        st["ptable"] = both[:G, :pc].contiguous()
        st["table"] = both[G:, :oc].contiguous()
        st["kc"] = normal(NB, BS, Hkv, D, s=0.5, dt=dt)
        st["vc"] = normal(NB, BS, Hkv, D, dt=dt)
        st["q"] = normal(Q, Hq, D, dt=dt)
        st["plens"], st["lens"] = _i32(pre, dev), _cumsum(own_lens, dev)
        st["groups"] = _cumsum(_groups(case), dev)
        st["longest"] = max(own_lens)
        st["scale"] = 1.0 / math.sqrt(D)
        if own:  # the workspace that a serving program allocates once and keeps
            from decode_attention_kv_gb300 import kvd
            st["workspace"] = kvd.workspace(kvd.attend_paged_prefix_workspace_bytes(
                Q, G, Hq, Hkv, BS, pc, oc, D, dt))
        return st
    R, V, use = case["R"], case["V"], case["use"]
    st["logits"] = normal(R, V, s=3.0, dt=_DT[case["dtype"]])
    pick = torch.rand((5, R), generator=g, device=dev)
    temp = uniform(R, 0.5, 1.3)
    # one row in sixteen is greedy, one in four does without one of the filters
    st["temp"] = torch.where(pick[0] < 0.0625, torch.zeros_like(temp), temp)
    k = torch.exp(uniform(R, 0.0, math.log(1000.0))).to(torch.int32)
    st["k"] = torch.where(pick[1] < 0.25, torch.zeros_like(k), k) if "k" in use else None
    p = uniform(R, 0.5, 0.999)
    st["p"] = torch.where(pick[2] < 0.25, torch.ones_like(p), p) if "p" in use else None
    m = uniform(R, 0.001, 0.1)
    st["m"] = torch.where(pick[3] < 0.25, torch.zeros_like(m), m) if "m" in use else None
    st["u"] = pick[4].contiguous()
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _own(op, st)
    return {"plan": _plan_twice, "rotate": _rotate, "prefix": _prefix, "sample": _sample,
            "probs": _probs}[op](st)


def _own(op, st):
    from decode_attention_kv_gb300 import kvd
    if op == "plan":
        # the step's tokens, then a step that keeps none of them
        state = (st["table"], st["held"], st["free"], st["count"])
        BS = st["case"]["BS"]
        lens, slots, pos = kvd.plan_pages(*state, st["kept"], st["new"], BS, st["N"],
                                          pos_base=st["base"])
        back, _, _ = kvd.plan_pages(*state, st["kept"], st["none"], BS, 0)
        return {"lens": lens, "slots": slots, "pos": pos, "back": back, "table": st["table"],
                "held": st["held"], "free": st["free"], "count": st["count"]}
    if op == "rotate":
        c = st["case"]
        q = kvd.rotate_append_paged(st["qkv"], st["kc"], st["vc"], st["slots"], st["pos"],
                                    st["freqs"], q_weight=st["wq"], k_weight=st["wk"], eps=1e-6,
                                    interleaved=not c["half"], rotary_scale=st["stretch"])
        return {"q": q, "kc": st["kc"], "vc": st["vc"]}
    if op == "prefix":
        Q, Hq, _ = st["q"].shape
        lse = torch.empty((Q, Hq), dtype=torch.float32, device="cuda")
        out = kvd.attend_paged_prefix(st["q"], st["kc"], st["vc"], st["ptable"], st["plens"],
                                      st["groups"], st["table"], st["lens"], scale=st["scale"],
                                      lse=lse, workspace=st["workspace"])
        return {"out": out, "lse": lse}
    if op == "sample":
        return {"tokens": kvd.sample(st["logits"], st["u"], temperature=st["temp"], top_k=st["k"],
                                     top_p=st["p"], min_p=st["m"])}
    return {"probs": kvd.filter_probs(st["logits"], temperature=st["temp"], top_k=st["k"],
                                      top_p=st["p"], min_p=st["m"])}


def _plan_twice(st):
    lens, slots, pos = _plan(st, st["kept"], st["new"], st["N"], st["base"])
    back, _, _ = _plan(st, st["kept"], st["none"], 0, None)
    return {"lens": lens, "slots": slots, "pos": pos, "back": back, "table": st["table"],
            "held": st["held"], "free": st["free"], "count": st["count"]}


def _plan(st, kept, new, N, base):
    """Pages for kept + new tokens a sequence, in sequence order, from the free list's end."""
    BS, table, free = st["case"]["BS"], st["table"], st["free"]
    Q, cols = table.shape
    dev = table.device
    kept, held = kept.long(), st["held"].long()
    n = (new[1:] - new[:-1]).long()
    need = (kept + n + BS - 1) // BS
    grow, give = (need - held).clamp(min=0), (held - need).clamp(min=0)
    count = st["count"].long()
    col = torch.arange(cols, device=dev)
    # given back, the last sequence's last page first
    end = give.flip(0).cumsum(0).flip(0)                      # given by this sequence and those behind
    back = (col >= need[:, None]) & (col < held[:, None])
    at = count + (end - give)[:, None] + (held[:, None] - 1 - col)
    at = torch.where(back, at, free.numel())                  # a place behind the list for the others
    pool = torch.cat([free, free.new_zeros(1)])
    pool[at.reshape(-1)] = table.reshape(-1)
    free.copy_(pool[:-1])
    count = count + end[:1]
    # taken: in order, as long as there are enough
    run = grow.cumsum(0)
    served = (grow == 0) | ((run <= count) & (need <= cols))
    grow = torch.where(served, grow, 0)
    take = (col >= held[:, None]) & (col < (held + grow)[:, None])
    at = count - 1 - ((run - grow)[:, None] + col - held[:, None])
    table.copy_(torch.where(take, free[at.clamp(0, free.numel() - 1)], table))
    st["held"].copy_(torch.where(served, need, held))
    st["count"].copy_(count - grow.sum())
    total = torch.where(served, kept + n, kept)
    lens = torch.cat([total.new_zeros(1), total.cumsum(0)]).to(torch.int32)
    i = torch.arange(N, device=dev)
    seq = torch.searchsorted(new[1:].long(), i, right=True)
    t = i - new.long()[seq] + kept[seq]
    ok = served[seq]
    slots = table.long()[seq, (t // BS).clamp(max=cols - 1)] * BS + t % BS
    if base is not None:
        t = t + base.long()[seq]
    minus = torch.full_like(t, -1)
    return (lens, torch.where(ok, slots, minus).to(torch.int32),
            torch.where(ok, t, minus).to(torch.int32))


def _turn(x, weight, st):
    """Norm over the head, then the rotation; fp32."""
    c = st["case"]
    Dr = c["Dr"]
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = st["pos"].double()[:, None] * st["freqs"][None, :]  # far positions: 64 bits
    cos = (torch.cos(angle) * st["stretch"]).float()[:, None]
    sin = (torch.sin(angle) * st["stretch"]).float()[:, None]
    if c["half"]:
        a, b = x[..., :Dr // 2], x[..., Dr // 2:Dr]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:Dr:2], x[..., 1:Dr:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., Dr:]], -1)


def _rotate(st):
    c = st["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    dt = st["qkv"].dtype
    x = st["qkv"].float()
    q = _turn(x[:, :Hq], st["wq"], st).to(dt)
    k = _turn(x[:, Hq:Hq + Hkv], st["wk"], st).to(dt)
    rows = st["slots"].long()
    st["kc"].view(-1, Hkv, D)[rows] = k
    st["vc"].view(-1, Hkv, D)[rows] = st["qkv"][:, Hq + Hkv:]
    return {"q": q, "kc": st["kc"], "vc": st["vc"]}


def _prefix(st):
    c = st["case"]
    Q, Hq, D = st["q"].shape
    Hkv, BS = c["Hkv"], c["BS"]
    g = Hq // Hkv
    dev = st["q"].device
    kf, vf = st["kc"].reshape(-1, Hkv, D), st["vc"].reshape(-1, Hkv, D)
    q = st["q"].float().reshape(Q, Hkv, g, D)
    # a sequence's own keys
    t = torch.arange(st["longest"], device=dev)
    rows = st["table"].long()[:, t // BS] * BS + t % BS                   # [Q, L]
    n = (st["lens"][1:] - st["lens"][:-1]).long()
    k = kf[rows].float().permute(0, 2, 3, 1)                             # [Q, Hkv, D, L]
    s = (q @ k) * st["scale"]
    s = s.masked_fill((t >= n[:, None])[:, None, None], -math.inf)       # [Q, Hkv, g, L]
    v = vf[rows].float().transpose(1, 2)                                 # [Q, Hkv, L, D]
    outs, lses = [], []
    s0 = 0
    for i, (m, P) in enumerate(zip(_groups(c), _prefix_lens(c))):
        t = torch.arange(P, device=dev)
        rows = st["ptable"].long()[i, t // BS] * BS + t % BS
        pk = kf[rows].float().permute(1, 2, 0)                           # [Hkv, D, P]
        pv = vf[rows].float().transpose(0, 1)                            # [Hkv, P, D]
        qi = q[s0:s0 + m].transpose(0, 1).reshape(Hkv, m * g, D)
        ps = (qi @ pk * st["scale"]).reshape(Hkv, m, g, P).transpose(0, 1)
        si = s[s0:s0 + m]
        top = torch.maximum(ps.amax(-1, keepdim=True), si.amax(-1, keepdim=True)
                            if si.shape[-1] else ps.amax(-1, keepdim=True))
        pe, e = torch.exp(ps - top), torch.exp(si - top)
        total = pe.sum(-1, keepdim=True) + e.sum(-1, keepdim=True)
        o = (pe.transpose(0, 1).reshape(Hkv, m * g, P) @ pv).reshape(Hkv, m, g, D).transpose(0, 1)
        o = (o + e @ v[s0:s0 + m]) / total
        outs.append(o.reshape(m, Hq, D))
        lses.append((torch.log(total) + top).reshape(m, Hq))
        s0 += m
    return {"out": torch.cat(outs).to(st["q"].dtype), "lse": torch.cat(lses)}


def _kept(st):
    """Rows in falling order: (weights in 64 bits, zero where a filter drops them; the order)."""
    x, R, V = st["logits"].double(), *st["logits"].shape
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    at = torch.arange(V, device=x.device)
    temp = st["temp"].double()[:, None]
    greedy = temp == 0
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, torch.ones_like(temp), temp))
    keep = ~greedy | (at == 0)
    if st["k"] is not None:
        k = st["k"].long()[:, None]
        keep &= (k <= 0) | (at < k)
    w = w * keep
    if st["p"] is not None:
        p = st["p"].double()[:, None]
        run = w.cumsum(1)
        keep &= (p >= 1) | (run - w < p * run[:, -1:])
    if st["m"] is not None:
        keep &= w >= st["m"].double()[:, None]
    keep[:, 0] = True
    return w * keep, order


def _sample(st):
    w, order = _kept(st)
    w = torch.zeros_like(w).scatter_(1, order, w)
    run = w.cumsum(1)
    above = run > st["u"].double()[:, None] * run[:, -1:]
    return {"tokens": above.long().argmax(1).to(torch.int32)}


def _probs(st):
    w, order = _kept(st)
    p = torch.zeros_like(w).scatter_(1, order, w / w.sum(1, keepdim=True))
    return {"probs": p.to(st["logits"].dtype)}


# ------------------------------------------------------------------ the work

def work(case):
    op = case["op"]
    if op == "plan":
        Q, BS = case["Q"], case["BS"]
        kept, new = _lens(Q, case["klo"], case["khi"]), _lens(Q, case["lo"], case["hi"])
        pages = sum(-(-(k + n) // BS) - -(-k // BS) for k, n in zip(kept, new))
        if case["short"]:
            pages = pages * 3 // 4
        # twice: lengths in and out, pages held; a number taken and given back per page; two a token
        return {"bytes": 4 * (2 * 6 * Q + 4 * pages + 2 * sum(new)), "flops": 0}
    es = _ES[case["dtype"]]
    if op == "rotate":
        N, Hq, Hkv, D, Dr = (case[k] for k in ("N", "Hq", "Hkv", "D", "Dr"))
        flops = N * (Hq + Hkv) * (3 * Dr + (4 * D if case["norm"] else 0))
        return {"bytes": 2 * N * (Hq + 2 * Hkv) * D * es + 8 * N, "flops": flops}
    if op == "prefix":
        Q, Hq, Hkv, D = (case[k] for k in ("Q", "Hq", "Hkv", "D"))
        own_lens, pre = sum(_lens(Q, case["lo"], case["hi"])), _prefix_lens(case)
        pairs = own_lens + sum(m * P for m, P in zip(_groups(case), pre))
        nbytes = 2 * (own_lens + sum(pre)) * Hkv * D * es + 2 * Q * Hq * D * es + Q * Hq * 4
        return {"bytes": nbytes, "flops": 4 * Hq * D * pairs}
    R, V = case["R"], case["V"]
    if op == "sample":
        return {"bytes": R * (V * es + 24), "flops": 4 * R * V}
    return {"bytes": R * (2 * V * es + 16), "flops": 5 * R * V}


# ------------------------------------------------------------------ 64 bits, by the definitions

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "rotate":
        N, Hq, Hkv, D, Dr = (case[k] for k in ("N", "Hq", "Hkv", "D", "Dr"))
        x = st["qkv"].double()
        pos, f = st["pos"].double(), st["freqs"]
        q, k = x[:, :Hq].clone(), x[:, Hq:Hq + Hkv].clone()
        for y, w in ((q, st["wq"]), (k, st["wk"])):
            if w is not None:
                y /= torch.sqrt(torch.mean(y ** 2, dim=2, keepdim=True) + 1e-6)
                y *= w.double()
            for i in range(Dr // 2):
                a, b = (i, i + Dr // 2) if case["half"] else (2 * i, 2 * i + 1)
                z = torch.polar(torch.full_like(pos, st["stretch"]), pos * f[i])[:, None]
                z = z * torch.complex(y[:, :, a], y[:, :, b])
                y[:, :, a], y[:, :, b] = z.real, z.imag
        kc, vc = st["kc"].double(), st["vc"].double()
        page, slot = st["slots"].long() // case["BS"], st["slots"].long() % case["BS"]
        kc[page, slot] = k
        vc[page, slot] = x[:, Hq + Hkv:]
        return {"q": q, "kc": kc, "vc": vc}
    if op == "prefix":
        Q, Hq, Hkv, D, BS = (case[k] for k in ("Q", "Hq", "Hkv", "D", "BS"))
        g = Hq // Hkv
        out = torch.empty((Q, Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.empty((Q, Hq), dtype=torch.float64, device="cuda")
        ends, first = st["lens"].tolist(), st["groups"].tolist()

        def rows(cache, table, n, h):
            return cache[table[:-(-n // BS)].long(), :, h].reshape(-1, D)[:n].double()

        for i, P in enumerate(_prefix_lens(case)):
            for h in range(Hkv):
                pk = rows(st["kc"], st["ptable"][i], P, h)
                pv = rows(st["vc"], st["ptable"][i], P, h)
                for b in range(first[i], first[i + 1]):
                    n = ends[b + 1] - ends[b]
                    k = torch.cat([pk, rows(st["kc"], st["table"][b], n, h)])
                    v = torch.cat([pv, rows(st["vc"], st["table"][b], n, h)])
                    s = st["scale"] * (st["q"][b, h * g:(h + 1) * g].double() @ k.T)
                    z = torch.logsumexp(s, 1)
                    lse[b, h * g:(h + 1) * g] = z
                    out[b, h * g:(h + 1) * g] = torch.exp(s - z[:, None]) @ v
        return {"out": out, "lse": lse}
    R, V = st["logits"].shape
    tokens = torch.zeros(R, dtype=torch.int32)
    probs = torch.zeros((R, V), dtype=torch.float64)
    for r in range(R):
        x = st["logits"][r].double().cpu()
        T = float(st["temp"][r])
        best = int(torch.nonzero(x == x.max())[0])
        w = torch.zeros(V, dtype=torch.float64)
        if T == 0.0:
            w[best] = 1.0
        else:
            e = torch.exp((x - x[best]) / T)
            order = torch.argsort(-x, stable=True)
            k = int(st["k"][r]) if st["k"] is not None else 0
            if k > 0:
                order = order[:k]
            total = float(e[order].sum())
            if st["p"] is not None and float(st["p"][r]) < 1.0:
                # the shortest beginning that reaches the share
                reach = torch.cumsum(e[order], 0)
                m = int(torch.searchsorted(reach, float(st["p"][r]) * total)) + 1
                order = order[:m]
            if st["m"] is not None:
                order = order[e[order] >= float(st["m"][r])]
            w[order] = e[order]
            w[best] = 1.0
        run = torch.cumsum(w, 0)
        tokens[r] = int(torch.searchsorted(run, float(st["u"][r]) * float(run[-1]), right=True))
        probs[r] = w / run[-1]
    return {"tokens": tokens} if op == "sample" else {"probs": probs}
