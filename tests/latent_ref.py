"""Plain 64-bit forms of the latent-cache operators and bounds of their errors.

Bounds (u = half a step of the type relative to the value: bf16 2^-8, fp32
2^-24).  A score is a sum of D products in fp32; each of its additions is off
by at most 2^-24 of the partial sums (2^-23 where a matrix unit truncates), so
it is off by at most d = D * 2^-23 * scale * sum |q k|.  A weight exp(s) / sum
is then off by a factor exp(2 d) at most.  The weighted sum over n keys adds n
* 2^-23; weights rounded to bf16 for a matrix unit add 2^-8 of each term; the
result is rounded once.  With A = sum_k w_k |v_k|:
  |out - ref| <= A * (exp(2 d) - 1 + n * 2^-23 + [bf16] 2^-8 + 2^-20) + u |ref|
  |lse - ref| <= d + n * 2^-24 + 2^-20 * (1 + |ref|)
(2^-20 covers the exponential's and logarithm's own few units in the last
place and the merge of partial results)."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def attention(q, k, v, scale, seen):
    """q [r, D], k [n, D], v [n, Dv] float64, seen [r, n] bool: out, lse, and
    the two parts of their bounds (A [r, Dv], d [r])."""
    n = k.shape[0]
    if n == 0:
        z = torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64, device=q.device)
        inf = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
        return z, inf, z.clone(), torch.zeros_like(inf)
    s = (scale * (q @ k.T)).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, 1)
    some = torch.isfinite(lse)
    w = torch.exp(s - torch.where(some, lse, torch.zeros_like(lse))[:, None])
    d = (abs(scale) * (q.abs() @ k.abs().T)).masked_fill(~seen, 0.0).amax(1)
    return w @ v, lse, w @ v.abs(), d * q.shape[1] * 2.0 ** -23


def check(name, out, lse, ref, ref_lse, A, d, n, dtype):
    """out, lse of the kernels against ref within the bounds above."""
    out, lse = out.double(), lse.double()
    none = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), none), f"{name}: rows without keys differ"
    assert bool((out[none] == 0).all()), f"{name}: a row without keys is not zero"
    assert bool(torch.isfinite(out).all()), f"{name}: non-finite output"
    u = U[dtype]
    soft = torch.exp(2 * d)[..., None] - 1 + n * 2.0 ** -23 + 2.0 ** -20
    if dtype == torch.bfloat16:
        soft = soft + 2.0 ** -8
    tol = A * soft + u * ref.abs() + 1e-30
    over = ((out - ref).abs() / tol)
    assert float(over.max()) <= 1.0, f"{name}: output {float(over.max()):.3g} of its bound"
    ltol = d + n * 2.0 ** -24 + 2.0 ** -20 * (1 + ref_lse.abs())
    some = ~none
    if bool(some.any()):
        lover = ((lse - ref_lse).abs()[some] / ltol[some])
        assert float(lover.max()) <= 1.0, f"{name}: lse {float(lover.max()):.3g} of its bound"


class LatentCase:
    """A paged latent cache with random pages; every slot that no sequence
    holds is NaN or infinite."""

    def __init__(self, lens, T, H, R, BS, dtype, seed=0, offsets=None, spare=2, device="cuda",
                 k_scale=1.0):
        g = torch.Generator()
        g.manual_seed(seed)
        P, Q = 64, len(lens)
        self.lens, self.T, self.H, self.R, self.P, self.BS = lens, T, H, R, P, BS
        self.dtype, self.device = dtype, device
        offsets = offsets or [0] * Q
        pages = [-(-n // BS) for n in lens]
        cols = max(1, max(o + p for o, p in zip(offsets, pages)) + spare)
        NB = sum(pages) + 3
        perm = torch.randperm(NB, generator=g)
        table = torch.full((Q, cols), -7, dtype=torch.int32)
        latent = torch.full((NB, BS, 1, R), math.nan)
        rope = torch.full((NB, BS, 1, P), math.inf)
        at = 0
        self.rows = []
        for b, n in enumerate(lens):
            ids = perm[at:at + pages[b]]
            at += pages[b]
            table[b, offsets[b]:offsets[b] + pages[b]] = ids.to(torch.int32)
            c = (torch.randn(n, R, generator=g) * k_scale).to(dtype).float()
            r = torch.randn(n, P, generator=g).to(dtype).float()
            for j, i in enumerate(ids.tolist()):
                part = slice(j * BS, min(n, (j + 1) * BS))
                latent[i, :part.stop - part.start, 0] = c[part]
                rope[i, :part.stop - part.start, 0] = r[part]
            self.rows.append((c.double().to(device), r.double().to(device)))
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        self.table = table.to(device)
        self.latent = latent.to(dtype).to(device)
        self.rope = rope.to(dtype).to(device)
        self.seq_lens = torch.tensor(ends, dtype=torch.int32, device=device)
        self.seq_offset = torch.tensor([o * BS for o in offsets], dtype=torch.int32, device=device)
        self.ql = torch.randn(Q, T, H, R, generator=g).to(dtype).to(device)
        self.qr = torch.randn(Q, T, H, P, generator=g).to(dtype).to(device)
        self.scale = 1.0 / math.sqrt(R + P)

    def reference(self, drop=()):
        """drop: (sequence, logical page) pairs whose tokens do not count."""
        Q, T, H, R, P = len(self.lens), self.T, self.H, self.R, self.P
        dev = self.device
        out = torch.zeros((Q, T, H, R), dtype=torch.float64, device=dev)
        A = torch.zeros_like(out)
        lse = torch.full((Q, T, H), -math.inf, dtype=torch.float64, device=dev)
        d = torch.zeros_like(lse)
        for b, n in enumerate(self.lens):
            c, r = self.rows[b]
            q = torch.cat([self.ql[b].double(), self.qr[b].double()], -1).reshape(T * H, R + P)
            t = torch.arange(T, device=dev).repeat_interleave(H)
            j = torch.arange(n, device=dev)
            seen = j[None, :] <= (n - T + t)[:, None]
            for db, page in drop:
                if db == b:
                    seen &= (j // self.BS != page)[None, :]
            o, z, a, e = attention(q, torch.cat([c, r], 1), c, self.scale, seen)
            out[b], A[b] = o.view(T, H, R), a.view(T, H, R)
            lse[b], d[b] = z.view(T, H), e.view(T, H)
        return out, lse, A, d
