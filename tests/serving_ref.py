"""Plain forms of the serving step's operators: pages in Python integers, the others
in 64 bits."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}

NO_PAGES, TABLE_COLS, SEQLENS, POS_RANGE, BLOCK_RANGE = 512, 4, 8, 1, 2


# ------------------------------------------------------------------ pages

def plan(table, held, free, count, kept, new, BS, N, F, base=None):
    """kvd_plan_pages over Python lists, in place; returns seq_lens, slots, positions, bits."""
    Q, cols = len(held), len(table[0]) if table else 0
    bits, good, need = 0, [], []
    lens_ok = Q == 0 or (new[0] == 0 and sorted(new) == list(new) and new[-1] <= N)
    usable = lens_ok and 0 <= count[0] <= F
    if not lens_ok:
        bits |= SEQLENS
        new = [0] * (Q + 1)
    if not 0 <= count[0] <= F:
        bits |= POS_RANGE
    for q in range(Q):
        s0, s1 = new[q], new[q + 1]
        ok, n = True, 0
        if kept[q] < 0 or not 0 <= held[q] <= cols or kept[q] > held[q] * BS or \
                kept[q] + s1 - s0 > 2 ** 31 - 1:
            ok, bits = False, bits | POS_RANGE
        else:
            n = -(-(kept[q] + s1 - s0) // BS)
        good.append(ok)
        need.append(n)
    back = [(q, c) for q in reversed(range(Q)) if good[q]
            for c in reversed(range(need[q], held[q]))]
    returns = usable and count[0] + len(back) <= F
    if usable and not returns:
        bits |= NO_PAGES
    if returns:
        for q, c in back:
            free[count[0]] = table[q][c]
            count[0] += 1
    avail = count[0] if usable else 0
    wanted, asked, lens, served = 0, 0, [0], []
    taken = 0
    for q in range(Q):
        ok, grow = good[q] and usable, 0
        if usable and good[q] and need[q] > held[q]:
            grow = need[q] - held[q]
            if need[q] > cols:
                ok, grow, bits = False, 0, bits | TABLE_COLS
            wanted += grow
            if grow and wanted > avail:
                ok, grow, bits = False, 0, bits | NO_PAGES
        n = (kept[q] if good[q] else 0) + (new[q + 1] - new[q] if ok else 0)
        asked += n
        if n and asked > 2 ** 31 - 1:
            ok, grow, n, bits = False, 0, 0, bits | SEQLENS
        lens.append(lens[-1] + n)
        for c in range(held[q], held[q] + grow):
            table[q][c] = free[avail - 1 - taken]
            taken += 1
        if ok and (need[q] > held[q] or (need[q] < held[q] and returns)):
            held[q] = need[q]
        served.append(ok)
    if usable:
        count[0] = avail - taken
    slots, pos = [-1] * N, [-1] * N
    for q in range(Q):
        if not served[q]:
            continue
        for i in range(new[q], new[q + 1]):
            t = kept[q] + i - new[q]
            page = table[q][t // BS]
            p = t + (base[q] if base else 0)
            if page < 0 or page * BS + t % BS > 2 ** 31 - 1:
                bits |= BLOCK_RANGE
            elif not 0 <= p <= 2 ** 31 - 1:
                bits |= POS_RANGE
            else:
                slots[i], pos[i] = page * BS + t % BS, p
    return lens, slots, pos, bits


# ------------------------------------------------------------------ rotation

def rotate(x, weight, pos, freqs, interleaved, m, eps):
    """x [N, H, D] float64: (result, the size that its error goes by): norm, then
    rotation of the first 2 * len(freqs) dims."""
    D, Dr = x.shape[-1], 2 * len(freqs)
    y = x
    if weight is not None:
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    size = y.abs().clone()
    out = y.clone()
    angle = pos.double()[:, None] * freqs.double()[None]
    c, s = (torch.cos(angle) * m)[:, None], (torch.sin(angle) * m)[:, None]
    a, b = (slice(0, Dr, 2), slice(1, Dr, 2)) if interleaved else (slice(0, Dr // 2),
                                                                  slice(Dr // 2, Dr))
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    size[..., a] = size[..., b] = abs(m) * (y[..., a].abs() + y[..., b].abs())
    return out, size


def check_rotated(name, got, ref, size, D, dtype):
    """fp32 arithmetic: the sum of D squares is off by at most D 2^-24 of itself, so its
    root by half of that; root, division, two products: 2^-24 each and a last place more;
    cos and sin with the angle's 2^-25 and the factor: 4 * 2^-24; two products and a sum:
    3 * 2^-24.  (D / 2 + 14) 2^-24 of |a| + |b| in all, then one rounding."""
    tol = size * (D / 2 + 14) * 2.0 ** -24 + U[dtype] * ref.abs() + 1e-30
    over = float(((got.double() - ref).abs() / tol).max())
    assert over <= 1.0, f"{name}: {over:.3g} of its bound"


# ------------------------------------------------------------------ sampling

def kept_weights(x, T, k, p, m):
    """One row x [V] float64 (no NaN): the weights that stay, in index order, 64 bits."""
    V = x.numel()
    order = torch.argsort(-x, stable=True)
    best = float(x.max())
    w = torch.where(x == best, torch.ones_like(x),
                    torch.exp((x - best) / T) if T > 0 else torch.zeros_like(x))
    stay = order[:1] if T == 0 else order[:k] if 0 < k < V else order
    if T > 0 and p < 1:
        run = torch.cumsum(w[stay], 0)
        before = run - w[stay]
        keep = before < p * float(run[-1])
        keep[0] = True
        stay = stay[keep]
    if T > 0:
        stay = stay[w[stay] >= min(m, 1.0)]
    out = torch.zeros_like(w)
    out[stay] = w[stay]
    return out


def draw(w, u):
    run = torch.cumsum(w, 0)
    return int(torch.nonzero(run > u * float(run[-1]))[0])
