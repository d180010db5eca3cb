"""Lengths that are not a cumulative sum: what they refuse, and what they leave."""
import pytest
import torch

from test_gpu_expanded import Packed

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


# ------------------------------------------------------------------ expanded

def expanded(kvd, lens, c, sequences):
    """The call with the q_lens given: rows of `sequences` as with good lengths
    (which are the keys' own), all others left as they were."""
    good, gl, bits = c.call(kvd)
    assert bits == 0
    c.ql = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse, bits = c.call(kvd)
    assert bits == kvd.DEV_SEQLENS
    keep = torch.zeros(out.shape[0], dtype=torch.bool, device="cuda")
    for b in sequences:
        keep[lens[b]:lens[b + 1]] = True
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], gl[keep])
    assert bool((out[~keep] == 7).all()) and bool((lse[~keep] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens, sequences", [
    ([0, 300, 0, 300], [0]),            # the third would take the first one's rows again
    ([0, 300, 299, 302], [0]),
    ([0, 100, 300, 200, 300], [0, 1]),
    ([0, 300, 100, 200, 300], [0]),
    ([0, 5000, 100, 300], []),          # past the queries, then decreasing
    ([0, -4, 100, 300], []),
    ([0, 100, 5000], [0]),              # past the queries: only that pair is bad
    ([3, 100, 300], [1]),               # not from zero: only that pair is bad
], ids=str)
def test_expanded_decreasing(kvd, lens, sequences, dtype):
    Q = len(lens) - 1
    # the keys, and the queries of the good call, are those of the pairs kept
    nq = [max(0, lens[b + 1] - lens[b]) if b in sequences else 0 for b in range(Q)]
    first = lens[sequences[0]] if sequences else 0
    if first:
        nq[0] = first                   # the good call's first sequence, rows that are then left
    c = Packed(nq, nq, 2, 64, 64, dtype, seed=Q)
    c.q = torch.cat([c.q, c.q[:1].repeat(302 - c.q.shape[0], 1, 1)]) if c.q.shape[0] < 302 else c.q
    expanded(kvd, lens, c, sequences)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_expanded_decreasing_among_many(kvd, dtype):
    """More sequences than one warp looks through; two places where it falls."""
    nq = [(i * 7) % 20 for i in range(300)]
    c = Packed(nq, nq, 1, 64, 64, dtype, seed=2)
    lens = c.ql.tolist()
    lens[201] -= 150
    lens[250] -= 1000
    expanded(kvd, lens, c, range(200))


def test_expanded_decreasing_all_along(kvd):
    """As many falling pairs as there may be sequences: nothing but the first is found."""
    nq = [3] + [0] * 16383
    for dtype in (BF, F32):
        c = Packed(nq, nq, 1, 64, 64, dtype, seed=3)
        expanded(kvd, ([0, 3] + [2, 3] * 8192)[:16385], c, [0])


# ------------------------------------------------------------------ append

def append(kvd, lens, N):
    """Appends rows 1, 2, .. N of all ones times their number at token 0 of every
    sequence, each with pages of its own; returns what every token then holds."""
    Q, BS, cols, R, P = len(lens) - 1, 4, 8, 64, 8
    table = torch.arange(Q * cols, dtype=torch.int32).view(Q, cols).cuda()
    latent, rope = torch.zeros(Q * cols, BS, 1, R).cuda(), torch.zeros(Q * cols, BS, 1, P).cuda()
    rows = torch.arange(1.0, N + 1, device="cuda")[:, None]
    status = kvd.status_tensor()
    kvd.append_latent(latent, rope, table, None, rows.repeat(1, R), rows.repeat(1, P),
                      torch.tensor(lens, dtype=torch.int32).cuda(),
                      torch.zeros(Q, dtype=torch.int32).cuda(), status)
    assert bool((latent == latent[..., :1]).all()) and bool((rope == latent[..., :1]).all())
    return latent[..., 0].view(Q, cols * BS).long().tolist(), int(status.item())


def held(lens, rows):
    """Tokens of every sequence where `rows` (counted from 0) are written."""
    want = [[0] * 32 for _ in lens[1:]]
    for r, b in rows:
        want[b][r - lens[b]] = r + 1
    return want


def test_append_past_the_rows(kvd):
    """A sequence whose rows end behind the N given has none of them written."""
    got, bits = append(kvd, [0, 3, 5, 9], 8)
    assert bits == kvd.DEV_SEQLENS
    assert got == held([0, 3, 5, 9], [(0, 0), (1, 0), (2, 0), (3, 1), (4, 1)])


def test_append_not_from_zero(kvd):
    """Nothing is written at all."""
    got, bits = append(kvd, [1, 3, 5], 8)
    assert bits == kvd.DEV_SEQLENS and got == held([1, 3, 5], [])


@pytest.mark.parametrize("lens", [[0, 2, 1, 6, 9], [0, 5, 3, 3, 8], [0, 4, 8, 6, 7, 8],
                                  [0, 7, -1, 8], [0, 20, 5, 6]], ids=str)
def test_append_decreasing(kvd, lens):
    """Rows below the smallest length that new_lens falls to are written where
    they belong, the others once at most, to a sequence whose pair holds them."""
    N = 8
    got, bits = append(kvd, lens, N)
    assert bits == kvd.DEV_SEQLENS
    low = min(b for a, b in zip(lens, lens[1:]) if b < a)
    holds = [[b for b in range(len(lens) - 1) if 0 <= lens[b] <= r < lens[b + 1] <= N]
             for r in range(N)]
    for r in range(N):
        at = [(b, t) for b, row in enumerate(got) for t, v in enumerate(row) if v == r + 1]
        assert len(at) <= 1
        assert all(b in holds[r] and t == r - lens[b] for b, t in at)
        if r < low:
            assert len(at) == len(holds[r])
    written = sum(v != 0 for row in got for v in row)
    assert written == sum(any(v == r + 1 for row in got for v in row) for r in range(N))
