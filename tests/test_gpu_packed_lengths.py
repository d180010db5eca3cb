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
