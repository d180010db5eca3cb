"""kvd_sample and kvd_filter_probs: tails of weights at the end of what a draw resolves."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


@pytest.mark.parametrize("V", [5000, 128000, 2 ** 20])
@pytest.mark.parametrize("half_units", [0.25, 0.998, 1.002, 1.4, 2.9])
def test_flat_tails(kvd, V, half_units):
    """One logit and a tail of equal ones whose weight is this many times 2^-43: counted in whole
    multiples of 2^-42, each of them is off by up to half of that, all to one side.  Weights are
    otherwise right to 2^-28, so with E(v) the running sum in 64 bits and n = V
      E(v - 1) - b <= u E(V) <= E(v) + b,  b = (2^-28 + n 2^-43) E(V)
    for the token v that is drawn; below 2^-43 none of the tail is.  Probabilities do not go by
    these units."""
    w = half_units * 2.0 ** -43
    logits = torch.full((1, V), math.log(w), device="cuda")
    best = V // 3
    logits[0, best] = 0.0
    tail = math.exp(float(logits[0, 0]))
    u = torch.tensor([0.0, 2.0 ** -24, 0.25, 0.5, 1 - 2.0 ** -23, 1 - 2.0 ** -24], device="cuda")
    R = len(u)
    rows = logits.repeat(R, 1)
    total = 1.0 + (V - 1) * tail
    bound = (2.0 ** -28 + V * 2.0 ** -43) * total
    status = kvd.status_tensor()
    for v, x in zip(kvd.sample(rows, u, dev_status=status).tolist(), u.double().tolist()):
        end = (v + 1) * tail + (1.0 - tail if v >= best else 0.0)
        before = end - (1.0 if v == best else tail)
        assert before - bound <= x * total <= end + bound
        assert v == best or half_units > 1
    # top-p's border in the same way: the largest, then the tail by index
    p = torch.tensor([0.5, 1 - 2.0 ** -20, 1 - 2.0 ** -23, 1 - 2.0 ** -24], device="cuda")
    kept = (kvd.filter_probs(rows[:4].contiguous(), top_p=p, dev_status=status) > 0).sum(1).tolist()
    for n, x in zip(kept, p.double().tolist()):
        end = 1.0 + (n - 1) * tail
        before = end - (1.0 if n == 1 else tail)
        assert before - bound <= x * total <= end + bound
    probs = kvd.filter_probs(logits, dev_status=status)[0].double()
    assert int(status.item()) == 0
    want = torch.full((V,), tail, dtype=torch.float64, device="cuda")
    want[best] = 1.0
    # the sum that they are divided by is off by its tail's units
    assert float((probs / (want / total) - 1).abs().max()) <= 3 * 2.0 ** -24 + 2.0 ** -28 + V * 2.0 ** -43
