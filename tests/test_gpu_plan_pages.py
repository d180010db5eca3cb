"""kvd_plan_pages against a sequential form in Python integers: everything equal."""
import random

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


class State:
    """A cache's tables as Python lists and as device tensors."""

    def __init__(self, Q, cols, F, BS, held, seed):
        rng = random.Random(seed)
        pages = list(range(F))
        rng.shuffle(pages)
        self.BS, self.F = BS, F
        self.held = list(held)
        self.table = [[-5] * cols for _ in range(Q)]
        for q, n in enumerate(held):
            for c in range(min(max(n, 0), cols)):
                self.table[q][c] = pages.pop()
        self.count = [len(pages)]
        self.free = pages + [-9] * (F - len(pages))

    def device(self):
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        t = i(self.table) if self.table else torch.zeros((0, 3), dtype=torch.int32, device="cuda")
        return t, i(self.held), i(self.free), i(self.count)


def same(kvd, st, dev, kept, new, N, base=None):
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    status = kvd.status_tensor()
    got = kvd.plan_pages(*dev, i(kept), i(new), st.BS, N, pos_base=None if base is None else i(base),
                         dev_status=status)
    lens, slots, pos, bits = ref.plan(st.table, st.held, st.free, st.count, kept, new, st.BS, N,
                                      st.F, base)
    assert got[0].tolist() == lens
    assert got[1].tolist() == slots
    assert got[2].tolist() == pos
    assert int(status.item()) == bits
    assert dev[0].tolist() == st.table
    assert dev[1].tolist() == st.held
    assert dev[2].tolist() == st.free
    assert dev[3].tolist() == st.count
    return lens


def cum(x):
    out = [0]
    for n in x:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("Q,BS", [(1, 1), (1, 16), (3, 7), (64, 16), (300, 24), (1025, 16),
                                  (2500, 128)])
def test_steps(kvd, Q, BS):
    """A run of steps: prompts, tokens, rejected drafts, requests that end and begin;
    the pool runs out now and then."""
    rng = random.Random(Q + BS)
    cols = 12
    st = State(Q, cols, max(3, Q * 5), BS, [0] * Q, seed=Q)
    dev = st.device()
    lens = [0] * Q
    for step in range(8):
        kept, new = [], []
        for q in range(Q):
            k = lens[q]
            r = rng.random()
            if r < 0.1:
                k = 0
            elif r < 0.3:
                k = max(0, k - rng.randint(0, 3))
            kept.append(k)
            new.append(rng.choice([0, 1, 1, 1, 4, rng.randint(0, 3 * BS)]))
        new = cum(new)
        N = new[-1] + rng.choice([0, 0, 5])
        base = [rng.randint(0, 50) for _ in range(Q)] if step % 2 else None
        ends = same(kvd, st, dev, kept, new, N, base)
        lens = [b - a for a, b in zip(ends, ends[1:])]
        owned = [p for q in range(Q) for p in st.table[q][:st.held[q]]] + st.free[:st.count[0]]
        assert sorted(owned) == list(range(st.F))  # no page lost, none twice


def test_taking_and_giving_back_leaves_the_list(kvd):
    st = State(40, 30, 900, 16, [2] * 40, seed=1)
    dev = st.device()
    before = (list(st.free), list(st.count), list(st.held))
    same(kvd, st, dev, [20] * 40, cum([17 * (q % 5) for q in range(40)]), 17 * 80)
    same(kvd, st, dev, [20] * 40, [0] * 41, 0)
    assert before == (st.free, st.count, st.held)


def test_one_long_sequence(kvd):
    """Many pages of one sequence: shared out by page, not by sequence."""
    st = State(2, 40000, 45000, 1, [0, 0], seed=2)
    same(kvd, st, st.device(), [0, 0], [0, 39999, 40001], 40001)


@pytest.mark.parametrize("Q", [3, 700])
def test_many_tokens(kvd, Q):
    """More tokens than the planning kernel looks up itself: a pool that runs out, bad
    pages, padding, and what refuses every sequence."""
    n = 30000 // Q
    for kind in range(4):
        st = State(Q, -(-n // 16) + 3, Q * (-(-n // 16)) * 3 // 4 + Q, 16, [1] * Q, seed=kind)
        kept, new = [5] * Q, cum([n - q % 7 for q in range(Q)])
        N, base = new[-1] + 100, [q for q in range(Q)]
        if kind == 1:
            st.table[1][0] = -4
            base[0] = -7
        elif kind == 2:
            new[Q // 2] = new[Q // 2 + 1] + 1
        elif kind == 3:
            st.count = [-1]
        same(kvd, st, st.device(), kept, new, N, base)


def test_padding_and_no_tokens(kvd):
    st = State(3, 4, 10, 8, [1, 0, 2], seed=3)
    dev = st.device()
    same(kvd, st, dev, [3, 0, 9], [0, 0, 0, 0], 0)
    same(kvd, st, dev, [3, 0, 9], [0, 0, 0, 0], 6)
    same(kvd, st, dev, [3, 0, 9], [0, 2, 2, 5], 9)


def test_no_sequences(kvd):
    st = State(0, 3, 4, 8, [], seed=4)
    same(kvd, st, st.device(), [], [0], 3)


@pytest.mark.parametrize("Q", [5, 1030])
def test_bad_sequences_are_left_alone(kvd, Q):
    """Each kind of bad argument, the others served."""
    for kind in range(9):
        st = State(Q, 6, 8 * Q, 8, [2] * Q, seed=kind)
        kept, n = [10] * Q, [3] * Q
        new, bad = cum(n), Q // 2
        N = new[-1]
        if kind == 0:
            kept[bad] = -3  # with its three tokens a length of zero
        elif kind == 1:
            kept[bad] = 17  # more than its pages hold
        elif kind == 2:
            st.held[bad] = 7
        elif kind == 3:
            st.held[bad] = -1
        elif kind == 4:
            new[bad] = new[bad + 1] + 2  # falls
        elif kind == 5:
            new[-1] = N + 4
        elif kind == 6:
            new[0] = 1
        elif kind == 7:
            kept[bad], new = 10, cum([3] * bad + [60] + [3] * (Q - bad - 1))  # past the columns
            N = new[-1]
        else:
            st.count = [8 * Q + 1]
        same(kvd, st, st.device(), kept, new, N)


def test_no_room_for_pages_given_back(kvd):
    st = State(3, 4, 8, 8, [2, 2, 2], seed=5)
    st.count = [5]
    dev = st.device()
    same(kvd, st, dev, [1, 16, 0], [0, 0, 1, 1], 1)
    st.count = [2]
    same(kvd, st, st.device(), [1, 16, 0], [0, 0, 1, 1], 1)


def test_lengths_and_slots_past_32_bits(kvd):
    BS = 1 << 20
    st = State(3, 2000, 40, BS, [0, 0, 0], seed=6)
    for q in range(3):  # shared pages: lengths that add up to more than 2^31
        st.held[q] = 1025
        st.table[q][:1025] = [3000] * 1025
    kept = [1 << 30, 1 << 30, 5]
    same(kvd, st, st.device(), kept, [0, 1, 2, 3], 3)


def test_positions_past_32_bits(kvd):
    st = State(2, 2, 4, 8, [1, 1], seed=7)
    same(kvd, st, st.device(), [3, 3], [0, 2, 4], 4, base=[2 ** 31 - 4, -4])


def test_graph_and_streams(kvd):
    """Captured once and replayed: the state moves on by itself."""
    Q, BS = 6, 4
    st = State(Q, 20, 200, BS, [0] * Q, seed=8)
    dev = st.device()
    kept = torch.zeros(Q, dtype=torch.int32, device="cuda")
    new = torch.arange(Q + 1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            lens, slots, pos = kvd.plan_pages(*dev, kept, new, BS, Q)
            kept.copy_(lens[1:] - lens[:-1])
    have = [0] * Q
    for step in range(9):
        graph.replay()
        torch.cuda.synchronize()
        a, b, c, bits = ref.plan(st.table, st.held, st.free, st.count, have, list(range(Q + 1)), BS,
                                 Q, st.F)
        have = [y - x for x, y in zip(a, a[1:])]
        assert (lens.tolist(), slots.tolist(), pos.tolist(), bits) == (a, b, c, 0)
        assert dev[0].tolist() == st.table and dev[3].tolist() == st.count


@pytest.mark.parametrize("Q", [2, 1030])
def test_a_list_without_entries(kvd, Q):
    """No page to take: sequences that need one are refused, the others go on."""
    table = torch.arange(Q, dtype=torch.int32, device="cuda")[:, None].repeat(1, 3)
    held = torch.ones(Q, dtype=torch.int32, device="cuda")
    held[0] = 0
    kept = torch.full((Q,), 2, dtype=torch.int32, device="cuda")
    kept[0] = 0
    new = torch.arange(Q + 1, dtype=torch.int32, device="cuda")
    empty, count = torch.empty(0, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    status = kvd.status_tensor()
    lens, slots, pos = kvd.plan_pages(table, held, empty, count, kept, new, 4, Q, dev_status=status)
    assert int(status.item()) == kvd.DEV_NO_PAGES
    assert lens.tolist() == [0] + [3 * i for i in range(Q)]
    assert slots.tolist() == [-1] + [4 * i + 2 for i in range(1, Q)]
    assert pos.tolist() == [-1] + [2] * (Q - 1) and held.tolist() == [0] + [1] * (Q - 1)
    assert int(count) == 0
