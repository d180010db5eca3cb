"""kvd_plan_pages: every page has one owner, whatever is refused; expectations are
worked out here, step by step, and do not come from a plain form of the call."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cum(x):
    out = [0]
    for n in x:
        out.append(out[-1] + n)
    return out


def once(table, held, free, count, sequences, pages):
    """The held pages of these sequences and the free list: each of `pages` exactly once."""
    table, held = table.tolist(), held.tolist()
    owned = [p for q in sequences for p in table[q][:held[q]]] + free.tolist()[:int(count)]
    assert sorted(owned) == sorted(pages)


@pytest.mark.parametrize("Q", [3, 200, 700, 1030])
@pytest.mark.parametrize("new", [0, 3])
def test_lengths_past_32_bits_with_pages_too_many(kvd, Q, new):
    """Two long sequences (of pages of their own kind, all the same) fill 2^31 - 1 tokens; the
    ones behind them are refused, hold two pages each, and need one.  The second one goes
    onto the list, and is no longer held."""
    BS, cols = 1 << 19, 2050
    small = Q - 2
    table = torch.full((Q, cols), -1, dtype=torch.int32, device="cuda")
    table[:2] = 1999
    pages = list(range(2 * small))
    table[2:, :2] = i32(pages).view(small, 2)
    held = i32([2048, 2048] + [2] * small)
    F = 4 * small + 5  # room for a list with pages in it twice
    extra = list(range(1000000, 1000003))
    free = torch.full((F,), -9, dtype=torch.int32, device="cuda")
    free[:3] = i32(extra)
    count = i32([3])
    kept = [2 ** 30, 2 ** 30 - 1] + [5] * small
    counts = [0, 0] + [new] * small
    status = kvd.status_tensor()
    lens, slots, pos = kvd.plan_pages(table, held, free, count, i32(kept), i32(cum(counts)), BS,
                                      new * small, dev_status=status)
    assert int(status.item()) == kvd.DEV_SEQLENS
    assert lens.tolist() == [0, 2 ** 30] + [2 ** 31 - 1] * (Q - 1)
    assert slots.tolist() == [-1] * (new * small) == pos.tolist()
    once(table, held, free, count, range(2, Q), pages + extra)
    assert held.tolist() == [2048, 2048] + [1] * small
    # the last sequence's page was pushed first
    assert free.tolist()[:3 + small] == extra + [2 * i + 1 for i in reversed(range(small))]
    # the second long request is over: those behind it go on, with the pages that they have
    status.zero_()
    held[1], kept[1] = 0, 0
    lens, slots, pos = kvd.plan_pages(table, held, free, count, i32(kept), i32(cum(counts)), BS,
                                      new * small, dev_status=status)
    assert int(status.item()) == 0
    assert lens.tolist() == [0, 2 ** 30] + [2 ** 30 + (5 + new) * i for i in range(Q - 1)]
    once(table, held, free, count, range(2, Q), pages + extra)
    assert pos.tolist() == [5 + i for i in range(new)] * small
    # and a step in which they grow takes every page of the list at most once
    counts = [0, 0] + [BS if i < 2 else 0 for i in range(small)]
    lens, _, _ = kvd.plan_pages(table, held, free, count, i32(kept), i32(cum(counts)), BS,
                                sum(counts), dev_status=status)
    assert int(status.item()) == 0
    once(table, held, free, count, range(2, Q), pages + extra)


@pytest.mark.parametrize("Q", [4, 1030])
def test_a_sequence_past_the_columns_asks_for_nothing(kvd, Q):
    """The first sequence needs more columns than there are; the list holds three pages.  The
    second and third get one and two, the fourth is refused for want of pages, and all that
    need some behind it."""
    BS, cols = 4, 3
    table = torch.full((Q, cols), -1, dtype=torch.int32, device="cuda")
    held, kept = i32([0] * Q), i32([0] * Q)
    free, count = i32([7, 8, 9]), i32([3])
    counts = [BS * cols + 1, 1, BS + 1, 1] + [1] * (Q - 4)
    status = kvd.status_tensor()
    lens, slots, pos = kvd.plan_pages(table, held, free, count, kept, i32(cum(counts)), BS,
                                      sum(counts), dev_status=status)
    assert int(status.item()) == kvd.DEV_TABLE_COLS | kvd.DEV_NO_PAGES
    assert lens.tolist() == [0, 0, 1] + [2 + BS] * (Q - 2)
    assert held.tolist() == [0, 1, 2] + [0] * (Q - 3) and int(count) == 0
    assert table[1, 0].item() == 9 and table[2, :2].tolist() == [8, 7]
    first = BS * cols + 1
    assert slots.tolist() == [-1] * first + [36, 32, 33, 34, 35, 28] + [-1] * (Q - 3)
    assert pos.tolist() == [-1] * first + [0, 0, 1, 2, 3, 4] + [-1] * (Q - 3)


def test_what_was_refused_counts_against_those_behind(kvd):
    """Two pages for sequences that need one, two and one: the second is refused, and the third,
    though a page is left."""
    status = kvd.status_tensor()
    table = torch.full((3, 3), -1, dtype=torch.int32, device="cuda")
    held, free, count = i32([0] * 3), i32([5, 6]), i32([2])
    lens, _, _ = kvd.plan_pages(table, held, free, count, i32([0] * 3), i32([0, 1, 6, 7]), 4, 7,
                                dev_status=status)
    assert int(status.item()) == kvd.DEV_NO_PAGES
    assert lens.tolist() == [0, 1, 1, 1] and held.tolist() == [1, 0, 0] and int(count) == 1
