"""Page operations on rows that do not stand as the calls themselves leave them: lengths ahead of their pages, pages behind an
empty entry."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402
from test_pages_gpu import BAD_BLOCK, NO_PAGES, Model, i32  # noqa: E402


@pytest.mark.parametrize("batch", [1, 2, 3, 16, 17, 31, 32, 33, 100])
def test_reserve_fills_entries_below_the_length(batch):
    """A length set before its pages are taken: all entries below length and new tokens are filled."""
    m = Model(60 * batch, batch, 600, layers=1, widths=(8,))
    rng = np.random.default_rng(batch)
    for s in range(batch):
        held = int(rng.integers(0, 4))
        m.table[s, :held] = [m.take() for _ in range(held)]
        m.lens[s] = (130, 128, 64 * held, 2000, 64 * held + 1)[s % 5]
    m.upload()
    add = rng.integers(0, 200, batch)
    add[::3] = 0
    m.reserve(add)
    assert m.bits == 0 and m.held(0) == -(-(130 + int(add[0])) // 64)
    m.check()
    m.reserve(add)  # nothing more
    m.check()


def test_reserve_of_long_rows():
    """Rows over several rounds of the count, one, two and forty sequences; what is left runs out on the way."""
    for batch, width in ((1, 9000), (2, 5000), (40, 700)):
        m = Model(12000, batch, width, layers=1, widths=(8,))
        for s in range(batch):
            held = (width - 5) * s // batch
            m.table[s, :held] = np.arange(held)  # (ids are only looked at)
            m.lens[s] = 64 * width - 64 * (s % 3)
        m.refs[:100] = 1
        m.upload()
        m.reserve(np.zeros(batch, np.int64))
        assert bool(m.bits & NO_PAGES) == (batch == 40)
        m.check(f"{batch} rows of {width}")


def test_reserve_leaves_rows_with_a_page_behind_an_empty_entry():
    m = Model(40, 6, 6)
    for s, row in enumerate(([0, -1, 1], [-1, -1, 2], [3, 4, -1, 5], [6, -1, -1, -1, -1, 7], [8], [9, -1, 10])):
        m.table[s, :len(row)] = row
        m.refs[[p for p in row if p >= 0]] = 1
    m.lens[:] = [64, 192, 100, 64, 64, 0]
    m.upload()
    add = [128, 0, 100, 200, 64, 65]
    b.lrkv_pages_reserve(m.d["refs"], m.d["table"], m.d["lens"], i32(add), status=m.status)
    m.bits = BAD_BLOCK  # rows 0 to 2; the last pages of rows 3 and 5 lie behind what is asked for
    for s in (3, 4, 5):
        for k in range(-(-(int(m.lens[s]) + add[s]) // 64)):
            if m.table[s, k] < 0:
                m.table[s, k] = m.take()
    m.check()


@pytest.mark.parametrize("rows", [128, 129, 256])
def test_reserve_of_more_than_32_bits_of_pages(rows):
    """Requests that sum to 2^31 pages and more (129 rows of 2^24 entries: 8.7 GB), and two that can be served."""
    table = torch.full((rows + 1, 1 << 24), -1, dtype=torch.int32, device="cuda")
    refs, lens, st = i32(np.zeros(70)), i32(np.zeros(rows + 1)), i32([0])
    add = torch.full((rows + 1,), 1 << 30, dtype=torch.int32, device="cuda")
    add[[3, rows]] = i32([64 * 40, 64 * 30])
    b.lrkv_pages_reserve(refs, table, lens, add, status=st)
    assert int(st) == NO_PAGES and (refs == 1).all()
    assert torch.equal(table[3, :40], i32(range(40))) and torch.equal(table[rows, :30], i32(range(40, 70)))
    assert int((table[:, :64] >= 0).sum()) == 70 and int((table[:, -1] >= 0).sum()) == 0
