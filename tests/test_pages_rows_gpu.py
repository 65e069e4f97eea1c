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


@pytest.mark.parametrize("cut", [65, 70, 127, 128])
def test_a_sequence_cut_inside_a_shared_page_goes_on_in_a_fork(cut):
    """Forks of 128 tokens share two full pages; the one cut to `cut` tokens is forked and given back, and what is appended
    and moved then reaches no row of the others."""
    H, d_h, r, d = 2, 64, 8, 128
    dims = b.make_dims(H, d_h, r, d)
    g = torch.Generator(device="cuda").manual_seed(cut)
    cache = b.PagedCache.empty(10, H, d_h, r)
    for t in cache.tensors():
        t.zero_()
    pools, st = b.Pools.of(cache), i32([0])
    W = (torch.randn(2 * (d_h + H * r), d, generator=g, device="cuda") * d ** -0.5).to(torch.bfloat16)
    refs, table, lens = i32(np.zeros(10)), torch.full((3, 4), -1, dtype=torch.int32, device="cuda"), i32([0, 0, 0])

    def append(s, first, n):
        t = torch.arange(first, first + n, device="cuda")
        x = torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16)
        b.lrkv_append(dims, x, W, (table[s][t // 64] * 64 + t % 64).int(), cache, status=st)

    def rows(s, n):
        return [t[table[s, :-(-n // 64)].long()].flatten(0, 1)[:n].clone() for t in cache.tensors()]

    b.lrkv_pages_reserve(refs, table, lens, i32([128, 0, 0]), status=st)
    append(0, 0, 128)
    lens[0] = 128
    b.lrkv_pages_fork(pools, refs, table, lens, i32([0]), i32([1]), status=st)
    assert torch.equal(table[0], table[1])
    b.lrkv_pages_free(refs, table, lens, i32([1]), keep_lens=i32([0, cut, 0]), status=st)
    parent = rows(0, 128)
    b.lrkv_pages_fork(pools, refs, table, lens, i32([1]), i32([2]), status=st)
    b.lrkv_pages_free(refs, table, lens, i32([1]), status=st)
    b.lrkv_pages_reserve(refs, table, lens, i32([0, 0, 60]), status=st)
    held = table[2, :-(-(cut + 60) // 64)].long()
    assert lens.tolist() == [128, 0, cut] and (refs[held[cut // 64:]] == 1).all()
    append(2, cut, 60)
    kept = rows(2, cut + 60)
    b.lrkv_cache_compact(pools, table, lens, i32([[0] * 20, [0] * 20, range(1, 60, 3)]), i32([0, 0, 20]), status=st)
    assert lens.tolist() == [128, 0, cut + 20] and int(st) == 0
    for x, y, z, k in zip(rows(0, 128), parent, rows(2, cut + 20), kept):
        assert torch.equal(x, y) and torch.equal(z[:cut], x[:cut]) and torch.equal(z[cut:], k[cut + 1:cut + 60:3])
    b.lrkv_pages_free(refs, table, lens, i32([0, 2]), status=st)
    assert (refs == 0).all() and (table == -1).all() and int(st) == 0
