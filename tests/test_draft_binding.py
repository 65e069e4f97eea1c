"""Arrays that the binding refuses before the library reads or writes them (no GPU needed): 64-bit integers, which torch makes
by default, strides, and other lengths."""
import pytest

torch = pytest.importorskip("torch")

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402

I32, I64 = torch.int32, torch.int64


def z(*s, t=I32):
    return torch.zeros(*s, dtype=t)


def bad_arrays(n):
    """What a call must not take for n 32-bit words."""
    return [z(n, t=I64), z(n, t=torch.float32), z(n, t=torch.int16), z(2 * n)[::2], z(n + 1), z(n - 1), z(n, 2),
            z(n, n).t()[0]]


def refused(call, *args, **kw):
    with pytest.raises(ValueError):
        call(*args, stream=0, **kw)


P = b.Pools.of(z(4, 64, 8, t=torch.bfloat16))
REFS, TABLE, LENS = z(4), z(3, 2), z(3)


@pytest.mark.parametrize("k", range(8))
def test_page_calls(k):
    bad = bad_arrays(3)[k]
    refused(b.lrkv_pages_reserve, REFS, TABLE, LENS, bad)
    refused(b.lrkv_pages_free, REFS, TABLE, LENS, z(2), keep_lens=bad)
    refused(b.lrkv_cache_compact, P, TABLE, LENS, z(3, 5), bad)
    refused(b.lrkv_cache_compact, P, TABLE, LENS, z(3, 5), z(3), new_lens=bad)
    refused(b.lrkv_pages_fork, P, REFS, TABLE, LENS, z(3), bad)
    refused(b.lrkv_pages_copy, P, z(3), P, bad)
    if k not in (4, 5):  # (lists may have any length)
        refused(b.lrkv_pages_free, REFS, TABLE, LENS, bad)
    refused(b.lrkv_pages_fork, P, REFS, TABLE, LENS, bad, z(3))
    refused(b.lrkv_pages_copy, P, bad, P, z(3))


@pytest.mark.parametrize("bad", [z(3, 5, t=I64), z(5, 3).t(), z(2, 5), z(4, 5), z(15)])
def test_paths(bad):
    refused(b.lrkv_cache_compact, P, TABLE, LENS, bad, z(3))


def test_empty_lists_are_taken():
    b.lrkv_pages_free(z(4), z(3, 2), z(3), z(0), stream=0)
    b.lrkv_pages_fork(P, z(4), z(3, 2), z(3), z(0), z(0), stream=0)
    b.lrkv_pages_copy(P, z(0), P, z(0), stream=0)


@pytest.mark.parametrize("k", range(8))
def test_rotation(k):
    """Positions may be of any number, row indices of theirs."""
    bad, plan, x = bad_arrays(3)[k], b.rope_plan(8), z(6, 2, 8, t=torch.bfloat16)
    if k not in (4, 5):
        refused(b.lrkv_rope, plan, x, x, bad)
    refused(b.lrkv_rope, plan, x, x, z(3), x_rows=bad)
    refused(b.lrkv_rope, plan, x, x, z(3), y_rows=bad)
    refused(b.lrkv_rope, plan, x, x, z(3), x_rows=z(3), y_rows=bad)


def test_no_rows_are_taken():
    b.lrkv_rope(b.rope_plan(8), z(6, 2, 8, t=torch.float32), z(6, 2, 8, t=torch.float32), z(0), x_rows=z(0), stream=0)


def tree(**kw):
    bf = torch.bfloat16
    cache = b.PagedCache(*(z(4, 64, 8, t=bf) for _ in range(4)))
    a = dict(table=TABLE, lens=LENS, mask=z(3, 5, t=I64), counts=z(3))
    a.update(kw)
    q, x = z(3, 5, 8, 64, t=bf), z(8, 64, 16, t=bf)
    return (b.make_dims(8, 64, 16, 512), q, x, x, cache, a["table"], a["lens"], a["mask"], a["counts"], q, z(256))


@pytest.mark.parametrize("bad", [z(3, 5, t=torch.float64), z(3, 5), z(3, 10), z(5, 3, t=I64).t(), z(3, 6, t=I64)[:, :5],
                                 z(15, t=I64), z(3, 4, t=I64), z(2, 5, t=I64)])
def test_tree_masks(bad):
    with pytest.raises(ValueError, match="64-bit"):
        b.lrkv_decode_tree(*tree(mask=bad), stream=0)


@pytest.mark.parametrize("k", range(8))
def test_tree_lengths(k):
    bad = bad_arrays(3)[k]
    refused(b.lrkv_decode_tree, *tree(counts=bad))
    refused(b.lrkv_decode_tree, *tree(lens=bad))


@pytest.mark.parametrize("bad", [z(3, 2, t=I64), z(2, 3).t(), z(3, 4)[:, :2], z(2, 2), z(4, 2), z(3, 2, t=torch.float32)])
def test_tree_tables(bad):
    refused(b.lrkv_decode_tree, *tree(table=bad))
