"""Launches of the rotation and of forks that calls of many rows or sequences take: several heads or rows a thread, lanes of a
warp shared by forks, more shared memory, pages found in a second search."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402
from test_pages_gpu import BAD_INDEX, Model  # noqa: E402
from test_rope_rows_gpu import BF, F32, check, positions, want64  # noqa: E402

# (n, heads, width, begin, d_rot): more units of eight values than threads run at once, whether all of a head or only its
# rotated part is taken; heads and rows that are no multiple of a thread's
LARGE = [(2601, 7, 136, 8, 128), (1203, 33, 48, 16, 32), (21001, 3, 72, 0, 40), (40003, 1, 64, 0, 64)]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,heads,width,begin,d_rot", LARGE)
def test_large_rotations(n, heads, width, begin, d_rot, half, dtype, transpose):
    g = torch.Generator().manual_seed(n + half)
    x = torch.randn(n, heads, width, generator=g).to(dtype)
    pos = positions(g, n, True)
    plan = b.rope_plan(d_rot, layout="half" if half else "interleaved", magnitude=1.25)
    y = torch.full_like(x, float("nan")).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.lrkv_rope(plan, x.cuda(), y, pos.cuda(), begin=begin, transpose=transpose, status=st)
    want, mag = want64(x.double(), pos, d_rot, begin, half, transpose, 1.25)
    check(y, want, mag, dtype, f"n {n}, {heads} heads of {width}")
    keep = [*range(begin), *range(begin + d_rot, width)]
    assert torch.equal(y.cpu()[..., keep], x[..., keep])
    z = x.cuda()
    b.lrkv_rope(plan, z, z, pos.cuda(), begin=begin, transpose=transpose, status=st)
    assert torch.equal(z, y) and int(st) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,heads,width,begin,d_rot", LARGE)
def test_large_rotations_of_picked_rows(n, heads, width, begin, d_rot, half, dtype):
    """Rows picked on both sides, some skipped, some out of range; the other rows stay."""
    g = torch.Generator().manual_seed(n + 10 * half)
    rows = n + 100
    x = torch.randn(rows, heads, width, generator=g).to(dtype)
    pos = positions(g, n, True)
    xr = torch.randint(0, rows, (n,), generator=g, dtype=torch.int32)
    yr = torch.randperm(rows, generator=g)[:n].to(torch.int32)
    out = torch.rand(n, generator=g)
    xr[out < 0.05], yr[(out > 0.05) & (out < 0.1)] = -1, -3
    xr[(out > 0.1) & (out < 0.15)], yr[(out > 0.15) & (out < 0.2)] = rows, 2 ** 31 - 1
    y = torch.full((rows, heads, width), 7.0, dtype=dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = b.rope_plan(d_rot, layout="half" if half else "interleaved")
    b.lrkv_rope(plan, x.cuda(), y, pos.cuda(), begin=begin, x_rows=xr.cuda(), y_rows=yr.cuda(), status=st)
    assert int(st) == b.DEV_BAD_SLOT
    done = (xr >= 0) & (xr < rows) & (yr >= 0) & (yr < rows)
    to = yr[done].long()
    want, mag = want64(x[xr[done].long()].double(), pos[done], d_rot, begin, half, False, 1.0)
    check(y[to.cuda()], want, mag, dtype, f"picked rows of n {n}, {heads} heads")
    rest = torch.ones(rows, dtype=torch.bool)
    rest[to] = False
    assert (y.cpu()[rest] == 7).all()


@pytest.mark.parametrize("n", [33, 40, 64, 65, 100, 300])
def test_many_forks(n):
    """Forks that share a warp, of parents of no pages up to many rounds of a fork's lanes, some forks left out."""
    m = Model(1500 + 3 * n, n + 6, 210, layers=2, widths=(8, 24))
    rng = np.random.default_rng(n)
    lens = [0, 64 * 200 + 3, 64, 1, 64 * 130, 4000]
    m.reserve(lens + [int(x) for x in rng.integers(0, 150, n)])
    m.lens[:6] = lens
    for s in range(6, n + 6):
        m.lens[s] = rng.integers(0, 64 * m.held(s) + 1)
    m.upload()
    parents, kids = rng.integers(0, 6, n), rng.permutation(n) + 6
    m.fork(parents, kids)
    assert m.bits == 0
    m.check("all")
    kids = kids.copy()
    kids[[3, n - 1]] = kids[[7, 20]]  # listed twice
    parents[11], kids[12] = kids[30], n + 6  # a child as a parent, an index out of range
    m.fork(parents, kids)
    assert m.bits == BAD_INDEX
    m.check("some left out")
    m.free(np.arange(n + 6))
    m.check()
    assert (m.refs == 0).all()


@pytest.mark.parametrize("n", [2049, 4097, 8192])
def test_forks_of_a_whole_batch(n):
    """More forks than a block's ordinary shared memory holds, each with a page of its own (found in a second search)."""
    batch = min(n + 2, 8192)
    m = Model(n + 40, batch, 3, layers=1, widths=(8,))
    m.reserve([100, 65] + [0] * (batch - 2))
    m.lens[:2] = [100, 65]
    m.upload()
    kids = np.random.default_rng(n).permutation(batch - 2) + 2
    kids = np.concatenate([kids, kids[:n - kids.size]])  # (of 8,192 the last two are listed twice)
    m.fork([i % 2 for i in range(n)], kids.tolist())
    assert m.bits == (BAD_INDEX if n == 8192 else 0)
    m.check()
    m.free(np.arange(batch))
    m.check()
    assert (m.refs == 0).all()
