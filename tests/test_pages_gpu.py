"""Page operations against a model on the host: tables, counts, lengths and every row's bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402

NO_PAGES, BAD_INDEX, BAD_SEQLEN, BAD_BLOCK = b.DEV_NO_PAGES, b.DEV_BAD_INDEX, b.DEV_BAD_SEQLEN, b.DEV_BAD_BLOCK


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Model:
    """The same state on the host and on the device: counts, table, lengths, pools [layers, blocks, 64, width]."""

    def __init__(self, blocks, batch, width, layers=2, widths=(8, 24, 16), seed=0):
        rng = np.random.default_rng(seed)
        self.refs = np.zeros(blocks, np.int32)
        self.table = np.full((batch, width), -1, np.int32)
        self.lens = np.zeros(batch, np.int32)
        self.pools = [rng.integers(-2 ** 15, 2 ** 15, (layers, blocks, 64, w)).astype(np.int16) for w in widths]
        self.d = dict(refs=i32(self.refs), table=i32(self.table), lens=i32(self.lens),
                      pools=[torch.from_numpy(p.copy()).cuda() for p in self.pools])
        self.own = b.Pools(self.d["pools"])
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.bits = 0

    def upload(self):
        for k in ("refs", "table", "lens"):
            self.d[k].copy_(torch.from_numpy(getattr(self, k)))
        for t, p in zip(self.d["pools"], self.pools):
            t.copy_(torch.from_numpy(p))

    def held(self, s):
        row = self.table[s]
        return int(np.argmax(row < 0)) if (row < 0).any() else row.size

    def take(self):
        free = np.flatnonzero(self.refs == 0)
        if not free.size:
            return None
        self.refs[free[0]] = 1
        return free[0]

    def reserve(self, add):
        b.lrkv_pages_reserve(self.d["refs"], self.d["table"], self.d["lens"], i32(add), status=self.status)
        for s, n in enumerate(add):
            want = -(-(int(self.lens[s]) + int(n)) // 64)
            if n < 0 or self.lens[s] < 0 or want > self.table.shape[1]:
                self.bits |= BAD_SEQLEN
                continue
            have = self.held(s)
            if want - have > (self.refs == 0).sum():
                self.bits |= NO_PAGES
                continue
            for k in range(have, want):
                self.table[s, k] = self.take()

    def drop(self, page):
        if page >= self.refs.size:
            self.bits |= BAD_BLOCK
        elif self.refs[page] <= 0:
            self.bits |= BAD_INDEX
        else:
            self.refs[page] -= 1

    def free(self, seqs, keep=None):
        b.lrkv_pages_free(self.d["refs"], self.d["table"], self.d["lens"], i32(seqs),
                          keep_lens=None if keep is None else i32(keep), status=self.status)
        for s in seqs:
            if not 0 <= s < len(self.lens):
                self.bits |= BAD_INDEX
                continue
            k = 0 if keep is None else int(keep[s])
            if k < 0:
                self.bits |= BAD_SEQLEN
                continue
            for j in range(-(-k // 64), self.table.shape[1]):
                if self.table[s, j] >= 0:
                    self.drop(self.table[s, j])
                    self.table[s, j] = -1
            self.lens[s] = min(self.lens[s], k)

    def fork(self, parents, children):
        b.lrkv_pages_fork(self.own, self.d["refs"], self.d["table"], self.d["lens"], i32(parents), i32(children),
                          status=self.status)
        B = len(self.lens)
        todo = []
        for i, (p, c) in enumerate(zip(parents, children)):
            if not (0 <= p < B and 0 <= c < B) or c in parents or list(children).count(c) > 1:
                self.bits |= BAD_INDEX
                continue
            L = int(self.lens[p])
            if not 0 <= L <= self.table.shape[1] * 64:
                self.bits |= BAD_SEQLEN
                continue
            row = self.table[p, :-(-L // 64)]
            if ((row < 0) | (row >= self.refs.size)).any():
                self.bits |= BAD_BLOCK
                continue
            todo.append((p, c, L))
        for _, c, _ in todo:
            for j in range(self.table.shape[1]):
                if self.table[c, j] >= 0:
                    self.drop(self.table[c, j])
            self.table[c] = -1
        new = []
        for p, c, L in todo:  # pages first, in the order of the call
            new.append(self.take() if L % 64 else -1)
        for (p, c, L), page in zip(todo, new):
            if page is None:
                self.bits |= NO_PAGES
                self.lens[c] = 0
                continue
            full = L // 64
            self.table[c, :full] = self.table[p, :full]
            np.add.at(self.refs, self.table[p, :full], 1)
            if L % 64:
                self.table[c, full] = page
                for t in self.pools:
                    t[:, page, :L % 64] = t[:, self.table[p, full], :L % 64]
            self.lens[c] = L

    def compact(self, path, n, in_place=True):
        out = None if in_place else i32(np.full(len(self.lens), -7))
        b.lrkv_cache_compact(self.own, self.d["table"], self.d["lens"], i32(path), i32(n), new_lens=out,
                             status=self.status)
        new = self.lens.copy()
        for s in range(len(self.lens)):
            L, k = int(self.lens[s]), int(n[s])
            if not 0 <= L <= self.table.shape[1] * 64:
                self.bits |= BAD_SEQLEN
                continue
            if not 0 <= k <= path.shape[1]:
                self.bits |= BAD_INDEX
                continue
            p, bad = path[s, :k].astype(np.int64), 0
            for i in range(k):
                if p[i] <= (p[i - 1] if i else -1) or p[i] < i:
                    bad |= BAD_INDEX
                elif L + p[i] >= self.table.shape[1] * 64:
                    bad |= BAD_SEQLEN
                else:
                    for at in (L + p[i], L + i):
                        if not 0 <= self.table[s, at // 64] < self.refs.size:
                            bad |= BAD_BLOCK
            self.bits |= bad
            if bad:
                continue
            slot = lambda at: (self.table[s, at // 64], at % 64)
            for i in range(k):
                f, t = slot(L + p[i]), slot(L + i)
                for x in self.pools:
                    x[:, t[0], t[1]] = x[:, f[0], f[1]]
            new[s] = L + k
        if in_place:
            self.lens = new
        else:
            assert np.array_equal(out.cpu().numpy(), new)

    def check(self, what=""):
        assert np.array_equal(self.d["table"].cpu().numpy(), self.table), what
        assert np.array_equal(self.d["refs"].cpu().numpy(), self.refs), what
        assert np.array_equal(self.d["lens"].cpu().numpy(), self.lens), what
        for t, p in zip(self.d["pools"], self.pools):
            assert np.array_equal(t.cpu().numpy(), p), what
        assert int(self.status.item()) == self.bits, (what, int(self.status.item()), self.bits)


@pytest.mark.parametrize("blocks,batch,width", [(1, 1, 1), (5, 2, 3), (40, 7, 9), (300, 40, 20), (2000, 100, 64)])
def test_reserve(blocks, batch, width):
    m = Model(blocks, batch, width, layers=1, widths=(8,))
    rng = np.random.default_rng(blocks)
    # pages that the caller keeps for itself
    m.refs[rng.random(blocks) < 0.2] = 3
    m.upload()
    for step in range(6):
        m.reserve(rng.integers(0, 64 * width // 3 + 2, batch))
        m.check(f"step {step}")
        for s in range(batch):  # the host takes some of it into use, as appends would
            m.lens[s] = rng.integers(m.lens[s], m.held(s) * 64 + 1)
        m.upload()


def test_reserve_takes_what_is_left_in_order():
    """Whole requests or none, in order; later ones that still fit are served."""
    m = Model(5, 4, 8)
    m.reserve([64 * 3, 64 * 4, 64 * 2, 1])
    assert m.bits == NO_PAGES
    m.check()
    assert (m.table[1] == -1).all() and m.held(0) == 3 and m.held(2) == 2 and m.held(3) == 0


def test_reserve_refuses_bad_lengths():
    m = Model(20, 5, 3)
    m.lens[:] = [0, -1, 64, 2 ** 31 - 1, 10]
    m.table[2, 0] = 7
    m.refs[7] = 1
    m.table[4, 0] = 8
    m.refs[8] = 1
    m.upload()
    m.reserve([193, 5, -1, 2 ** 31 - 1, 100])
    assert m.bits == BAD_SEQLEN
    m.check()


def test_pages_are_found_behind_many_taken_ones():
    """A pool of more pages than one round of the search covers, its last ones free (and not a multiple of 4)."""
    blocks = 16384 * 2 + 3
    m = Model(blocks, 3, 8, layers=1, widths=(8,))
    m.refs[:] = 1
    m.refs[[16383, 16384, blocks - 1, blocks - 2]] = 0
    m.upload()
    m.reserve([64, 65, 0])
    assert m.bits == 0 and m.table[1, 1] == blocks - 2
    m.check()
    m.reserve([64, 65, 129])
    assert m.bits == NO_PAGES
    m.check()


def random_state(seed, blocks=120, batch=12, width=9, layers=2):
    m = Model(blocks, batch, width, layers=layers, seed=seed)
    rng = np.random.default_rng(seed)
    m.reserve(rng.integers(0, 64 * width // 2, batch))
    for s in range(batch):
        m.lens[s] = rng.integers(0, m.held(s) * 64 + 1)
    m.lens[0] = m.held(0) * 64  # a full last page
    m.upload()
    return m, rng


@pytest.mark.parametrize("seed", range(6))
def test_random_runs(seed):
    """Reserve, compact, fork and free one after another on one state."""
    m, rng = random_state(seed, blocks=40 + 30 * seed)
    B = len(m.lens)
    for step in range(12):
        kind = rng.integers(0, 4)
        if kind == 0:
            m.reserve(rng.integers(0, 130, B))
        elif kind == 1:
            kids = rng.permutation(B)[:rng.integers(1, B // 2)]
            rest = [s for s in range(B) if s not in kids]
            m.fork(rng.choice(rest, kids.size), kids)
        elif kind == 2:
            seqs = rng.integers(0, B, rng.integers(1, 5))  # some listed twice
            m.free(seqs, None if rng.random() < 0.3 else rng.integers(0, 300, B))
        else:
            T = int(rng.integers(1, 40))
            room = [m.held(s) * 64 - int(m.lens[s]) for s in range(B)]
            path, n = np.zeros((B, T), np.int32), np.zeros(B, np.int32)
            for s in range(B):
                k = int(rng.integers(0, min(room[s], T) + 1)) if room[s] > 0 else 0
                path[s, :k] = np.sort(rng.permutation(room[s])[:k])
                n[s] = k
            m.compact(path, n, in_place=bool(rng.random() < 0.7))
        m.check(f"seed {seed}, step {step}, kind {kind}")
    # counts are what the table names
    assert np.array_equal(m.refs, np.bincount(m.table[m.table >= 0], minlength=m.refs.size))
    m.free(np.arange(B))
    m.check("all given back")
    assert (m.refs == 0).all()


def test_fork_refusals():
    m, _ = random_state(50)
    m.lens[5] = -3
    m.lens[6] = 64 * 9 + 1
    m.lens[7] = 70
    m.table[7, :2] = [3, 120]  # a bad page id in what would be passed on
    m.refs[:] = np.bincount(m.table[(m.table >= 0) & (m.table < 120)], minlength=120)
    m.upload()
    m.fork([0, 1, 1, 2, -1, 0, 12, 5, 6, 7], [1, 9, 9, 2, 3, -1, 4, 10, 10, 11])
    assert m.bits == BAD_INDEX | BAD_BLOCK
    m.check()
    m.fork([5, 6], [10, 3])
    assert m.bits == BAD_INDEX | BAD_BLOCK | BAD_SEQLEN
    m.check()


def test_a_child_that_stands_like_its_parent_is_left_alone_when_refused():
    """A refused fork writes no row, even where the child already has the parent's length and a last page of its own."""
    m = Model(10, 4, 4)
    m.reserve([100, 100, 0, 0])
    m.lens[:2] = 100
    m.upload()
    m.fork([0, 0, 1], [1, 2, 3])  # 1 is also a parent
    assert m.bits == BAD_INDEX
    m.check()


def test_fork_without_pages_leaves_an_empty_child():
    m = Model(4, 5, 4)
    m.reserve([130, 64, 0, 0, 0])
    m.lens[:] = [130, 64, 0, 0, 0]
    m.upload()
    m.fork([0, 1, 0], [2, 3, 4])
    assert m.bits == NO_PAGES and m.lens[2] == 0 and m.lens[3] == 64
    m.check()
    # what a child held is given back first, and is enough here
    m = Model(3, 3, 4)
    m.reserve([64, 100, 0])
    m.lens[:] = [64, 100, 0]
    m.upload()
    m.fork([1], [0])
    assert m.bits == 0
    m.check()


def test_free_refusals():
    m, _ = random_state(60)
    keep = np.full(12, 64)
    keep[3] = -1
    m.refs[m.table[4, 1]] = 0  # a count that the caller has lost
    m.table[5, 2] = 500
    m.upload()
    m.free([-1, 12, 3, 4, 4, 5], keep)
    assert m.bits & BAD_INDEX and m.bits & BAD_SEQLEN and m.bits & BAD_BLOCK
    m.check()


def test_compact_refusals():
    m, _ = random_state(70)
    m.reserve(np.full(12, 64))
    m.upload()
    path = np.tile(np.array([0, 3, 5, 9], np.int32), (12, 1))
    n = np.full(12, 4)
    path[1] = [0, 3, 3, 9]
    path[2] = [2, 1, 5, 9]
    path[3] = [-1, 1, 5, 9]
    n[4], n[5] = 5, -1
    path[6] = [0, 1, 2, 2 ** 31 - 1]
    m.lens[7] = -1
    m.lens[8] = 64 * 9 + 1
    m.table[9, (m.lens[9] + 9) // 64] = -1
    m.table[10, m.lens[10] // 64] = 120
    m.upload()
    m.compact(path, n, in_place=False)
    m.compact(path, n)
    assert m.bits & ~NO_PAGES == BAD_INDEX | BAD_SEQLEN | BAD_BLOCK
    m.check()


def test_long_paths_over_pages():
    """A thousand rows of each sequence, over many pages, each moved by little; rows of one 16-byte unit and of many."""
    m = Model(90, 2, 40, layers=3, widths=(8, 520))
    m.reserve([64 * 38, 64 * 38])
    m.lens[:] = [1, 130]
    m.upload()
    rng = np.random.default_rng(1)
    path = np.stack([np.sort(rng.permutation(1100)[:1024]) for _ in range(2)]).astype(np.int32)
    m.compact(path, np.array([1024, 1000]))
    m.check()


@pytest.mark.parametrize("layers,widths", [(1, (8,)), (3, (64, 8, 24)), (2, (576,)), (1, (128, 128, 1024, 1024))])
def test_copy(layers, widths):
    m = Model(30, 1, 1, layers=layers, widths=widths)
    o = Model(17, 1, 1, layers=layers, widths=widths, seed=5)
    src = [0, 29, -1, 7, 7, 30, 3, 4]
    dst = [16, 0, 3, 5, 6, 7, -2, 17]
    b.lrkv_pages_copy(m.own, i32(src), o.own, i32(dst), status=m.status)
    for s, t in zip(src, dst):
        if 0 <= s < 30 and 0 <= t < 17:
            for x, y in zip(m.pools, o.pools):
                y[:, t] = x[:, s]
    m.bits = BAD_BLOCK
    m.check()
    o.check()


def test_copy_beyond_32_bit_offsets():
    blocks = (1 << 31) // (64 * 1024) + 3
    pool = torch.zeros(1, blocks, 64, 1024, dtype=torch.bfloat16, device="cuda")
    pool[0, 1].normal_()
    p = b.Pools([pool])
    b.lrkv_pages_copy(p, i32([1]), p, i32([blocks - 1]))
    assert torch.equal(pool[0, 1], pool[0, blocks - 1]) and (pool[0, blocks - 2] == 0).all()
    page = pool[0, 1].clone()
    table, lens = i32([[1, blocks - 2, blocks - 1]]), i32([126])
    b.lrkv_cache_compact(p, table, lens, i32([[1, 3, 5, 60]]), i32([4]))  # rows 127, 129, 131, 186
    assert int(lens) == 130 and torch.equal(pool[0, 1], page)
    assert (pool[0, blocks - 2, :63] == 0).all() and torch.equal(pool[0, blocks - 2, 63], page[1])
    assert torch.equal(pool[0, blocks - 1, :2], page[[3, 58]]) and torch.equal(pool[0, blocks - 1, 2:], page[2:])


def test_layers_apart_and_other_caches():
    """Layers with a gap between them; the rows of a quantised and of a latent cache."""
    big = torch.randint(0, 100, (3, 9, 64, 16), dtype=torch.int16, device="cuda")
    p = b.Pools([big[:, :6]])
    before = big.clone()
    b.lrkv_pages_copy(p, i32([0]), p, i32([5]))
    before[:, 5] = before[:, 0]
    assert torch.equal(big, before)
    dims = b.make_dims(3, 64, 8, 192)
    q = b.QuantCache(torch.randint(0, 256, (4, 64, b.quant_row_bytes(dims)), dtype=torch.uint8, device="cuda"))
    kv = torch.randn(4, 64, 576, device="cuda").to(torch.bfloat16)
    for c, t in ((q, q.rows), (kv, kv)):
        pools = b.Pools.of(c)
        t0 = t.clone()
        b.lrkv_cache_compact(pools, i32([[2, 0]]), i32([63]), i32([[1, 2]]), i32([2]))
        t0[2, 63], t0[0, 0] = t0[0, 0].clone(), t0[0, 1].clone()
        assert torch.equal(t, t0)


def test_graph_replays():
    """Reserve, compact, fork and free captured once and replayed on a state that goes on."""
    m, _ = random_state(80, blocks=200)
    B = len(m.lens)
    d = m.d
    add, path, n = i32(np.full(B, 20)), i32(np.tile([1, 4, 6], (B, 1))), i32(np.full(B, 3))
    kids, par = i32([10, 11]), i32([2, 2])
    seqs = i32(np.arange(B))

    def step():
        b.lrkv_pages_reserve(d["refs"], d["table"], d["lens"], add, status=m.status)
        b.lrkv_cache_compact(m.own, d["table"], d["lens"], path, n, status=m.status)
        b.lrkv_pages_free(d["refs"], d["table"], d["lens"], seqs, keep_lens=d["lens"], status=m.status)
        b.lrkv_pages_fork(m.own, d["refs"], d["table"], d["lens"], par, kids, status=m.status)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    m.upload()
    for _ in range(5):
        g.replay()
    got = {k: d[k].clone() for k in ("refs", "table", "lens")}
    pools = [p.clone() for p in d["pools"]]
    m.upload()
    for _ in range(5):
        step()
    assert all(torch.equal(got[k], d[k]) for k in got) and all(torch.equal(x, y) for x, y in zip(pools, d["pools"]))
    assert int(m.status.item()) == 0
