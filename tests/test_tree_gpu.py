"""Attention of drafted tokens over the cache, against attention in 64 bits over what each token sees."""
import pytest
import torch

from attn64 import attend64, check

pytestmark = pytest.mark.gpu

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402

BAD_BLOCK, BAD_SEQLEN = b.DEV_BAD_BLOCK, b.DEV_BAD_SEQLEN
MARK = 7.0  # in rows of out that a call must not touch


def words(m):
    """Bool [.., 64] -> 64-bit words."""
    w = torch.zeros(m.shape[:-1], dtype=torch.int64)
    for j in range(64):
        w |= m[..., j].long() << j
    return w


class Case:
    """Pools with NaN in every row that no token uses; masks with bits behind the drafted tokens set."""

    def __init__(self, seed, H, d_h, r, d_rope, lens, drafted, T=None, mask="tree", cap=0, blocks=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        c = torch.Generator().manual_seed(seed)
        B, T = len(lens), T or max(drafted)
        self.H, self.d_h, self.r, self.d_rope, self.lens, self.drafted, self.T = H, d_h, r, d_rope, lens, drafted, T
        self.dims = b.make_dims(H, d_h, r, H * d_h, d_rope=d_rope)
        pages = [-(-(n + k) // 64) for n, k in zip(lens, drafted)]
        nb = blocks or sum(pages) + 2
        ids = (torch.randperm(sum(pages) + 2, generator=c) + (nb - sum(pages) - 2)).int()
        self.bt = torch.full((B, max(1, max(pages)) + cap), -1, dtype=torch.int32)
        at = 0
        for i, p in enumerate(pages):
            self.bt[i, :p] = ids[at:at + p]
            at += p
        self.slots = [self.bt[i, t // 64].long() * 64 + t % 64
                      for i, t in enumerate(torch.arange(n + k) for n, k in zip(lens, drafted))]
        used = torch.cat(self.slots).cuda()
        self.bt = self.bt.cuda()
        pools = []
        for s in ((d_h + d_rope,), (d_h,), (H, r), (H, r)):
            t = torch.full((nb * 64, *s), float("nan"), dtype=torch.bfloat16, device="cuda")
            t[used] = torch.randn(used.numel(), *s, generator=g, device="cuda").to(torch.bfloat16)
            pools.append(t.view(nb, 64, *s))
        self.cache = b.PagedCache(*pools)
        self.q = torch.randn(B, T, H, d_h + d_rope, generator=g, device="cuda").to(torch.bfloat16)
        fk = lambda: (torch.randn(H, d_h, r, generator=g, device="cuda") * r ** -0.5).to(torch.bfloat16)
        self.BK, self.BV = fk(), fk()
        m = torch.zeros(B, T, 64, dtype=torch.bool)
        for i in range(B):
            for k in range(T):
                if mask == "chain":
                    m[i, k, :k + 1] = True
                elif mask == "random":  # any set, the token itself or all drafted ones missing at times
                    m[i, k] = torch.rand(64, generator=c) < torch.rand(1, generator=c)
                elif mask == "none":
                    m[i, k, drafted[i]:] = True
                else:
                    if k:
                        m[i, k] = m[i, torch.randint(0, k, (1,), generator=c).item()]
                    m[i, k, k] = True
        self.seen = m.clone()
        m |= torch.arange(64) >= torch.tensor(drafted)[:, None, None]
        self.mask = words(m).cuda()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.sl, self.tl = i32(lens), i32(drafted)
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = b.alloc_workspace(b.decode_tree_workspace_bytes(self.dims, B, T))
        self.ws.fill_(255)
        self.out = torch.full((B, T, H, d_h), MARK, dtype=torch.bfloat16, device="cuda")

    def run(self, mask=True, lens=True, stream=None):
        b.lrkv_decode_tree(self.dims, self.q, self.BK, self.BV, self.cache, self.bt, self.sl,
                           self.mask if mask else None, self.tl if lens else None, self.out, self.ws, status=self.st,
                           stream=stream)
        return self.out

    def parts(self, i, k):
        """What drafted token k of sequence i sees."""
        s, L = self.slots[i], self.lens[i]
        at = torch.cat([s[:L], s[L:][self.seen[i, k, :self.drafted[i]]]]).cuda()
        return [t.view(-1, *t.shape[2:])[at].double() for t in self.cache.tensors()]

    def verify(self, seqs=None, what="tree", heads=None, every=1):
        for i in range(len(self.lens)) if seqs is None else seqs:
            n = self.drafted[i]
            assert (self.out[i, n:] == MARK).all(), f"rows behind the drafted tokens of sequence {i}"
            for k in {*range(0, n, every), n - 1} - {-1}:
                parts = self.parts(i, k)
                if parts[0].shape[0] == 0:
                    assert (self.out[i, k] == 0).all(), f"token {k} of sequence {i} sees nothing"
                    continue
                # probabilities are rounded to bf16 for the tensor cores; q~ goes there in two bf16 pieces
                want, bound = attend64(self.q[i, k].double(), self.BK.double(), self.BV.double(), parts, self.d_rope,
                                       eps_p=2.0 ** -8, eps_qt=2.0 ** -16)
                h = slice(None) if heads is None else heads
                check(self.out[i, k][h], want[h], bound[h], f"{what}: token {k} of {n}, {self.lens[i]} before")


CASES = [
    (1, 64, 8, 0, [0], [1], "tree"), (1, 128, 32, 64, [0, 1, 63], [1, 3, 64], "tree"), (3, 64, 8, 0, [64, 5], [64, 1], "random"),
    (8, 64, 16, 0, [256], [4], "chain"), (8, 64, 16, 0, [62, 63, 64, 65, 127], [2, 2, 2, 2, 2], "random"),
    (9, 64, 32, 0, [129, 0], [33, 7], "random"), (5, 128, 8, 64, [1000, 3], [17, 64], "tree"),
    (16, 128, 16, 0, [2000, 1, 700], [9, 16, 15], "tree"), (32, 128, 16, 64, [333, 4100], [26, 13], "tree"),
    (32, 128, 32, 0, [5000], [8], "chain"), (20, 64, 16, 64, [200] * 5, [5, 1, 3, 2, 4], "random"),
    (40, 128, 8, 0, [500, 0], [33, 1], "tree"), (128, 128, 16, 64, [640], [64], "tree"),
    (128, 64, 8, 0, [100, 30], [10, 20], "random"), (100, 128, 32, 0, [320], [3], "tree"),
    (128, 128, 32, 0, [192, 66], [2, 5], "chain"), (2, 128, 16, 0, [9000], [50], "tree"),
    (6, 64, 32, 64, [100, 20, 30], [40, 2, 64], "none"), (32, 128, 16, 0, [0] * 3, [64, 40, 9], "random"),
    (128, 128, 8, 0, [70], [1], "chain"), (128, 128, 16, 0, [1500], [1], "chain"), (7, 64, 16, 0, [31] * 70, [3] * 70, "tree"),
]


@pytest.mark.parametrize("H,d_h,r,d_rope,lens,drafted,mask", CASES,
                         ids=[f"H{c[0]}_dh{c[1]}_r{c[2]}_rope{c[3]}_L{c[4][0]}_B{len(c[4])}_T{max(c[5])}_{c[6]}" for c in CASES])
def test_matches_64_bits(H, d_h, r, d_rope, lens, drafted, mask):
    c = Case(H + r + lens[0], H, d_h, r, d_rope, lens, drafted, mask=mask)
    c.run()
    assert int(c.st.item()) == 0
    c.verify(every=1 if len(lens) < 10 else 2)
    first = c.out.clone()
    c.ws.fill_(0x7f)
    c.run()  # the same again, from another workspace content: bit for bit
    assert torch.equal(c.out, first)


def test_no_mask_is_a_chain_and_no_counts_are_all():
    c = Case(1, 8, 128, 16, 0, [100, 61, 0], [12, 12, 12], mask="chain")
    c.run()
    want = c.out.clone()
    c.out.fill_(MARK)
    c.run(mask=False, lens=False)
    assert torch.equal(c.out, want)
    c.verify()


def test_one_drafted_token_is_a_decode():
    """T = 1: lrkv_decode over one token more, within both calls' bounds."""
    c = Case(2, 32, 128, 16, 0, [300, 1, 5000], [1, 1, 1], mask="chain")
    c.run()
    c.verify()
    out = torch.empty_like(c.out[:, 0])
    ws = b.alloc_workspace(b.decode_workspace_bytes(c.dims, 3))
    b.lrkv_decode(c.dims, c.q[:, 0].contiguous(), c.BK, c.BV, c.cache, c.bt, c.sl + 1, out, ws)
    assert ((out.double() - c.out[:, 0].double()).norm() / out.double().norm()) <= 1e-2


@pytest.mark.parametrize("d_h,r,d_rope,H", [(128, 16, 0, 32), (64, 32, 64, 5), (128, 32, 0, 3), (64, 8, 0, 40)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_seen_does_not_reach_a_result(bad, d_h, r, d_rope, H):
    """A drafted token with non-finite keys and values: its own branch shows it, the others are as without it."""
    c = Case(3, H, d_h, r, d_rope, [90, 0], [24, 24], mask="random")
    c.seen[:, :, 5] = torch.arange(24) % 3 == 0
    c.mask = words(c.seen | (torch.arange(64) >= 24)).cuda()
    for kind in range(3):
        slots = torch.stack([c.slots[i][c.lens[i] + 5] for i in range(2)]).cuda()
        saved = [t.view(-1, *t.shape[2:])[slots] for t in c.cache.tensors()]
        k, v, zk, zv = (t.view(-1, *t.shape[2:]) for t in c.cache.tensors())
        if kind == 0:
            k[slots, 3] = bad
        elif kind == 1:
            v[slots, 7] = bad
        else:
            zv[slots, H - 1, 2] = bad
        c.out.fill_(MARK)
        c.run()
        for i in range(2):
            for q in range(24):
                got = c.out[i, q]
                if not c.seen[i, q, 5]:
                    if c.parts(i, q)[0].shape[0] == 0:
                        assert (got == 0).all()
                        continue
                    want, bound = attend64(c.q[i, q].double(), c.BK.double(), c.BV.double(), c.parts(i, q), c.d_rope,
                                           eps_qt=2.0 ** -16)
                    check(got, want, bound, f"kind {kind}, token {q} of sequence {i}")
                elif kind == 1:
                    col = torch.ones(d_h, dtype=torch.bool)
                    col[7] = False
                    assert not torch.isfinite(got[:, 7]).any() and torch.isfinite(got[:, col]).all()
                elif kind == 2:
                    assert not torch.isfinite(got[H - 1]).any() and torch.isfinite(got[:H - 1]).all()
                elif bad != bad:
                    assert torch.isnan(got).all()
        for t, s in zip((k, v, zk, zv), saved):
            t[slots] = s
    assert int(c.st.item()) == 0


def test_latents_of_other_heads_do_not_reach_a_head():
    """NaN and infinities in one head's latents, in the cached and in the drafted tokens."""
    c = Case(4, 16, 128, 16, 0, [200], [20])
    zk, zv = c.cache.zK.view(-1, 16, 16), c.cache.zV.view(-1, 16, 16)
    for t in (3, 150, 205):
        zk[c.slots[0][t].item(), 5, 1] = float("inf") if t == 3 else float("nan")
        zv[c.slots[0][t].item(), 9, 1] = float("inf")
    c.run()
    ok = [h for h in range(16) if h not in (5, 9)]
    keep5, keep9 = zk[:, 5].clone(), zv[:, 9].clone()
    zk[:, 5], zv[:, 9] = 0, 0
    c.verify(heads=ok)
    zk[:, 5], zv[:, 9] = keep5, keep9


def test_bad_lengths_and_pages():
    for sl, tl in (([-1, 184], None), ([100, 2 ** 31 - 1], None), (None, [-1, 8]), (None, [5, 9]), ([188, 188], None)):
        c = Case(5, 8, 64, 16, 0, [100, 184], [5, 8])
        sl, tl = sl or c.lens, tl or c.drafted
        c.sl.copy_(torch.tensor(sl))
        c.tl.copy_(torch.tensor(tl))
        c.run()
        assert int(c.st.item()) == BAD_SEQLEN
        good = [i for i in range(2) if sl[i] == c.lens[i] and tl[i] == c.drafted[i]]
        for i in range(2):
            assert i in good or (c.out[i] == 0).all()
        c.verify(seqs=good)
    for bad in (-1, 1000, 2 ** 31 - 1):
        c = Case(6, 8, 128, 16, 0, [300, 10], [5, 6], mask="chain")
        c.bt[0, 1] = bad
        c.run()
        assert int(c.st.item()) == BAD_BLOCK
        c.verify(seqs=[1])
        c.slots[0] = torch.cat([c.slots[0][:64], c.slots[0][128:]])  # its tokens are left out
        c.lens[0] -= 64
        c.verify(seqs=[0])
    # the only page of a sequence, and the page of the drafted tokens
    c = Case(7, 8, 128, 16, 0, [10, 64], [5, 6], mask="chain")
    c.bt[0, 0] = c.bt[1, 1] = -1
    c.run()
    assert int(c.st.item()) == BAD_BLOCK and (c.out[0, :5] == 0).all() and (c.out[0, 5:] == MARK).all()
    c.seen[1] = False
    c.verify(seqs=[1])


def test_no_drafted_tokens():
    c = Case(8, 8, 64, 16, 0, [50, 0, 70], [0, 0, 3], T=3)
    c.run()
    assert int(c.st.item()) == 0
    c.verify()


def test_sharp_and_flat_logits():
    """One token takes nearly all of the softmax, in every place of the row in turn; and all logits equal."""
    c = Case(9, 8, 128, 16, 0, [400], [12])
    k = c.cache.sK.view(-1, 128)
    for t in (0, 63, 64, 399, 401):
        old = k[c.slots[0][t].item()].clone()
        k[c.slots[0][t].item()] = (c.q[0, 3, 2] * 4).to(torch.bfloat16)
        c.run()
        c.verify(what=f"sharp at {t}")
        k[c.slots[0][t].item()] = old
    c.q.zero_()
    c.run()
    c.verify(what="flat")


def test_wide_table():
    c = Case(10, 16, 128, 16, 0, [200, 1], [10, 3], cap=3000)
    c.run()
    c.verify()


def test_rows_beyond_32_bit_offsets():
    """Pages whose latents start more than 2^31 elements into their pool."""
    H, r = 128, 32
    c = Case(11, H, 128, r, 0, [130, 40], [9, 2], blocks=(1 << 31) // (64 * H * r) + 8)
    assert int(c.bt.max()) * 64 * H * r > 1 << 31
    c.run()
    c.verify(every=4)


def test_streams_and_workspaces():
    """Two calls at once on two streams, each with a workspace of its own; and one after another in one workspace."""
    a, d = Case(12, 32, 128, 16, 0, [3000, 17], [16, 9]), Case(13, 8, 64, 8, 64, [900] * 9, [7] * 9)
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, st in zip((a, d), s):
            with torch.cuda.stream(st):
                c.run()
    torch.cuda.synchronize()
    a.verify(every=3)
    d.verify(every=3)
    ws = b.alloc_workspace(max(a.ws.nbytes, d.ws.nbytes))
    for c in (a, d):
        c.first = c.out.clone()
        c.out.fill_(MARK)
        c.ws = ws
    for _ in range(3):
        for c in (a, d):
            c.run()
    assert torch.equal(a.out, a.first) and torch.equal(d.out, d.first)


def test_graph_replays_with_other_lengths():
    c = Case(14, 16, 128, 16, 0, [700, 90, 0], [20, 11, 3])
    c.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for lens, drafted in (([700, 90, 0], [20, 11, 3]), ([64, 95, 1], [1, 6, 2]), ([716, 0, 0], [4, 20, 0])):
        c.sl.copy_(torch.tensor(lens))
        c.tl.copy_(torch.tensor(drafted))
        c.out.fill_(MARK)
        g.replay()
        got = c.out.clone()
        c.out.fill_(MARK)
        c.run()
        torch.cuda.synchronize()
        # (masks and pages fit the first lengths; drafted tokens are NaN or cached ones here, so only the equality is asked)
        assert torch.equal(got.nan_to_num(5.0), c.out.nan_to_num(5.0))
    c.sl.copy_(torch.tensor([700, 90, 0]))
    c.tl.copy_(torch.tensor([20, 11, 3]))
    c.out.fill_(MARK)
    g.replay()
    c.verify()


def test_workspace_is_checked():
    c = Case(15, 8, 64, 16, 0, [10], [4])
    need = b.decode_tree_workspace_bytes(c.dims, 1, 4)
    assert need > 0
    for ws in (c.ws[:need - 1], c.ws[16:]):
        with pytest.raises(b.LrkvError) as e:
            b.lrkv_decode_tree(c.dims, c.q, c.BK, c.BV, c.cache, c.bt, c.sl, c.mask, c.tl, c.out, ws)
        assert e.value.status in (1, 3)
    assert (c.out == MARK).all()


@pytest.mark.parametrize("H,d_h,r,d_rope,lens,T", [(32, 128, 16, 0, [4000, 200], 20), (32, 128, 32, 0, [3000], 8),
                                                   (8, 64, 16, 64, [900] * 8, 64), (128, 128, 16, 0, [700, 90], 64)])
def test_expired_wait_reports_timeout_and_gpu_stays_usable(monkeypatch, H, d_h, r, d_rope, lens, T):
    """With the debugging limit LRKV_DEBUG_WAIT_LIMIT_NS=0 the scan's waits give up as soon as something is not already
    there.  The call ends, reports LRKV_DEV_TIMEOUT and nothing else, and the next one is right to the bit."""
    c = Case(16, H, d_h, r, d_rope, lens, [T] * len(lens))
    c.run()
    assert int(c.st.item()) == 0
    want = c.out.clone()
    c.verify(every=7)
    monkeypatch.setenv("LRKV_DEBUG_WAIT_LIMIT_NS", "0")
    seen = 0
    for _ in range(5):
        c.run()
        seen |= int(c.st.item())
    assert seen == b.DEV_TIMEOUT
    monkeypatch.delenv("LRKV_DEBUG_WAIT_LIMIT_NS")
    c.st.zero_()
    c.out.fill_(MARK)
    c.run()
    assert int(c.st.item()) == 0 and torch.equal(c.out, want)


def test_many_short_sequences():
    """More tiles than the GPU takes at once, of a page or two each, one drafted token and several; odd head counts."""
    for H, r, T in ((33, 32, 1), (17, 16, 3)):
        c = Case(17, H, 128, r, 0, [5 * i % 130 for i in range(150)], [1 + i % T for i in range(150)])
        c.run()
        assert int(c.st.item()) == 0
        c.verify(seqs=range(0, 150, 7))


def test_consecutive_one_page_pieces_repeat_exactly():
    """CTAs with many pieces of one page each: the group of rows without a page goes ahead into the next piece, whose
    sums must not reach the piece before.  Every sequence is compared with 64 bits, and runs with one another."""
    c = Case(23, 33, 128, 16, 0, [7 * i % 60 for i in range(300)], [1 + i % 3 for i in range(300)])
    first = c.run().clone()
    assert int(c.st.item()) == 0
    c.verify(seqs=range(0, 300, 3))
    for _ in range(20):
        assert torch.equal(c.run(), first)


def test_workspace_stays_in_proportion():
    """The workspace grows with the queries, not with the rows of the kernel's tiles: for one drafted token at most
    32 rows a tile are kept."""
    dims = b.make_dims(128, 128, 16, 128 * 128)
    for T in (1, 8, 64):
        per_query = b.decode_tree_workspace_bytes(dims, 256, T) / (256 * T * 128)
        assert per_query <= 4 * (128 + 16 + 16 + 2) * (32 / min(32, 8 * T)) * 1.2 + 64, T
