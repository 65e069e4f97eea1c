"""Decode of a batch that shares a prefix, against attention in 64 bits over the prefix and the
sequence's own tokens."""
import pytest
import torch

from attn64 import attend64, check

pytestmark = pytest.mark.gpu

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402

BAD_BLOCK, BAD_SEQLEN = b.DEV_BAD_BLOCK, b.DEV_BAD_SEQLEN


class Case:
    """Pools with NaN in every row that no token uses."""

    def __init__(self, seed, H, d_h, r, d_rope, P, lens, cap=0, num_splits=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.H, self.d_h, self.r, self.d_rope, self.P, self.lens = H, d_h, r, d_rope, P, list(lens)
        B = len(lens)
        self.dims = b.make_dims(H, d_h, r, H * d_h, d_rope=d_rope, num_splits=num_splits)
        pp, pages = (P + 63) // 64, [(n + 63) // 64 for n in lens]
        nb = pp + sum(pages) + 2
        ids = torch.randperm(nb, generator=g, device="cuda").int()
        self.blocks = torch.full((max(1, pp) + cap,), -1, dtype=torch.int32, device="cuda")
        self.blocks[:pp] = ids[:pp]
        self.bt = torch.full((B, max(1, max(pages))), -1, dtype=torch.int32, device="cuda")
        at = pp
        for i, p in enumerate(pages):
            self.bt[i, :p] = ids[at:at + p]
            at += p
        mk = lambda *s: torch.randn(nb, 64, *s, generator=g, device="cuda").to(torch.bfloat16)
        pools = [mk(d_h + d_rope), mk(d_h), mk(H, r), mk(H, r)]
        self.pslots = self.at(self.blocks, P)
        self.slots = [self.at(self.bt[i], n) for i, n in enumerate(lens)]
        used = torch.zeros(nb * 64, dtype=torch.bool, device="cuda")
        for s in [self.pslots] + self.slots:
            used[s] = True
        for t in pools:
            t.view(nb * 64, -1)[~used] = float("nan")
        self.cache = b.PagedCache(*pools)
        self.q = torch.randn(B, H, d_h + d_rope, generator=g, device="cuda").to(torch.bfloat16)
        fk = lambda: (torch.randn(H, d_h, r, generator=g, device="cuda") * r ** -0.5).to(torch.bfloat16)
        self.BK, self.BV = fk(), fk()
        self.sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.pl = torch.tensor([P], dtype=torch.int32, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = b.alloc_workspace(b.decode_shared_workspace_bytes(self.dims, B, int(self.blocks.shape[0])))
        self.ws.fill_(255)
        self.out = torch.full((B, H, d_h), float("nan"), dtype=torch.bfloat16, device="cuda")

    def at(self, pages, n):
        t = torch.arange(n, device="cuda")
        return pages[t // 64].long() * 64 + t % 64

    def run(self, stream=None):
        b.lrkv_decode_shared(self.dims, self.q, self.BK, self.BV, self.cache, self.blocks, self.pl, self.bt, self.sl,
                             self.out, self.ws, status=self.st, stream=stream)
        return self.out

    def parts(self, i):
        s = torch.cat([self.pslots, self.slots[i]])
        k, v, zk, zv = self.cache.tensors()
        f = lambda t: t.view(-1, *t.shape[2:])[s].double()
        return f(k), f(v), f(zk), f(zv)

    def verify(self, out=None, seqs=None, what="decode_shared", rel_max=5e-3):
        out = self.out if out is None else out
        seqs = range(len(self.lens)) if seqs is None else seqs
        for i in seqs:
            # probabilities are rounded to bf16 for the tensor cores; so is q~ for a sequence's own tokens
            want, bound = attend64(self.q[i].double(), self.BK.double(), self.BV.double(), self.parts(i), self.d_rope,
                                   eps_p=2.0 ** -8, eps_qt=2.0 ** -8)
            check(out[i], want, bound, f"{what} P={self.P} sequence {i} of {self.lens[i]}", rel_max)


CASES = [
    (1, 64, 8, 0, 1, [0]), (1, 128, 32, 64, 300, [1, 0, 70]), (3, 64, 8, 0, 63, [5, 0]), (8, 64, 16, 0, 64, [64, 1, 0, 9]),
    (8, 64, 16, 0, 65, [2] * 5), (9, 64, 32, 0, 129, [33]), (5, 128, 8, 64, 1000, [100] * 7),
    (16, 128, 16, 0, 2000, list(range(0, 33))), (32, 128, 16, 0, 4100, [17] * 16), (32, 128, 32, 0, 777, [1] * 33),
    (20, 64, 16, 64, 200, [3] * 130), (40, 128, 8, 0, 500, [0] * 9), (128, 128, 16, 64, 640, [50, 0, 1]),
    (128, 64, 8, 0, 100, [10] * 20), (100, 128, 32, 0, 320, [7, 8]), (128, 128, 32, 0, 192, [66, 2]),
    (2, 128, 16, 0, 9000, [1, 2, 3]), (128, 128, 16, 0, 300, [66, 2, 0, 500]), (128, 128, 8, 0, 70, [1] * 17 + [300]),
]


@pytest.mark.parametrize("H,d_h,r,d_rope,P,lens", CASES,
                         ids=[f"H{c[0]}_dh{c[1]}_r{c[2]}_rope{c[3]}_P{c[4]}_B{len(c[5])}" for c in CASES])
def test_matches_64_bits(H, d_h, r, d_rope, P, lens):
    c = Case(H + r + P, H, d_h, r, d_rope, P, lens)
    c.run()
    assert int(c.st.item()) == 0
    c.verify()


def test_no_prefix():
    """prefix_len 0: the sequences' own tokens alone; a sequence without any gets zeros and a status bit."""
    c = Case(1, 8, 64, 16, 0, 0, [100, 3])
    c.run()
    assert int(c.st.item()) == 0
    c.verify()
    c = Case(2, 8, 64, 16, 0, 0, [100, 0])
    c.run()
    assert int(c.st.item()) == BAD_SEQLEN and (c.out[1] == 0).all()
    c.verify(seqs=[0])


def test_decode_of_128_heads_with_r_8():
    """The sequences' own scan by itself, lrkv_decode."""
    c = Case(22, 128, 128, 8, 0, 0, [300, 9, 64])
    b.lrkv_decode(c.dims, c.q, c.BK, c.BV, c.cache, c.bt, c.sl, c.out, c.ws, status=c.st)
    assert int(c.st.item()) == 0
    c.verify(what="decode")


def test_table_longer_than_the_prefix():
    c = Case(3, 16, 128, 16, 0, 200, [10, 0], cap=300)
    c.run()
    assert int(c.st.item()) == 0
    c.verify()


def test_bad_lengths_and_pages():
    for bad in (-1, 257):
        c = Case(4, 8, 64, 16, 0, 200, [10, 0])
        c.pl.fill_(bad)
        c.run()
        assert int(c.st.item()) == BAD_SEQLEN and (c.out == 0).all()
    c = Case(5, 8, 64, 16, 0, 200, [10, 20, 30])
    c.sl[1] = 65
    c.sl[2] = -1
    c.run()
    assert int(c.st.item()) == BAD_SEQLEN and (c.out[1:] == 0).all()
    c.verify(seqs=[0])
    for bad in (-1, 10 ** 6):
        c = Case(6, 8, 64, 16, 0, 200, [10, 0])
        c.blocks[1] = bad
        c.run()
        assert int(c.st.item()) == BAD_BLOCK
        c.pslots = torch.cat([c.pslots[:64], c.pslots[128:]])
        c.verify()


def test_sharp_and_flat_logits():
    c = Case(7, 16, 128, 16, 0, 1500, [40] * 20)
    c.q[:10] *= 20
    c.q[10:15] = 0
    c.run()
    c.verify(rel_max=1.0)  # (logits 20 times as large magnify q~'s rounding: the bound says by how much)


def test_queries_keep_more_than_one_rounding():
    """Two roundings to bf16 are left over a prefix, the probabilities' and the output's.  Rounding x = f 2^e, f
    spread evenly over [1, 2), is off by up to 2^-8 2^e: 2^-8 / sqrt 3 * sqrt E[f^-2] = 0.0016 of x, root mean
    square, and two of them 0.0023.  q~ rounded to bf16 as well would move logits of unit spread by as much again:
    0.0028."""
    for H, d_h, P in ((32, 128, 4096), (8, 64, 500)):
        c = Case(20, H, d_h, 16, 0, P, [0, 0])
        c.run()
        c.verify(rel_max=2.5e-3)


def test_prefix_partials_join_other_caches():
    """A prefix in bf16 pages, old own tokens in 8 bits, the newest in bf16: three partials, one merge."""
    H, d_h, r, P = 16, 128, 16, 500
    lens = [100, 30, 64, 1]
    c = Case(8, H, d_h, r, 0, P, lens)
    B = len(lens)
    qc = b.QuantCache.empty(c.dims, c.cache.num_blocks)
    old = [64, 0, 64, 0]
    slots = torch.cat([s[:n] for s, n in zip(c.slots, old)]).int()
    b.lrkv_cache_quantize(c.dims, c.cache, slots, qc, slots, status=c.st)
    b.lrkv_cache_dequantize(c.dims, qc, slots, c.cache, slots, status=c.st)  # what the 8-bit rows stand for
    parts = torch.full((3, B, H, d_h + r + 2), float("nan"), device="cuda")
    ws = b.alloc_workspace(max(b.decode_workspace_bytes(c.dims, B), b.decode_quant_workspace_bytes(c.dims, B)))
    b.lrkv_prefix_partials(c.dims, c.q, c.BK, c.cache, c.blocks, c.pl, parts[0], c.ws, status=c.st)
    b.lrkv_decode_quant_partials(c.dims, c.q, c.BK, qc, c.bt, torch.tensor(old, device="cuda").int(), parts[1], ws,
                                 status=c.st)
    new_bt = torch.full_like(c.bt, -1)
    new_bt[0, 0], new_bt[1, 0], new_bt[3, 0] = c.bt[0, 1], c.bt[1, 0], c.bt[3, 0]
    b.lrkv_decode_partials(c.dims, c.q, c.BK, c.cache, new_bt, torch.tensor([36, 30, 0, 1], device="cuda").int(),
                           parts[2], ws, status=c.st)
    b.lrkv_decode_merge(c.dims, parts, c.BV, c.out, status=c.st)
    assert int(c.st.item()) == 0
    c.verify(what="joined partials")
    # an empty prefix: empty partials, no status bit
    c.pl.fill_(0)
    b.lrkv_prefix_partials(c.dims, c.q, c.BK, c.cache, c.blocks, c.pl, parts[0], c.ws, status=c.st)
    assert int(c.st.item()) == 0
    assert torch.isneginf(parts[0, :, :, -2]).all() and (parts[0, :, :, -1] == 0).all()
    assert (parts[0, :, :, :-2] == 0).all()


def test_captured_and_replayed():
    c = Case(9, 32, 128, 16, 0, 1000, [30, 0, 64, 5])
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    c.verify()
    c.P, c.lens = 129, [1, 0, 9, 5]
    c.pl.fill_(c.P)
    c.sl.copy_(torch.tensor(c.lens, dtype=torch.int32))
    c.pslots = c.pslots[:c.P]
    c.slots = [s[:n] for s, n in zip(c.slots, c.lens)]
    graph.replay()
    torch.cuda.synchronize()
    c.verify()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.out.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    c.verify()


def test_runs_are_bitwise_repeatable():
    c = Case(10, 32, 128, 32, 0, 3001, [100] * 16)
    first = c.run().clone()
    for _ in range(5):
        assert torch.equal(c.run(), first)


@pytest.mark.parametrize("H,d_h,r,P,B,own", [(128, 64, 16, 6000, 64, 3), (32, 128, 32, 32768, 32, 20),
                                             (8, 128, 8, 20011, 40, 0)])
def test_many_pages_a_piece_repeated(H, d_h, r, P, B, own):
    """Many rounds of every buffer in one thread block, run after run: results may not depend on who came first."""
    c = Case(11, H, d_h, r, 0, P, [own] * B)
    first = c.run().clone()
    for _ in range(30):
        c.run()
        assert torch.equal(c.out, first)
    assert int(c.st.item()) == 0
    c.verify(seqs=[0, B - 1])


@pytest.mark.parametrize("H,d_h,r,P,lens", [(1, 64, 8, 90, [i % 5 for i in range(1000)]),
                                            (3, 128, 16, 130, [1 + i % 70 for i in range(257)])])
def test_many_sequences(H, d_h, r, P, lens):
    c = Case(12, H, d_h, r, 0, P, lens)
    c.run()
    assert int(c.st.item()) == 0
    c.verify(seqs=[0, 1, 15, 16, 127, 128, 129, len(lens) - 1])


@pytest.mark.parametrize("ns", [1, 3, 500])
def test_split_counts(ns):
    c = Case(13, 16, 128, 16, 0, 1500, [900, 0, 1, 40], num_splits=ns)
    c.run()
    assert int(c.st.item()) == 0
    c.verify(what=f"num_splits {ns}")


def test_pages_listed_twice_and_shared():
    """A page twice in the prefix, and again among a sequence's own."""
    c = Case(14, 16, 128, 16, 0, 200, [100, 70])
    c.blocks[2] = c.blocks[0]
    c.bt[1, 0] = c.blocks[1]
    c.pslots = c.at(c.blocks, 200)
    c.slots[1] = c.at(c.bt[1], 70)
    c.run()
    assert int(c.st.item()) == 0
    c.verify()


def test_a_nan_query_stays_in_its_head():
    c = Case(15, 9, 64, 16, 0, 300, [20, 0, 3])
    c.q[1, 4, 7] = float("nan")
    c.run()
    nan = torch.isnan(c.out)
    assert nan[1, 4].all() and int(nan.sum()) == 64
    keep = c.out.clone()
    c.q[1, 4, 7] = 1.0
    c.run()
    keep[1, 4] = c.out[1, 4]
    assert torch.equal(keep, c.out)
    c.verify()


def test_calls_on_two_streams():
    cases = [Case(16, 32, 128, 16, 0, 4000, [50] * 16), Case(17, 8, 64, 16, 0, 900, [5] * 4)]
    want = [c.run().clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c.out, w) and int(c.st.item()) == 0


def test_partials_of_a_bad_prefix_length():
    c = Case(18, 8, 64, 16, 0, 200, [1, 1])
    parts = torch.full((2, 8, 64 + 16 + 2), float("nan"), device="cuda")
    for bad in (-1, 257, 2 ** 31 - 1):
        c.st.zero_()
        c.pl.fill_(bad)
        b.lrkv_prefix_partials(c.dims, c.q, c.BK, c.cache, c.blocks, c.pl, parts, c.ws, status=c.st)
        assert int(c.st.item()) == BAD_SEQLEN
        assert torch.isneginf(parts[..., -2]).all() and (parts[..., -1] == 0).all() and (parts[..., :-2] == 0).all()


def test_small_workspaces_are_refused():
    c = Case(19, 8, 64, 16, 0, 200, [100, 3])
    need = b.decode_shared_workspace_bytes(c.dims, 2, int(c.blocks.shape[0]))
    c.ws = c.ws[:need]
    c.run()
    c.verify()
    c.ws = c.ws[:need - 1]
    with pytest.raises(b.LrkvError, match="workspace") as e:
        c.run()
    assert e.value.status == 3


@pytest.mark.parametrize("H,d_h,r,lens", [(32, 128, 16, [40] * 16), (128, 128, 8, [3, 200, 70]), (8, 64, 32, [0, 9])])
@pytest.mark.parametrize("graph", [False, True])
def test_calls_back_to_back_share_a_workspace(H, d_h, r, lens, graph):
    """Calls with other queries, lengths and prefixes, one behind the other in one workspace: a launch of a call may
    begin before the one in front of it has ended, and must still see what it left."""
    c = Case(21, H, d_h, r, 0, 700, lens)
    B = len(lens)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    qs = [torch.randn(B, H, d_h, generator=g, device="cuda").to(torch.bfloat16) for _ in range(6)]
    sls = [(c.sl - i).clamp(min=0) for i in range(6)]
    pls = [c.pl - 100 * i for i in range(6)]
    outs = [torch.empty_like(c.out) for _ in range(6)]

    def call(i, out):
        b.lrkv_decode_shared(c.dims, qs[i], c.BK, c.BV, c.cache, c.blocks, pls[i], c.bt, sls[i], out, c.ws,
                             status=c.st)

    want = []
    for i in range(6):
        call(i, outs[i])
        torch.cuda.synchronize()
        want.append(outs[i].clone())
    if graph:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            for i in range(6):
                call(i, outs[i])
    for _ in range(10):
        for o in outs:
            o.zero_()
        if graph:
            gr.replay()
        else:
            for i in range(6):
                call(i, outs[i])
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    assert int(c.st.item()) == 0


@pytest.mark.parametrize("start,step", [(0, 20), (0, 45), (0, 60), (10, 85), (0, 250), (250, -60), (0, 3)])
@pytest.mark.parametrize("d_h", [64, 128])
def test_large_logits_rise_from_page_to_page(start, step, d_h):
    """Logits of 2^15 log2 units and more whose page maxima rise by less than 2^-7 of their size: every one has to be
    compared in full, or probabilities overflow.

    Queries of one sign and rows of whole numbers make every dot product exact, latents of the keys are zero, so a
    logit is off only by the roundings of x = s * (scale log2 e): the factor's 2^-24 (which moves all logits of a row
    by one factor, differences of at most 2^10 by 2^-14) and those of x - m and m, |m| < 2^17, 2^-8 each, for a piece
    and once more in the merge: 4 * 2^-8 ln 2 of a probability, plus 2^-8 for its rounding to bf16."""
    H, r, P = 8, 16, 1000
    B = 2400  # 150 tiles of query rows: pieces of eight pages and more
    c = Case(23, H, d_h, r, 0, P, [0] * B)
    scale = 2.0 if d_h == 64 else 1.0
    c.dims = b.make_dims(H, d_h, r, H * d_h, softmax_scale=scale)
    sK = c.cache.sK.view(-1, d_h)
    page = torch.arange(P, device="cuda") // 64
    top = (start + step * page) % 256 if step > 0 else (start + step * page).clamp(min=0)
    within = torch.randint(0, 4, (P,), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    base = torch.full((P, d_h), 256.0 if d_h == 64 else 192.0, device="cuda")
    base[:, 0] = (top - within * 4).clamp(min=0).float()
    sK[c.pslots] = base.to(torch.bfloat16)
    c.cache.zK.zero_()
    c.q.fill_(1.0)
    logits = sK[c.pslots].double().sum(1) * scale
    assert logits.min() * 1.4427 > 2 ** 15 and logits.max() * 1.4427 < 2 ** 17
    c.run()
    assert int(c.st.item()) == 0
    sV, zV = c.cache.sV.view(-1, d_h)[c.pslots].double(), c.cache.zV.view(-1, H, r)[c.pslots].double()
    p = torch.softmax(logits, 0)
    V = sV[:, None] + torch.einsum("thr,hdr->thd", zV, c.BV.double())
    absV = sV.abs()[:, None] + torch.einsum("thr,hdr->thd", zV.abs(), c.BV.double().abs())
    want = torch.einsum("t,thd->hd", p, V)
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 4 * 2.0 ** -8 * 0.694 + 2.0 ** -13) * torch.einsum("t,thd->hd", p, absV)
    check(c.out[0], want, bound, f"page maxima from {start} by {step}", rel_max=1.0)
    assert (c.out == c.out[0]).all()


@pytest.mark.parametrize("H,d_h,r,d_rope,P,B,partials", [(32, 128, 16, 0, 20000, 16, False), (128, 128, 16, 64, 9000, 16, True),
                                                        (8, 64, 8, 0, 40000, 64, True), (32, 128, 32, 0, 65, 3, True)])
def test_expired_wait_reports_timeout_and_gpu_stays_usable(monkeypatch, H, d_h, r, d_rope, P, B, partials):
    """With the debugging limit LRKV_DEBUG_WAIT_LIMIT_NS=0 the scans' waits give up as soon as something is not already
    there.  The call ends, reports LRKV_DEV_TIMEOUT and nothing else, and the next one is right to the bit."""
    c = Case(24, H, d_h, r, d_rope, P, [70] * B)
    out = torch.empty(B, H, d_h + r + 2, device="cuda") if partials else c.out

    def call():
        if partials:
            b.lrkv_prefix_partials(c.dims, c.q, c.BK, c.cache, c.blocks, c.pl, out, c.ws, status=c.st)
        else:
            c.run()

    call()
    want = out.clone()
    if not partials:
        c.verify(seqs=[0, B - 1])
    assert int(c.st.item()) == 0 and torch.isfinite(want).all()
    monkeypatch.setenv("LRKV_DEBUG_WAIT_LIMIT_NS", "0")
    seen = 0
    for _ in range(5):
        call()
        seen |= int(c.st.item())
    assert seen == b.DEV_TIMEOUT
    monkeypatch.delenv("LRKV_DEBUG_WAIT_LIMIT_NS")
    c.st.zero_()
    out.fill_(float("nan"))
    call()
    assert int(c.st.item()) == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("H,d_h,r,d_rope,P,B", [(8, 64, 8, 0, 300, 3), (32, 128, 16, 0, 700, 16), (20, 128, 32, 64, 200, 5),
                                               (128, 64, 16, 0, 130, 40), (128, 128, 8, 64, 1000, 2)])
def test_nan_and_infinity_in_a_head_stay_in_it(H, d_h, r, d_rope, P, B):
    """Latents of one head that are not finite, of keys and of values: all other heads are as without them.  An
    infinity among a key's latents moves its token's logit to the infinity of q~'s sign: with the minus sign the token
    has no weight, with the plus sign the head's output is NaN."""
    c = Case(25, H, d_h, r, d_rope, P, [5] * B)
    zK, zV = c.cache.zK.view(-1, H, r), c.cache.zV.view(-1, H, r)

    def verify(i, heads, what):
        want, bound = attend64(c.q[i].double(), c.BK.double(), c.BV.double(), c.parts(i), d_rope)
        check(c.out[i][heads], want[heads], bound[heads], what)

    heads = torch.arange(H, device="cuda")
    for value, pool, tok in ((float("nan"), zK, 0), (float("inf"), zK, P - 1), (float("-inf"), zK, P // 2),
                             (float("nan"), zV, P // 3), (float("inf"), zV, P - 2)):
        h, t = (7 * tok) % H, c.pslots[tok]
        keep = pool[t, h, 1].clone()
        pool[t, h, 1] = value
        c.run()
        assert int(c.st.item()) == 0
        for i in (0, B // 2, B - 1):
            verify(i, heads != h, f"heads beside one with {value}")
        if value != value:
            assert torch.isnan(c.out[:, h]).all()
        elif pool is zV:
            assert not torch.isfinite(c.out[:, h]).any()
        else:
            qt = torch.einsum("bd,d->b", c.q[:, h, :d_h].double(), c.BK[h, :, 1].double())
            plus = qt * value > 0
            assert torch.isnan(c.out[plus, h]).all()
            slots = c.pslots
            c.pslots = torch.cat([slots[:tok], slots[tok + 1:]])  # (the reference without that token)
            for i in torch.nonzero(~plus).flatten().tolist():
                verify(i, heads == h, "a head without one token")
            c.pslots = slots
        pool[t, h, 1] = keep


@pytest.mark.parametrize("H,d_h,r,d_rope,P,factor", [(16, 128, 16, 0, 1500, 20), (32, 128, 8, 0, 3000, 8),
                                                    (8, 64, 32, 64, 700, 20), (128, 64, 16, 0, 5000, 30)])
def test_sharp_logits_over_a_prefix_alone(H, d_h, r, d_rope, P, factor):
    """Without tokens of the sequences' own q~ enters in two bf16 pieces: two roundings to half a step of 2^-8, 2^-16
    left, so large queries move no logit much.  The outputs' roundings are 0.0016 of them, root mean square; the
    probabilities', where a few tokens have all the weight, at most 2^-8 each: sqrt(0.0016^2 + 0.0039^2) = 0.0042.
    (Logits 20% off take up 6 to 14 times the elementwise bound, and 2% off leave a relative error of up to 0.007.)"""
    c = Case(26, H, d_h, r, d_rope, P, [0] * 3)
    c.q *= factor
    c.run()
    assert int(c.st.item()) == 0
    for i in range(3):
        want, bound = attend64(c.q[i].double(), c.BK.double(), c.BV.double(), c.parts(i), d_rope, eps_p=2.0 ** -8,
                               eps_qt=2.0 ** -16)
        check(c.out[i], want, bound, f"queries times {factor}, sequence {i}", rel_max=4.3e-3)


@pytest.mark.parametrize("P,lens", [(0, [9000, 7000, 1]), (700, [3000] * 6)])
def test_expired_wait_of_128_heads(monkeypatch, P, lens):
    """The same for the tensor-core scan of 128 heads, by itself (lrkv_decode) and as the sequences' own scan."""
    c = Case(27, 128, 128, 16, 0, P, lens)

    def call():
        if P:
            c.run()
        else:
            b.lrkv_decode(c.dims, c.q, c.BK, c.BV, c.cache, c.bt, c.sl, c.out, c.ws, status=c.st)

    call()
    assert int(c.st.item()) == 0
    want = c.out.clone()
    c.verify(seqs=[0, len(lens) - 1])
    monkeypatch.setenv("LRKV_DEBUG_WAIT_LIMIT_NS", "0")
    seen = 0
    for _ in range(5):
        call()
        seen |= int(c.st.item())
    assert seen == b.DEV_TIMEOUT
    monkeypatch.delenv("LRKV_DEBUG_WAIT_LIMIT_NS")
    c.st.zero_()
    c.out.fill_(float("nan"))
    call()
    assert int(c.st.item()) == 0
    assert torch.equal(c.out, want)
