"""Quantised cache on the GPU: rows written and read back, and the decode over them, against
implementations in 64 bits."""
import numpy as np
import pytest
import torch

from attn64 import attend64, check

pytestmark = pytest.mark.gpu

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402

PAGE, BLOCK = 64, 32
BAD_BLOCK, BAD_SEQLEN, BAD_SLOT = b.DEV_BAD_BLOCK, b.DEV_BAD_SEQLEN, b.DEV_BAD_SLOT


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def widths(H, d_h, r, d_rope):
    return [d_h + d_rope, d_h, H * r, H * r]


def layout(H, d_h, r, d_rope):
    """Byte offsets of the parts, of the scales, blocks per part, bytes of a row."""
    off, at = [], 0
    for w in widths(H, d_h, r, d_rope):
        off.append(at)
        at += (w + 15) // 16 * 16
    blocks = [(w + BLOCK - 1) // BLOCK for w in widths(H, d_h, r, d_rope)]
    units = (at + sum(blocks) + 15) // 16
    return off, at, blocks, 16 * (units | 1)


def quantise64(x):
    """x [n, w] float64 (bf16 values) -> (q int64 [n, w], scale byte int64 [n, blocks])."""
    x = x.cpu().numpy()
    n, w = x.shape
    nb = (w + BLOCK - 1) // BLOCK
    q, e = np.zeros((n, w), np.int64), np.zeros((n, nb), np.int64)
    for i in range(nb):
        v = x[:, i * BLOCK:(i + 1) * BLOCK]
        bad = ~np.isfinite(v).all(1)
        amax = np.abs(np.where(np.isfinite(v), v, 0)).max(1)
        k = np.maximum(np.frexp(amax)[1] - 7, -126)  # amax = f 2^(k + 7), f in [1/2, 1)
        k = np.where(amax == 0, -126, k)
        qq = np.clip(np.rint(np.where(np.isfinite(v), v, 0) / np.exp2(k.astype(float))[:, None]), -127, 127)
        q[:, i * BLOCK:(i + 1) * BLOCK] = np.where(bad[:, None], 0, qq)
        e[:, i] = np.where(bad, 255, k + 127)
    return q, e


def values64(rows, H, d_h, r, d_rope):
    """Rows [n, bytes] (uint8) -> the four parts in float64, z as [n, H, r]."""
    off, at, blocks, _ = layout(H, d_h, r, d_rope)
    out = []
    for i, w in enumerate(widths(H, d_h, r, d_rope)):
        e = rows[:, at:at + blocks[i]].long().repeat_interleave(BLOCK, 1)[:, :w]
        v = (rows[:, off[i]:off[i] + w].double() - 128) * ((e - 127 + 1023) << 52).view(torch.float64)
        v = torch.where(e == 255, torch.full_like(v, float("nan")), torch.where(e == 0, torch.zeros_like(v), v))
        out.append(v if i < 2 else v.view(-1, H, r))
        at += blocks[i]
    return out


def bf16_cache(g, blocks, H, d_h, r, d_rope, scale=1.0):
    mk = lambda *s: (torch.randn(blocks, PAGE, *s, generator=g, device="cuda") * scale).to(torch.bfloat16)
    return b.PagedCache(mk(d_h + d_rope), mk(d_h), mk(H, r), mk(H, r))


def flat(cache, H, r):
    return [t.view(-1, t.shape[2] if t.dim() == 3 else H * r) for t in cache.tensors()]


SHAPES = [(1, 64, 8, 0), (3, 64, 8, 64), (8, 64, 16, 0), (5, 128, 32, 0), (33, 128, 16, 64), (32, 128, 32, 0),
          (128, 128, 16, 0), (128, 128, 32, 64), (7, 128, 8, 0)]


@pytest.mark.parametrize("H,d_h,r,d_rope", SHAPES)
@pytest.mark.parametrize("n", [1, 37, 300])
def test_rows_written_and_read_back(H, d_h, r, d_rope, n):
    """Every byte as computed in 64 bits; reading back gives exactly the values; other rows stay."""
    g = gen(H * 1000 + n)
    dims = b.make_dims(H, d_h, r, H * d_h, d_rope=d_rope)
    nb = (n + 63) // 64 + 1
    cache = bf16_cache(g, nb, H, d_h, r, d_rope)
    for t in cache.tensors():  # sizes over a wide range, zeros, and the largest finite value
        f = t.view(nb * PAGE, -1)
        f *= torch.exp2(torch.randint(-40, 40, (f.shape[0], 1), generator=g, device="cuda").float()).to(torch.bfloat16)
        f[:: 7] = 0
        f[3] = torch.finfo(torch.bfloat16).max
        f[5] *= 2.0 ** -100
    rb = b.quant_row_bytes(dims)
    assert rb == layout(H, d_h, r, d_rope)[3] and rb % 32 == 16
    qc = b.QuantCache(torch.full((nb, PAGE, rb), 77, dtype=torch.uint8, device="cuda"))
    src = torch.randperm(nb * PAGE, generator=g, device="cuda")[:n].int()
    dst = torch.randperm(nb * PAGE, generator=g, device="cuda")[:n].int()
    if n > 10:
        src[4], dst[9] = -1, -7
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.lrkv_cache_quantize(dims, cache, src, qc, dst, status=st)
    live = (src >= 0) & (dst >= 0)
    s, d = src[live].long(), dst[live].long()
    rows = qc.rows.view(-1, rb)
    off, at, blocks, _ = layout(H, d_h, r, d_rope)
    for i, f in enumerate(flat(cache, H, r)):
        q, e = quantise64(f[s].double())
        w = f.shape[1]
        assert np.array_equal(rows[d, off[i]:off[i] + w].cpu().numpy().astype(np.int64), q + 128), i
        assert np.array_equal(rows[d, at:at + blocks[i]].cpu().numpy().astype(np.int64), e), i
        at += blocks[i]
    rest = torch.ones(nb * PAGE, dtype=torch.bool, device="cuda")
    rest[d] = False
    assert (rows[rest] == 77).all()
    back = b.PagedCache(*(torch.full_like(t, -3.0) for t in cache.tensors()))
    to = torch.randperm(nb * PAGE, generator=g, device="cuda")[:n].int()
    b.lrkv_cache_dequantize(dims, qc, dst, back, to, status=st)
    # (a negative source slot skipped the write, so that row of the 8-bit cache holds the fill)
    read = dst >= 0
    want = values64(rows[dst[read].long()], H, d_h, r, d_rope)
    rest = torch.ones(nb * PAGE, dtype=torch.bool, device="cuda")
    rest[to[read].long()] = False
    for f, w in zip(flat(back, H, r), want):
        assert torch.equal(f[to[read].long()].double(), w.reshape(w.shape[0], -1))
        assert (f[rest] == -3.0).all()
    assert int(st.item()) == 0


def test_error_of_a_value_is_half_a_step():
    H, d_h, r = 32, 128, 32
    g = gen(5)
    dims = b.make_dims(H, d_h, r, H * d_h)
    cache = bf16_cache(g, 4, H, d_h, r, 0)
    qc = b.QuantCache.empty(dims, 4)
    slots = torch.arange(256, dtype=torch.int32, device="cuda")
    b.lrkv_cache_quantize(dims, cache, slots, qc, slots)
    for f, v in zip(flat(cache, H, r), values64(qc.rows.view(256, -1), H, d_h, r, 0)):
        x = f.double().view(256, -1, BLOCK)
        amax = x.abs().amax(2, keepdim=True)
        step = torch.exp2(torch.floor(torch.log2(amax)) - 6)
        assert ((v.reshape(x.shape) - x).abs() <= step / 2).all()


def test_blocks_with_nan_or_infinity_read_as_nan():
    H, d_h, r = 3, 64, 8
    g = gen(6)
    dims = b.make_dims(H, d_h, r, H * d_h)
    cache = bf16_cache(g, 1, H, d_h, r, 0)
    cache.sK[0, 3, 40] = float("nan")
    cache.zV[0, 4, 2, 1] = float("-inf")
    qc = b.QuantCache.empty(dims, 1)
    slots = torch.arange(64, dtype=torch.int32, device="cuda")
    b.lrkv_cache_quantize(dims, cache, slots, qc, slots)
    back = b.PagedCache.empty(1, H, d_h, r)
    b.lrkv_cache_dequantize(dims, qc, slots, back, slots)
    nan = [torch.isnan(t) for t in back.tensors()]
    assert nan[0][0, 3, 32:].all() and int(nan[0].sum()) == 32
    assert nan[3][0, 4].all() and int(nan[3].sum()) == H * r
    assert not nan[1].any() and not nan[2].any()


def test_slots_out_of_range_are_reported_and_skipped():
    H, d_h, r = 8, 64, 16
    g = gen(7)
    dims = b.make_dims(H, d_h, r, H * d_h)
    cache = bf16_cache(g, 2, H, d_h, r, 0)
    for src, dst in (([0, 128, 5], [0, 1, 2]), ([0, 1, 5], [0, 64, 2])):
        qc = b.QuantCache(torch.full((1, PAGE, b.quant_row_bytes(dims)), 9, dtype=torch.uint8, device="cuda"))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        b.lrkv_cache_quantize(dims, cache, torch.tensor(src, device="cuda").int(), qc,
                              torch.tensor(dst, device="cuda").int(), status=st)
        assert int(st.item()) == BAD_SLOT
        assert (qc.rows[0, 1] == 9).all() and (qc.rows[0, 0] != 9).any() and (qc.rows[0, 2] != 9).any()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.lrkv_cache_dequantize(dims, qc, torch.tensor([64, 0], device="cuda").int(), cache,
                            torch.tensor([0, 128], device="cuda").int(), status=st)
    assert int(st.item()) == BAD_SLOT


# ------------------------------------------------------------------ decode
class Case:
    """A quantised cache with random pages and queries; rows behind the sequences' ends hold 0xff."""

    def __init__(self, seed, H, d_h, r, d_rope, lens, spare=2, num_splits=0, cap=None):
        g = gen(seed)
        self.H, self.d_h, self.r, self.d_rope, self.lens = H, d_h, r, d_rope, lens
        self.dims = b.make_dims(H, d_h, r, H * d_h, d_rope=d_rope, num_splits=num_splits)
        pages = [(n + 63) // 64 for n in lens]
        nb = sum(pages) + spare
        ids = torch.randperm(nb, generator=g, device="cuda")
        self.bt = torch.full((len(lens), cap or max(1, max(pages))), -1, dtype=torch.int32, device="cuda")
        rb = b.quant_row_bytes(self.dims)
        self.qc = b.QuantCache(torch.full((nb, PAGE, rb), 255, dtype=torch.uint8, device="cuda"))
        at, slots = 0, []
        for i, (n, p) in enumerate(zip(lens, pages)):
            self.bt[i, :p] = ids[at:at + p].int()
            at += p
            t = torch.arange(n, device="cuda")
            slots.append(self.bt[i][t // 64].long() * 64 + t % 64)
        self.slots = slots
        total = sum(lens)
        cache = bf16_cache(g, (total + 63) // 64 or 1, H, d_h, r, d_rope)
        all_slots = torch.cat(slots).int()
        b.lrkv_cache_quantize(self.dims, cache, torch.arange(total, device="cuda").int(), self.qc, all_slots)
        self.q = torch.randn(len(lens), H, d_h + d_rope, generator=g, device="cuda").to(torch.bfloat16)
        mk = lambda: (torch.randn(H, d_h, r, generator=g, device="cuda") * r ** -0.5).to(torch.bfloat16)
        self.BK, self.BV = mk(), mk()
        self.sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = b.alloc_workspace(b.decode_quant_workspace_bytes(self.dims, len(lens)))
        self.out = torch.full((len(lens), H, d_h), float("nan"), dtype=torch.bfloat16, device="cuda")

    def run(self, stream=None):
        b.lrkv_decode_quant(self.dims, self.q, self.BK, self.BV, self.qc, self.bt, self.sl, self.out, self.ws,
                            status=self.st, stream=stream)
        return self.out

    def parts(self, i):
        rows = self.qc.rows.view(-1, self.qc.rows.shape[2])[self.slots[i]]
        return values64(rows, self.H, self.d_h, self.r, self.d_rope)

    def verify(self, out=None, seqs=None, what="decode_quant", rel_max=5e-3):
        out = self.out if out is None else out
        for i in range(len(self.lens)) if seqs is None else seqs:
            # probabilities: bf16 for the shared rows' products; q~: fp16 for the latents'
            want, bound = attend64(self.q[i].double(), self.BK.double(), self.BV.double(), self.parts(i), self.d_rope,
                                   eps_p=2.0 ** -8, eps_qt=2.0 ** -11)
            check(out[i], want, bound, f"{what} sequence {i} of {self.lens[i]} tokens", rel_max)


DECODE = [
    (1, 64, 8, 0, [1]), (1, 128, 32, 64, [5000]), (3, 64, 8, 0, [1, 15, 16, 17, 63, 64, 65]), (7, 64, 32, 0, [200, 3]),
    (8, 64, 8, 0, [256]), (8, 64, 16, 0, [2048] * 3 + [1, 777]), (9, 128, 8, 0, [130, 31]),
    (16, 128, 16, 64, [1500, 300, 1]), (17, 128, 32, 64, [300, 5]), (32, 128, 32, 0, [3000, 1290, 64]),
    (32, 64, 16, 0, list(range(1, 200, 3))), (40, 128, 16, 0, [999]), (64, 128, 32, 0, [400, 2]),
    (100, 128, 32, 0, [700, 33]), (104, 64, 32, 64, [65]), (109, 128, 32, 0, [300, 70]), (128, 128, 16, 0, [2048, 777, 130]),
    (128, 128, 32, 64, [500, 9]), (128, 64, 8, 0, [1000, 1]), (96, 128, 8, 64, [640]),
]


@pytest.mark.parametrize("H,d_h,r,d_rope,lens", DECODE, ids=[f"H{c[0]}_dh{c[1]}_r{c[2]}_rope{c[3]}_B{len(c[4])}" for c in DECODE])
def test_decode_matches_64_bits(H, d_h, r, d_rope, lens):
    c = Case(H + r + len(lens), H, d_h, r, d_rope, lens)
    c.run()
    assert int(c.st.item()) == 0
    c.verify()


@pytest.mark.parametrize("ns", [1, 2, 7, 500])
def test_split_counts(ns):
    c = Case(11, 16, 128, 16, 0, [900, 40, 1], num_splits=ns)
    c.run()
    c.verify(what=f"num_splits {ns}")


def test_values_of_very_different_size():
    """Tokens whose rows differ by 2^+-30, large scales among the values and small ones: the weights
    of the latents' products are kept relative to their own largest."""
    c = Case(12, 8, 128, 16, 0, [300])
    off, at, blocks, _ = layout(8, 128, 16, 0)
    rows = c.qc.rows.view(-1, c.qc.rows.shape[2])
    first = at + blocks[0]  # scales of s^V, then (after z^K's) z^V
    zv = at + blocks[0] + blocks[1] + blocks[2]
    for i, e in ((0, 157), (1, 100), (2, 1), (50, 150), (299, 97)):
        rows[c.slots[0][i], first:first + blocks[1]] = e
        rows[c.slots[0][i], zv:zv + blocks[3]] = e
    c.run()
    c.verify()


def test_sharp_logits_and_zero_queries():
    c = Case(13, 8, 64, 16, 0, [500, 90])
    c.q[0] *= 30  # one token takes nearly everything
    c.q[1] = 0    # a plain mean
    c.run()
    c.verify(rel_max=1.0)  # (logits 30 times as large magnify q~'s rounding: the bound says by how much)


def test_bad_lengths_and_pages():
    c = Case(14, 8, 64, 16, 0, [100, 70, 128, 64], cap=3)
    c.sl = torch.tensor([100, 0, 193, 64], dtype=torch.int32, device="cuda")
    c.run()
    assert int(c.st.item()) == BAD_SEQLEN
    assert (c.out[1] == 0).all() and (c.out[2] == 0).all()
    c.verify(seqs=[0, 3])
    # a page id out of range: reported, its tokens left out
    for bad in (-1, c.qc.num_blocks):
        c = Case(15, 8, 64, 16, 0, [200, 70])
        c.bt[0, 1] = bad
        c.run()
        assert int(c.st.item()) == BAD_BLOCK
        keep = torch.cat([c.slots[0][:64], c.slots[0][128:]])
        c.slots[0] = keep
        c.lens[0] = len(keep)
        c.verify()


def test_nan_block_reaches_its_sequence_only():
    c = Case(16, 8, 64, 16, 0, [100, 100])
    off, at, blocks, _ = layout(8, 64, 16, 0)
    c.qc.rows.view(-1, c.qc.rows.shape[2])[c.slots[0][17], at + blocks[0]] = 255  # a block of s^V
    c.run()
    assert torch.isnan(c.out[0][:, :32]).all()
    c.verify(seqs=[1])


def test_partials_and_merge():
    """Partials of two parts of the tokens (one empty for a sequence) merge to the whole."""
    H, d_h, r, lens = 16, 128, 32, [500, 64, 130]
    c = Case(17, H, d_h, r, 0, lens)
    first = torch.tensor([256, 64, 0], dtype=torch.int32, device="cuda")
    tail_bt = torch.full_like(c.bt, -1)
    tail_bt[0, :4], tail_bt[2, :3] = c.bt[0, 4:8], c.bt[2, :3]
    tail = torch.tensor([244, 0, 130], dtype=torch.int32, device="cuda")
    parts = torch.full((2, 3, H, d_h + r + 2), float("nan"), device="cuda")
    b.lrkv_decode_quant_partials(c.dims, c.q, c.BK, c.qc, c.bt, first, parts[0], c.ws, status=c.st)
    b.lrkv_decode_quant_partials(c.dims, c.q, c.BK, c.qc, tail_bt, tail, parts[1], c.ws, status=c.st)
    assert torch.isneginf(parts[1, 1, :, -2]).all() and (parts[1, 1, :, -1] == 0).all()
    b.lrkv_decode_merge(c.dims, parts, c.BV, c.out, status=c.st)
    assert int(c.st.item()) == 0
    c.verify()


def test_captured_and_replayed_on_another_stream():
    """A captured call reads lengths, pages and rows as they are at each replay; the workspace is
    shared with eager calls between the replays."""
    c = Case(18, 32, 128, 16, 0, [1000, 333, 2])
    side = torch.cuda.Stream()
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run()
    c.out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    c.verify()
    c.lens = [64, 1, 128]
    c.sl.copy_(torch.tensor([64, 1, 65], dtype=torch.int32))
    c.lens = [64, 1, 2]
    c.sl.copy_(torch.tensor(c.lens, dtype=torch.int32))
    for i, n in enumerate(c.lens):
        c.slots[i] = c.slots[i][:n]
    other = Case(19, 8, 64, 16, 0, [70])
    other.ws = c.ws
    other.run()
    graph.replay()
    torch.cuda.synchronize()
    c.verify()
    other.verify()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    c.verify()


def test_runs_are_bitwise_repeatable():
    c = Case(20, 32, 128, 32, 0, [4000, 100])
    first = c.run().clone()
    for _ in range(5):
        assert torch.equal(c.run(), first)


def test_append_quantise_decode_step():
    """A decode step as a user runs it: the newest rows appended to a bf16 staging page, quantised into
    the sequences' pages, attended over with the old ones."""
    H, d_h, r, d, B = 8, 64, 16, 512, 3
    g = gen(21)
    c = Case(21, H, d_h, r, 0, [100, 65, 64])
    W = (torch.randn(2 * (d_h + H * r), d, generator=g, device="cuda") * d ** -0.5).to(torch.bfloat16)
    X = torch.randn(B, d, generator=g, device="cuda").to(torch.bfloat16)
    staging = b.PagedCache.empty(1, H, d_h, r)
    idx = torch.arange(B, dtype=torch.int32, device="cuda")
    b.lrkv_append(c.dims, X, W, idx, staging, status=c.st)
    last = torch.stack([s[-1] for s in c.slots]).int()
    b.lrkv_cache_quantize(c.dims, staging, idx, c.qc, last, status=c.st)
    c.run()
    assert int(c.st.item()) == 0
    y = X.double() @ W.double().t()
    got = c.parts(1)[0][-1]
    assert (got - y[1, :d_h]).abs().max() <= y[1, :d_h].abs().max() * (2.0 ** -7 + 2.0 ** -7)
    c.verify()


@pytest.mark.parametrize("H,d_h,r,lens", [(1, 64, 8, [1 + 7 * (i % 90) for i in range(300)]),
                                          (8, 128, 16, [2000] * 3 + [1] * 170 + [900]),
                                          (16, 64, 32, [33] * 1100)], ids=["one_head", "uneven", "1100_sequences"])
def test_more_sequences_than_thread_blocks(H, d_h, r, lens):
    c = Case(22, H, d_h, r, 0, lens)
    c.run()
    assert int(c.st.item()) == 0
    c.verify(seqs=[0, 1, 2, 31, 32, 33, 127, 128, 151, 152, 153, len(lens) - 2, len(lens) - 1])


@pytest.mark.parametrize("H,d_h,r,d_rope,ns", [(8, 64, 8, 64, 1), (112, 128, 32, 64, 3), (2, 128, 16, 0, 0)])
def test_long_sequences_in_few_pieces(H, d_h, r, d_rope, ns):
    """Many rounds of each ring of buffers in one segment."""
    c = Case(23, H, d_h, r, d_rope, [12001], num_splits=ns)
    c.run()
    assert int(c.st.item()) == 0
    first = c.out.clone()
    c.verify()
    for _ in range(3):
        assert torch.equal(c.run(), first)


def test_cleared_rows():
    """Rows as in memory that was cleared stand for zeros: among others, as a whole sequence, as its start."""
    c = Case(24, 9, 64, 16, 0, [100, 70, 300])
    rows = c.qc.rows.view(-1, c.qc.rows.shape[2])
    rows[c.slots[0][::3]] = 0
    rows[c.slots[1]] = 0
    rows[c.slots[2][:200]] = 0
    c.run()
    assert int(c.st.item()) == 0 and (c.out[1] == 0).all()
    c.verify()


def test_pages_listed_twice_and_shared():
    """The same page twice in a sequence, and in two sequences."""
    c = Case(25, 16, 128, 16, 0, [200, 190])
    c.bt[0, 2] = c.bt[0, 0]
    c.bt[1, :2] = c.bt[0, :2]
    for i, n in enumerate(c.lens):
        t = torch.arange(n, device="cuda")
        c.slots[i] = c.bt[i][t // 64].long() * 64 + t % 64
    c.run()
    assert int(c.st.item()) == 0
    c.verify()


def test_a_nan_query_stays_in_its_head():
    c = Case(26, 9, 64, 16, 0, [200, 40])
    c.q[0, 3, 5] = float("nan")
    c.run()
    nan = torch.isnan(c.out)
    assert nan[0, 3].all() and int(nan.sum()) == 64
    keep = c.out.clone()
    c.q[0, 3, 5] = 1.0
    c.run()
    keep[0, 3] = c.out[0, 3]
    assert torch.equal(keep, c.out)
    c.verify()


def test_calls_on_two_streams():
    """Two calls at once, each with a workspace of its own."""
    cases = [Case(27, 32, 128, 32, 0, [3000, 700]), Case(28, 8, 64, 16, 0, [5000] * 4)]
    want = [c.run().clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c.out, w) and int(c.st.item()) == 0


def test_small_workspaces_are_refused():
    c = Case(29, 8, 64, 16, 0, [100, 3])
    need = b.decode_quant_workspace_bytes(c.dims, 2)
    c.ws = c.ws[:need]
    c.run()
    c.verify()
    c.ws = c.ws[:need - 1]
    with pytest.raises(b.LrkvError, match="workspace") as e:
        c.run()
    assert e.value.status == 3


@pytest.mark.parametrize("H,d_h,r,lens", [(32, 128, 16, [900, 30]), (128, 128, 16, [200] * 9), (8, 64, 8, [1, 600])])
@pytest.mark.parametrize("graph", [False, True])
def test_calls_back_to_back_share_a_workspace(H, d_h, r, lens, graph):
    """Rows written and decoded with other queries, lengths and values, call behind call in one workspace."""
    c = Case(30, H, d_h, r, 0, lens)
    g = gen(31)
    qs = [torch.randn(len(lens), H, d_h, generator=g, device="cuda").to(torch.bfloat16) for _ in range(6)]
    sls = [(c.sl - 7 * i).clamp(min=1) for i in range(6)]
    last = torch.stack([s[0] for s in c.slots]).int()
    news = [bf16_cache(g, 1, H, d_h, r, 0) for _ in range(6)]
    src = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(c.out) for _ in range(6)]

    def call(i, out):
        b.lrkv_cache_quantize(c.dims, news[i], src, c.qc, last, status=c.st)
        b.lrkv_decode_quant(c.dims, qs[i], c.BK, c.BV, c.qc, c.bt, sls[i], out, c.ws, status=c.st)

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


def test_offsets_beyond_32_bits():
    """The same rows in the last pages of pools of more than 2^31 elements and 2^32 bytes as in small ones: written,
    read back, decoded, and as a shared prefix."""
    H, d_h, r, n, big = 128, 64, 32, 150, 8300
    g = gen(32)
    dims = b.make_dims(H, d_h, r, H * d_h)
    small = bf16_cache(g, 3, H, d_h, r, 0)
    large = b.PagedCache.empty(big, H, d_h, r)
    assert large.zK.numel() > 2 ** 31 and big * b.quant_block_bytes(dims) > 2 ** 32
    for s, t in zip(small.tensors(), large.tensors()):
        t[big - 3:] = s
    q = torch.randn(1, H, d_h, generator=g, device="cuda").to(torch.bfloat16)
    BK, BV = ((torch.randn(H, d_h, r, generator=g, device="cuda") * r ** -0.5).to(torch.bfloat16) for _ in range(2))
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    own = torch.tensor([64], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    results = []
    for cache in (small, large):
        nb = cache.num_blocks
        pages = torch.arange(nb - 3, nb, device="cuda", dtype=torch.int32)
        slots = torch.arange((nb - 3) * PAGE, (nb - 3) * PAGE + n, device="cuda", dtype=torch.int32)
        qc = b.QuantCache.empty(dims, nb)
        b.lrkv_cache_quantize(dims, cache, slots, qc, slots, status=st)
        out = torch.empty(2, 1, H, d_h, dtype=torch.bfloat16, device="cuda")
        ws = b.alloc_workspace(max(b.decode_quant_workspace_bytes(dims, 1), b.decode_shared_workspace_bytes(dims, 1, 2)))
        b.lrkv_decode_quant(dims, q, BK, BV, qc, pages[None], sl, out[0], ws, status=st)
        b.lrkv_decode_shared(dims, q, BK, BV, cache, pages[:2], torch.full_like(sl, 100), pages[None, 2:], own, out[1], ws,
                             status=st)
        for t in cache.tensors():
            t[nb - 3:] = 0
        b.lrkv_cache_dequantize(dims, qc, slots, cache, slots, status=st)
        off, at, blocks, _ = layout(H, d_h, r, 0)  # (the row's padding is not written)
        results.append([qc.rows[nb - 3:].view(-1, qc.rows.shape[2])[:n, :at + sum(blocks)].clone(), out] +
                       [t[nb - 3:].clone() for t in cache.tensors()])
        assert int(st.item()) == 0
        del qc
    for x, y in zip(*results):
        assert torch.equal(x, y)


@pytest.mark.parametrize("H,d_h,r,d_rope", [(8, 64, 8, 0), (9, 128, 16, 64), (32, 128, 32, 0), (72, 64, 16, 0),
                                            (128, 128, 32, 64)])
@pytest.mark.parametrize("shift", [14, 18, 24, 60, -14, -18, -24, -60])
def test_factors_and_latents_of_any_ratio(H, d_h, r, d_rope, shift):
    """B^K times 2^k with z^K times 2^-k is the same model: q~ is then 2^k times what it was, and nothing else
    changes.  Powers of two round nothing, so not a bit of the output may change either."""
    c = Case(33, H, d_h, r, d_rope, [300, 5, 2, 1])
    want = c.run().clone()
    c.verify(seqs=[0, 1])
    off, at, blocks, _ = layout(H, d_h, r, d_rope)
    first = at + blocks[0] + blocks[1]
    for s in c.slots:
        e = c.qc.rows.view(-1, c.qc.rows.shape[2])[s, first:first + blocks[2]].int() - shift
        assert 1 <= int(e.min()) and int(e.max()) <= 254
        c.qc.rows.view(-1, c.qc.rows.shape[2])[s, first:first + blocks[2]] = e.to(torch.uint8)
    c.BK = (c.BK.float() * 2.0 ** shift).to(torch.bfloat16)
    c.run()
    assert int(c.st.item()) == 0
    c.verify()
    assert torch.equal(c.out, want)


@pytest.mark.parametrize("H,d_h,r,d_rope,lens", [(32, 128, 32, 0, [20000, 9000]), (128, 128, 16, 64, [4000, 3000, 1]),
                                                 (8, 64, 8, 0, [30000] + [50] * 200), (128, 128, 32, 0, [6000])])
def test_expired_wait_reports_timeout_and_gpu_stays_usable(monkeypatch, H, d_h, r, d_rope, lens):
    """With the debugging limit LRKV_DEBUG_WAIT_LIMIT_NS=0 the scan's waits give up as soon as something is not already
    there.  The call ends, reports LRKV_DEV_TIMEOUT and nothing else, and the next one is right to the bit."""
    c = Case(34, H, d_h, r, d_rope, lens)
    want = c.run().clone()
    c.verify(seqs=[0, len(lens) - 1])
    monkeypatch.setenv("LRKV_DEBUG_WAIT_LIMIT_NS", "0")
    seen = 0
    for _ in range(5):
        c.run()
        seen |= int(c.st.item())
    assert seen == b.DEV_TIMEOUT
    monkeypatch.delenv("LRKV_DEBUG_WAIT_LIMIT_NS")
    c.st.zero_()
    c.out.fill_(float("nan"))
    c.run()
    assert int(c.st.item()) == 0
    assert torch.equal(c.out, want)
