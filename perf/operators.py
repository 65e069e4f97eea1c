"""Operators over the compressed cache that are measured one by one, with their plain forms.

Three operators, each on the paged cache of shared rows s and per-head latents z_h
(K_h = s^K + B_h^K z^K_h, V_h = s^V + B_h^V z^V_h):

  store   rows of a bf16 cache are quantised into 8-bit rows (blocks of 32 values with one
          power-of-two scale each) and read back into bf16 pages;
  quant   one decode step per sequence over a cache of such 8-bit rows;
  shared  one decode step for a batch whose sequences share a long prefix, held and read once,
          and go on in pages of their own.

A quantised row of a token is, in bytes,
  [s^K (d_h + d_rope) | s^V (d_h) | z^K (H r, padded to 16) | z^V (H r, padded to 16) | scales]
padded to an odd number of 16-byte units.  Each of the four parts is cut into blocks of 32
values (the last one may be shorter); block i of a part has the scale byte e_i, and a value is
(byte - 128) * 2^(e_i - 127).  Scale bytes stand in the parts' order.
"""
import math
import random

import torch

own = False

PAGE = 64
BLOCK = 32


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the newest rows of 16 sequences, written as a decode step writes them
        dict(name="store-step", op="store", H=32, d_h=128, r=32, d_rope=0, n=16),
        # one prefill chunk of two prompts, with the positional key
        dict(name="store-chunk", op="store", H=32, d_h=128, r=16, d_rope=64, n=1000),
        # pages of idle sequences moved to 8 bits and back
        dict(name="store-pages", op="store", H=32, d_h=128, r=32, d_rope=0, n=65536),
        # the smallest call: one short sequence, eight heads
        dict(name="quant-small", op="quant", H=8, d_h=64, r=8, d_rope=0, B=1, L_min=256, L=256),
        # one layer of a 12-layer backbone
        dict(name="quant-backbone", op="quant", H=8, d_h=64, r=16, d_rope=0, B=16, L_min=2048, L=2048),
        # ragged batch with the positional key, from one token on
        dict(name="quant-ragged", op="quant", H=32, d_h=128, r=16, d_rope=64, B=24, L_min=1, L=8191),
        # long context
        dict(name="quant-longctx", op="quant", H=32, d_h=128, r=32, d_rope=0, B=4, L_min=16384, L=32768),
        # many heads
        dict(name="quant-heads", op="quant", H=128, d_h=128, r=16, d_rope=0, B=8, L_min=8192, L=8192),
        # a short system prompt, a few short answers
        dict(name="shared-small", op="shared", H=8, d_h=64, r=16, d_rope=0, B=4, P=500, L_min=0, L=64),
        # a chat batch behind one system prompt
        dict(name="shared-chat", op="shared", H=32, d_h=128, r=16, d_rope=0, B=16, P=8192, L_min=1, L=512),
        # many samples of one long document
        dict(name="shared-doc", op="shared", H=32, d_h=128, r=32, d_rope=0, B=32, P=32768, L_min=1, L=256),
        # a wide batch of many heads, with the positional key
        dict(name="shared-wide", op="shared", H=128, d_h=128, r=16, d_rope=64, B=48, P=4001, L_min=0, L=200),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    most = {"store": 65536 * 2500, "quant": 8 * 8192 * 4500, "shared": 2e12}
    while True:
        c = dict(op=rng.choice(["store", "quant", "shared"]), H=_log_int(rng, 1, 128), d_h=rng.choice([64, 128]),
                 r=rng.choice([8, 16, 32]), d_rope=rng.choice([0, 0, 64]))
        if c["r"] == 32 and c["H"] >= 105:
            c["H"] = c["H"] // 8 * 8
        if c["op"] == "store":
            c["n"] = _log_int(rng, 1, 65536)
            if c["n"] * row_bytes(c) <= most["store"]:
                return c
            continue
        c["B"] = _log_int(rng, 1, 64)
        if c["op"] == "quant":
            c["L"] = _log_int(rng, 1, 32768)
            c["L_min"] = rng.randint(1, c["L"])
            if sum(lengths(c)) * row_bytes(c) <= most["quant"]:
                return c
            continue
        c["P"] = _log_int(rng, 1, 32768)
        c["L"] = _log_int(rng, 1, 2048)
        c["L_min"] = rng.randint(0, c["L"])
        if work(c)["flops"] <= most["shared"] and c["B"] * c["H"] * c["P"] <= 48 << 20:
            return c


def lengths(case):
    """The sequences' own lengths: whole numbers spread over [L_min, L], fixed by the case."""
    rng = random.Random(case["B"] * 1000003 + case["L_min"] * 101 + case["L"])
    return [rng.randint(case["L_min"], case["L"]) for _ in range(case["B"])]


def _widths(case):
    hr = case["H"] * case["r"]
    return [case["d_h"] + case["d_rope"], case["d_h"], hr, hr]


def _offsets(case):
    """Byte offsets of the four parts, of the scales, and each part's number of blocks."""
    w = _widths(case)
    off, at = [], 0
    for x in w:
        off.append(at)
        at += -(-x // 16) * 16
    blocks = [-(-x // BLOCK) for x in w]
    return off, at, blocks


def row_bytes(case):
    _, at, blocks = _offsets(case)
    units = -(-(at + sum(blocks)) // 16)
    return 16 * (units | 1)


def work(case):
    H, d_h, r = case["H"], case["d_h"], case["r"]
    dk, w = d_h + case["d_rope"], sum(_widths(case))
    bf16_row, q_row = 2 * w, row_bytes(case)
    if case["op"] == "store":
        return {"bytes": case["n"] * (bf16_row + q_row + bf16_row + 12), "flops": 3 * case["n"] * w}
    B, own_tokens = case["B"], sum(lengths(case))
    io = 2 * B * H * (dk + d_h) + 4 * H * d_h * r
    per_pair = 2 * (dk + d_h + 2 * r)  # flops of one (query, key) pair of one head
    up = 4 * B * H * d_h * r
    if case["op"] == "quant":
        return {"bytes": own_tokens * q_row + io, "flops": own_tokens * H * per_pair + up}
    return {"bytes": (case["P"] + own_tokens) * bf16_row + io,
            "flops": (B * case["P"] + own_tokens) * H * per_pair + up}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _pools(case, g, blocks):
    """bf16 pages: unit normal with channels of somewhat different size, as projections give."""
    H, d_h, r = case["H"], case["d_h"], case["r"]
    out = []
    for shape in ((d_h + case["d_rope"],), (d_h,), (H, r), (H, r)):
        ch = torch.exp(0.25 * _normal(g, *shape))
        out.append((_normal(g, blocks, PAGE, *shape) * ch).to(torch.bfloat16))
    return out


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda")


def _pages_of(lens):
    return [-(-n // PAGE) for n in lens]


def _table(g, lens, first, ids):
    """[B, most pages] int32 page ids of the sequences, taken from ids in order; -1 where unused."""
    pages = _pages_of(lens)
    t = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32, device="cuda")
    at = first
    for b, p in enumerate(pages):
        t[b, :p] = ids[at:at + p].to(torch.int32)
        at += p
    return t


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _quantise(x):
    """x [n, w] (bf16 values): bytes [n, w] and scale bytes [n, blocks], as in the heading."""
    n, w = x.shape
    blocks = -(-w // BLOCK)
    v = torch.zeros(n, blocks * BLOCK, dtype=torch.float32, device=x.device)
    v[:, :w] = x.float()
    v = v.view(n, blocks, BLOCK)
    amax = v.abs().amax(2)
    # the scale's exponent puts the largest magnitude into [64, 128)
    e = torch.where(torch.isfinite(amax), ((amax.view(torch.int32) >> 23) - 6).clamp(min=1), 255)
    inv = ((254 - e.clamp(max=253)) << 23).view(torch.float32)
    q = torch.round(v * inv[..., None]).clamp(-127, 127)
    q = torch.nan_to_num(q, nan=0.0)
    return (q + 128).to(torch.uint8).view(n, -1)[:, :w], e.to(torch.uint8)


def _values(q, e, w):
    n = q.shape[0]
    blocks = e.shape[1]
    v = torch.zeros(n, blocks * BLOCK, dtype=torch.float32, device=q.device)
    v[:, :w] = q.float() - 128
    s = (e.to(torch.int32) << 23).view(torch.float32)
    return (v.view(n, blocks, BLOCK) * s[..., None]).view(n, -1)[:, :w]


def _pack(case, parts, rb):
    """bf16 parts [n, w_i] -> quantised rows [n, rb]."""
    off, soff, blocks = _offsets(case)
    rows = torch.zeros(parts[0].shape[0], rb, dtype=torch.uint8, device=parts[0].device)
    for i, x in enumerate(parts):
        q, e = _quantise(x)
        rows[:, off[i]:off[i] + q.shape[1]] = q
        at = soff + sum(blocks[:i])
        rows[:, at:at + blocks[i]] = e
    return rows


def _unpack(case, rows):
    """Quantised rows [n, rb] -> the four parts' values in 32 bits."""
    off, soff, blocks = _offsets(case)
    out = []
    for i, w in enumerate(_widths(case)):
        at = soff + sum(blocks[:i])
        out.append(_values(rows[:, off[i]:off[i] + w], rows[:, at:at + blocks[i]], w))
    return out


def _inputs(case, seed):
    g = _gen(seed)
    H, d_h, r = case["H"], case["d_h"], case["r"]
    s = dict(case=case)
    if case["op"] == "store":
        n = case["n"]
        blocks = _pages_of([n])[0]
        s["src"] = _pools(case, g, blocks)
        s["dst"] = [torch.zeros_like(p) for p in s["src"]]
        for k in ("src_slots", "row_slots", "dst_slots"):
            s[k] = _perm(g, blocks * PAGE)[:n].to(torch.int32)
        s["rows"] = torch.zeros(blocks, PAGE, row_bytes(case), dtype=torch.uint8, device="cuda")
        return s
    lens = lengths(case)
    B = case["B"]
    s["lens"] = lens
    s["q"] = _normal(g, B, H, d_h + case["d_rope"]).to(torch.bfloat16)
    s["BK"] = (_normal(g, H, d_h, r) * r ** -0.5).to(torch.bfloat16)
    s["BV"] = (_normal(g, H, d_h, r) * r ** -0.5).to(torch.bfloat16)
    own_pages = sum(_pages_of(lens))
    prefix = _pages_of([case["P"]])[0] if case["op"] == "shared" else 0
    ids = _perm(g, own_pages + prefix + 1)
    s["block_table"] = _table(g, lens, prefix, ids)
    s["seq_lens"] = _i32(lens)
    s["out"] = torch.empty(B, H, d_h, dtype=torch.bfloat16, device="cuda")
    if case["op"] == "shared":
        s["pools"] = _pools(case, g, own_pages + prefix + 1)
        s["prefix_blocks"] = ids[:prefix].to(torch.int32)
        s["prefix_len"] = _i32([case["P"]])
        return s
    rb = row_bytes(case)
    rows = torch.empty(own_pages + 1, PAGE, rb, dtype=torch.uint8, device="cuda")
    for first in range(0, own_pages + 1, 256):  # in pieces: the values in 32 bits are large
        last = min(own_pages + 1, first + 256)
        part = _pools(case, g, last - first)
        rows[first:last] = _pack(case, [p.reshape((last - first) * PAGE, -1) for p in part], rb).view(last - first, PAGE, rb)
    s["rows"] = rows
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from compressed_kv_cache_lrkv_gb300 import binding as b
        H, d_h = case["H"], case["d_h"]
        s["dims"] = b.make_dims(H, d_h, case["r"], H * d_h, d_rope=case["d_rope"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] == "store":
            s["src_cache"], s["dst_cache"] = b.PagedCache(*s["src"]), b.PagedCache(*s["dst"])
            s["qcache"] = b.QuantCache(s["rows"])
        elif case["op"] == "quant":
            s["qcache"] = b.QuantCache(s["rows"])
            s["ws"] = b.alloc_workspace(b.decode_quant_workspace_bytes(s["dims"], case["B"]))
        else:
            s["cache"] = b.PagedCache(*s["pools"])
            s["ws"] = b.alloc_workspace(
                b.decode_shared_workspace_bytes(s["dims"], case["B"], int(s["prefix_blocks"].shape[0])))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from compressed_kv_cache_lrkv_gb300 import binding as b
    op = s["case"]["op"]
    if op == "store":
        b.lrkv_cache_quantize(s["dims"], s["src_cache"], s["src_slots"], s["qcache"], s["row_slots"], status=s["status"])
        b.lrkv_cache_dequantize(s["dims"], s["qcache"], s["row_slots"], s["dst_cache"], s["dst_slots"],
                                status=s["status"])
        return s["dst"]
    if op == "quant":
        b.lrkv_decode_quant(s["dims"], s["q"], s["BK"], s["BV"], s["qcache"], s["block_table"], s["seq_lens"],
                            s["out"], s["ws"], status=s["status"])
    else:
        b.lrkv_decode_shared(s["dims"], s["q"], s["BK"], s["BV"], s["cache"], s["prefix_blocks"], s["prefix_len"],
                             s["block_table"], s["seq_lens"], s["out"], s["ws"], status=s["status"])
    return s["out"]


def _slots(pages, n):
    """Token slots 0 .. n - 1 of a sequence with these pages."""
    t = torch.arange(n, device="cuda")
    return pages[t // PAGE].long() * PAGE + t % PAGE


def _attend(case, q, qt, sK, sV, zK, zV):
    """Softmax statistics of queries [B, H, dk], q~ [B, H, r] over tokens [n, ...] in 32 bits."""
    n, H, r = sK.shape[0], case["H"], case["r"]
    scale = (case["d_h"] + case["d_rope"]) ** -0.5
    zK, zV = zK.view(n, H, r), zV.view(n, H, r)
    s = (torch.matmul(q, sK.t()) + torch.einsum("bhr,thr->bht", qt, zK)) * scale
    m = s.amax(2, keepdim=True)
    p = torch.exp(s - m)
    return m, p.sum(2, keepdim=True), torch.matmul(p, sV), torch.einsum("bht,thr->bhr", p, zV)


def _join(parts, BV):
    """Statistics of the parts of the tokens -> outputs."""
    m = torch.cat([p[0] for p in parts], 2).amax(2, keepdim=True)
    w = [torch.exp(p[0] - m) for p in parts]
    l = sum(x * p[1] for x, p in zip(w, parts))
    os = sum(x * p[2] for x, p in zip(w, parts))
    oz = sum(x * p[3] for x, p in zip(w, parts))
    return (os + torch.einsum("bhr,hdr->bhd", oz, BV)) / l


def _run_plain(s):
    case = s["case"]
    if case["op"] == "store":
        src = [p.view(-1, w)[s["src_slots"].long()] for p, w in zip(s["src"], _widths(case))]
        rows = s["rows"].view(-1, s["rows"].shape[2])
        rows[s["row_slots"].long()] = _pack(case, src, rows.shape[1])
        back = _unpack(case, rows[s["row_slots"].long()])
        for d, x in zip(s["dst"], back):
            d.view(-1, x.shape[1])[s["dst_slots"].long()] = x.to(torch.bfloat16)
        return s["dst"]
    q, BK, BV = s["q"].float(), s["BK"].float(), s["BV"].float()
    qt = torch.einsum("bhd,hdr->bhr", q[..., :case["d_h"]], BK)
    out = s["out"]
    if case["op"] == "quant":
        rows = s["rows"].view(-1, s["rows"].shape[2])
        for b, n in enumerate(s["lens"]):
            parts = _unpack(case, rows[_slots(s["block_table"][b], n)])
            out[b:b + 1] = _join([_attend(case, q[b:b + 1], qt[b:b + 1], *parts)], BV).to(torch.bfloat16)
        return out
    flat = [p.view(-1, w) for p, w in zip(s["pools"], _widths(case))]

    def tokens(pages, n):
        at = _slots(pages, n)
        return [p[at].float() for p in flat]

    pre = _attend(case, q, qt, *tokens(s["prefix_blocks"], case["P"]))
    for b, n in enumerate(s["lens"]):
        parts = [[x[b:b + 1] for x in pre]]
        if n:
            parts.append(_attend(case, q[b:b + 1], qt[b:b + 1], *tokens(s["block_table"][b], n)))
        out[b:b + 1] = _join(parts, BV).to(torch.bfloat16)
    return out


# ------------------------------------------------------------------ the definition, in 64 bits
def _power(k):
    """2^k in 64 bits, exactly (pow is not exact on every device)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _exact_blocks(x):
    """x [n, w] -> what the 8-bit blocks stand for: each block of 32 rounded to multiples of the
    power of two that puts its largest magnitude into [64, 128), at most 127 of them."""
    out = x.double().clone()
    for c in range(0, x.shape[1], BLOCK):
        v = out[:, c:c + BLOCK]
        top = v.abs().amax(1, keepdim=True)
        k = torch.frexp(top).exponent - 7  # top = f 2^k 128 with f in [1/2, 1)
        step = _power(k.clamp(min=-126))
        out[:, c:c + BLOCK] = (v / step).round().clamp(-127, 127) * step
    return out


def _exact_values(case, rows):
    """Rows [n, bytes] -> values in 64 bits, column by column of the format."""
    off, at, blocks = _offsets(case)
    r = rows.double()
    out = []
    for i, w in enumerate(_widths(case)):
        col = torch.arange(w, device=rows.device)
        e = rows[:, at:at + blocks[i]][:, col // BLOCK].long() - 127
        out.append((r[:, off[i]:off[i] + w] - 128.0) * _power(e))
        at += blocks[i]
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "store":
        res = []
        for p, d, w in zip(s["src"], s["dst"], _widths(case)):
            want = torch.zeros(d.numel() // w, w, dtype=torch.float64, device="cuda")
            want[s["dst_slots"].long()] = _exact_blocks(p.reshape(-1, w)[s["src_slots"].long()])
            res.append(want.view(d.shape))
        return res
    H, d_h, r = case["H"], case["d_h"], case["r"]
    BK, BV, q = s["BK"].double(), s["BV"].double(), s["q"].double()

    def features(parts):
        """Every head's keys and values, formed in full."""
        sK, sV, zK, zV = parts
        n = sK.shape[0]
        K = torch.einsum("thr,hdr->htd", zK.view(n, H, r), BK) + sK[:, :d_h]
        if case["d_rope"]:
            K = torch.cat([K, sK[None, :, d_h:].expand(H, -1, -1)], 2)
        return K, torch.einsum("thr,hdr->htd", zV.view(n, H, r), BV) + sV

    def stats(x, feats):
        """Over tokens in pieces: (max, sum, weighted values) of queries x [b, H, dk]."""
        t = torch.einsum("bhd,htd->bht", x, feats[0]) / math.sqrt(d_h + case["d_rope"])
        top = t.max(2).values
        e = torch.exp(t - top[..., None])
        return top, e.sum(2), torch.einsum("bht,htd->bhd", e, feats[1])

    def merge(a, b):
        if a is None:
            return b
        top = torch.maximum(a[0], b[0])
        fa, fb = torch.exp(a[0] - top), torch.exp(b[0] - top)
        return top, a[1] * fa + b[1] * fb, a[2] * fa[..., None] + b[2] * fb[..., None]

    def read(pages, first, last):
        t = torch.arange(first, last, device="cuda")
        at = pages[t // PAGE].long() * PAGE + t % PAGE
        if case["op"] == "quant":
            return _exact_values(case, s["rows"].view(-1, s["rows"].shape[2])[at])
        return [p.view(-1, w)[at].double() for p, w in zip(s["pools"], _widths(case))]

    step = 4096
    pre = None
    if case["op"] == "shared":
        for first in range(0, case["P"], step):
            pre = merge(pre, stats(q, features(read(s["prefix_blocks"], first, min(case["P"], first + step)))))
    res = []
    for b, n in enumerate(s["lens"]):
        st = None if pre is None else tuple(x[b:b + 1] for x in pre)
        for first in range(0, n, step):
            st = merge(st, stats(q[b:b + 1], features(read(s["block_table"][b], first, min(n, first + step)))))
        res.append(st[2] / st[1][..., None])
    return torch.cat(res)
