"""Operators of decoding with drafted tokens over the compressed cache, measured one by one, with
their plain forms.

Three operators on the paged cache of shared rows s and per-head latents z_h
(K_h = s^K + B_h^K z^K_h, V_h = s^V + B_h^V z^V_h):

  tree   one step over up to 64 drafted tokens per sequence: each attends to the sequence's cached
         tokens and to the drafted ones that its mask names (its ancestors and itself);
  rope   rotation of part of the heads of rows (queries, cached positional keys that move), in pairs
         of neighbours or of halves, with frequencies scaled for long contexts;
  pages  pages with reference counts: taken for drafted tokens, accepted rows moved together and the
         rest given back (step); sequences forked and freed (fork); whole pages copied (copy).

A page that no sequence holds has count 0, a table entry without a page is -1, and pages are taken
lowest first, for the sequences in their order.
"""
import math
import random

import torch

own = False

PAGE = 64


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest step: one short sequence, a chain of four drafted tokens
        dict(name="tree-small", op="tree", H=8, d_h=64, r=16, d_rope=0, B=1, T=4, tree=False, L_min=256, L=256),
        # one layer of a 12-layer backbone, a small tree for each sequence
        dict(name="tree-backbone", op="tree", H=8, d_h=64, r=16, d_rope=0, B=16, T=16, tree=True, L_min=2048, L=2048),
        # ragged batch with the positional key, trees of 26
        dict(name="tree-ragged", op="tree", H=32, d_h=128, r=16, d_rope=64, B=24, T=26, tree=True, L_min=1, L=8191),
        # long context, a chain of eight
        dict(name="tree-longctx", op="tree", H=32, d_h=128, r=32, d_rope=0, B=4, T=8, tree=False, L_min=16384, L=32768),
        # many heads and the widest trees
        dict(name="tree-heads", op="tree", H=128, d_h=128, r=16, d_rope=0, B=8, T=64, tree=True, L_min=8192, L=8192),
        # the queries of one decode step: the positional part of every head
        dict(name="rope-step", op="rope", n=16, heads=32, width=192, begin=128, d_rot=64, half=False, scaling="none",
             transpose=False, fp32=False, slots=False),
        # the queries of a prefill chunk of two prompts
        dict(name="rope-chunk", op="rope", n=8192, heads=32, width=192, begin=128, d_rot=64, half=False,
             scaling="none", transpose=False, fp32=False, slots=False),
        # cached positional keys of a long context, turned on to new positions in new slots
        dict(name="rope-keys", op="rope", n=65536, heads=1, width=64, begin=0, d_rot=64, half=False, scaling="parts",
             transpose=False, fp32=False, slots=True),
        # a gradient in 32 bits through half-paired rotation of whole heads, odd sizes
        dict(name="rope-grad", op="rope", n=4095, heads=12, width=128, begin=0, d_rot=128, half=True,
             scaling="linear", transpose=True, fp32=True, slots=False),
        # a 12-layer backbone after a step with drafted tokens: pages, accepted rows, pages back
        dict(name="pages-step", op="pages", kind="step", layers=12, H=8, d_h=64, r=16, d_rope=0, B=16, T=32, L_min=1,
             L=2048),
        # four prompts, sixteen samples of each
        dict(name="pages-fork", op="pages", kind="fork", layers=4, H=32, d_h=128, r=32, d_rope=0, B=4, forks=16,
             L_min=2048, L=8192),
        # idle sequences' pages moved to another pool
        dict(name="pages-copy", op="pages", kind="copy", layers=1, H=32, d_h=128, r=32, d_rope=0, n=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        c = dict(op=rng.choice(["tree", "tree", "rope", "pages"]))
        if c["op"] == "rope":
            c["n"] = _log_int(rng, 1, 65536)
            c["heads"] = _log_int(rng, 1, 128)
            c["d_rot"] = rng.choice([8, 16, 32, 64, 64, 96, 128, 128])
            c["begin"] = rng.choice([0, 0, 8, 64, 128])
            c["width"] = c["begin"] + c["d_rot"] + rng.choice([0, 0, 8, 40])
            c["half"] = rng.random() < 0.5
            c["scaling"] = rng.choice(["none", "linear", "parts"])
            c["transpose"] = rng.random() < 0.3
            c["fp32"] = rng.random() < 0.3
            c["slots"] = rng.random() < 0.3
            if c["n"] * c["heads"] * c["width"] * (4 if c["fp32"] else 2) <= 8192 * 32 * 192 * 2:
                return c
            continue
        c.update(H=_log_int(rng, 1, 128), d_h=rng.choice([64, 128]), r=rng.choice([8, 16, 32]),
                 d_rope=rng.choice([0, 0, 64]))
        if c["op"] == "tree":
            c["B"] = _log_int(rng, 1, 48)
            c["T"] = _log_int(rng, 1, 64)
            c["tree"] = rng.random() < 0.7
            c["L"] = _log_int(rng, 1, 32768)
            c["L_min"] = rng.randint(0, c["L"])
            if work(c)["flops"] <= 2.2e11 and sum(lengths(c)) * row_bytes(c) <= 55e7:
                return c
            continue
        c["kind"] = rng.choice(["step", "fork", "copy"])
        c["layers"] = _log_int(rng, 1, 16)
        if c["kind"] == "copy":
            c["n"] = _log_int(rng, 1, 1024)
            if c["n"] * c["layers"] * PAGE * row_bytes(c) <= 1024 * PAGE * 4608:
                return c
            continue
        c["B"] = _log_int(rng, 1, 64)
        c["L"] = _log_int(rng, 1, 8192)
        c["L_min"] = rng.randint(1, c["L"])
        if c["kind"] == "step":
            c["T"] = _log_int(rng, 1, 64)
        else:
            c["forks"] = _log_int(rng, 1, 16)
        pages = sum(_pages_of(lengths(c))) + c["B"] * c.get("forks", 1) + c["B"]
        if pages * c["layers"] * PAGE * row_bytes(c) <= 1 << 30:
            return c


def lengths(case):
    """The sequences' cached tokens: whole numbers spread over [L_min, L], fixed by the case."""
    rng = random.Random(case["B"] * 1000003 + case["L_min"] * 101 + case["L"])
    return [rng.randint(case["L_min"], case["L"]) for _ in range(case["B"])]


def trees(case):
    """Per sequence the drafted tokens' masks (bit j: token j is seen), as many as it has drafted; the
    first sequence has T, others down to half of that."""
    rng = random.Random(case["T"] * 7907 + case["B"])
    out = []
    for b in range(case["B"]):
        n = case["T"] if b == 0 else rng.randint((case["T"] + 1) // 2, case["T"])
        masks = []
        for i in range(n):
            # a child of a token not far behind, so that paths get some depth
            parent = i - 1 if not case["tree"] else rng.randint(max(0, i // 2 - 2), i - 1) if i else -1
            masks.append((masks[parent] if i else 0) | 1 << i)
        out.append(masks)
    return out


def accepted(case):
    """Per sequence the drafted tokens kept, increasing: the first ones as they stand, later ones from
    behind the places that are written (so that a second pass finds the same rows)."""
    rng = random.Random(case["T"] * 31 + case["B"])
    out = []
    for b in range(case["B"]):
        n = rng.randint(0, min(8, case["T"]))
        keep = rng.randint(0, n)
        rest = n - keep
        if case["T"] - n < rest:
            keep, rest = n, 0
        out.append(list(range(keep)) + sorted(rng.sample(range(n, case["T"]), rest)))
    return out


def _widths(case):
    hr = case["H"] * case["r"]
    return [case["d_h"] + case["d_rope"], case["d_h"], hr, hr]


def row_bytes(case):
    return 2 * sum(_widths(case))


def _pages_of(lens):
    return [-(-n // PAGE) for n in lens]


def work(case):
    if case["op"] == "rope":
        e = 4 if case["fp32"] else 2
        n = case["n"] * case["heads"]
        return {"bytes": 2 * e * n * case["width"] + case["n"] * (4 + 8 * case["slots"]), "flops": 3 * n * case["d_rot"]}
    if case["op"] == "tree":
        H, d_h, r = case["H"], case["d_h"], case["r"]
        dk, lens, tr = d_h + case["d_rope"], lengths(case), trees(case)
        rows = sum(len(m) for m in tr)
        pairs = sum(len(m) * n + sum(bin(x).count("1") for x in m) for m, n in zip(tr, lens))
        tokens = sum(lens) + rows
        return {"bytes": tokens * row_bytes(case) + 2 * rows * H * (dk + d_h) + 4 * H * d_h * r + 8 * rows,
                "flops": pairs * H * 2 * (dk + d_h + 2 * r) + 4 * rows * H * d_h * r}
    row = row_bytes(case) * case["layers"]
    if case["kind"] == "copy":
        return {"bytes": case["n"] * (2 * PAGE * row + 8), "flops": 0}
    lens = lengths(case)
    if case["kind"] == "fork":
        tails = sum(n % PAGE for n in lens) * case["forks"]
        return {"bytes": 2 * tails * row + 16 * case["forks"] * sum(_pages_of(lens)), "flops": 0}
    moved = sum(1 for p in accepted(case) for i, x in enumerate(p) if i != x)
    return {"bytes": 2 * moved * row + 32 * case["B"] * (2 + -(-case["T"] // PAGE)), "flops": 0}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 23)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _pools(case, g, blocks, layers=None):
    """bf16 pages: unit normal with channels of somewhat different size, as projections give."""
    H, d_h, r = case["H"], case["d_h"], case["r"]
    out = []
    for shape in ((d_h + case["d_rope"],), (d_h,), (H, r), (H, r)):
        ch = torch.exp(0.25 * _normal(g, *shape))
        each = [(_normal(g, blocks, PAGE, *shape) * ch).to(torch.bfloat16) for _ in range(layers or 1)]
        out.append(each[0] if layers is None else torch.stack(each))
    return out


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(pages, ids, width, rows=None):
    """[rows, width] int32 page ids of the sequences, taken from ids in order; -1 where unused."""
    t = torch.full((rows or len(pages), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, p in enumerate(pages):
        t[b, :p] = ids[at:at + p].to(torch.int32)
        at += p
    return t


# scaled for contexts of eight times the length that the frequencies were made for
ROPE = dict(base=10000.0, factor=8.0, original=8192.0, low=1.0, high=32.0)


def _tree_inputs(case, g):
    H, d_h, r, B, T = (case[k] for k in ("H", "d_h", "r", "B", "T"))
    lens, masks = lengths(case), trees(case)
    pages = _pages_of([n + len(m) for n, m in zip(lens, masks)])
    s = dict(lens=lens, drafted=[len(m) for m in masks])
    s["q"] = _normal(g, B, T, H, d_h + case["d_rope"]).to(torch.bfloat16)
    s["BK"] = (_normal(g, H, d_h, r) * r ** -0.5).to(torch.bfloat16)
    s["BV"] = (_normal(g, H, d_h, r) * r ** -0.5).to(torch.bfloat16)
    s["pools"] = _pools(case, g, sum(pages) + 1)
    s["block_table"] = _table(pages, _perm(g, sum(pages) + 1), max(1, max(pages)))
    s["seq_lens"], s["tree_lens"] = _i32(lens), _i32(s["drafted"])
    words = [[x - (1 << 64) if x >> 63 else x for x in m] + [0] * (T - len(m)) for m in masks]
    s["mask"] = torch.tensor(words, dtype=torch.int64, device="cuda")
    s["out"] = torch.zeros(B, T, H, d_h, dtype=torch.bfloat16, device="cuda")
    return s


def _rope_inputs(case, g):
    n, heads, width = case["n"], case["heads"], case["width"]
    kind = torch.float32 if case["fp32"] else torch.bfloat16
    rows = -(-(n + n // 8) // PAGE) * PAGE if case["slots"] else n
    s = dict(x=_normal(g, rows, heads, width).to(kind), y=torch.zeros(rows, heads, width, dtype=kind, device="cuda"),
             x_rows=None, y_rows=None)
    if case["slots"]:  # keys that move on by up to a context's length, either way
        s["x_rows"], s["y_rows"] = (_perm(g, rows)[:n].to(torch.int32) for _ in range(2))
        s["positions"] = torch.randint(-131072, 131072, (n,), generator=g, device="cuda", dtype=torch.int32)
    else:
        first = torch.randint(0, 1 << 17, (1,), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = first + torch.arange(n, device="cuda", dtype=torch.int32) % 4096
    return s


def _pages_inputs(case, g):
    s = {}
    if case["kind"] == "copy":
        s["pools"] = _pools(case, g, case["n"], case["layers"])
        s["other"] = [torch.zeros_like(p) for p in s["pools"]]
        s["src"], s["dst"] = (_perm(g, case["n"]).to(torch.int32) for _ in range(2))
        return s
    lens, B = lengths(case), case["B"]
    pages = _pages_of(lens)
    rows = B * (1 + case.get("forks", 0))
    spare = B * (case["forks"] if case["kind"] == "fork" else 1 + case["T"] // PAGE) + 3
    blocks = sum(pages) + spare
    s["pools"] = _pools(case, g, blocks, case["layers"])
    s["table"] = _table(pages, _perm(g, blocks), max(pages) + 2, rows)
    s["seq_lens"] = _i32(lens + [0] * (rows - B))
    held = s["table"].flatten()
    s["refs"] = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    s["refs"][held[held >= 0].long()] = 1
    if case["kind"] == "fork":
        s["children"] = torch.arange(B, rows, dtype=torch.int32, device="cuda")
        s["parents"] = _perm(g, rows - B).to(torch.int32) % B
        return s
    T, path = case["T"], accepted(case)
    s["new_tokens"] = torch.full((B,), T, dtype=torch.int32, device="cuda")
    s["path"] = _i32([p + [0] * (T - len(p)) for p in path])
    s["path_lens"] = _i32([len(p) for p in path])
    s["new_lens"] = torch.zeros_like(s["seq_lens"])
    s["all"] = torch.arange(B, dtype=torch.int32, device="cuda")
    return s


def _inputs(case, seed):
    make = {"tree": _tree_inputs, "rope": _rope_inputs, "pages": _pages_inputs}[case["op"]]
    return dict(make(case, _gen(seed)), case=case)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from compressed_kv_cache_lrkv_gb300 import binding as b
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] == "tree":
            s["dims"] = b.make_dims(case["H"], case["d_h"], case["r"], case["H"] * case["d_h"], d_rope=case["d_rope"])
            s["cache"] = b.PagedCache(*s["pools"])
            s["ws"] = b.alloc_workspace(b.decode_tree_workspace_bytes(s["dims"], case["B"], case["T"]))
        elif case["op"] == "rope":
            s["plan"] = b.rope_plan(case["d_rot"], layout="half" if case["half"] else "interleaved", base=ROPE["base"],
                                    scaling=case["scaling"], factor=ROPE["factor"], original_len=ROPE["original"],
                                    low=ROPE["low"], high=ROPE["high"], magnitude=_magnitude(case))
        else:
            s["own_pools"] = b.Pools.of(b.LayeredCache(*s["pools"]))
            if case["kind"] == "copy":
                s["own_other"] = b.Pools.of(b.LayeredCache(*s["other"]))
    return s


def _magnitude(case):
    return 0.1 * math.log(ROPE["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if case["op"] == "tree":
        (_tree_own if own else _tree_plain)(s)
        return s["out"]
    if case["op"] == "rope":
        (_rope_own if own else _rope_plain)(s)
        return s["y"]
    (_pages_own if own else _pages_plain)(s)
    # cache rows are moved, not computed: returned as their bits
    if case["kind"] == "copy":
        return [p.view(torch.int16) for p in s["other"]]
    res = [p.view(torch.int16) for p in s["pools"]] + [s["table"], s["refs"], s["seq_lens"]]
    return res + [s["new_lens"]] if case["kind"] == "step" else res


def _tree_own(s):
    from compressed_kv_cache_lrkv_gb300 import binding as b
    b.lrkv_decode_tree(s["dims"], s["q"], s["BK"], s["BV"], s["cache"], s["block_table"], s["seq_lens"], s["mask"],
                       s["tree_lens"], s["out"], s["ws"], status=s["status"])


def _rope_own(s):
    from compressed_kv_cache_lrkv_gb300 import binding as b
    b.lrkv_rope(s["plan"], s["x"], s["y"], s["positions"], begin=s["case"]["begin"], x_rows=s["x_rows"],
                y_rows=s["y_rows"], transpose=s["case"]["transpose"], status=s["status"])


def _pages_own(s):
    from compressed_kv_cache_lrkv_gb300 import binding as b
    kind = s["case"]["kind"]
    if kind == "copy":
        b.lrkv_pages_copy(s["own_pools"], s["src"], s["own_other"], s["dst"], status=s["status"])
    elif kind == "fork":
        b.lrkv_pages_free(s["refs"], s["table"], s["seq_lens"], s["children"], status=s["status"])
        b.lrkv_pages_fork(s["own_pools"], s["refs"], s["table"], s["seq_lens"], s["parents"], s["children"],
                          status=s["status"])
    else:
        b.lrkv_pages_reserve(s["refs"], s["table"], s["seq_lens"], s["new_tokens"], status=s["status"])
        b.lrkv_cache_compact(s["own_pools"], s["table"], s["seq_lens"], s["path"], s["path_lens"],
                             new_lens=s["new_lens"], status=s["status"])
        b.lrkv_pages_free(s["refs"], s["table"], s["new_lens"], s["all"], keep_lens=s["new_lens"], status=s["status"])


def _slots(pages, n):
    """Token slots 0 .. n - 1 of a sequence with these pages."""
    t = torch.arange(n, device="cuda")
    return pages[t // PAGE].long() * PAGE + t % PAGE


def _tree_plain(s):
    case = s["case"]
    H, d_h, r = case["H"], case["d_h"], case["r"]
    q, BK, BV = s["q"].float(), s["BK"].float(), s["BV"].float()
    qt = torch.einsum("bihd,hdr->bihr", q[..., :d_h], BK)
    flat = [p.view(-1, w) for p, w in zip(s["pools"], _widths(case))]
    scale = (d_h + case["d_rope"]) ** -0.5
    bits = torch.arange(PAGE, device="cuda")
    for b, (L, n) in enumerate(zip(s["lens"], s["drafted"])):
        at = _slots(s["block_table"][b], L + n)
        sK, sV, zK, zV = (p[at].float() for p in flat)
        zK, zV = zK.view(-1, H, r), zV.view(-1, H, r)
        t = (torch.matmul(q[b, :n], sK.t()) + torch.einsum("ihr,thr->iht", qt[b, :n], zK)) * scale
        seen = torch.ones(n, L + n, dtype=torch.bool, device="cuda")
        seen[:, L:] = (s["mask"][b, :n, None] >> bits[:n] & 1).bool()
        t = t.masked_fill(~seen[:, None], -math.inf)
        m = t.amax(2, keepdim=True)
        p = torch.exp(t - torch.where(m == -math.inf, 0.0, m))
        o = torch.matmul(p, sV) + torch.einsum("ihr,hdr->ihd", torch.einsum("iht,thr->ihr", p, zV), BV)
        total = p.sum(2, keepdim=True)
        s["out"][b, :n] = torch.where(total > 0, o / total, 0.0).to(torch.bfloat16)


def _frequencies(case):
    """Turning speeds of the pairs in 64 bits (radians a position)."""
    i = torch.arange(case["d_rot"] // 2, dtype=torch.float64, device="cuda")
    f = ROPE["base"] ** (-2.0 * i / case["d_rot"])
    if case["scaling"] == "linear":
        return f / ROPE["factor"]
    if case["scaling"] == "parts":
        turns = ROPE["original"] * f / (2 * math.pi)
        kept = ((turns - ROPE["low"]) / (ROPE["high"] - ROPE["low"])).clamp(0, 1)
        return f * kept + f / ROPE["factor"] * (1 - kept)
    return f


def _rope_plain(s):
    case = s["case"]
    angle = s["positions"].double()[:, None] * _frequencies(case)
    if case["transpose"]:
        angle = -angle
    c, si = ((f(angle) * _magnitude(case)).float()[:, None] for f in (torch.cos, torch.sin))
    x = (s["x"] if s["x_rows"] is None else s["x"][s["x_rows"].long()]).float()
    lo, hi = case["begin"], case["begin"] + case["d_rot"]
    part = x[..., lo:hi]
    if case["half"]:
        x0, x1 = part.chunk(2, -1)
        turned = torch.cat([x0 * c - x1 * si, x0 * si + x1 * c], -1)
    else:
        x0, x1 = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([x0 * c - x1 * si, x0 * si + x1 * c], -1).flatten(-2)
    y = torch.cat([x[..., :lo], turned, x[..., hi:]], -1).to(s["y"].dtype)
    if s["y_rows"] is None:
        s["y"].copy_(y)
    else:
        s["y"][s["y_rows"].long()] = y


def _take(refs, wanted):
    """The lowest free pages for the places where wanted is true, in order (enough are free)."""
    free = torch.cumsum((refs == 0).long(), 0)
    rank = torch.cumsum(wanted.flatten().long(), 0).view(wanted.shape)
    return torch.searchsorted(free, rank.clamp(min=1)).clamp(max=refs.numel() - 1)


def _free_plain(refs, table, lens, rows, keep):
    rows = rows.long()
    sub = table[rows]
    kept = (keep[rows] + PAGE - 1) // PAGE if keep is not None else torch.zeros_like(rows)
    gone = (torch.arange(table.shape[1], device="cuda") >= kept[:, None]) & (sub >= 0)
    refs.scatter_add_(0, sub.clamp(min=0).flatten().long(), -gone.flatten().to(refs.dtype))
    table[rows] = torch.where(gone, -1, sub)
    if keep is None:
        lens[rows] = 0


def _pages_plain(s):
    case, table, refs, lens = s["case"], s.get("table"), s.get("refs"), s.get("seq_lens")
    kind = case["kind"]
    if kind == "copy":
        for d, p in zip(s["other"], s["pools"]):
            d[:, s["dst"].long()] = p[:, s["src"].long()]
        return
    col = torch.arange(table.shape[1], device="cuda")
    flat = [p.view(p.shape[0], -1, w) for p, w in zip(s["pools"], _widths(case))]
    if kind == "fork":
        _free_plain(refs, table, lens, s["children"], None)
        parents, kids = s["parents"].long(), s["children"].long()
        L = lens[parents].long()
        full, tail = L // PAGE, L % PAGE
        rows = torch.where(col < full[:, None], table[parents], -1)
        refs.scatter_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).flatten().to(refs.dtype))
        new = _take(refs, tail > 0)
        refs.scatter_add_(0, new, (tail > 0).to(refs.dtype))
        old = table[parents].gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
        rows = torch.where((col == full[:, None]) & (tail > 0)[:, None], new[:, None].to(torch.int32), rows)
        table[kids] = rows
        lens[kids] = lens[parents]
        t = torch.arange(PAGE, device="cuda")
        live = t < tail[:, None]
        # (a row that is not copied is written onto itself, in its own page)
        src = torch.where(live, old[:, None] * PAGE + t, new[:, None] * PAGE + t)
        dst = new[:, None] * PAGE + t
        keep = (tail > 0)
        src, dst = src[keep].flatten(), dst[keep].flatten()
        for p in flat:
            p[:, dst] = p[:, src]
        return
    need = (lens + s["new_tokens"] + PAGE - 1) // PAGE
    wanted = (col < need[:, None]) & (table < 0)
    page = _take(refs, wanted)
    table.copy_(torch.where(wanted, page.to(torch.int32), table))
    refs.scatter_add_(0, page.flatten(), wanted.flatten().to(refs.dtype))
    i = torch.arange(case["T"], device="cuda")
    live = i < s["path_lens"][:, None]

    def slot(at):
        return table.gather(1, (at // PAGE).long()).long() * PAGE + at % PAGE

    to = lens[:, None] + torch.where(live, i, 0)
    src = slot(torch.where(live, lens[:, None] + s["path"], to))[live]
    dst = slot(to)[live]
    for p in flat:
        p[:, dst] = p[:, src]
    s["new_lens"].copy_(lens + s["path_lens"])
    _free_plain(refs, table, None, s["all"], s["new_lens"])


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    if case["op"] == "pages":  # nothing is computed
        return None
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    H, d_h, r = case["H"], case["d_h"], case["r"]
    BK, BV, q = s["BK"].double(), s["BV"].double(), s["q"].double()
    res = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, masks in enumerate(trees(case)):
        L, n = s["lens"][b], len(masks)
        top = torch.full((n, H), -math.inf, dtype=torch.float64, device="cuda")
        total, acc = torch.zeros_like(top), torch.zeros(n, H, d_h, dtype=torch.float64, device="cuda")
        for first in range(0, L + n, 2048):
            t = torch.arange(first, min(L + n, first + 2048), device="cuda")
            at = s["block_table"][b][t // PAGE].long() * PAGE + t % PAGE
            sK, sV, zK, zV = (p.reshape(-1, w)[at].double() for p, w in zip(s["pools"], _widths(case)))
            # every head's keys and values, formed in full
            K = torch.einsum("thr,hdr->htd", zK.view(-1, H, r), BK) + sK[:, :d_h]
            if case["d_rope"]:
                K = torch.cat([K, sK[None, :, d_h:].expand(H, -1, -1)], 2)
            V = torch.einsum("thr,hdr->htd", zV.view(-1, H, r), BV) + sV
            x = torch.einsum("ihd,htd->iht", q[b, :n], K) / math.sqrt(d_h + case["d_rope"])
            hide = torch.tensor([[j >= L and not m >> (j - L) & 1 for j in range(first, min(L + n, first + 2048))]
                                 for m in masks], device="cuda") if first + 2048 > L else None
            if hide is not None:
                x = x.masked_fill(hide[:, None], -math.inf)
            new = torch.maximum(top, x.max(2).values)
            base = torch.where(new == -math.inf, 0.0, new)
            e, f = torch.exp(x - base[..., None]), torch.exp(top - base)
            total = total * f + e.sum(2)
            acc = acc * f[..., None] + torch.einsum("iht,htd->ihd", e, V)
            top = new
        res[b, :n] = torch.where(total[..., None] > 0, acc / total[..., None], 0.0)
    return res


def _exact_rope(case, s):
    """Pairs as complex numbers, times e^(i angle)."""
    x = s["x"].double()
    y = torch.zeros_like(x)
    src = torch.arange(case["n"], device="cuda") if s["x_rows"] is None else s["x_rows"].long()
    dst = torch.arange(case["n"], device="cuda") if s["y_rows"] is None else s["y_rows"].long()
    m, lo = case["d_rot"] // 2, case["begin"]
    i = torch.arange(m, device="cuda")
    a, b = (lo + i, lo + m + i) if case["half"] else (lo + 2 * i, lo + 2 * i + 1)
    speed = []
    for k in range(m):
        f = math.exp(-2.0 * k / case["d_rot"] * math.log(ROPE["base"]))
        kept = 1.0
        if case["scaling"] == "linear":
            kept = 0.0
        elif case["scaling"] == "parts":
            kept = (ROPE["original"] * f / math.tau - ROPE["low"]) / (ROPE["high"] - ROPE["low"])
            kept = min(1.0, max(0.0, kept))
        speed.append(f * (kept + (1.0 - kept) / ROPE["factor"]))
    angle = s["positions"].double()[:, None] * torch.tensor(speed, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, _magnitude(case)), -angle if case["transpose"] else angle)[:, None]
    rows = x[src]
    z = torch.complex(rows[..., a], rows[..., b]) * turn
    rows[..., a], rows[..., b] = z.real, z.imag
    y[dst] = rows
    return y
