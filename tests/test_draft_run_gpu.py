"""Steps with drafted tokens as a server takes them: pages, append, rotated queries, verification, accepted rows kept, the
rest given back, a fork; after each step the cache holds exactly the accepted rows, and a plain decode sees them."""
import pytest
import torch

from attn64 import attend64, check

pytestmark = pytest.mark.gpu

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("H,d_h,r,T", [(8, 64, 16, 7), (20, 128, 16, 33)])
def test_serving_steps(H, d_h, r, T):
    g = torch.Generator(device="cuda").manual_seed(H)
    c = torch.Generator().manual_seed(H)
    d, dr, B, W, blocks = 256, 64, 5, 8, 40
    dims = b.make_dims(H, d_h, r, d, d_rope=dr)
    cache = b.PagedCache.empty(blocks, H, d_h, r, d_rope=dr)
    for t in cache.tensors():
        t.fill_(float("nan"))
    pools, plan = b.Pools.of(cache), b.rope_plan(dr)
    Wc = (torch.randn(2 * (d_h + H * r) + dr, d, generator=g, device="cuda") * d ** -0.5).to(BF)
    BK, BV = ((torch.randn(H, d_h, r, generator=g, device="cuda") * r ** -0.5).to(BF) for _ in range(2))
    refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = b.alloc_workspace(max(b.decode_tree_workspace_bytes(dims, B, T), b.decode_workspace_bytes(dims, B)))
    history = [[] for _ in range(B)]  # accepted (hidden row, position) of each sequence
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")

    def slots_of(s, first, n):
        t = torch.arange(first, first + n, device="cuda")
        return (table[s][t // 64] * 64 + t % 64).int()

    def rows(s):
        at = slots_of(s, 0, len(history[s])).long()
        return [t.view(-1, *t.shape[2:])[at].double() for t in cache.tensors()]

    # prompts of the first three sequences
    prompt = [70, 3, 64, 0, 0]
    b.lrkv_pages_reserve(refs, table, lens, i32(prompt), status=st)
    for s, n in enumerate(prompt):
        if n:
            x = torch.randn(n, d, generator=g, device="cuda").to(BF)
            pos = torch.arange(n, dtype=torch.int32, device="cuda")
            b.lrkv_append(dims, x, Wc, slots_of(s, 0, n), cache, status=st, positions=pos)
            history[s] = [(x[i], i) for i in range(n)]
    lens.copy_(i32(prompt))
    live, kids = [0, 1, 2], [3, 4]
    for step in range(4):
        if step == 1:  # two samples more of the first prompt
            b.lrkv_pages_fork(pools, refs, table, lens, i32([0, 0]), i32(kids), status=st)
            for k in kids:
                history[k] = list(history[0])
            live = [0, 1, 2, 3, 4]
        drafted = [T if s in live else 0 for s in range(B)]
        b.lrkv_pages_reserve(refs, table, lens, i32(drafted), status=st)
        parent = [[-1] + [int(torch.randint(0, i, (1,), generator=c)) for i in range(1, T)] for _ in range(B)]
        depth, seen = torch.zeros(B, T, dtype=torch.int64), torch.zeros(B, T, 64, dtype=torch.bool)
        for s in range(B):
            for i in range(T):
                if i:
                    seen[s, i], depth[s, i] = seen[s, parent[s][i]], depth[s, parent[s][i]] + 1
                seen[s, i, i] = True
        mask = (seen.long() << torch.arange(64)).sum(2).cuda()
        hidden = torch.randn(B, T, d, generator=g, device="cuda").to(BF)
        base = [len(h) for h in history]
        pos = (lens.cpu()[:, None] + depth).to(torch.int32).cuda()
        for s in live:
            b.lrkv_append(dims, hidden[s], Wc, slots_of(s, base[s], T), cache, status=st, positions=pos[s].contiguous())
        q = torch.randn(B, T, H, d_h + dr, generator=g, device="cuda").to(BF)
        flat = q.view(B * T, H, d_h + dr)
        b.lrkv_rope(plan, flat, flat, pos.view(-1), begin=d_h, status=st)
        out = torch.zeros(B, T, H, d_h, dtype=BF, device="cuda")
        b.lrkv_decode_tree(dims, q, BK, BV, cache, table, lens, mask, i32(drafted), out, ws, status=st)
        for s in live:
            at = slots_of(s, 0, base[s] + T).long()
            for i in (0, T // 2, T - 1):
                keep = torch.cat([torch.arange(base[s]), base[s] + torch.nonzero(seen[s, i]).flatten()]).cuda()
                parts = [t.view(-1, *t.shape[2:])[at[keep]].double() for t in cache.tensors()]
                want, bound = attend64(q[s, i].double(), BK.double(), BV.double(), parts, dr, eps_qt=2.0 ** -16)
                check(out[s, i], want, bound, f"step {step}, sequence {s}, token {i}")
        # a path of the tree is accepted, of any length
        path, n = torch.zeros(B, T, dtype=torch.int32), [0] * B
        for s in live:
            p = torch.nonzero(seen[s, int(torch.randint(0, T, (1,), generator=c))]).flatten()
            p = p[:int(torch.randint(0, p.numel() + 1, (1,), generator=c))]
            path[s, :p.numel()], n[s] = p.int(), p.numel()
            history[s] += [(hidden[s, i], int(pos[s, i])) for i in p.tolist()]
        b.lrkv_cache_compact(pools, table, lens, path.cuda(), i32(n), status=st)
        b.lrkv_pages_free(refs, table, lens, i32(list(range(B))), keep_lens=lens, status=st)
        assert lens.tolist() == [len(h) for h in history] and int(st.item()) == 0
        held = table[table >= 0].long()
        assert torch.equal(refs.cpu(), torch.bincount(held.cpu(), minlength=blocks).int())
        assert (table >= 0).sum(1).tolist() == [-(-len(h) // 64) for h in history]
        # the cache holds the accepted rows, as an append of them alone writes them
        other = b.PagedCache.empty(2 * W, H, d_h, r, d_rope=dr)
        for s in live:
            x = torch.stack([h[0] for h in history[s]])
            p = i32([h[1] for h in history[s]])
            assert p.tolist() == list(range(len(p)))  # depths follow the prompt without gaps
            b.lrkv_append(dims, x, Wc, torch.arange(len(p), dtype=torch.int32, device="cuda"), other, positions=p)
            for t, u in zip(rows(s), other.tensors()):
                u = u.view(-1, *u.shape[2:])[:len(p)].double()
                # (the append of few rows and of many sums in another order)
                assert (t - u).abs().max() <= 2.0 ** -6 * max(1.0, float(u.abs().max()))
        # a plain decode over them
        q1 = torch.randn(B, H, d_h + dr, generator=g, device="cuda").to(BF)
        o1 = torch.empty(B, H, d_h, dtype=BF, device="cuda")
        sub = i32(live).long()
        b.lrkv_decode(dims, q1[sub], BK, BV, cache, table[sub], lens[sub], o1[:len(live)], ws, status=st)
        for k, s in enumerate(live):
            want, bound = attend64(q1[s].double(), BK.double(), BV.double(), rows(s), dr)
            check(o1[k], want, bound, f"decode after step {step}, sequence {s}")
    b.lrkv_pages_free(refs, table, lens, i32(list(range(B))), status=st)
    assert (refs == 0).all() and (table == -1).all() and (lens == 0).all() and int(st.item()) == 0
