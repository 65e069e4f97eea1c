"""Drafted tokens, rotary positions and pages: arguments that are refused on the host (no GPU needed), and the plan of a
rotation."""
import ctypes
import math

import numpy as np
import pytest

from compressed_kv_cache_lrkv_gb300 import binding as b

R = ctypes.byref
GOOD = b.make_dims(8, 64, 16, 512)
CACHE = b.Cache(16, 16, 16, 16, 4)


def test_tree_arguments():
    lib = b.load()
    base = dict(dims=GOOD, q=16, BK=16, BV=16, cache=CACHE, bt=16, mb=1, sl=16, mask=16, tl=16, B=1, T=4, out=16)

    def call(**kw):
        a = dict(base, **kw)
        c = R(a["cache"]) if a["cache"] else None
        return lib.lrkv_decode_tree(R(a["dims"]), a["q"], a["BK"], a["BV"], c, a["bt"], a["mb"], a["sl"], a["mask"],
                                    a["tl"], a["B"], a["T"], a["out"], 256, 1 << 40, None, None)

    assert call(B=0) == 0
    assert call(T=0) == 2 and call(T=65) == 2 and call(T=-1) == 2 and b"T " in lib.lrkv_last_error()
    assert call(B=-1) == 1 and call(B=65536, T=1) == 1 and call(B=1024, T=64) == 1
    assert call(dims=b.make_dims(8, 96, 16, 512)) == 2 and call(dims=b.make_dims(8, 64, 16, 512, d_rope=32)) == 2
    assert call(cache=None) == 1 and call(cache=b.Cache(16, 16, 16, 0, 4)) == 1
    assert call(mb=0) == 1 and call(mb=1 << 25) == 1
    for k in ("q", "BK", "BV", "out"):
        assert call(**{k: None}) == 1 and call(**{k: 24}) == 1, k
    assert call(bt=None) == 1 and call(sl=None) == 1 and call(mask=20) == 1
    assert b.decode_tree_workspace_bytes(GOOD, 1, 65) == 0 and b.decode_tree_workspace_bytes(GOOD, -1, 1) == 0


def spec(**kw):
    d = dict(d_rot=64, layout=0, scaling=0, reserved=0, base=0.0, factor=0.0, original_len=0.0, low=0.0, high=0.0,
             magnitude=0.0)
    d.update(kw)
    return b.RopeSpec(**d)


def test_rope_plan_arguments():
    lib = b.load()
    plan = b.RopePlan()

    def make(**kw):
        return lib.lrkv_rope_make_plan(R(spec(**kw)), R(plan))

    assert make() == 0 and lib.lrkv_rope_make_plan(None, R(plan)) == 1 and lib.lrkv_rope_make_plan(R(spec()), None) == 1
    for d in (0, 4, 12, 264, -8):
        assert make(d_rot=d) == 2, d
    nan, inf = float("nan"), float("inf")
    assert make(layout=2) == 1 and make(layout=-1) == 1 and make(scaling=3) == 1 and make(scaling=-1) == 1
    for x in (1.0, 0.5, -3.0, nan, inf):
        assert make(base=x) == 1, x
    assert make(magnitude=nan) == 1 and make(magnitude=1e300) == 1
    for x in (0.0, 0.99, nan, inf):
        assert make(scaling=1, factor=x) == 1 and make(factor=x) == 0, x
    parts = dict(scaling=2, factor=4.0, original_len=100.0, low=1.0, high=32.0)
    assert make(**parts) == 0
    for k, v in (("original_len", 0.0), ("original_len", nan), ("low", -1.0), ("high", 1.0), ("high", inf), ("low", nan)):
        assert make(**dict(parts, **{k: v})) == 1, (k, v)


@pytest.mark.parametrize("d_rot,kw", [(64, {}), (128, dict(base=500000.0, scaling="linear", factor=8.0)),
                                      (96, dict(scaling="parts", factor=8.0, original_len=8192.0)), (8, {}), (256, {})])
def test_rope_plan_speeds(d_rot, kw):
    """Fractions of a turn against the formula in Python's floats: within a few steps of double precision, what
    the check itself can tell, and half a step of the table, 2^-65 of a turn (a speed of 2^-19 of a turn has 2^-70 as
    its eight steps of double precision, so the table's own step is the larger part there)."""
    plan = b.rope_plan(d_rot, **kw)
    base, factor = kw.get("base", 10000.0), kw.get("factor", 1.0)
    for i in range(d_rot // 2):
        f = base ** (-2.0 * i / d_rot)
        if kw.get("scaling") == "linear":
            f /= factor
        elif kw.get("scaling") == "parts":
            g = min(1.0, max(0.0, (8192.0 * f / math.tau - 1.0) / 31.0))
            f = g * f + (1 - g) * f / factor
        assert abs(plan.turn[i] / 2.0 ** 64 - f / math.tau) <= 8 * 2.0 ** -53 * f + 2.0 ** -65, i
    assert all(plan.turn[i] == 0 for i in range(d_rot // 2, 128)) and plan.magnitude == 1.0
    # pair 0 turns by 1 / 2 pi of a turn where nothing is scaled: its 64 bits, from pi's published digits
    if not kw:
        assert abs(plan.turn[0] - 2935890503282001226) <= 2


def test_rope_arguments():
    lib = b.load()
    plan = b.rope_plan(64)
    base = dict(plan=plan, dtype=0, n=4, heads=2, width=128, begin=64, x=(16, 4, 256, 128, None),
                y=(4096, 4, 256, 128, None), pos=16, tr=0)

    def call(**kw):
        a = dict(base, **kw)
        x, y = (R(b.RowsStruct(*a[k])) if a[k] else None for k in "xy")
        return lib.lrkv_rope(R(a["plan"]) if a["plan"] else None, a["dtype"], a["n"], a["heads"], a["width"], a["begin"],
                             x, y, a["pos"], a["tr"], None, None)

    assert call(n=0) == 0
    assert call(plan=None) == 1 and call(plan=b.RopePlan()) == 1 and call(x=None) == 1 and call(y=None) == 1
    assert call(dtype=2) == 2 and call(tr=2) == 1 and call(n=-1) == 1 and call(heads=0) == 1 and call(heads=65536) == 1
    assert call(width=100) == 2 and call(begin=4) == 2 and call(begin=72) == 2 and call(begin=-8) == 2
    assert call(width=1032) == 2 and call(pos=None) == 1
    for k in "xy":
        for bad in ((0, 4, 256, 128, None), (24, 4, 256, 128, None), (16, 4, 252, 128, None), (16, 4, 256, 4, None),
                    (16, 4, -256, 128, None), (16, 3, 256, 128, None), (16, 0, 256, 128, 16)):
            assert call(**{k: bad}) == 1, (k, bad)
    # y's rows or heads on top of one another
    for bad in ((16, 4, 128, 128, None), (16, 4, 256, 64, None), (16, 4, 0, 128, None), (16, 4, 256, 0, None),
                (16, 4, 128, 256, None)):
        assert call(y=bad) == 1 and b"overlap" in lib.lrkv_last_error(), bad


def pools(**kw):
    s = b.PoolsStruct()
    d = dict(num_pools=2, num_layers=2, num_blocks=4, base=(16, 32, 0, 0), row_bytes=(32, 16, 0, 0),
             layer_bytes=(4 * 64 * 32, 4 * 64 * 16, 0, 0))
    d.update(kw)
    for k in ("num_pools", "num_layers", "num_blocks"):
        setattr(s, k, d[k])
    for k in ("base", "row_bytes", "layer_bytes"):
        for i, v in enumerate(d[k]):
            getattr(s, k)[i] = v
    return s


BAD_POOLS = [dict(num_pools=0), dict(num_pools=5), dict(num_layers=0), dict(num_blocks=0), dict(num_blocks=(1 << 24) + 1),
             dict(base=(16, 0, 0, 0)), dict(base=(16, 24, 0, 0)), dict(row_bytes=(32, 8, 0, 0)),
             dict(row_bytes=(32, 0, 0, 0)), dict(layer_bytes=(4 * 64 * 32, 4 * 64 * 16 - 16, 0, 0))]


def test_pages_arguments():
    lib = b.load()
    assert lib.lrkv_pages_reserve(4, 16, 16, 1, 16, 16, 0, None, None) == 0
    for bad in ((0, 16, 16, 1, 16, 16, 1), (4, None, 16, 1, 16, 16, 1), (4, 20, 16, 1, 16, 16, 1),
                (4, 16, None, 1, 16, 16, 1), (4, 16, 16, 0, 16, 16, 1), (4, 16, 16, 1 << 25, 16, 16, 1),
                (4, 16, 16, 1, None, 16, 1), (4, 16, 16, 1, 16, None, 1), (4, 16, 16, 1, 16, 16, -1),
                (4, 16, 16, 1, 16, 16, 8193)):
        assert lib.lrkv_pages_reserve(*bad, None, None) == 1, bad
    p = pools()
    assert lib.lrkv_pages_fork(R(p), 16, 16, 1, 16, 1, 16, 16, 0, None, None) == 0
    for bad in ((None, 16, 1, 16, 1, 16, 16, 1), (16, None, 1, 16, 1, 16, 16, 1), (16, 16, 0, 16, 1, 16, 16, 1),
                (16, 16, 1, None, 1, 16, 16, 1), (16, 16, 1, 16, 0, 16, 16, 1), (16, 16, 1, 16, 1, None, 16, 1),
                (16, 16, 1, 16, 1, 16, None, 1), (16, 16, 1, 16, 1, 16, 16, -1), (16, 16, 1, 16, 1, 16, 16, 8193)):
        assert lib.lrkv_pages_fork(R(p), *bad, None, None) == 1, bad
    assert lib.lrkv_pages_free(4, 16, 16, 1, 16, 1, 16, 0, None, None, None) == 0
    for bad in ((4, None, 16, 1, 16, 1, 16, 1), (4, 16, 16, 1, 16, 1, None, 1), (4, 16, 16, 1, 16, 0, 16, 1),
                (4, 16, 16, 1, 16, 1, 16, -1), (4, 16, None, 1, 16, 1, 16, 1)):
        assert lib.lrkv_pages_free(*bad, None, None, None) == 1, bad
    assert lib.lrkv_pages_copy(R(p), 16, R(p), 16, 0, None, None) == 0
    assert lib.lrkv_pages_copy(R(p), None, R(p), 16, 1, None, None) == 1
    assert lib.lrkv_pages_copy(R(p), 16, R(p), 16, -1, None, None) == 1
    for other in (pools(num_pools=1), pools(num_layers=1), pools(row_bytes=(16, 16, 0, 0))):
        assert lib.lrkv_pages_copy(R(p), 16, R(other), 16, 1, None, None) == 1 and b"differ" in lib.lrkv_last_error()
    assert lib.lrkv_cache_compact(R(p), 16, 1, 16, 0, 16, 16, 4, None, None, None) == 0
    for bad in ((16, 1, 16, 1, None, 16, 4), (16, 1, 16, 1, 16, None, 4), (16, 1, 16, 1, 16, 16, 0),
                (16, 1, 16, 1, 16, 16, 1025), (None, 1, 16, 1, 16, 16, 4), (16, 1, 16, -1, 16, 16, 4)):
        assert lib.lrkv_cache_compact(R(p), *bad, None, None, None) == 1, bad
    for kw in BAD_POOLS:
        bad = pools(**kw)
        assert lib.lrkv_pages_fork(R(bad), 16, 16, 1, 16, 1, 16, 16, 1, None, None) == 1, kw
        assert lib.lrkv_pages_copy(R(bad), 16, R(p), 16, 1, None, None) == 1, kw
        assert lib.lrkv_pages_copy(R(p), 16, R(bad), 16, 1, None, None) == 1, kw
        assert lib.lrkv_cache_compact(R(bad), 16, 1, 16, 1, 16, 16, 4, None, None, None) == 1, kw


def test_binding_checks():
    torch = pytest.importorskip("torch")
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)
    bf = torch.bfloat16
    with pytest.raises(ValueError):  # a transposed pool
        b.Pools.of(z(64, 4, 8, t=bf).transpose(0, 1))
    with pytest.raises(ValueError):  # pages of another size
        b.Pools.of(z(4, 32, 8, t=bf))
    with pytest.raises(ValueError):
        b.Pools([z(1, 4, 64, 8, t=bf), z(1, 5, 64, 8, t=bf)])
    p = b.Pools.of(b.LayeredCache(*(z(3, 4, 64, 8, t=bf) for _ in range(4))))
    assert (p.c.num_pools, p.c.num_layers, p.c.num_blocks) == (4, 3, 4) and p.c.row_bytes[2] == 16
    assert p.c.layer_bytes[1] == 4 * 64 * 16
    assert b.Pools.of(b.PagedCache(*(z(4, 64, 8, t=bf) for _ in range(4)))).c.num_layers == 1
    assert b.Pools.of(b.QuantCache(z(4, 64, 48, t=torch.uint8))).c.row_bytes[0] == 48
    with pytest.raises(ValueError):
        b.lrkv_pages_reserve(z(4, t=torch.int64), z(2, 3), z(2), z(2), stream=0)
    with pytest.raises(ValueError):
        b.lrkv_pages_reserve(z(4), z(3, 2).t(), z(2), z(2), stream=0)
    with pytest.raises(ValueError):
        b.lrkv_pages_reserve(z(4), z(2, 3), z(3), z(3), stream=0)
    with pytest.raises(ValueError):
        b.lrkv_pages_fork(p, z(5), z(2, 3), z(2), z(1), z(1), stream=0)
    plan = b.rope_plan(8)
    x = z(4, 2, 8, t=bf)
    for bad in (dict(x=x.float()), dict(y=z(4, 3, 8, t=bf)), dict(x=x[..., 0]), dict(x=z(4, 2, 16, t=bf)[..., ::2]),
                dict(x_rows=z(3)), dict(x=x.half(), y=x.half())):
        a = dict(dict(x=x, y=x, x_rows=None), **bad)
        with pytest.raises(ValueError):
            b.lrkv_rope(plan, a["x"], a["y"], z(4), x_rows=a["x_rows"], stream=0)
    cache = b.PagedCache(*(z(4, 64, 8, t=bf) for _ in range(4)))
    with pytest.raises(ValueError, match="64-bit"):
        b.lrkv_decode_tree(GOOD, z(1, 2, 8, 64, t=bf), x, x, cache, z(1, 1), z(1), z(1, 2), z(1), x, x, stream=0)
    with pytest.raises(KeyError):
        b.rope_plan(64, layout="other")
