"""lrkv_rope against the rotation in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def speeds(d_rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0, **_):
    """Radians a position, in long double (more than 64 bits of the angle matter at far positions)."""
    i = np.arange(d_rot // 2, dtype=np.longdouble)
    f = np.longdouble(base) ** (-2 * i / np.longdouble(d_rot))
    if scaling == "linear":
        return f / np.longdouble(factor)
    if scaling == "parts":
        tau = 8 * np.arctan(np.longdouble(1))
        g = np.clip((np.longdouble(original_len) * f / tau - low) / (np.longdouble(high) - low), 0, 1)
        return g * f + (1 - g) * f / np.longdouble(factor)
    return f


def want64(x, pos, d_rot, begin, half, transpose, m, **kw):
    """x [n, heads, width] (64 bits), pos [n] -> rotated rows, and the magnitudes |m| (|x0| + |x1|) of each value's pair."""
    tau = 8 * np.arctan(np.longdouble(1))
    turns = pos.numpy().astype(np.longdouble)[:, None] * (speeds(d_rot, **kw) / tau)
    ang = ((turns - np.floor(turns)) * tau).astype(np.float64)
    ang = torch.from_numpy(-ang if transpose else ang)[:, None]
    c, s = torch.cos(ang) * m, torch.sin(ang) * m
    k = d_rot // 2
    i = torch.arange(k)
    p0, p1 = (begin + i, begin + k + i) if half else (begin + 2 * i, begin + 2 * i + 1)
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., p0] = x[..., p0] * c - x[..., p1] * s
    y[..., p1] = x[..., p0] * s + x[..., p1] * c
    mag[..., p0] = mag[..., p1] = abs(m) * (x[..., p0].abs() + x[..., p1].abs())
    return y, mag


def check(got, want, mag, dtype, what):
    """Half a step of the result's rounding (2^-8 of it in bf16, 2^-24 in fp32) and 9 x 2^-24 of the pair's magnitude: the
    angle in fp32 (rounded, times a rounded constant: 3 x 2^-24 x pi / 4), the polynomials (2 roundings, 4e-9 left out),
    the magnitude (2 roundings) and the products and their sum (2)."""
    bound = (2.0 ** -8 if dtype is BF else 2.0 ** -24) * want.abs() + 9 * 2.0 ** -24 * mag
    err = (got.double().cpu() - want).abs()
    assert torch.isfinite(got).all(), what
    over = (err / bound.clamp(min=1e-300)).where(err > 0, torch.zeros_like(err)).max().item()
    print(f"{what}: {over:.3f} of the bound")
    assert over <= 1.0, what


def positions(g, n, far):
    if far:
        p = torch.randint(-2 ** 31, 2 ** 31, (n,), generator=g)
        p[:4] = torch.tensor([0, -1, 2 ** 31 - 1, -2 ** 31])[:n]
        return p.to(torch.int32)
    return torch.randint(0, 1 << 17, (n,), generator=g).to(torch.int32)


CASES = [
    (1, 1, 64, 0, 64, False, BF, {}), (1, 1, 8, 0, 8, True, BF, {}), (3, 5, 24, 8, 8, False, F32, {}),
    (3, 5, 24, 8, 8, True, F32, {}), (16, 32, 192, 128, 64, False, BF, {}), (7, 128, 128, 0, 128, True, BF, {}),
    (130, 3, 72, 0, 24, True, BF, dict(scaling="linear", factor=4.0)),
    (130, 3, 72, 24, 40, False, F32, dict(scaling="parts", factor=8.0, original_len=8192.0, magnitude=1.2079441541679836)),
    (65, 1, 256, 0, 256, True, F32, dict(base=500000.0)), (1000, 12, 128, 64, 64, True, BF, dict(base=1e6)),
    (5000, 9, 192, 128, 64, False, BF, dict(scaling="parts", factor=2.0, original_len=4096.0, low=2.0, high=8.0)),
    (2, 300, 1024, 512, 96, True, BF, {}), (20000, 1, 64, 0, 64, False, BF, dict(magnitude=-0.5)),
]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("n,heads,width,begin,d_rot,half,dtype,kw", CASES)
def test_matches_64_bits(n, heads, width, begin, d_rot, half, dtype, kw, transpose):
    g = torch.Generator().manual_seed(n * heads + d_rot)
    x = torch.randn(n, heads, width, generator=g).to(dtype)
    pos = positions(g, n, far=n % 2 == 1)
    plan = b.rope_plan(d_rot, layout="half" if half else "interleaved", **kw)
    y = torch.full_like(x, float("nan")).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.lrkv_rope(plan, x.cuda(), y, pos.cuda(), begin=begin, transpose=transpose, status=st)
    assert int(st.item()) == 0
    m = float(np.float32(kw.get("magnitude", 1.0)))
    args = {k: v for k, v in kw.items() if k != "magnitude"}
    want, mag = want64(x.double(), pos, d_rot, begin, half, transpose, m, **args)
    check(y, want, mag, dtype, f"n {n}, {heads} heads of {width}")
    keep = [*range(begin), *range(begin + d_rot, width)]
    assert torch.equal(y.cpu()[..., keep], x[..., keep])
    # in place: the same values, the rest not touched
    z = x.cuda()
    b.lrkv_rope(plan, z, z, pos.cuda(), begin=begin, transpose=transpose)
    assert torch.equal(z, y)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_and_row_indices(dtype):
    """A slice of wider rows to [heads][rows] order, rows picked on both sides; untouched rows and columns stay."""
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(40, 6, 96, generator=g).to(dtype).cuda()
    x = wide[:, 1:4, 16:80]
    store = torch.full((3, 30, 72), 7.0, dtype=dtype, device="cuda")
    y = store.transpose(0, 1)[..., 8:]
    xr = torch.tensor([39, 0, 5, 5, -1, 7, 40, 3], dtype=torch.int32)
    yr = torch.tensor([2, 29, 0, 4, 6, -5, 8, 30], dtype=torch.int32)
    pos = torch.tensor([1, 2, 3, 4, 5, 6, 7, 100000], dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = b.rope_plan(16, layout="half")
    b.lrkv_rope(plan, x, y, pos.cuda(), begin=8, x_rows=xr.cuda(), y_rows=yr.cuda(), status=st)
    assert int(st.item()) == b.DEV_BAD_SLOT
    done = [0, 1, 2, 3]
    want, mag = want64(x.cpu().double()[xr[done].long()], pos[done], 16, 8, True, False, 1.0)
    check(y[yr[done].long()], want, mag, dtype, "picked rows")
    rest = [r for r in range(30) if r not in (2, 29, 0, 4)]
    assert (store[:, rest] == 7).all() and (store[..., :8] == 7).all()


def test_broadcast_input():
    """One row and one head read for all (strides 0)."""
    x = torch.randn(1, 1, 64).cuda()
    y = torch.empty(9, 4, 64, device="cuda")
    pos = torch.arange(9, dtype=torch.int32)
    b.lrkv_rope(b.rope_plan(64), x.expand(9, 4, 64), y, pos.cuda())
    want, mag = want64(x.cpu().double().expand(9, 4, 64), pos, 64, 0, False, False, 1.0)
    check(y, want, mag, F32, "broadcast")


def test_gradient():
    """<R x, u> = <x, R^T u>, differences of the forward (linear: exact up to rounding), and R^T R = m^2."""
    g = torch.Generator().manual_seed(9)
    n, heads, w = 50, 3, 128
    x, u = (torch.randn(n, heads, w, generator=g).cuda() for _ in range(2))
    pos = positions(g, n, True).cuda()
    plan = b.rope_plan(w, layout="half", scaling="linear", factor=3.0, magnitude=1.5)
    f = lambda a, tr=False: (lambda o: (b.lrkv_rope(plan, a, o, pos, transpose=tr), o)[1])(torch.empty_like(a))
    gx = f(u, True).double()
    # a value is off by at most (2^-24 + 9 x 2^-24) x 1.5 (|x0| + |x1|); |x0| + |x1| <= sqrt(2) |pair| there and in
    # the product with u's pair; two sides
    tol = 10 * 2.0 ** -24 * 1.5 * 2 * 2 * float(x.double().norm() * u.double().norm())
    assert abs(float((f(x).double() * u.double()).sum() - (x.double() * gx).sum())) <= tol
    h, k = 2.0 ** -6, (7, 1, 70)
    xp, xm = x.clone(), x.clone()
    xp[k] += h
    xm[k] -= h
    step = (xp[k] - xm[k]).double()
    diff = float(((f(xp).double() - f(xm).double()) * u.double()).sum() / step)
    # two values change, each rounded to 10 x 2^-24 of 1.5 x 2 x the largest magnitude, divided by 2 h
    bound = 4 * 10 * 2.0 ** -24 * 1.5 * 2 * float(x.abs().max() * u.abs().max()) / (2 * h)
    assert abs(diff - float(gx[k])) <= bound + 1e-6 * abs(diff)
    back = f(f(x), True).double() / 2.25
    assert (back - x.double()).abs().max() <= 4 * 10 * 2.0 ** -24 * 2 * float(x.abs().max())


def test_same_rotation_as_the_append():
    """Rows appended at position 0 and turned by lrkv_rope equal rows appended at their positions, up to the rounding
    of the row in between (half a step each)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    H, d_h, r, d, n = 2, 64, 8, 128, 40
    dims = b.make_dims(H, d_h, r, d, d_rope=64)
    N = 2 * (d_h + H * r) + 64
    X = torch.randn(n, d, generator=g, device="cuda").to(BF)
    W = (torch.randn(N, d, generator=g, device="cuda") * d ** -0.5).to(BF)
    slots = torch.arange(n, dtype=torch.int32, device="cuda") + 9
    pos = torch.randint(0, 100000, (n,), generator=g, device="cuda").to(torch.int32)
    caches = [b.PagedCache.empty(1, H, d_h, r, d_rope=64) for _ in range(2)]
    for c, p in zip(caches, (pos, torch.zeros_like(pos))):
        c.sK.zero_()
        b.lrkv_append(dims, X, W, slots, c, positions=p)
    keys = caches[1].sK.view(-1, 1, d_h + 64)
    before = keys.clone()
    b.lrkv_rope(b.rope_plan(64), keys, keys, pos, begin=d_h, x_rows=slots, y_rows=slots)
    at = slots.long()
    a, c = caches[0].sK.view(-1, d_h + 64)[at].double(), keys[at, 0].double()
    pair = before[at, 0, d_h:].double().view(n, 32, 2).abs().sum(2).repeat_interleave(2, 1)
    # the unrotated pair is off by 2^-8 of each value, both results by 2^-8 of themselves, fp32 parts below 2^-18
    bound = 2.0 ** -8 * (pair + a[:, d_h:].abs() + c[:, d_h:].abs()) + 2.0 ** -18 * pair
    assert ((a - c)[:, d_h:].abs() <= bound).all() and torch.equal(a[:, :d_h], c[:, :d_h])
    other = torch.ones(64, dtype=torch.bool)
    other[at.cpu()] = False
    assert (keys.view(64, -1)[other.cuda()] == 0).all()


def test_rows_beyond_32_bit_offsets():
    """A row whose values lie more than 2^31 elements and 2^32 bytes into its tensor."""
    n = (1 << 31) // 64 + 100
    x = torch.zeros(n, 1, 64, dtype=BF, device="cuda")
    rows = torch.tensor([n - 1, 3], dtype=torch.int32, device="cuda")
    vals = torch.randn(2, 1, 64).to(BF)
    x[rows.long()] = vals.cuda()
    pos = torch.tensor([12345, -7], dtype=torch.int32)
    b.lrkv_rope(b.rope_plan(64), x, x, pos.cuda(), x_rows=rows, y_rows=rows)
    want, mag = want64(vals.double(), pos, 64, 0, False, False, 1.0)
    check(x[rows.long()], want, mag, BF, "far rows")


def test_stream_and_graph():
    x = torch.randn(33, 4, 64).cuda()
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    plan = b.rope_plan(64, layout="half")
    y, z = torch.empty_like(x), torch.zeros_like(x)
    b.lrkv_rope(plan, x, y, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.lrkv_rope(plan, x, z, pos)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, z)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        b.lrkv_rope(plan, x, z, pos)
    x.normal_()
    pos += 1000
    gr.replay()
    b.lrkv_rope(plan, x, y, pos)
    torch.cuda.synchronize()
    assert torch.equal(y, z)


def test_non_finite_values_stay_in_their_pair():
    x = torch.randn(2, 2, 64).to(BF).cuda()
    x[0, 1, 6] = float("inf")
    x[1, 0, 40] = float("nan")
    y = torch.empty_like(x)
    b.lrkv_rope(b.rope_plan(64), x, y, torch.tensor([5, 9], dtype=torch.int32, device="cuda"))
    bad = ~torch.isfinite(y)
    assert bad.sum() <= 4 and bad[0, 1, 6:8].all() and bad[1, 0, 40:42].all()
