"""Quantised cache and shared prefix: arguments that are refused on the host (no GPU needed)."""
import ctypes

import pytest

from compressed_kv_cache_lrkv_gb300 import binding as b

GOOD = b.make_dims(8, 64, 16, 512)
CACHE = b.Cache(16, 16, 16, 16, 4)
ROWS = b.QuantCacheStruct(16, 4)
R = ctypes.byref


def test_row_bytes():
    """Four parts, z padded to 16 bytes, a scale byte per 32 values, an odd number of 16-byte units."""
    for H, d_h, r, rope in [(1, 64, 8, 0), (3, 64, 8, 64), (8, 64, 16, 0), (5, 128, 32, 0), (32, 128, 32, 0),
                            (128, 128, 16, 64)]:
        dims = b.make_dims(H, d_h, r, H * d_h, d_rope=rope)
        z, blocks = (H * r + 15) // 16 * 16, (d_h + rope) // 32 + d_h // 32 + 2 * ((H * r + 31) // 32)
        need = 2 * d_h + rope + 2 * z + blocks
        rb = b.quant_row_bytes(dims)
        assert need <= rb < need + 32 and rb % 32 == 16
        assert b.quant_block_bytes(dims) == 64 * rb
    assert b.quant_row_bytes(b.make_dims(8, 96, 8, 512)) == 0
    assert b.decode_quant_workspace_bytes(b.make_dims(8, 96, 8, 512), 1) == 0
    assert b.decode_shared_workspace_bytes(b.make_dims(8, 96, 8, 512), 1, 1) == 0


@pytest.mark.parametrize("write", [True, False])
def test_store_arguments(write):
    lib = b.load()

    def call(dims=GOOD, n=1, cache=CACHE, bf=16, rows=ROWS, qs=16):
        c, r = (R(cache) if cache else None), (R(rows) if rows else None)
        if write:
            return lib.lrkv_cache_quantize(R(dims), n, c, bf, r, qs, None, None)
        return lib.lrkv_cache_dequantize(R(dims), n, r, qs, c, bf, None, None)

    assert call(n=0) == 0 and call(n=0, bf=None, qs=None) == 0
    assert call(dims=b.make_dims(8, 64, 12, 512)) == 2
    assert call(n=-1) == 1 and b"n_tok" in lib.lrkv_last_error()
    assert call(cache=None) == 1 and call(rows=None) == 1
    assert call(cache=b.Cache(16, 16, 0, 16, 4)) == 1 and call(cache=b.Cache(16, 24, 16, 16, 4)) == 1
    assert call(rows=b.QuantCacheStruct(0, 4)) == 1
    assert call(rows=b.QuantCacheStruct(24, 4)) == 1 and b"aligned" in lib.lrkv_last_error()
    assert call(rows=b.QuantCacheStruct(16, 0)) == 1 and call(rows=b.QuantCacheStruct(16, (1 << 24) + 1)) == 1
    assert call(bf=None) == 1 and call(qs=None) == 1 and b"slots" in lib.lrkv_last_error()


def test_decode_quant_arguments():
    lib = b.load()
    base = dict(dims=GOOD, q=16, BK=16, BV=16, rows=ROWS, bt=16, mb=1, sl=16, B=1, out=16)

    def call(partials=False, **kw):
        a = dict(base, **kw)
        r = R(a["rows"]) if a["rows"] else None
        if partials:
            return lib.lrkv_decode_quant_partials(R(a["dims"]), a["q"], a["BK"], r, a["bt"], a["mb"], a["sl"], a["B"],
                                                  a["out"], 256, 1 << 40, None, None)
        return lib.lrkv_decode_quant(R(a["dims"]), a["q"], a["BK"], a["BV"], r, a["bt"], a["mb"], a["sl"], a["B"],
                                     a["out"], 256, 1 << 40, None, None)

    for p in (False, True):
        assert call(p, B=0) == 0
        assert call(p, B=-1) == 1 and call(p, B=65536) == 1
        assert call(p, dims=b.make_dims(8, 64, 16, 512, softmax_scale=float("nan"))) == 1
        assert call(p, dims=b.make_dims(129, 64, 16, 512)) == 2
        assert call(p, rows=None) == 1 and call(p, rows=b.QuantCacheStruct(8, 4)) == 1
        assert call(p, mb=0) == 1 and call(p, mb=1 << 25) == 1
        assert call(p, mb=1 << 24, B=60000) == 1 and b"2^34" in lib.lrkv_last_error()
        for k in ("q", "BK", "out"):
            assert call(p, **{k: None}) == 1 and call(p, **{k: 24}) == 1, k
        assert call(p, bt=None) == 1 and call(p, sl=None) == 1
    assert call(BV=None) == 1 and call(BV=40) == 1


def test_shared_arguments():
    lib = b.load()
    base = dict(dims=GOOD, q=16, BK=16, BV=16, cache=CACHE, pb=16, mp=1, pl=16, bt=16, mb=1, sl=16, B=1, out=16)

    def call(partials=False, **kw):
        a = dict(base, **kw)
        c = R(a["cache"]) if a["cache"] else None
        if partials:
            return lib.lrkv_prefix_partials(R(a["dims"]), a["q"], a["BK"], c, a["pb"], a["mp"], a["pl"], a["B"],
                                            a["out"], 256, 1 << 40, None, None)
        return lib.lrkv_decode_shared(R(a["dims"]), a["q"], a["BK"], a["BV"], c, a["pb"], a["mp"], a["pl"], a["bt"],
                                      a["mb"], a["sl"], a["B"], a["out"], 256, 1 << 40, None, None)

    for p in (False, True):
        assert call(p, B=0) == 0
        assert call(p, B=-1) == 1 and call(p, B=65536) == 1
        assert call(p, dims=b.make_dims(8, 64, 16, 512, d_rope=32)) == 2
        assert call(p, cache=None) == 1 and call(p, cache=b.Cache(16, 16, 16, 0, 4)) == 1
        assert call(p, mp=0) == 1 and call(p, mp=1 << 25) == 1 and b"max_prefix_blocks" in lib.lrkv_last_error()
        assert call(p, pb=None) == 1 and call(p, pl=None) == 1 and b"prefix_len" in lib.lrkv_last_error()
        for k in ("q", "BK", "out"):
            assert call(p, **{k: None}) == 1 and call(p, **{k: 24}) == 1, k
    assert call(BV=None) == 1 and call(bt=None) == 1 and call(sl=None) == 1 and call(mb=0) == 1


def test_binding_checks_row_width_and_slot_counts():
    torch = pytest.importorskip("torch")
    rows = torch.zeros(2, 64, b.quant_row_bytes(GOOD) + 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        b.QuantCache(rows).struct(GOOD)
    with pytest.raises(ValueError):
        b._same_length(torch.zeros(3), torch.zeros(4))


def test_refused_dims_leave_nothing_behind():
    """Dims that the library refuses are reported as its refusal, and good dims of the same heads and widths are taken
    afterwards."""
    torch = pytest.importorskip("torch")
    good = b.make_dims(24, 64, 16, 1536)
    rows = torch.zeros(2, 64, b.quant_row_bytes(good), dtype=torch.uint8)
    x = torch.zeros(64, dtype=torch.uint8)
    i = torch.zeros(1, 1, dtype=torch.int32)
    for bad, status in ((b.make_dims(24, 64, 16, 12), 2), (b.make_dims(24, 64, 16, 1536, softmax_scale=float("nan")), 1),
                        (b.make_dims(24, 64, 16, 1536, num_splits=-1), 1)):
        with pytest.raises(b.LrkvError) as e:
            b.lrkv_decode_quant(bad, x, x, x, b.QuantCache(rows), i, i[0], x, x, stream=0)
        assert e.value.status == status
    assert b.QuantCache(rows).struct(good).num_blocks == 2


def test_binding_refuses_rows_that_are_not_whole_bytes_in_order():
    """Rows are addressed as [num_blocks, 64, row bytes] from the first one on: views of the right size that lie
    otherwise, and other types, are refused; a slice of whole pages is not."""
    torch = pytest.importorskip("torch")
    rb = b.quant_row_bytes(GOOD)
    rows = torch.zeros(4, 64, 2 * rb, dtype=torch.uint8)
    for bad in (rows[:, :, :rb], torch.zeros(8, 64, rb, dtype=torch.uint8)[::2],
                torch.zeros(64, 2, rb, dtype=torch.uint8).transpose(0, 1),
                torch.zeros(2, 64, rb // 2, dtype=torch.bfloat16), torch.zeros(2, 64, rb, dtype=torch.int8)):
        with pytest.raises(ValueError, match="contiguous uint8"):
            b.QuantCache(bad).struct(GOOD)
    whole = torch.zeros(8, 64, rb, dtype=torch.uint8)
    assert b.QuantCache(whole[2:5]).struct(GOOD).num_blocks == 3
    assert b.QuantCache(whole[2:5].view(3, -1)).struct(GOOD).num_blocks == 3
