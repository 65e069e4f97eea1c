"""The MLA decode again and again on the same inputs: no status, and every part of the result written, whatever the caches hold
(a part that a call does not write shows as NaN)."""
import pytest
import torch

from test_mla_gpu import DC, DK

pytestmark = pytest.mark.gpu

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402


def repeated(H, lens, runs):
    g = torch.Generator(device="cuda").manual_seed(H + len(lens))
    pages = [-(-n // 64) for n in lens]
    kv = torch.randn(sum(pages), 64, DK, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(len(lens), H, DK, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randperm(sum(pages), generator=g, device="cuda").int()
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device="cuda")
    for s, part in enumerate(ids.split(pages)):
        table[s, :pages[s]] = part
    dims = b.make_mla_dims(H, 5120)
    out = torch.empty(len(lens), H, DC, dtype=torch.bfloat16, device="cuda")
    ws = b.alloc_workspace(b.mla_decode_workspace_bytes(dims, len(lens)))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    other = torch.empty(48 << 20, device="cuda")  # larger than L2, the kernels' code with it
    written = torch.ones((), dtype=torch.bool, device="cuda")
    for i in range(runs):
        ws.fill_(255)  # NaNs
        other.fill_(i)
        b.lrkv_mla_decode(dims, q, kv, table, sl, out, ws, status=st)
        written &= torch.isfinite(out).all()
    assert int(st) == 0 and bool(written)


@pytest.mark.parametrize("H,lens", [(128, [4096] * 152), (128, [700] * 76), (16, [300] * 90), (128, [16384, 9000]), (1, [64 * 3] * 200)])
def test_every_wait_ends(H, lens):
    """Caches without the kernel's code: one warp may be tiles behind another."""
    repeated(H, lens, 200)
