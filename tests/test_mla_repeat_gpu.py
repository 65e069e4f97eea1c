"""The MLA decode again and again on the same inputs: the same bits and no status, whatever the caches hold and whatever the
workspace held before (a part that a call does not write would show as NaN)."""
import pytest
import torch

from gpu_util import REL_L2_TOL
from test_mla_gpu import DC, DK

pytestmark = pytest.mark.gpu

from compressed_kv_cache_lrkv_gb300 import binding as b  # noqa: E402


def attend(q, kv, table, lens, scale):
    """softmax(q . row scale) over each sequence's rows, summed over the rows' latent part, in 64 bits."""
    out = torch.zeros(*q.shape[:2], DC, dtype=torch.float64, device="cuda")
    for s, n in enumerate(lens):
        rows = kv[table[s, :-(-n // 64)].long()].flatten(0, 1)[:n].double()
        out[s] = torch.softmax(q[s].double() @ rows.T * scale, 1) @ rows[:, :DC]
    return out


def repeated(H, lens, runs, flush):
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
    first, same = None, torch.ones((), dtype=torch.bool, device="cuda")
    for i in range(runs):
        ws.fill_(255)  # NaNs
        if flush:
            other.fill_(i)
        b.lrkv_mla_decode(dims, q, kv, table, sl, out, ws, status=st)
        if first is None:
            first = out.clone()
        same &= (out.view(torch.int16) == first.view(torch.int16)).all()
    assert int(st) == 0 and bool(same)
    want = attend(q, kv, table, lens, 192 ** -0.5)
    assert float((first.double() - want).norm() / want.norm()) <= REL_L2_TOL


@pytest.mark.parametrize("H,lens", [(32, [300] * 90), (128, [300] * 200), (128, [100, 64, 1, 130] * 100),
                                    (16, [1000] * 100)])
def test_more_sequences_than_pairs(H, lens):
    """A pair's CTAs may be a tile apart where one still stores a sequence's sums: the logits that one of them sends are
    those of the tile, not the probabilities written over them."""
    repeated(H, lens, 100, flush=False)


@pytest.mark.parametrize("H,lens", [(128, [4096] * 152), (128, [700] * 76), (16, [300] * 90), (128, [16384, 9000]), (1, [64 * 3] * 200)])
def test_every_wait_ends(H, lens):
    """Caches without the kernel's code: one warp may be tiles behind another."""
    repeated(H, lens, 200, flush=True)
