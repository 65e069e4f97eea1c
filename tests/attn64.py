"""Attention over s/z parts in 64 bits (torch, expanded per-head keys and values), with a bound on
what the kernels' roundings may add."""
import torch


def attend64(q, BK, BV, parts, d_rope=0, eps_p=2.0 ** -8, eps_qt=2.0 ** -8):
    """One sequence: q [H, d_h + d_rope], parts = (sK [n, d_k], sV [n, d_h], zK [n, H, r], zV) as
    float64 -> (out [H, d_h], bound [H, d_h]).

    The bound, from half a step of each rounding (eps = finfo.eps / 2 of the type):
      - the output's own: 2^-8 |out| (bf16);
      - each probability's, to the type of its product: eps_p of sum_t p_t |V_t| (the same
        products with magnitudes, the up-projection included);
      - q~'s, to the type of its product: a logit moves by at most d = scale * eps_qt * sum_j
        |q~_j z_j|, all logits' sums in fp32 by (d_k + r) 2^-24 sum |q k| more, so a normalised
        probability by a factor within e^(+-2 d_max);
      - sums over n tokens and r latents in fp32: (n + r) 2^-24 of the same magnitudes, and
        2^-20 for the approximate exponential (2 ulp) and the merges' factors.
    """
    H, r = BK.shape[0], BK.shape[2]
    d_h = BK.shape[1]
    sK, sV, zK, zV = parts
    n = sK.shape[0]
    scale = (d_h + d_rope) ** -0.5
    qt = torch.einsum("hd,hdr->hr", q[:, :d_h], BK)
    K = sK[:, None, :d_h] + torch.einsum("thr,hdr->thd", zK, BK)
    V = sV[:, None] + torch.einsum("thr,hdr->thd", zV, BV)
    t = torch.einsum("hd,thd->ht", q[:, :d_h], K)
    if d_rope:
        t = t + q[:, d_h:] @ sK[:, d_h:].t()
    p = torch.softmax(t * scale, 1)
    out = torch.einsum("ht,thd->hd", p, V)
    mag_z = torch.einsum("hr,thr->ht", qt.abs(), zK.abs())
    mag_s = q.abs() @ sK.abs().t()
    d = scale * (eps_qt * mag_z + (sK.shape[1] + r) * 2.0 ** -24 * (mag_s + mag_z))
    # q~ itself is summed in fp32 over d_h products
    qt_mag = torch.einsum("hd,hdr->hr", q[:, :d_h].abs(), BK.abs())
    d = d + scale * d_h * 2.0 ** -24 * torch.einsum("hr,thr->ht", qt_mag, zK.abs())
    dmax = d.amax(1, keepdim=True)
    absV = sV.abs()[:, None] + torch.einsum("thr,hdr->thd", zV.abs(), BV.abs())
    A = torch.einsum("ht,thd->hd", p, absV)
    rel = eps_p + torch.expm1(2 * dmax) + (n + r) * 2.0 ** -24 + 2.0 ** -20
    return out, 2.0 ** -8 * out.abs() + rel * A


def check(got, want, bound, what="", rel_max=5e-3):
    """Elementwise |got - want| <= bound, and the decode's parity bar on the relative L2 error; prints
    the largest share of the bound used."""
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = ((got - want).abs() / bound.clamp(min=1e-30)).amax().item()
    rel = ((got - want).norm() / want.norm().clamp(min=1e-300)).item()
    print(f"{what}: {over:.3f} of the bound, rel_l2 {rel:.2e}")
    assert over <= 1.0 and rel <= rel_max, f"{what}: {over:.3f} of the bound, rel_l2 {rel:.2e}"
