"""Inputs and bounds for the tests of latent attention."""
import numpy as np
import torch

# half steps of the types
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def cu(lens, device="cpu"):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=device)


def packed(lens_q, lens_k, H, Dk, Ds, Dv, dtype, seed, pad=0, spread=1.5):
    """Packed inputs (CPU); `pad` rows of NaN behind the last sequence."""
    g = torch.Generator().manual_seed(seed)
    tq, tk = sum(lens_q), sum(lens_k)

    def n(rows, *shape):
        x = torch.randn(rows + pad, *shape, generator=g)
        if pad:
            x[rows:] = float("nan")
        return x.to(dtype)

    return dict(q=n(tq, H, Dk), k=n(tk, H, Dk), v=n(tk, H, Dv), q_shared=n(tq, H, Ds) if Ds else None,
                k_shared=n(tk, Ds) if Ds else None, d_out=n(tq, H, Dv), cu_q=cu(lens_q), cu_k=cu(lens_k),
                scale=spread * (Dk + Ds) ** -0.5)


def score_error(D, scale, size=4.5):
    """How far fp32 accumulation can move a score of D products of values up to about `size` in
    size: half a step each for D additions, on partial sums of at most sum |q k| (4.5 x 0.8 x D
    bounds the sum of |q k| for normal inputs; one factor at its mean size)."""
    return D * 2.0 ** -24 * abs(scale) * size * 0.8 * D


def check(got, ref, moved, dtype, D, scale, n_sum, what):
    """Elementwise: |got - ref| <= (half step of the type) x moved, plus what fp32 statistics and sums give."""
    got = got.detach().to("cpu", torch.float64)
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), what
    fp32 = 2 * score_error(D, scale) + (n_sum + 8) * 2.0 ** -24
    bound = moved * (HALF[dtype] * 1.02 + fp32) + 1e-30
    over = ((got - ref).abs() / bound).max().item() if got.numel() else 0.0
    assert over <= 1.0, f"{what}: {over:.3f} times the bound"
    if dtype == torch.float32 and got.numel() and ref.norm() > 0:
        rel = ((got - ref).norm() / ref.norm()).item()
        assert rel <= 1e-5, f"{what}: rel-L2 {rel:.2e}"


def check_lse(got, ref, D, scale, what="lse"):
    got = got.detach().to("cpu", torch.float64)
    empty = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), empty) and not torch.isnan(got).any(), what
    if (~empty).any():
        off = (got - ref)[~empty].abs().max().item()
        assert off <= score_error(D, scale) + 4e-6 * (1 + ref[~empty].abs().max().item()), (what, off)


def paged(lens, T, H, Dl, Ds, page, dtype, seed, spare=3, garbage=True, scale=192 ** -0.5):
    """A paged cache holding the sequences in shuffled pages; everything that belongs to no token is
    NaN if `garbage`; table entries past a sequence's pages are out of range."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = [-(-n // page) for n in lens]
    P, W = sum(per) + spare, max(max(per), 1)
    pages = torch.full((P, page, Dl + Ds), float("nan") if garbage else 1.0)
    ids = torch.randperm(P, generator=g).tolist()
    table = torch.full((B, W), 1 << 30, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        for i in range(per[b]):
            table[b, i] = ids[at]
            m = min(page, n - i * page)
            pages[ids[at], :m] = torch.randn(m, Dl + Ds, generator=g)
            at += 1
    return dict(q=torch.randn(B, T, H, Dl, generator=g).to(dtype),
                q_shared=torch.randn(B, T, H, Ds, generator=g).to(dtype) if Ds else None,
                pages=pages.to(dtype), table=table, lens=torch.tensor(lens, dtype=torch.int32), scale=scale)
