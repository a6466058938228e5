"""Latent attention and draft verification near the largest sizes that their calls take: tensors of more than 2^31
elements, whose last rows have the bits (or the tokens) of a call on those rows alone."""
import pytest
import torch

import gated_delta_rule_rda_b200 as rda

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,grads", [(BF16, True), (F32, False)])
def test_packed_batch_whose_values_pass_32_bits(cuda_device, dtype, grads):
    """total H (Dk + Ds) just below 2^31 with Dv = 2 Dk: v and out have almost 2^32 elements."""
    H, Dk, Dv, T, N = 64, 64, 128, 1000, 523
    total = T * N
    assert (1 << 31) * 0.99 < total * H * Dk < 1 << 31 < total * H * Dv
    torch.manual_seed(7)
    n = lambda *s: torch.empty(*s, dtype=dtype, device="cuda").normal_()
    q, k, v = n(total, H, Dk), n(total, H, Dk), n(total, H, Dv)
    cu = torch.arange(0, total + 1, T, dtype=torch.int32, device="cuda")
    out, lse = rda.rda_latent_prefill(q, k, v, cu, scale=0.125, return_lse=True)
    last = slice(total - 2 * T, total)
    c2 = cu[:3].contiguous()
    # the same rules for sizes have to hold for the part: as many sequences as make the same choices
    part = [t[total - 40 * T:] for t in (q, k, v)]
    o2, l2 = rda.rda_latent_prefill(*part, cu[:41].contiguous(), scale=0.125, return_lse=True)
    assert torch.equal(o2[-2 * T:], out[last]) and torch.equal(l2[-2 * T:], lse[last])
    assert torch.isfinite(out[last].float()).all()
    if grads:
        d = n(total, H, Dv)
        g = rda.rda_latent_backward(q, k, v, out, lse, d, cu, scale=0.125)
        g2 = rda.rda_latent_backward(*(t[last] for t in (q, k, v, out, lse, d)), c2, scale=0.125)
        assert all(torch.equal(g2[m], g[m][last]) for m in ("dq", "dk", "dv"))


@pytest.mark.parametrize("V", [1 << 30, (1 << 30) - 1])
def test_largest_vocabulary(cuda_device, V):
    """Equal weights: the sums are whole numbers, and u V is exact."""
    p = torch.ones(1, 1, V, device="cuda")
    x = torch.zeros(1, 0, dtype=torch.int32, device="cuda")
    for u, want in ((0.0, 0), (0.75, int(0.75 * V)), (1 - 2.0 ** -24, int((1 - 2.0 ** -24) * V))):
        tok, kept = rda.rda_verify_drafts(x, p, torch.full((1, 1), u, device="cuda"))
        assert tok.tolist() == [[want]] and kept.tolist() == [0]


def test_probabilities_past_32_bits(cuda_device):
    B, T, V = 1100, 7, 259840
    assert B * (T + 1) * V > 1 << 31
    torch.manual_seed(8)
    p = torch.rand(B, T + 1, V, device="cuda")
    q = torch.rand(B, T, V, device="cuda")
    x = torch.randint(0, V, (B, T), dtype=torch.int32, device="cuda")
    u = torch.rand(B, T + 1, device="cuda")
    tok, kept = rda.rda_verify_drafts(x, p, u, q)
    s = slice(B - 64, B)
    tok2, kept2 = rda.rda_verify_drafts(x[s], p[s], u[s], q[s])
    assert torch.equal(tok[s], tok2) and torch.equal(kept[s], kept2) and (kept > 0).any()
    assert ((tok >= 0).sum(1) == kept + 1).all()
