"""The draw of rda_verify_drafts where the drawn token lies far from the row's start, against the fp64 oracle."""
import pytest
import torch

import gated_delta_rule_rda_b200 as rda
from oracle import latent

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [5000, 140000])      # one kernel, two kernels
def test_tokens_drawn_from_every_slice(cuda_device, V):
    """Uniforms spread over a flat row: each sequence draws from another slice, whose start one thread finds and all
    of its CTA use.  Many times over, with the same result."""
    B = 160
    g = torch.Generator().manual_seed(V)
    p = torch.rand(B, 1, V, generator=g)
    u = (torch.arange(B)[:, None] + 0.5) / B
    x = torch.zeros(B, 0, dtype=torch.int32)
    ref, _ = latent.verify(x, p, u, None)
    assert len({t[0] // 1024 for t in ref}) >= 0.9 * (V + 1023) // 1024
    c = [t.cuda() for t in (x, p, u)]
    for _ in range(20):
        tok, kept = rda.rda_verify_drafts(*c)
        assert tok.cpu().tolist() == ref and not kept.any()
