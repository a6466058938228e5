"""Latent attention at the sizes that choose its kernels and paths, against the fp64 oracle."""
import pytest
import torch

import gated_delta_rule_rda_b200 as rda
from latent_util import check, check_lse, cu, packed
from oracle import latent
from test_parity_latent import BF16, F32, dev, forward, gradients, oracle_forward, oracle_gradients

pytestmark = pytest.mark.gpu
NAMES = ("dq", "dk", "dv", "dq_shared", "dk_shared")


def test_gradients_whose_delta_is_formed_again(cuda_device):
    """81 to 160 keys in reach of a query tile: two steps of keys, and a pass ahead over both.  Many such tiles at
    once and many times over: no wait runs out, and the bits are the same."""
    lens = [81, 96, 128, 159, 160, 161, 400]
    x = packed(lens, lens, 24, 128, 64, 128, BF16, seed=101)
    d = dev(x)
    out, lse = forward(d)
    ws = rda.new_workspace(rda.rda_latent_backward_workspace_bytes(sum(lens), sum(lens), 24, 128, 64, 128, len(lens)), "cuda")
    g, rg = gradients(d, out, lse, workspace=ws), oracle_gradients(x, True)
    for n in NAMES:
        check(g[n], rg[n], rg[n + "_round"], BF16, 192, x["scale"], 3 * 800, n)
    for _ in range(40):
        g2 = gradients(d, out, lse, workspace=ws)
        assert all(torch.equal(g[n], g2[n]) for n in NAMES)
    assert rda.rda_read_device_error(ws) == 0
