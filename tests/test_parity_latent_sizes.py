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


def compare(x, causal, what=NAMES):
    """Forward and gradients of packed inputs against the oracle; returns them."""
    lq, lk = x["cu_q"].diff(), x["cu_k"].diff()
    D, dtype = x["q"].shape[2] + (x["q_shared"].shape[2] if x["q_shared"] is not None else 0), x["q"].dtype
    d = dev(x)
    ws = rda.new_workspace(1 << 28, "cuda")
    out, lse = forward(d, causal=causal, workspace=ws)
    r, rg = oracle_forward(x, causal), oracle_gradients(x, causal)
    check(out, r["out"], r["out_round"], dtype, D, x["scale"], int(lk.max()), "out")
    check_lse(lse, r["lse"], D, x["scale"])
    g = gradients(d, out, lse, causal=causal, workspace=ws)
    for n in what:
        if n in rg:
            check(g[n], rg[n], rg[n + "_round"], dtype, D, x["scale"], 3 * int(max(lq.max(), lk.max())), n)
    assert rda.rda_read_device_error(ws) == 0
    out2, lse2 = forward(d, causal=causal, workspace=ws)
    g2 = gradients(d, out, lse, causal=causal, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and all(g[n] is None or torch.equal(g[n], g2[n]) for n in g)
    return d, out, lse, g


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Dk,Ds,Dv", [(128, 64, 128), (64, 0, 64), (64, 64, 128), (128, 0, 64)])
@pytest.mark.parametrize("lens", [
    [100, 1, 90],          # 3 x 37 tiles of 64 rows: 16 rows a CTA forward, 32 in the gradients
    [101, 1, 90],          # 4 x 37 = 148: 64 and 64
    [330, 0, 301, 8],      # 5 x 37 tiles of 128: 64
    [331, 0, 301, 8],      # 6 x 37 = 222: 128
])
def test_fp32_rows_of_a_cta(cuda_device, lens, Dk, Ds, Dv, causal):
    """fp32 on either side of each change in the rows that a CTA takes."""
    compare(packed(lens, lens, 37, Dk, Ds, Dv, F32, seed=sum(lens) + Dk + Ds + Dv), causal)


@pytest.mark.parametrize("lq,lk", [([60, 3, 0, 70], [500, 131, 64, 70]), ([400, 130, 65, 70], [40, 130, 0, 1])])
def test_fp32_queries_and_keys_that_differ(cuda_device, lq, lk):
    """Few rows on one side and many on the other: each side's gradients by kernels of their own size."""
    compare(packed(lq, lk, 40, 128, 64, 128, F32, seed=len(lk) + lk[0]), True)


def test_fp32_rows_behind_the_last_sequence_many_heads(cuda_device):
    """NaN behind the sequences of a batch that 64 and 128 rows a CTA take."""
    for lens, pad in (([130, 77, 64], 30), ([300, 257, 1, 90], 100)):
        x = packed(lens, lens, 40, 128, 64, 128, F32, seed=pad, pad=pad)
        d, n = dev(x), sum(lens)
        out = torch.full((n + pad, 40, 128), 7.0, device="cuda")
        lse = torch.full((n + pad, 40), 7.0, device="cuda")
        forward(d, out=out, lse=lse)
        y = {m: t[:n] if isinstance(t, torch.Tensor) and len(t) == n + pad else t for m, t in x.items()}
        r, rg = oracle_forward(y, True), oracle_gradients(y, True)
        assert (out[n:] == 7).all() and (lse[n:] == 7).all()
        check(out[:n], r["out"], r["out_round"], F32, 192, x["scale"], 300, "out")
        g = gradients(d, out, lse)
        for m in NAMES:
            check(g[m][:n], rg[m], rg[m + "_round"], F32, 192, x["scale"], 900, m)


def alone(x, n):
    """Sequence n of packed inputs by itself (device tensors), and the rows of its queries and keys."""
    sq, sk = slice(*x["cu_q"][n:n + 2].tolist()), slice(*x["cu_k"][n:n + 2].tolist())
    one = {m: t[sk if m in ("k", "v", "k_shared") else sq].contiguous() if isinstance(t, torch.Tensor) else t
           for m, t in x.items()}
    one["cu_q"], one["cu_k"] = cu([sq.stop - sq.start], "cuda"), cu([sk.stop - sk.start], "cuda")
    return one, sq, sk


@pytest.mark.parametrize("lq,lk", [
    ([300, 77, 5], [300, 77, 5]),                              # 4 places x 37 heads = 148 CTAs: by their places
    ([300, 77, 0, 5], [300, 77, 0, 5]),                        # 5 x 37: in order
    ([700, 0, 33, 513, 256, 1], [700, 40, 161, 600, 256, 0]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_bf16_tiles_in_order(cuda_device, lq, lk, causal):
    """Tiles ordered by their work and not: the oracle's results, and each sequence's bits are those of a call by itself."""
    x = packed(lq, lk, 37, 128, 64, 128, BF16, seed=len(lq) + causal)
    d, out, lse, g = compare(x, causal)
    for n in range(len(lq)):
        one, sq, sk = alone(d, n)
        if not lq[n] or not lk[n]:
            continue
        o1, l1 = forward(one, causal=causal)
        g1 = gradients(one, o1, l1, causal=causal)
        assert torch.equal(o1, out[sq]) and torch.equal(l1, lse[sq])
        assert all(torch.equal(g1[m], g[m][sq if m in ("dq", "dq_shared") else sk]) for m in NAMES)


@pytest.mark.parametrize("count,H", [(512, 1), (513, 1), (600, 2), (1100, 1), (1100, 2)])
def test_bf16_more_sequences_than_threads(cuda_device, count, H):
    """More tiles than the ordering CTA has threads (512 and 256), and more sequences than it keeps offsets of (1024);
    one head by places from 513 sequences on; empty sequences among them, and some of several tiles."""
    lq = [(7 * i) % 13 if i % 97 else 300 + i % 5 for i in range(count)]
    lk = [n + i % 3 if i % 11 else 0 for i, n in enumerate(lq)]
    x = packed(lq, lk, H, 64, 64, 64, BF16, seed=count + H)
    d, out, lse, g = compare(x, True)
    for n in (0, 1, 97, 98, count - 2):
        one, sq, sk = alone(d, n)
        if not lq[n] or not lk[n]:
            continue
        o1, l1 = forward(one)
        g1 = gradients(one, o1, l1)
        assert torch.equal(o1, out[sq]) and torch.equal(l1, lse[sq])
        assert all(torch.equal(g1[m], g[m][sq if m in ("dq", "dq_shared") else sk]) for m in NAMES)


def test_fp32_alone_and_packed(cuda_device):
    """fp32 splits keys by the whole batch's size: a sequence's results are the same bits from run to run (`compare`), and
    alone and packed both within the bound."""
    lens = [257, 64, 190]
    x = packed(lens, lens, 2, 128, 64, 128, F32, seed=14)
    d, _, _, _ = compare(x, True)
    r, rg = oracle_forward(x, True), oracle_gradients(x, True)
    for n in range(3):
        one, s, _ = alone(d, n)
        o1, l1 = forward(one)
        check(o1, r["out"][s], r["out_round"][s], F32, 192, x["scale"], 257, "out")
        check_lse(l1, r["lse"][s], 192, x["scale"])
        g1 = gradients(one, o1, l1)
        for m in NAMES:
            check(g1[m], rg[m][s], rg[m + "_round"][s], F32, 192, x["scale"], 900, m)
