"""The fp64 oracle of latent attention and draft verification, pinned on the
CPU by closed forms, autograd, differences and each other."""
import numpy as np
import pytest
import torch

from latent_util import cu, packed, paged
from oracle import latent


def test_equal_keys_average_the_values():
    x = packed([3], [5], 2, 64, 64, 64, torch.float32, 1)
    x["k"][:] = x["k"][:1]
    x["k_shared"][:] = x["k_shared"][:1]
    r = latent.prefill(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], x["scale"], x["q_shared"], x["k_shared"])
    for i in range(3):
        assert torch.allclose(r["out"][i], x["v"][:i + 3].double().mean(0), atol=1e-12)


def test_one_key_gives_its_value_and_no_gradient_to_scores():
    x = packed([1], [1], 3, 64, 0, 128, torch.float32, 2)
    r = latent.prefill(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], x["scale"])
    assert torch.equal(r["out"], x["v"].double())
    g = latent.backward(x["q"], x["k"], x["v"], x["d_out"], x["cu_q"], x["cu_k"], x["scale"])
    assert g["dq"].abs().max() < 1e-13 and g["dk"].abs().max() < 1e-13
    assert torch.equal(g["dv"], x["d_out"].double())


def test_rows_without_keys():
    x = packed([4, 2], [2, 0], 1, 64, 0, 64, torch.float32, 3)
    r = latent.prefill(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], x["scale"])
    assert torch.isinf(r["lse"][[0, 1, 4, 5]]).all() and (r["out"][[0, 1, 4, 5]] == 0).all()
    assert torch.isfinite(r["lse"][2:4]).all()


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_against_autograd_and_differences(causal):
    x = packed([5, 1, 4], [7, 1, 3], 2, 64, 64, 64, torch.float32, 4)
    names = ["q", "k", "v", "q_shared", "k_shared"]
    leaves = {n: x[n].double().requires_grad_(True) for n in names}

    def loss(t):
        total = 0.0
        for n in range(3):
            sq, sk = slice(int(x["cu_q"][n]), int(x["cu_q"][n + 1])), slice(int(x["cu_k"][n]), int(x["cu_k"][n + 1]))
            lq, lk = sq.stop - sq.start, sk.stop - sk.start
            s = torch.einsum("ihd,jhd->hij", t["q"][sq], t["k"][sk]) + torch.einsum("ihd,jd->hij", t["q_shared"][sq],
                                                                                 t["k_shared"][sk])
            s = x["scale"] * s
            if causal:
                s = s.masked_fill(torch.arange(lk)[None] > torch.arange(lq)[:, None] + lk - lq, -1e30)
            p = torch.softmax(s, -1)
            if causal:
                p = p * (s > -1e29)
            total = total + (torch.einsum("hij,jhd->ihd", p, t["v"][sk]) * x["d_out"][sq].double()).sum()
        return total

    ref = torch.autograd.grad(loss(leaves), [leaves[n] for n in names])
    g = latent.backward(x["q"], x["k"], x["v"], x["d_out"], x["cu_q"], x["cu_k"], x["scale"], x["q_shared"],
                        x["k_shared"], causal)
    plain = {n: leaves[n].detach() for n in names}
    rng = np.random.default_rng(0)
    for n, r in zip(names, ref):
        assert torch.allclose(g["d" + n], r, atol=1e-12), n
        for _ in range(4):
            at = tuple(int(rng.integers(s)) for s in r.shape)
            e = torch.zeros_like(r)
            e[at] = 1e-5
            diff = (loss({**plain, n: plain[n] + e}) - loss({**plain, n: plain[n] - e})) / 2e-5
            assert abs(diff - g["d" + n][at]) < 1e-7, (n, at)


def test_absorbed_equals_expanded():
    """q . (W c) = (W^T q) . c, and sum_j p_j (W c_j) = W sum_j p_j c_j."""
    torch.manual_seed(5)
    n, H, Dl, Ds, Dk, T = 9, 2, 128, 64, 64, 3
    d = paged([n], T, H, Dl, Ds, 16, torch.float64, 6)
    c = d["pages"][d["table"][0, 0], :n]
    wk, wv = torch.randn(H, Dk, Dl, dtype=torch.float64), torch.randn(H, Dk, Dl, dtype=torch.float64)
    q = torch.randn(T, H, Dk, dtype=torch.float64)
    exp = latent.prefill(q, torch.einsum("hdl,jl->jhd", wk, c[:, :Dl]), torch.einsum("hdl,jl->jhd", wv, c[:, :Dl]),
                         cu([T]), cu([n]), 0.05, d["q_shared"][0], c[:, Dl:])
    ab = latent.decode(torch.einsum("hdl,thd->thl", wk, q)[None], d["pages"], d["table"], d["lens"], 0.05, d["q_shared"])
    assert torch.allclose(torch.einsum("hdl,thl->thd", wv, ab["out"][0]), exp["out"], atol=1e-9)
    assert torch.allclose(ab["lse"][0], exp["lse"], atol=1e-9)


def test_decode_drops_bad_pages_and_cuts_lengths():
    d = paged([20, 5], 2, 1, 128, 0, 16, torch.float64, 7)
    d["table"][0, 1] = -4
    a = latent.decode(d["q"], d["pages"], d["table"], torch.tensor([99, -1]), 0.1)
    # 99 is cut to 32, all of the second page's tokens are gone
    ref = torch.softmax(0.1 * d["q"][0, 0] @ d["pages"][d["table"][0, 0]].T, 1) @ d["pages"][d["table"][0, 0]]
    assert torch.allclose(a["out"][0, 0], ref) and (a["out"][1] == 0).all() and torch.isinf(a["lse"][1]).all()


def test_verify_keeps_what_the_rule_keeps():
    p = [[[0.5, 0.5, 0.0], [0.0, 0.25, 0.75], [0.2, 0.3, 0.5]]]
    q = [[[0.25, 0.75, 0.0], [0.5, 0.5, 0.0]]]
    # draft 0: 0.6 x 0.75 < 0.5 kept; draft 1: p = 0 refused; residual max(p - q, 0) = (0, 0, 0.75)
    assert latent.verify([[1, 0]], p, [[0.6, 0.0, 0.1]], q) == ([[1, 2, -1]], [1])
    # every draft kept: from the last row, 0.2 <= 0.45 < 0.5
    assert latent.verify([[0, 1]], p, [[0.99, 0.49, 0.45]], q) == ([[0, 1, 1]], [2])
    # drafts chosen outright: 0.6 > 0.5 refused, token 1 out of the residual
    assert latent.verify([[1, 1]], p, [[0.6, 0.0, 0.99]]) == ([[0, -1, -1]], [0])
    # none, outside the vocabulary, and a residual of nothing
    assert latent.verify([[1, 1]], p, [[0.0, 0.0, 0.6]], q, [0]) == ([[1, -1, -1]], [0])
    assert latent.verify([[7, 1]], p, [[0.0, 0.0, 0.2]]) == ([[0, -1, -1]], [0])
    assert latent.verify([[2]], [[[0.5, 0.5, 0.0]] * 2], [[0.5, 0.7]], [[[0.5, 0.5, 0.0]]]) == ([[1, -1]], [0])


def test_verify_follows_the_target():
    """The first token's distribution is the target's, whatever the draft's."""
    rng = np.random.default_rng(8)
    n = 40000
    p, q = np.array([0.1, 0.6, 0.3]), np.array([0.5, 0.2, 0.3])
    x = rng.choice(3, size=(n, 1), p=q)
    tokens, _ = latent.verify(x, np.broadcast_to(p, (n, 2, 3)), rng.random((n, 2)), np.broadcast_to(q, (n, 1, 3)))
    got = np.bincount([t[0] for t in tokens], minlength=3) / n
    # four standard deviations of a frequency
    assert np.all(np.abs(got - p) < 4 * np.sqrt(p * (1 - p) / n))
