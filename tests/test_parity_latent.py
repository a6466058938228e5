"""Latent attention on the GPU against the fp64 oracle: the expanded form, its
gradients and the absorbed form over pages, elementwise within what the
rounded terms allow."""
import math

import pytest
import torch

import gated_delta_rule_rda_b200 as rda
from latent_util import check, check_lse, cu, packed, paged
from oracle import latent

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def dev(x):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}


def forward(x, **kw):
    return rda.rda_latent_prefill(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], scale=x["scale"],
                                  q_shared=x["q_shared"], k_shared=x["k_shared"], return_lse=True, **kw)


def gradients(x, out, lse, **kw):
    return rda.rda_latent_backward(x["q"], x["k"], x["v"], out, lse, x["d_out"], x["cu_q"], x["cu_k"], scale=x["scale"],
                                   q_shared=x["q_shared"], k_shared=x["k_shared"], **kw)


def oracle_forward(x, causal):
    return latent.prefill(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], x["scale"], x["q_shared"], x["k_shared"], causal)


def oracle_gradients(x, causal):
    return latent.backward(x["q"], x["k"], x["v"], x["d_out"], x["cu_q"], x["cu_k"], x["scale"], x["q_shared"],
                           x["k_shared"], causal)


LENS = {
    "one token": ([1], [1]),
    "tile edges": ([63, 64, 65, 128, 129], [63, 64, 65, 128, 129]),
    "odd": ([200, 1, 37, 0, 96], [200, 1, 37, 0, 96]),
    "prefix": ([5, 130, 1, 64], [261, 131, 97, 64]),
    "more queries": ([70, 3, 10], [20, 0, 1]),
    "long": ([700], [700]),
    "many": ([3, 0, 1, 7, 2, 0, 0, 11, 5, 1, 1, 1, 4, 9, 2, 130, 1], [3, 5, 1, 7, 2, 0, 1, 11, 5, 1, 2, 1, 4, 9, 2, 130, 1]),
}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", list(LENS))
def test_lengths(cuda_device, dtype, causal, lens):
    lq, lk = LENS[lens]
    x = packed(lq, lk, 3, 128, 64, 128, dtype, seed=len(lens) + causal)
    d = dev(x)
    out, lse = forward(d, causal=causal)
    r = oracle_forward(x, causal)
    check(out, r["out"], r["out_round"], dtype, 192, x["scale"], max(lk), "out")
    check_lse(lse, r["lse"], 192, x["scale"])
    g, rg = gradients(d, out, lse, causal=causal), oracle_gradients(x, causal)
    for n in ("dq", "dk", "dv", "dq_shared", "dk_shared"):
        if rg[n].norm() > 1e-9:
            check(g[n], rg[n], rg[n + "_round"], dtype, 192, x["scale"], 3 * max(lq + lk), n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Dk,Ds,Dv", [(64, 0, 64), (64, 64, 64), (64, 64, 128), (128, 0, 64), (128, 0, 128), (64, 0, 128),
                                      (128, 64, 64)])
def test_dims(cuda_device, dtype, Dk, Ds, Dv):
    lq, lk = [150, 40, 1], [150, 75, 300]
    x = packed(lq, lk, 2, Dk, Ds, Dv, dtype, seed=Dk + Ds + Dv)
    d = dev(x)
    out, lse = forward(d)
    r = oracle_forward(x, True)
    check(out, r["out"], r["out_round"], dtype, Dk + Ds, x["scale"], 300, "out")
    check_lse(lse, r["lse"], Dk + Ds, x["scale"])
    g, rg = gradients(d, out, lse), oracle_gradients(x, True)
    for n in ("dq", "dk", "dv") + (("dq_shared", "dk_shared") if Ds else ()):
        check(g[n], rg[n], rg[n + "_round"], dtype, Dk + Ds, x["scale"], 900, n)
    if not Ds:
        assert g["dq_shared"] is None and g["dk_shared"] is None


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sharp_softmax_and_growing_maximum(cuda_device, dtype):
    """Scores that grow along the keys by far more than the exponent's range in one tile: the running
    maximum moves in every tile, and early tiles vanish."""
    x = packed([300], [300], 1, 64, 0, 64, dtype, seed=9)
    x["k"] = (x["k"].float() * torch.linspace(0.1, 6, 300)[:, None, None]).to(dtype)
    x["scale"] = 0.5
    d = dev(x)
    out, lse = forward(d)
    r = oracle_forward(x, True)
    # scores reach ~6 x 64 x 0.5 x 0.8: six times the size that check()'s bound takes
    check(out, r["out"], r["out_round"], dtype, 64, 6 * x["scale"], 300, "out")
    check_lse(lse, r["lse"], 64, 6 * x["scale"])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_behind_the_last_sequence(cuda_device, dtype):
    """Garbage behind the last sequence reaches no result, and results there stay as they were."""
    lq, lk, pad = [70, 33], [70, 50], 40
    x = packed(lq, lk, 2, 128, 64, 128, dtype, seed=11, pad=pad)
    y = packed(lq, lk, 2, 128, 64, 128, dtype, seed=11)
    d = dev(x)
    for n in ("q", "k", "v", "q_shared", "k_shared", "d_out"):
        y[n] = x[n][:len(x[n]) - pad]
    out = torch.full((sum(lq) + pad, 2, 128), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((sum(lq) + pad, 2), 7.0, device="cuda")
    forward(d, out=out, lse=lse)
    r, rg = oracle_forward(y, True), oracle_gradients(y, True)
    assert (out[sum(lq):] == 7).all() and (lse[sum(lq):] == 7).all()
    check(out[:sum(lq)], r["out"], r["out_round"], dtype, 192, x["scale"], 70, "out")
    out[sum(lq):] = float("nan")
    lse[sum(lq):] = float("nan")
    g = gradients(d, out, lse)
    for n in ("dq", "dk", "dv", "dq_shared", "dk_shared"):
        check(g[n][:len(rg[n])], rg[n], rg[n + "_round"], dtype, 192, x["scale"], 300, n)


def test_gradients_write_no_row_behind_the_last_sequence(cuda_device):
    for dtype in (F32, BF16):
        lq, pad = [33], 40
        x = dev(packed(lq, lq, 2, 128, 64, 128, dtype, seed=12, pad=pad))
        out, lse = forward(x, out=torch.zeros(73, 2, 128, dtype=dtype, device="cuda"))
        lib, P = rda.lib, rda._ptr
        g = {n: torch.full_like(x[n], 7.0) for n in ("q", "k", "v", "q_shared", "k_shared")}
        ws = rda.new_workspace(rda.rda_latent_backward_workspace_bytes(73, 73, 2, 128, 64, 128, 1), "cuda")
        code = lib.rda_latent_backward(P(x["q"]), P(x["q_shared"]), P(x["k"]), P(x["k_shared"]), P(x["v"]), P(out), P(lse),
                                       P(x["d_out"]), P(x["cu_q"]), P(x["cu_k"]), 1, 73, 73, P(g["q"]), P(g["q_shared"]),
                                       P(g["k"]), P(g["k_shared"]), P(g["v"]), rda._dtype_code(x["q"]), 2, 128, 64, 128,
                                       x["scale"], 1, P(ws), ws.numel(), rda._stream(None))
        assert code == 0
        torch.cuda.synchronize()
        for n, t in g.items():
            assert (t[33:] == 7).all() and torch.isfinite(t[:33]).all(), (dtype, n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lead", [3, 400])
def test_sequences_in_the_middle_of_a_batch(cuda_device, dtype, lead):
    """Offsets that begin behind 0: only the sequences they name are computed and written."""
    lens = [lead, 130, 300, 77]
    x = packed(lens, lens, 2, 128, 64, 128, dtype, seed=14)
    d, (lo, hi) = dev(x), (lead, lead + 430)
    part = {**d, "cu_q": d["cu_q"][1:4].contiguous(), "cu_k": d["cu_k"][1:4].contiguous()}
    whole, wl = forward(d)
    out = torch.full_like(whole, 7.0)
    lse = torch.full_like(wl, 7.0)
    forward(part, out=out, lse=lse)
    r, rg = oracle_forward(x, True), oracle_gradients(x, True)
    check(out[lo:hi], r["out"][lo:hi], r["out_round"][lo:hi], dtype, 192, x["scale"], 300, "out")
    for t in (out, lse):
        assert (t[:lo] == 7).all() and (t[hi:] == 7).all()
    lib, P = rda.lib, rda._ptr
    g = {n: torch.full_like(d[n], 7.0) for n in ("q", "q_shared", "k", "k_shared", "v")}
    total = sum(lens)
    ws = rda.new_workspace(rda.rda_latent_backward_workspace_bytes(total, total, 2, 128, 64, 128, 2), "cuda")
    assert lib.rda_latent_backward(P(d["q"]), P(d["q_shared"]), P(d["k"]), P(d["k_shared"]), P(d["v"]), P(whole), P(wl),
                                   P(d["d_out"]), P(part["cu_q"]), P(part["cu_k"]), 2, total, total, P(g["q"]),
                                   P(g["q_shared"]), P(g["k"]), P(g["k_shared"]), P(g["v"]), rda._dtype_code(d["q"]), 2, 128,
                                   64, 128, x["scale"], 1, P(ws), ws.numel(), rda._stream(None)) == 0
    torch.cuda.synchronize()
    for n, t in g.items():
        assert (t[:lo] == 7).all() and (t[hi:] == 7).all(), n
        check(t[lo:hi], rg["d" + n][lo:hi], rg["d" + n + "_round"][lo:hi], dtype, 192, x["scale"], 900, n)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_out_of_bounds_stay_inside(cuda_device, dtype):
    """cu_seqlens that a caller got wrong are kept inside the tensors."""
    x = packed([50], [50], 1, 64, 0, 64, dtype, seed=13)
    d = dev(x)
    d["cu_q"] = torch.tensor([-7, 90], dtype=torch.int32, device="cuda")
    d["cu_k"] = torch.tensor([-1, 1 << 30], dtype=torch.int32, device="cuda")
    out, lse = forward(d)
    r = oracle_forward(x, True)
    check(out, r["out"], r["out_round"], dtype, 64, x["scale"], 50, "out")
    d["cu_q"] = torch.tensor([40, 10], dtype=torch.int32, device="cuda")
    forward(d)
    gradients(d, out, lse)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_repeatable_and_bit_equal_alone_or_packed(cuda_device, dtype):
    """A sequence's results do not hang on what it is packed with, nor on when it runs."""
    lens = [257, 64, 190]
    d = dev(packed(lens, lens, 2, 128, 64, 128, dtype, seed=14))
    out, lse = forward(d)
    g = gradients(d, out, lse)
    for _ in range(3):
        out2, lse2 = forward(d)
        g2 = gradients(d, out2, lse2)
        assert torch.equal(out, out2) and torch.equal(lse, lse2) and all(torch.equal(g[n], g2[n]) for n in g)
    s = slice(257, 321)
    one = {n: t[s].contiguous() if isinstance(t, torch.Tensor) else t for n, t in d.items()}
    one["cu_q"] = one["cu_k"] = cu([64], "cuda")
    o1, l1 = forward(one)
    g1 = gradients(one, o1, l1)
    assert torch.equal(o1, out[s]) and torch.equal(l1, lse[s]) and all(torch.equal(g1[n], g[n][s]) for n in g)


def test_gradient_by_differences(cuda_device):
    """fp32, the loss through the kernel itself at q +- e d against <dq, d>."""
    x = dev(packed([40, 9], [50, 9], 2, 64, 64, 64, F32, seed=15))
    out, lse = forward(x)
    g = gradients(x, out, lse)
    for n in ("q", "k", "v", "q_shared", "k_shared"):
        torch.manual_seed(3)
        d = torch.randn_like(x[n])
        e = 1e-2

        def loss(sign):
            o, _ = forward({**x, n: x[n] + sign * e * d})
            return (o.double() * x["d_out"].double()).sum().item()

        want = (g["d" + n].double() * d.double()).sum().item()
        got = (loss(1) - loss(-1)) / (2 * e)
        # second-order term of a central difference: e^2 / 6 x third derivative (of the size of the loss's terms),
        # and fp32 noise of the loss over 2 e
        size = (g["d" + n].double().abs() * d.double().abs()).sum().item()
        assert abs(got - want) <= (e * e * 10 + 2.0 ** -24 * 100 / e) * size, n


def test_large_grid_of_one_head(cuda_device):
    """Every tile of a longer sequence, one head, against torch in fp64 on the GPU."""
    T = 2500
    x = dev(packed([T], [T], 1, 128, 64, 128, BF16, seed=16))
    out, lse = forward(x)
    q = torch.cat([x["q"][:, 0], x["q_shared"][:, 0]], 1).double()
    k = torch.cat([x["k"][:, 0], x["k_shared"]], 1).double()
    s = (x["scale"] * q @ k.T).masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    p = torch.softmax(s, 1)
    ref = p @ x["v"][:, 0].double()
    check(out[:, 0], ref.cpu(), (p @ x["v"][:, 0].double().abs() + ref.abs()).cpu(), BF16, 192, x["scale"], T, "out")
    check_lse(lse[:, 0], torch.logsumexp(s, 1).cpu(), 192, x["scale"])


# ---------------------------------------------------------------- absorbed form
def absorbed(d, **kw):
    return rda.rda_latent_decode(d["q"], d["pages"], d["table"], d["lens"], scale=d["scale"], q_shared=d["q_shared"],
                                 return_lse=True, **kw)


def check_absorbed(x, out, lse, dtype):
    r = latent.decode(x["q"], x["pages"], x["table"], x["lens"], x["scale"], x["q_shared"])
    D = x["pages"].shape[2]
    check(out, r["out"], r["out_round"], dtype, D, x["scale"], int(x["lens"].max()), "out")
    check_lse(lse, r["lse"], D, x["scale"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H,lens", [
    (1, 16, [1]), (1, 16, [63, 64, 65, 1, 0]), (1, 1, [300, 7]), (1, 5, [129, 128, 127]), (2, 40, [70, 2, 1, 131]),
    (8, 16, [8, 9, 200, 3, 0]), (8, 3, [1000]), (3, 24, [64, 640]), (1, 128, [100, 33]), (5, 13, [257, 5, 6]),
])
def test_decode_lengths(cuda_device, dtype, T, H, lens):
    x = paged(lens, T, H, 512, 64, 64, dtype, seed=T * 100 + H)
    out, lse = absorbed(dev(x))
    check_absorbed(x, out, lse, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Dl,Ds,page", [(512, 0, 16), (256, 64, 32), (128, 64, 48), (384, 0, 128), (512, 64, 80),
                                        (256, 0, 256), (512, 64, 16)])
def test_decode_dims_and_pages(cuda_device, dtype, Dl, Ds, page):
    x = paged([100, 259, 16, 1], 2, 9, Dl, Ds, page, dtype, seed=Dl + Ds + page)
    ws = rda.new_workspace(rda.rda_latent_decode_workspace_bytes(4, 2, 9, Dl, Ds), "cuda")
    out, lse = absorbed(dev(x), workspace=ws)
    check_absorbed(x, out, lse, dtype)
    assert rda.rda_read_device_error(ws) == 0


@pytest.mark.parametrize("T,H", [(5, 16), (2, 33), (1, 80), (3, 27), (8, 12)])
@pytest.mark.parametrize("Dl,Ds,page", [(512, 64, 16), (512, 0, 64), (384, 64, 32), (256, 64, 64), (128, 64, 16)])
def test_decode_more_rows_than_a_tile(cuda_device, T, H, Dl, Ds, page):
    """More than 64 rows are split over CTAs, evenly and not."""
    x = paged([300, 8, 1000, 64], T, H, Dl, Ds, page, BF16, seed=T + H + Dl)
    out, lse = absorbed(dev(x))
    check_absorbed(x, out, lse, BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_bad_pages_and_lengths(cuda_device, dtype):
    """Pages outside the cache drop their tokens, lengths are cut, and the error word says so."""
    x = paged([100, 40, 64, 30], 1, 16, 512, 64, 16, dtype, seed=21)
    ws = rda.new_workspace(rda.rda_latent_decode_workspace_bytes(4, 1, 16, 512, 64), "cuda")
    x["table"][0, 2] = -1
    x["table"][2, 0] = x["pages"].shape[0]
    out, lse = absorbed(dev(x), workspace=ws)
    check_absorbed(x, out, lse, dtype)
    assert rda.rda_read_device_error(ws) == 1
    x["lens"][1] = -5
    x["lens"][3] = 1 << 30
    x["table"][3] = torch.arange(x["table"].shape[1], dtype=torch.int32)
    x["pages"] = torch.nan_to_num(x["pages"])
    out, lse = absorbed(dev(x), workspace=ws)
    check_absorbed(x, out, lse, dtype)
    assert rda.rda_read_device_error(ws) == 1 and rda.rda_read_device_error(ws) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_long_and_ragged_batch(cuda_device, dtype):
    """Sequences that are split over many CTAs next to short ones; the same bits every time."""
    x = paged([5000, 3, 777, 0, 64, 1200], 2, 16, 512, 64, 64, dtype, seed=22)
    d = dev(x)
    out, lse = absorbed(d)
    check_absorbed(x, out, lse, dtype)
    for _ in range(3):
        o2, l2 = absorbed(d)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_many_short_sequences(cuda_device, dtype):
    lens = [(7 * i) % 23 for i in range(300)]
    x = paged(lens, 1, 4, 256, 64, 16, dtype, seed=23)
    out, lse = absorbed(dev(x))
    check_absorbed(x, out, lse, dtype)


def test_decode_most_rows(cuda_device):
    """8 tokens of 1024 heads: more row tiles than the batch can be split for."""
    x = paged([70, 9], 8, 1024, 128, 64, 16, BF16, seed=94)
    out, lse = absorbed(dev(x))
    check_absorbed(x, out, lse, BF16)


def test_decode_largest_batch(cuda_device):
    B, Dl, page = 65535, 128, 16
    g = torch.Generator(device="cuda").manual_seed(95)
    pages = torch.randn(3000, page, Dl, generator=g, device="cuda").to(BF16)
    table = torch.randint(0, 3000, (B, 2), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(0, 33, (B,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(B, 1, 1, Dl, generator=g, device="cuda").to(BF16)
    scale = Dl ** -0.5
    out, lse = rda.rda_latent_decode(q, pages, table, lens, scale=scale, return_lse=True)
    for lo in range(0, B, 8192):                       # the definition in 64 bits, a part at a time
        c = pages[table[lo:lo + 8192].long()].flatten(1, 2).double()
        s = scale * (c @ q[lo:lo + 8192, 0, 0].double()[..., None])[..., 0]
        s = s.masked_fill(torch.arange(32, device="cuda") >= lens[lo:lo + 8192, None], -math.inf)
        p = torch.nan_to_num(torch.softmax(s, 1))      # no token: no weight
        ref = (p[:, None] @ c)[:, 0]
        moved = (p[:, None] @ c.abs())[:, 0] + ref.abs()
        check(out[lo:lo + 8192, 0, 0], ref.cpu(), moved.cpu(), BF16, Dl, scale, 32, "out")
        check_lse(lse[lo:lo + 8192, 0, 0], torch.logsumexp(s, 1).cpu(), Dl, scale)


def test_decode_cache_past_32_bit_offsets(cuda_device):
    """A cache of more than 2^32 bytes and 2^31 elements, with the sequence's pages at its end."""
    D, page = 576, 64
    P = (1 << 31) // (D * page) + 40
    pages = torch.zeros(P, page, D, dtype=BF16, device="cuda")
    x = paged([150], 1, 16, 512, 64, page, BF16, seed=24, spare=0, garbage=False)
    m = x["pages"].shape[0]
    pages[P - m:] = x["pages"].cuda()
    d = dev(x)
    d["pages"], d["table"] = pages, d["table"] + (P - m)
    out, lse = absorbed(d)
    check_absorbed(x, out, lse, BF16)


def test_decode_shared_pages(cuda_device):
    """The same page twice in a table, and in two sequences."""
    x = paged([64, 64], 1, 16, 512, 64, 16, BF16, seed=25)
    x["table"][0, 3] = x["table"][0, 0]
    x["table"][1] = x["table"][0]
    out, lse = absorbed(dev(x))
    check_absorbed(x, out, lse, BF16)


# ---------------------------------------------------------------- streams, graphs, devices
def test_streams_and_graphs(cuda_device):
    """Two streams with a workspace each, and a captured graph replayed on new inputs."""
    pre = [dev(packed([200 + i], [200 + i], 4, 128, 64, 128, BF16, seed=30 + i)) for i in range(4)]
    dec = [dev(paged([900 + i, 20], 1, 16, 512, 64, 64, BF16, seed=40 + i)) for i in range(4)]
    ref = []
    for a, b in zip(pre, dec):
        o, l = forward(a)
        ref.append((o, l, gradients(a, o, l), absorbed(b)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None] * 4
    for _ in range(3):
        for i, (a, b) in enumerate(zip(pre, dec)):
            with torch.cuda.stream(streams[i % 2]):
                o, l = forward(a)
                got[i] = (o, l, gradients(a, o, l), absorbed(b))
        torch.cuda.synchronize()
        for r, g in zip(ref, got):
            assert torch.equal(r[0], g[0]) and torch.equal(r[1], g[1]) and all(torch.equal(r[2][n], g[2][n]) for n in r[2])
            assert torch.equal(r[3][0], g[3][0]) and torch.equal(r[3][1], g[3][1])
    # capture, then replay with other contents of the same buffers
    a, b = pre[0], dec[0]
    ws = rda.new_workspace(1 << 26, "cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = forward(a, workspace=ws)
        g = gradients(a, o, l, workspace=ws)
        od, ld = absorbed(b, workspace=ws)
    new = packed([200], [200], 4, 128, 64, 128, BF16, seed=50)
    for n in ("q", "k", "v", "q_shared", "k_shared", "d_out"):
        a[n].copy_(new[n])
    b["lens"].copy_(torch.tensor([333, 7], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    eo, el = forward(a)
    eg = gradients(a, eo, el)
    ed, eld = absorbed(b)
    assert torch.equal(o, eo) and torch.equal(l, el) and all(torch.equal(g[n], eg[n]) for n in g)
    assert torch.equal(od, ed) and torch.equal(ld, eld)


def test_calls_wait_for_what_came_before(cuda_device):
    """Inputs written right before each call, by kernels and by copies, on the same buffers and the same workspace:
    eager, and in two captured graphs that share the workspace, with a branch that joins before the calls."""
    pre = [dev(packed([300, 40, 129], [300, 40, 129], 4, 128, 64, 128, BF16, seed=70 + i)) for i in range(2)]
    dec = [dev(paged([700, 90, 1], 2, 16, 512, 64, 16, BF16, seed=80 + i)) for i in range(2)]
    names = ("q", "k", "v", "q_shared", "k_shared", "d_out")
    ws = rda.new_workspace(1 << 27, "cuda")

    def calls(a, b):
        o, l = forward(a, workspace=ws)
        g = gradients(a, o, l, workspace=ws)
        od, ld = absorbed(b, workspace=ws)
        return [o, l, *(g[n] for n in sorted(g)), od, ld]

    ref = [calls(a, b) for a, b in zip(pre, dec)]
    torch.cuda.synchronize()
    a = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in pre[0].items()}
    b = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in dec[0].items()}
    pinned = [x["lens"].cpu().pin_memory() for x in dec]

    def fill(i, by_kernel):
        for n in names:
            torch.mul(pre[i][n], 1, out=a[n]) if by_kernel else a[n].copy_(pre[i][n])
        for n in ("q", "pages", "table", "q_shared"):
            b[n].zero_()
            torch.mul(dec[i][n], 1, out=b[n]) if by_kernel else b[n].copy_(dec[i][n])
        b["lens"].copy_(pinned[i], non_blocking=True)

    got = []
    for i in range(12):
        fill(i % 2, i % 4 < 2)
        got.append(calls(a, b))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, ref[i % 2])), i
    graphs = []
    side = torch.cuda.Stream()
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                fill(i, i == 0)
            main.wait_stream(side)
            out = calls(a, b)
        graphs.append((graph, out))
    for i in (0, 1, 1, 0, 1, 0):
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(graphs[i][1], ref[i])), i


def test_memory_made_for_a_call_on_another_stream(cuda_device):
    """`stream=` another than the current one: results and workspaces made by the call stay whole while the
    current stream allocates and writes."""
    a = dev(packed([500, 260], [500, 260], 8, 128, 64, 128, BF16, seed=90))
    b = dev(paged([3000, 90], 2, 16, 512, 64, 64, BF16, seed=91))
    ref = [*forward(a), *absorbed(b)]
    rg = gradients(a, ref[0], ref[1])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        o = [*forward(a, stream=s), *absorbed(b, stream=s)]
        g = gradients(a, o[0], o[1], stream=s)
        got.append((o, g))
        for n in (1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24):
            torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for o, g in got:
        assert all(torch.equal(x, y) for x, y in zip(o, ref)) and all(torch.equal(g[n], rg[n]) for n in g)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_scales_that_are_not_positive(cuda_device, dtype, scale):
    x = packed([150, 40], [150, 90], 2, 128, 64, 128, dtype, seed=92)
    x["scale"] = scale
    out, lse = forward(dev(x))
    r, rg = oracle_forward(x, True), oracle_gradients(x, True)
    check(out, r["out"], r["out_round"], dtype, 192, scale, 150, "out")
    check_lse(lse, r["lse"], 192, scale)
    g = gradients(dev(x), out, lse)
    for n in ("dq", "dk", "dv", "dq_shared", "dk_shared"):
        check(g[n], rg[n], rg[n + "_round"], dtype, 192, scale, 3 * 240, n)
    y = paged([100, 30], 2, 16, 512, 64, 16, dtype, seed=93, scale=scale)
    out, lse = absorbed(dev(y))
    check_absorbed(y, out, lse, dtype)


def test_binding_refusals(cuda_device):
    x = dev(packed([10], [10], 2, 64, 64, 64, BF16, seed=60))
    with pytest.raises(ValueError):
        forward({**x, "k": x["k"][:, :1].contiguous()})
    with pytest.raises(TypeError):
        forward({**x, "v": x["v"].float()})
    with pytest.raises(ValueError):
        forward({**x, "q": x["q"].transpose(0, 1).contiguous().transpose(0, 1)})
    with pytest.raises(ValueError):
        forward({**x, "k_shared": None})
    with pytest.raises(ValueError):
        forward({**x, "cu_k": x["cu_k"].cpu()})
    with pytest.raises(rda.RdaError) as e:
        forward({**x, "q": torch.zeros(10, 2, 96, dtype=BF16, device="cuda"),
                 "k": torch.zeros(10, 2, 96, dtype=BF16, device="cuda")})
    assert e.value.code == 2
    with pytest.raises(rda.RdaError) as e:
        forward(x, workspace=torch.zeros(128, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4


def test_empty_calls(cuda_device):
    z = lambda *s: torch.zeros(*s, dtype=BF16, device="cuda")
    c0 = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = rda.rda_latent_prefill(z(0, 2, 64), z(0, 2, 64), z(0, 2, 64), c0, scale=1.0, return_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    g = rda.rda_latent_backward(z(0, 2, 64), z(0, 2, 64), z(0, 2, 64), out, lse, out, c0, scale=1.0)
    assert g["dq"].shape == (0, 2, 64)
    # queries without a single key anywhere, and keys without a query
    c1 = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    c2 = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    out, lse = rda.rda_latent_prefill(z(5, 2, 64) + 1, z(0, 2, 64), z(0, 2, 64), c1, c2, scale=1.0, return_lse=True)
    assert (out == 0).all() and torch.isinf(lse).all()
    g = rda.rda_latent_backward(z(5, 2, 64) + 1, z(0, 2, 64), z(0, 2, 64), out, lse, out + 1, c1, c2, scale=1.0)
    assert (g["dq"] == 0).all()
    o0, l0 = out[:0], lse[:0]
    g = rda.rda_latent_backward(z(0, 2, 64), z(5, 2, 64), z(5, 2, 64), o0, l0, o0, c2, c1, scale=1.0)
    assert (g["dk"] == 0).all() and (g["dv"] == 0).all()
    o, l = rda.rda_latent_decode(z(2, 1, 4, 128), z(0, 16, 128), torch.zeros(2, 0, dtype=torch.int32, device="cuda"),
                                 torch.zeros(2, dtype=torch.int32, device="cuda"), scale=1.0, return_lse=True)
    assert (o == 0).all() and torch.isinf(l).all()
