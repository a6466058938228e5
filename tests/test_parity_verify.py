"""Draft verification on the GPU against the fp64 oracle (whole numbers: equal),
and the whole of a speculative step: prompt, drafts, verification, replay."""
import pytest
import torch

import gated_delta_rule_rda_b200 as rda
import rda_gen
from latent_util import cu, packed, paged
from oracle import latent

pytestmark = pytest.mark.gpu


def inputs(B, T, V, seed, sharp=2.5, near=0.5):
    g = torch.Generator().manual_seed(seed)
    base = sharp * torch.randn(B, T + 1, V, generator=g)
    p = torch.softmax(base, -1)
    q = torch.softmax(base[:, :T] + near * torch.randn(B, T, V, generator=g), -1)
    u = torch.rand(B, T + 1, generator=g)
    x = torch.multinomial(q.reshape(-1, V), 1, generator=g).reshape(B, T).int() if T else torch.zeros(B, 0, dtype=torch.int32)
    return x, p, u, q


def run(x, p, u, q=None, n=None, **kw):
    c = lambda t: None if t is None else t.cuda()
    tok, acc = rda.rda_verify_drafts(c(x), c(p), c(u), draft_probs=c(q), num_drafts=c(n), **kw)
    return tok.cpu().tolist(), acc.cpu().tolist()


@pytest.mark.parametrize("V", [1, 3, 17, 1000, 1023, 1024, 1025, 4096, 32000, 259840])
@pytest.mark.parametrize("B,T", [(1, 0), (1, 3), (5, 7), (2, 32)])
def test_equal_to_the_oracle(cuda_device, V, B, T):
    if V * B * T > 4e6:
        B, T = 2, 3
    x, p, u, q = inputs(B, T, V, seed=V + B + T)
    assert run(x, p, u, q) == latent.verify(x, p, u, q)
    assert run(x, p, u) == latent.verify(x, p, u)


@pytest.mark.parametrize("V", [8192, 8193, 9001, 16385, 40000, 65537, 131072, 131073, 131076])
def test_vocabularies_around_the_changes_of_launch(cuda_device, V):
    """One CTA, clusters of 2, 4 and 8, two kernels; and a residual of nothing in each."""
    x, p, u, q = inputs(3, 2, V, seed=V)
    assert run(x, p, u, q) == latent.verify(x, p, u, q)
    same = p[:, :2].contiguous()                       # the target nowhere above the draft
    never = torch.cat([torch.ones(3, 2), u[:, 2:]], 1) * 0.999999
    x[:, 0] = -1                                       # refused, then drawn from the target itself
    assert run(x, p, never, same) == latent.verify(x, p, never, same)


def test_ragged_counts_and_bad_tokens(cuda_device):
    x, p, u, q = inputs(8, 5, 777, seed=2, near=0.05)
    n = torch.tensor([0, 1, 2, 3, 4, 5, 9, -3], dtype=torch.int32)
    assert run(x, p, u, q, n) == latent.verify(x, p, u, q, n)
    x[3, 0], x[4, 1], x[5, 4] = -1, 777, 1 << 30
    assert run(x, p, u, q, n) == latent.verify(x, p, u, q, n)
    assert run(x, p, u, None, n) == latent.verify(x, p, u, None, n)


def test_corners(cuda_device):
    """Uniforms of 0 and next to 1, equal distributions (a residual of nothing), zero rows, a single heavy
    token at either end, weights in one slice alone."""
    V = 3000
    x, p, u, q = inputs(6, 2, V, seed=3)
    for value in (0.0, 1 - 2.0 ** -24):
        u[:] = value
        assert run(x, p, u, q) == latent.verify(x, p, u, q)
        assert run(x, p, u) == latent.verify(x, p, u)
    x, p, u, q = inputs(6, 2, V, seed=4)
    q[:] = p[:, :2]
    u[:, :2] = 1.0            # u q < p fails where q = p: refused, and nothing is left
    assert run(x, p, u, q) == latent.verify(x, p, u, q)
    p[:] = 0
    assert run(x, p, u, q) == latent.verify(x, p, u, q)
    for at in (0, V - 1, 1023, 1024, 2047):
        p[:] = 0
        p[:, :, at] = 0.7
        assert run(x, p, u, q) == latent.verify(x, p, u, q)
    p[:] = 0
    p[:, :, 1024:2048] = torch.rand(6, 3, 1024)
    assert run(x, p, u, q) == latent.verify(x, p, u, q)


def test_unaligned_rows(cuda_device):
    """Rows that start anywhere: an odd vocabulary, and tensors that are a slice of a buffer."""
    x, p, u, q = inputs(3, 4, 1001, seed=5)
    assert run(x, p, u, q) == latent.verify(x, p, u, q)
    x, p, u, q = inputs(3, 4, 1000, seed=6)
    buf = torch.zeros(p.numel() + 1, device="cuda")
    view = buf[1:].view(p.shape).copy_(p)
    tok, acc = rda.rda_verify_drafts(x.cuda(), view, u.cuda(), draft_probs=q.cuda())
    assert (tok.cpu().tolist(), acc.cpu().tolist()) == latent.verify(x, p, u, q)


def test_graph_and_streams(cuda_device):
    x, p, u, q = (t.cuda() for t in inputs(16, 7, 5000, seed=7))
    ws = rda.new_workspace(rda.rda_verify_drafts_workspace_bytes(16, 7, 5000), "cuda")
    rda.rda_verify_drafts(x, p, u, q, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tok, acc = rda.rda_verify_drafts(x, p, u, q, workspace=ws)
    x2, p2, u2, q2 = inputs(16, 7, 5000, seed=8)
    for a, b in ((x, x2), (p, p2), (u, u2), (q, q2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert (tok.cpu().tolist(), acc.cpu().tolist()) == latent.verify(x2, p2, u2, q2)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(s[i % 2]):
            got.append(rda.rda_verify_drafts(x, p, u, q))
    torch.cuda.synchronize()
    for t, a in got:
        assert torch.equal(t, tok) and torch.equal(a, acc)


def test_calls_wait_for_what_came_before(cuda_device):
    """Inputs written right before each call, on the same buffers and the same workspace."""
    sets = [inputs(4, 3, 3001, seed=20 + i) for i in range(3)]
    ref = [latent.verify(*(t.cpu() for t in s)) for s in sets]
    sets = [[t.cuda() for t in s] for s in sets]
    buf = [torch.empty_like(t) for t in sets[0]]
    ws = rda.new_workspace(rda.rda_verify_drafts_workspace_bytes(4, 3, 3001), "cuda")
    got = []
    for i in range(12):
        for b, t in zip(buf, sets[i % 3]):
            b.copy_(t) if i % 2 else torch.mul(t, 1, out=b)
        got.append(rda.rda_verify_drafts(*buf, workspace=ws))
    for i, (tok, acc) in enumerate(got):
        assert (tok.cpu().tolist(), acc.cpu().tolist()) == ref[i % 3]


def test_a_speculative_step(cuda_device):
    """A hybrid's serving step as it would be used: the prompt through both kinds of layer, its latents into
    pages, drafted tokens through both kinds in one pass each, verification, and the recurrent state taken back
    to the accepted tokens -- against the same tokens run one by one."""
    dev, bf = "cuda", torch.bfloat16
    torch.manual_seed(0)
    B, H, D, Dl, Ds, page, prompt, T, V = 3, 16, 128, 512, 64, 16, [50, 17, 90], 4, 1000
    # latent layer: prompt in the expanded form, then into pages
    W = -(-(max(prompt) + T) // page)
    pages = torch.zeros(B * W, page, Dl + Ds, dtype=bf, device=dev)
    table = torch.randperm(B * W, device=dev).int().view(B, W)
    lat = torch.randn(sum(prompt) + B * T, Dl + Ds, device=dev).to(bf)
    wk, wv = (torch.randn(H, D, Dl, device=dev).to(bf) * Dl ** -0.5 for _ in range(2))
    at = [0]
    for b, n in enumerate(prompt):
        for j in range(n + T):
            pages[table[b, j // page], j % page] = lat[at[-1] + j]
        at.append(at[-1] + n + T)
    tokens = torch.cat([torch.arange(at[b], at[b] + prompt[b]) for b in range(B)]).to(dev)
    c = lat[tokens]
    k = torch.einsum("hdl,jl->jhd", wk.float(), c[:, :Dl].float()).to(bf).contiguous()
    v = torch.einsum("hdl,jl->jhd", wv.float(), c[:, :Dl].float()).to(bf).contiguous()
    q, qs = torch.randn(sum(prompt), H, D, device=dev).to(bf), torch.randn(sum(prompt), H, Ds, device=dev).to(bf)
    scale = (D + Ds) ** -0.5
    out, _ = rda.rda_latent_prefill(q, k, v, cu(prompt, dev), scale=scale, q_shared=qs, k_shared=c[:, Dl:].contiguous())
    # the last prompt token again, absorbed, one token a sequence: the same attention up to bf16 operands
    last = torch.tensor([sum(prompt[:b + 1]) - 1 for b in range(B)], device=dev)
    ql = torch.einsum("hdl,bhd->bhl", wk.float(), q[last].float()).to(bf).contiguous()[:, None]
    one, _ = rda.rda_latent_decode(ql, pages, table, torch.tensor(prompt, dtype=torch.int32, device=dev), scale=scale,
                                   q_shared=qs[last][:, None])
    got = torch.einsum("hdl,bhl->bhd", wv.float(), one[:, 0].float())
    # roundings of k, v, q.W, p (twice) and out (twice): 8 half steps of 2^-8, as relative 2-norms
    assert ((got - out[last].float()).norm() / out[last].float().norm()) < 8 * 2.0 ** -8
    # RDA layer: prompt, then T drafted tokens in one pass on a copy of the state
    vin = rda_gen.varlen_inputs(lengths=prompt, H=H, Dk=D, Dv=D, dtype=bf, seed=3).to(dev)
    _, state = rda.rda_prefill_varlen(vin.q, vin.k, vin.v, vin.log_alpha, vin.beta, vin.cu_seqlens)
    din = rda_gen.fixed_inputs(B, T, H, D, D, dtype=bf, seed=4).to(dev)
    drafted = state.clone()
    o_all = rda.rda_decode_tokens(din.q, din.k, din.v, din.log_alpha, din.beta, drafted)
    # latent layer: the drafted tokens in one pass against one by one
    lens = torch.tensor([n + T for n in prompt], dtype=torch.int32, device=dev)
    qT, qsT = torch.randn(B, T, H, Dl, device=dev).to(bf), torch.randn(B, T, H, Ds, device=dev).to(bf)
    oT, lseT = rda.rda_latent_decode(qT, pages, table, lens, scale=scale, q_shared=qsT, return_lse=True)
    for t in range(T):
        o1, l1 = rda.rda_latent_decode(qT[:, t:t + 1].contiguous(), pages, table, lens - T + t + 1, scale=scale,
                                       q_shared=qsT[:, t:t + 1].contiguous(), return_lse=True)
        # p and out are rounded on both sides
        assert (oT[:, t:t + 1].float() - o1.float()).norm() <= 4 * 2.0 ** -8 * o1.float().norm()
        assert (lseT[:, t:t + 1] - l1).abs().max() < 1e-4
    # verification, then the state after the accepted tokens alone
    x, p, u, qp = (t.to(dev) for t in inputs(B, T, V, seed=9, near=1.0))
    tok, kept = rda.rda_verify_drafts(x, p, u, qp)
    assert (tok.cpu().tolist(), kept.cpu().tolist()) == latent.verify(x.cpu(), p.cpu(), u.cpu(), qp.cpu())
    keep = (torch.arange(T, device=dev)[None] < kept[:, None])[..., None]
    replay = state.clone()
    rda.rda_decode_tokens(din.q, din.k, din.v, torch.where(keep, din.log_alpha, 0.0), torch.where(keep, din.beta, 0.0),
                          replay)
    for b in range(B):
        s = state[b:b + 1].clone()
        for t in range(int(kept[b])):
            rda.rda_decode_step(din.q[b:b + 1, t].contiguous(), din.k[b:b + 1, t].contiguous(),
                                din.v[b:b + 1, t].contiguous(), din.log_alpha[b:b + 1, t].contiguous(),
                                din.beta[b:b + 1, t].contiguous(), s)
        assert (replay[b:b + 1] - s).norm() <= 1e-5 * s.norm()
    assert torch.isfinite(o_all.float()).all()
