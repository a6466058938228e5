"""Cases, plain forms and 64-bit definitions of latent attention (prefill, its gradients, paged decode) and of draft
verification.

``run`` with ``own`` false computes an operator with elementary torch operations in 32 bits (64 where a choice of a
token hangs on it); with ``own`` true it makes the calls of ``gated_delta_rule_rda_b200``.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------------------------------
def listed():
    attn = dict(heads=16, dk=128, ds=64, dv=128, dtype="bf16", causal=True)
    return [
        # the smallest prompt in fp32, held to fp32 accuracy: parity runs and unit tests of a model
        dict(name="prefill f32 T256 H2", op="prefill", lens_q="256", lens_k="256", heads=2, dk=64, ds=64, dv=64,
             dtype="f32", causal=True),
        # one 4096-token prompt of the 16-head model
        dict(name="prefill T4096 H16", op="prefill", lens_q="4096", lens_k="4096", **attn),
        # a serving batch: new prompts and continued ones (more keys than queries), odd lengths, an empty one
        dict(name="prefill packed ragged", op="prefill", lens_q="1531,64,1,777,0,2048,300,129",
             lens_k="1531,1999,1025,777,512,2048,2801,129", **attn),
        # a long prompt
        dict(name="prefill T8192 H16", op="prefill", lens_q="8192", lens_k="8192", **attn),
        # a training step's microbatch of packed documents
        dict(name="backward packed ragged", op="backward", lens_q="911,260,64,1,333", lens_k="911,260,64,1,333", **attn),
        # a training step over one 4096-token sequence
        dict(name="backward T4096 H16", op="backward", lens_q="4096", lens_k="4096", **attn),
        # one user, one token: latency
        dict(name="decode B1 L4096", op="decode", batch=1, tokens=1, heads=16, dl=512, ds=64, page=64, longest=4096,
             ragged=False, dtype="bf16"),
        # a full serving batch of single tokens
        dict(name="decode B256 L4096", op="decode", batch=256, tokens=1, heads=16, dl=512, ds=64, page=64, longest=4096,
             ragged=True, dtype="bf16"),
        # drafted tokens verified in one pass (8 a sequence)
        dict(name="decode B32 T8 ragged", op="decode", batch=32, tokens=8, heads=16, dl=512, ds=64, page=32, longest=8192,
             ragged=True, dtype="bf16"),
        # the 40-head model, small pages, odd lengths
        dict(name="decode B24 H40", op="decode", batch=24, tokens=2, heads=40, dl=512, ds=64, page=16, longest=5001,
             ragged=True, dtype="bf16"),
        # one user's drafts of a small vocabulary: latency
        dict(name="verify B1 T3 V32000", op="verify", batch=1, drafts=3, vocab=32000, draft_probs=True),
        # a serving batch's drafts over the 259,840-row vocabulary
        dict(name="verify B64 T7 V259840", op="verify", batch=64, drafts=7, vocab=259840, draft_probs=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "backward", "decode", "verify"])
    if op in ("prefill", "backward"):
        dtype = "f32" if rng.random() < 0.25 else "bf16"
        heads = rng.choice([1, 2, 3, 8, 16, 40])
        # a sequence of one key alone has gradients of zero for its query and key: nothing to compare
        longest = _spread(rng, 1 if op == "prefill" else 16, 1200 if dtype == "f32" else 4096)
        seqs = rng.randint(1, 9)
        cap = (2.0e8 if op == "prefill" else 5.0e7) * (0.25 if dtype == "f32" else 1.0)
        lq, lk, pairs = [], [], 0
        for _ in range(seqs):
            a = rng.randint(0, longest) if rng.random() < 0.9 and (lq or op == "prefill") else longest
            b = a if rng.random() < 0.6 or op == "backward" and rng.random() < 0.7 else a + rng.randint(0, longest)
            if pairs + a * b * heads > cap and lq:
                break
            a = min(a, int(math.sqrt(cap / heads)))
            b = min(b, int(cap / heads / max(a, 1)))
            lq.append(a)
            lk.append(b)
            pairs += a * b * heads
        if sum(lq) == 0:
            lq[0], lk[0] = 1 + rng.randint(0, 200), 1 + rng.randint(0, 400)
        return dict(op=op, lens_q=",".join(map(str, lq)), lens_k=",".join(map(str, lk)), heads=heads,
                    dk=rng.choice([64, 128, 128]), ds=rng.choice([0, 64, 64]), dv=rng.choice([64, 128, 128]),
                    dtype=dtype, causal=rng.random() < 0.8)
    if op == "decode":
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        tokens = rng.choice([1, 1, 1, 2, 3, 4, 8])
        heads = rng.choice([1, 2, 5, 16, 16, 40, 128])
        longest = _spread(rng, tokens, 16384)
        room = min(400_000, 40_000_000 // (tokens * heads)) // (4 if dtype == "f32" else 1)
        batch = max(1, min(_spread(rng, 1, 256), room // longest))
        return dict(op=op, batch=batch, tokens=tokens, heads=heads, dl=rng.choice([256, 512, 512]),
                    ds=rng.choice([0, 64, 64]), page=rng.choice([16, 32, 48, 64, 128]), longest=longest,
                    ragged=rng.random() < 0.8, dtype=dtype)
    vocab = _spread(rng, 17, 259840)
    drafts = rng.randint(0, 8)
    batch = max(1, min(_spread(rng, 1, 128), 60_000_000 // (vocab * (drafts + 1))))
    return dict(op=op, batch=batch, drafts=drafts, vocab=vocab, draft_probs=rng.random() < 0.75)


def _lens(case, key):
    return [int(x) for x in case[key].split(",")]


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    n = 0
    for a, b in zip(_lens(case, "lens_q"), _lens(case, "lens_k")):
        if not case["causal"]:
            n += a * b
        elif b >= a:
            n += a * (b - a) + a * (a + 1) // 2
        else:
            n += b * (b + 1) // 2
    return n


def _decode_lens(case, seed):
    if not case["ragged"]:
        return [case["longest"]] * case["batch"]
    g = torch.Generator().manual_seed(seed * 7 + 3)
    lo = min(case["tokens"], case["longest"])
    x = torch.randint(lo, case["longest"] + 1, (case["batch"],), generator=g).tolist()
    x[0] = case["longest"]
    return x


def work(case):
    op = case["op"]
    if op in ("prefill", "backward"):
        e = 2 if case["dtype"] == "bf16" else 4
        tq, tk, h = sum(_lens(case, "lens_q")), sum(_lens(case, "lens_k")), case["heads"]
        dk, ds, dv = case["dk"], case["ds"], case["dv"]
        ins = e * (tq * h * (dk + ds) + tk * (h * (dk + dv) + ds))
        out = e * tq * h * dv + 4 * tq * h
        if op == "prefill":
            return {"bytes": ins + out, "flops": 2 * h * (dk + ds + dv) * _pairs(case)}
        return {"bytes": 2 * ins + out + e * tq * h * dv, "flops": 2 * h * (3 * (dk + ds) + 2 * dv) * _pairs(case)}
    if op == "decode":
        e = 2 if case["dtype"] == "bf16" else 4
        # ragged lengths are uniform between `tokens` and `longest`
        mean = (case["tokens"] + case["longest"]) / 2 if case["ragged"] else case["longest"]
        n, rows = case["batch"] * mean, case["batch"] * case["tokens"] * case["heads"]
        return {"bytes": e * (n * (case["dl"] + case["ds"]) + rows * (2 * case["dl"] + case["ds"])) + 4 * rows,
                "flops": 2 * case["tokens"] * case["heads"] * (2 * case["dl"] + case["ds"]) * n}
    rows = 2 if case["draft_probs"] and case["drafts"] else 1
    return {"bytes": 4 * case["batch"] * (rows * case["vocab"] + 4 * case["drafts"] + 3),
            "flops": 3 * case["batch"] * case["vocab"]}


# --------------------------------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------------------------------
def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    op = case["op"]
    s = dict(case=dict(case), workspace=None)
    if op in ("prefill", "backward"):
        dt, h = DTYPES[case["dtype"]], case["heads"]
        lq, lk = _lens(case, "lens_q"), _lens(case, "lens_k")
        tq, tk = sum(lq), sum(lk)

        def n(*shape):
            return torch.randn(*shape, generator=g, device=DEVICE).to(dt)

        s.update(q=n(tq, h, case["dk"]), k=n(tk, h, case["dk"]), v=n(tk, h, case["dv"]),
                 q_shared=n(tq, h, case["ds"]) if case["ds"] else None,
                 k_shared=n(tk, case["ds"]) if case["ds"] else None,
                 cu_q=_cu(lq), cu_k=_cu(lk), max_q=max(lq), max_k=max(lk),
                 scale=1.5 * (case["dk"] + case["ds"]) ** -0.5)
        if op == "backward":
            # what the forward pass left: its outputs and log-sum-exps
            o, lse = _attention(s, torch.float32)[:2]
            s.update(out=o.to(dt), lse=lse, d_out=n(tq, h, case["dv"]))
    elif op == "decode":
        dt, b, t, h = DTYPES[case["dtype"]], case["batch"], case["tokens"], case["heads"]
        dl, ds, page = case["dl"], case["ds"], case["page"]
        lens = _decode_lens(case, seed)
        per = [-(-x // page) for x in lens]
        width = max(per)
        pages = sum(per) + 3
        ids = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32).tolist()
        table = torch.full((b, width), -1, dtype=torch.int32)
        at = 0
        for i, m in enumerate(per):
            table[i, :m] = torch.tensor(ids[at:at + m], dtype=torch.int32)
            at += m
        s.update(q=torch.randn(b, t, h, dl, generator=g, device=DEVICE).to(dt),
                 q_shared=torch.randn(b, t, h, ds, generator=g, device=DEVICE).to(dt) if ds else None,
                 pages=torch.randn(pages, page, dl + ds, generator=g, device=DEVICE).to(dt),
                 table=table.to(DEVICE), lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE),
                 scale=192 ** -0.5)
    else:
        b, t, v = case["batch"], case["drafts"], case["vocab"]
        # the target's probabilities, and a draft model's that are near them
        base = 2.5 * torch.randn(b, t + 1, v, generator=g, device=DEVICE)
        s["target"] = torch.softmax(base, -1)
        near = torch.softmax(base[:, :t] + 0.5 * torch.randn(b, t, v, generator=g, device=DEVICE), -1)
        s["uniforms"] = torch.rand(b, t + 1, generator=g, device=DEVICE)
        pick = torch.rand(b, t, 1, generator=g, device=DEVICE, dtype=torch.float64)
        cum = near.double().cumsum(-1)
        s["tokens"] = (cum <= pick * cum[..., -1:]).sum(-1).clamp(max=v - 1).to(torch.int32)
        s["draft"] = near if case["draft_probs"] else None
    if own:
        s["workspace"] = _workspace(case, s)
    return s


# --------------------------------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------------------------------
def _workspace(case, s):
    """The scratch memory that a program keeps for calls of these sizes."""
    import gated_delta_rule_rda_b200 as rda
    op = case["op"]
    if op in ("prefill", "backward"):
        sizes = (s["q"].shape[0], s["k"].shape[0], case["heads"], case["dk"], case["ds"], case["dv"], s["cu_q"].numel() - 1)
        size = (rda.rda_latent_prefill_workspace_bytes if op == "prefill" else rda.rda_latent_backward_workspace_bytes)(*sizes)
    elif op == "decode":
        size = rda.rda_latent_decode_workspace_bytes(case["batch"], case["tokens"], case["heads"], case["dl"], case["ds"])
    else:
        size = rda.rda_verify_drafts_workspace_bytes(case["batch"], case["drafts"], case["vocab"])
    return rda.new_workspace(size, DEVICE)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import gated_delta_rule_rda_b200 as rda
        if op == "prefill":
            return rda.rda_latent_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], scale=s["scale"],
                                          q_shared=s["q_shared"], k_shared=s["k_shared"], causal=c["causal"],
                                          return_lse=True, workspace=s["workspace"])
        if op == "backward":
            return rda.rda_latent_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["d_out"], s["cu_q"], s["cu_k"],
                                           scale=s["scale"], q_shared=s["q_shared"], k_shared=s["k_shared"],
                                           causal=c["causal"], workspace=s["workspace"])
        if op == "decode":
            return rda.rda_latent_decode(s["q"], s["pages"], s["table"], s["lens"], scale=s["scale"],
                                         q_shared=s["q_shared"], return_lse=True, workspace=s["workspace"])
        return rda.rda_verify_drafts(s["tokens"], s["target"], s["uniforms"], draft_probs=s["draft"],
                                     workspace=s["workspace"])
    if op == "prefill":
        o, lse = _attention(s, torch.float32)[:2]
        return o.to(s["q"].dtype), lse
    if op == "backward":
        return _gradients(s)
    if op == "decode":
        return _decode(s)
    return _verify(s)


# --------------------------------------------------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------------------------------------------------
def _padded(x, cu, longest):
    """Rows of packed sequences as [sequences, longest, ...] (other rows repeat some row), and which are real."""
    at = torch.arange(longest, device=x.device)
    real = at[None] < (cu[1:] - cu[:-1])[:, None]
    return x[(cu[:-1, None] + at[None]).clamp(max=max(x.shape[0] - 1, 0)).long()], real


def _packed(x, cu, total):
    """The inverse of _padded: [total, ...]."""
    t = torch.arange(total, device=x.device, dtype=torch.int32)
    n = torch.searchsorted(cu, t, right=True) - 1
    return x[n, t - cu[n]]


def _whole(part, shared):
    """Per-head vectors with the shared part behind them, in 32 bits."""
    if shared is None:
        return part.float()
    if shared.dim() == part.dim() - 1:
        shared = shared[:, None].expand(-1, part.shape[1], -1)
    return torch.cat([part.float(), shared.float()], -1)


def _attention(s, kind):
    """Outputs and log-sum-exps in `kind`, and what the gradients use of the way there."""
    cu_q, cu_k = s["cu_q"], s["cu_k"]
    q, real_q = _padded(_whole(s["q"], s["q_shared"]).to(kind), cu_q, s["max_q"])
    k, real_k = _padded(_whole(s["k"], s["k_shared"]).to(kind), cu_k, s["max_k"])
    v, _ = _padded(s["v"].to(kind), cu_k, s["max_k"])
    seen = (real_q[:, :, None] & real_k[:, None, :])
    if s["case"]["causal"]:
        more = ((cu_k[1:] - cu_k[:-1]) - (cu_q[1:] - cu_q[:-1]))[:, None, None]
        i = torch.arange(s["max_q"], device=q.device)[None, :, None]
        j = torch.arange(s["max_k"], device=q.device)[None, None, :]
        seen = seen & (j <= i + more)
    x = torch.matmul(q.transpose(1, 2), k.permute(0, 2, 3, 1)).mul_(s["scale"])
    x.masked_fill_(~seen[:, None], -math.inf)
    top = x.amax(-1, keepdim=True) if x.shape[-1] else x.new_full((*x.shape[:-1], 1), -math.inf)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, 1.0))
    o = _packed(torch.matmul(p, v.transpose(1, 2)).transpose(1, 2), cu_q, s["q"].shape[0])
    lse = _packed((top + total.log())[..., 0].transpose(1, 2), cu_q, s["q"].shape[0])
    return o, lse.contiguous(), q, k, v, p, real_q


def _gradients(s):
    dt, ds = s["q"].dtype, s["case"]["ds"]
    dk = s["case"]["dk"]
    o, _, q, k, v, p, real_q = _attention(s, torch.float32)
    d_out = _padded(s["d_out"].float(), s["cu_q"], s["max_q"])[0]
    d_out = d_out * real_q[:, :, None, None]
    o = _padded(o, s["cu_q"], s["max_q"])[0]
    delta = (d_out * o).sum(-1).transpose(1, 2)[..., None]
    d = d_out.transpose(1, 2)
    dv = torch.matmul(p.transpose(2, 3), d).transpose(1, 2)
    dx = torch.matmul(d, v.permute(0, 2, 3, 1)).sub_(delta).mul_(p).mul_(s["scale"])
    dq = torch.matmul(dx, k.transpose(1, 2)).transpose(1, 2)
    dk_all = torch.matmul(dx.transpose(2, 3), q.transpose(1, 2)).transpose(1, 2)
    tq, tk = s["q"].shape[0], s["k"].shape[0]
    dq, dk_all, dv = _packed(dq, s["cu_q"], tq), _packed(dk_all, s["cu_k"], tk), _packed(dv, s["cu_k"], tk)
    return dict(dq=dq[..., :dk].contiguous().to(dt), dk=dk_all[..., :dk].contiguous().to(dt), dv=dv.to(dt),
                dq_shared=dq[..., dk:].contiguous().to(dt) if ds else None,
                dk_shared=dk_all[..., dk:].sum(1).to(dt) if ds else None)


def _decode(s):
    q = s["q"] if s["q_shared"] is None else torch.cat([s["q"], s["q_shared"]], -1)
    b, t, h, _ = q.shape
    dl = s["case"]["dl"]
    c = s["pages"][s["table"].clamp(min=0).long()].flatten(1, 2).float()
    x = torch.matmul(q.float().flatten(1, 2), c.transpose(1, 2)).mul_(s["scale"]).view(b, t, h, -1)
    last = (s["lens"][:, None] - t + torch.arange(t, device=q.device))[:, :, None, None]
    x.masked_fill_(torch.arange(c.shape[1], device=q.device) > last, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, 1.0))
    o = torch.matmul(p.flatten(1, 2), c[..., :dl]).view(b, t, h, dl)
    return o.to(s["q"].dtype), (top + total.log())[..., 0]


def _verify(s):
    x, p, u, q = s["tokens"].long(), s["target"], s["uniforms"].double(), s["draft"]
    b, t = x.shape
    px = p[:, :t].gather(2, x[..., None])[..., 0].double()
    qx = q.gather(2, x[..., None])[..., 0].double() if q is not None else torch.ones_like(px)
    kept = (u[:, :t] * qx < px).long().cumprod(1).sum(1)
    each = torch.arange(b, device=x.device)
    w = p[each, kept].double()
    if t:
        at = kept.clamp(max=t - 1)
        if q is not None:
            other = q[each, at].double()
        else:
            other = torch.zeros_like(w).scatter_(1, x[each, at][:, None], 2.0)
        rest = (w - other).clamp(min=0.0)
        rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, w)
        w = torch.where((kept < t)[:, None], rest, w)
    cum = w.cumsum(1)
    new = (cum <= u[:, t:] * cum[:, -1:]).sum(1)
    at = torch.arange(t + 1, device=x.device)
    out = torch.cat([x, x.new_zeros(b, 1)], 1)
    out = torch.where(at == kept[:, None], new[:, None], torch.where(at < kept[:, None], out, -1))
    return out.int(), kept.int()


# --------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------------------------------------------------
def _head64(q, k, v, scale, causal):
    """One sequence, one head: outputs and log-sum-exps of rows that see at least one key."""
    x = scale * (q @ k.T)
    if causal:
        i = torch.arange(q.shape[0], device=q.device)[:, None] + (k.shape[0] - q.shape[0])
        x = torch.where(torch.arange(k.shape[0], device=q.device)[None] <= i, x, -math.inf)
    lse = torch.logsumexp(x, 1)
    return torch.exp(x - lse[:, None]) @ v, lse


def exact(case, seed):
    op = case["op"]
    if op == "verify":
        return None  # whole numbers: they have to be equal
    s = prepare(case, seed)
    if op == "decode":
        b, t, h, dl = s["q"].shape
        o = torch.zeros(b, t, h, dl, dtype=torch.float64, device=DEVICE)
        lse = torch.full((b, t, h), -math.inf, dtype=torch.float64, device=DEVICE)
        lens, table = s["lens"].tolist(), s["table"].cpu()
        for i in range(b):
            n = lens[i]
            rows = s["pages"][table[i, :-(-n // case["page"])].long().to(DEVICE)].flatten(0, 1)[:n].double()
            for j in range(t):
                m = n - t + j + 1
                if m <= 0:
                    continue
                w = s["q"][i, j].double() @ rows[:m, :dl].T
                if case["ds"]:
                    w = w + s["q_shared"][i, j].double() @ rows[:m, dl:].T
                w = w * s["scale"]
                lse[i, j] = torch.logsumexp(w, 1)
                o[i, j] = torch.softmax(w, 1) @ rows[:m, :dl]
        return o, lse
    back = op == "backward"
    names = [n for n in ("q", "k", "v", "q_shared", "k_shared") if s[n] is not None]
    x = {n: s[n].double().requires_grad_(back) for n in names}
    o = torch.zeros(*s["q"].shape[:2], case["dv"], dtype=torch.float64, device=DEVICE)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEVICE)
    sums = {n: torch.zeros_like(x[n]) for n in names}
    q0 = k0 = 0
    for a, b in zip(_lens(case, "lens_q"), _lens(case, "lens_k")):
        first = max(0, a - b) if case["causal"] else (0 if b else a)  # rows before it see nothing
        for h in range(case["heads"] if a > first else 0):
            q, k, v = x["q"][q0 + first:q0 + a, h], x["k"][k0:k0 + b, h], x["v"][k0:k0 + b, h]
            if case["ds"]:
                q = torch.cat([q, x["q_shared"][q0 + first:q0 + a, h]], 1)
                k = torch.cat([k, x["k_shared"][k0:k0 + b]], 1)
            oh, lh = _head64(q, k, v, s["scale"], case["causal"])
            if back:
                got = torch.autograd.grad(oh, [q, k, v], s["d_out"][q0 + first:q0 + a, h].double())
                dk = case["dk"]
                sums["q"][q0 + first:q0 + a, h] += got[0][:, :dk]
                sums["k"][k0:k0 + b, h] += got[1][:, :dk]
                sums["v"][k0:k0 + b, h] += got[2]
                if case["ds"]:
                    sums["q_shared"][q0 + first:q0 + a, h] += got[0][:, dk:]
                    sums["k_shared"][k0:k0 + b] += got[1][:, dk:]
            else:
                o[q0 + first:q0 + a, h], lse[q0 + first:q0 + a, h] = oh, lh
        q0, k0 = q0 + a, k0 + b
    if back:
        return {"d" + n: sums.get(n) for n in ("q", "k", "v", "q_shared", "k_shared")}
    return o, lse
