"""Plain fp64 oracle of latent attention (expanded, its gradients, absorbed over
pages) and of draft verification (test infrastructure only, like the rest of
this package).

Written from the definitions in ``include/rda.h``, one sequence and head at a
time.  Besides each result the functions return, elementwise, what a rounding
of the terms that the kernels round can move it by at most (``*_round``: for
one half step of relative size 1 in every rounded term; a test multiplies it by
the half step of the type).
"""
import numpy as np
import torch


def _t(x):
    return None if x is None else torch.as_tensor(x).detach().to("cpu", torch.float64)


def _seen(lq, lk, causal):
    i, j = torch.arange(lq)[:, None], torch.arange(lk)[None, :]
    return (j <= i + lk - lq) if causal else torch.ones(lq, lk, dtype=torch.bool)


def softmax_rows(s, seen):
    """(p, lse) of the visible scores; rows that see nothing: 0 and -inf."""
    s = torch.where(seen, s, torch.tensor(-np.inf, dtype=torch.float64))
    if s.shape[1] == 0:
        return s, torch.full((s.shape[0],), -np.inf, dtype=torch.float64)
    top = s.max(1, keepdim=True).values
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(s - top)
    l = e.sum(1, keepdim=True)
    p = e / torch.where(l > 0, l, torch.ones_like(l))
    return p, (top + torch.log(l))[:, 0]


def _parts(x, shared, sl, h):
    y = x[sl, h]
    if shared is None:
        return y
    z = shared[sl, h] if shared.dim() == 3 else shared[sl]
    return torch.cat([y, z], 1)


def prefill(q, k, v, cu_q, cu_k, scale, q_shared=None, k_shared=None, causal=True):
    """dict: out, lse, out_round (Sum p |v| + |out|: the probabilities and the result rounded)."""
    q, k, v, q_shared, k_shared = map(_t, (q, k, v, q_shared, k_shared))
    H, Dv = q.shape[1], v.shape[2]
    out = torch.zeros(q.shape[0], H, Dv, dtype=torch.float64)
    rnd = torch.zeros_like(out)
    lse = torch.full((q.shape[0], H), -np.inf, dtype=torch.float64)
    for n in range(len(cu_q) - 1):
        sq, sk = slice(int(cu_q[n]), int(cu_q[n + 1])), slice(int(cu_k[n]), int(cu_k[n + 1]))
        for h in range(H):
            x, y, z = _parts(q, q_shared, sq, h), _parts(k, k_shared, sk, h), v[sk, h]
            p, l = softmax_rows(scale * x @ y.T, _seen(len(x), len(y), causal))
            out[sq, h], lse[sq, h] = p @ z, l
            rnd[sq, h] = p @ z.abs() + (p @ z).abs()
    return dict(out=out, lse=lse, out_round=rnd)


def backward(q, k, v, d_out, cu_q, cu_k, scale, q_shared=None, k_shared=None, causal=True):
    """dict: dq, dk, dv, dq_shared, dk_shared and their ``_round``: p, ds, the forward's
    result (in delta) and the gradient itself rounded."""
    q, k, v, d_out, q_shared, k_shared = map(_t, (q, k, v, d_out, q_shared, k_shared))
    H, Dk = q.shape[1], q.shape[2]
    g = dict(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    if k_shared is not None:
        g.update(dq_shared=torch.zeros_like(q_shared), dk_shared=torch.zeros_like(k_shared))
    r = {n + "_round": torch.zeros_like(x) for n, x in g.items()}
    for n in range(len(cu_q) - 1):
        sq, sk = slice(int(cu_q[n]), int(cu_q[n + 1])), slice(int(cu_k[n]), int(cu_k[n + 1]))
        for h in range(H):
            x, y, z, d = _parts(q, q_shared, sq, h), _parts(k, k_shared, sk, h), v[sk, h], d_out[sq, h]
            p, _ = softmax_rows(scale * x @ y.T, _seen(len(x), len(y), causal))
            o = p @ z
            ds = p * (d @ z.T - (d * o).sum(1, keepdim=True))
            moved = ds.abs() + p * (d.abs() * o.abs()).sum(1, keepdim=True)
            g["dv"][sk, h] = p.T @ d
            r["dv_round"][sk, h] = p.T @ d.abs()
            dx, dy = scale * ds @ y, scale * ds.T @ x
            rx, ry = abs(scale) * moved @ y.abs(), abs(scale) * moved.T @ x.abs()
            g["dq"][sq, h], g["dk"][sk, h] = dx[:, :Dk], dy[:, :Dk]
            r["dq_round"][sq, h], r["dk_round"][sk, h] = rx[:, :Dk], ry[:, :Dk]
            if k_shared is not None:
                g["dq_shared"][sq, h], r["dq_shared_round"][sq, h] = dx[:, Dk:], rx[:, Dk:]
                g["dk_shared"][sk] += dy[:, Dk:]
                r["dk_shared_round"][sk] += ry[:, Dk:]
    for name, x in g.items():
        r[name + "_round"] += x.abs()
    return {**g, **r}


def decode(q, pages, table, lens, scale, q_shared=None):
    """dict: out, lse, out_round.  Pages outside the cache drop their tokens; lengths are
    cut to [0, table width x page size]."""
    q, pages, q_shared = _t(q), _t(pages), _t(q_shared)
    B, T, H, Dl = q.shape
    P, size, _ = pages.shape
    out = torch.zeros(B, T, H, Dl, dtype=torch.float64)
    rnd, lse = torch.zeros_like(out), torch.full((B, T, H), -np.inf, dtype=torch.float64)
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * size)
        rows, at = [], []
        for j in range(n):
            page = int(table[b, j // size])
            if 0 <= page < P:
                rows.append(pages[page, j % size])
                at.append(j)
        if not rows:
            continue
        c, at = torch.stack(rows), torch.tensor(at)
        for t in range(T):
            x = q[b, t] if q_shared is None else torch.cat([q[b, t], q_shared[b, t]], 1)
            seen = (at <= n - T + t)[None, :].expand(H, -1)
            p, lse[b, t] = softmax_rows(scale * x @ c.T, seen)
            out[b, t] = p @ c[:, :Dl]
            rnd[b, t] = p @ c[:, :Dl].abs() + out[b, t].abs()
    return dict(out=out, lse=lse, out_round=rnd)


def verify(draft, target_probs, uniforms, draft_probs=None, num_drafts=None):
    """(tokens, num_accepted) as lists of ints, by the definition, a token at a time."""
    draft, p, u = np.asarray(draft), np.asarray(target_probs, np.float64), np.asarray(uniforms, np.float64)
    q = None if draft_probs is None else np.asarray(draft_probs, np.float64)
    B, T = draft.shape
    V = p.shape[2]
    tokens, kept = [], []
    for b in range(B):
        n = T if num_drafts is None else min(max(int(num_drafts[b]), 0), T)
        k = 0
        while k < n:
            x = int(draft[b, k])
            if not 0 <= x < V or not u[b, k] * (1.0 if q is None else q[b, k, x]) < p[b, k, x]:
                break
            k += 1
        w = p[b, k]
        if k < n:
            if q is not None:
                rest = np.maximum(w - q[b, k], 0.0)
            else:
                rest = w.copy()
                if 0 <= int(draft[b, k]) < V:
                    rest[int(draft[b, k])] = 0.0
            if rest.sum() > 0:
                w = rest
        cum = np.cumsum(w)
        past = np.nonzero(cum > u[b, T] * cum[-1])[0]
        heavy = np.nonzero(w > 0)[0]
        new = int(past[0]) if len(past) else int(heavy[-1]) if len(heavy) else -1
        tokens.append([int(t) for t in draft[b, :k]] + [new] + [-1] * (T - k))
        kept.append(k)
    return tokens, kept
