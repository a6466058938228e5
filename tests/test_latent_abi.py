"""Argument checks of the latent-attention and verification calls on the host
(CPU only: nothing here reaches a CUDA runtime function)."""
import ctypes

import pytest
import torch

import gated_delta_rule_rda_b200 as rda

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
P = 1 << 20          # stands for a 256-byte aligned device address; never dereferenced
BIG = 1 << 40


def prefill(**kw):
    a = dict(q=P, qs=P, k=P, ks=P, v=P, cu_q=P, cu_k=P, n=2, tq=10, tk=10, out=P, lse=P, dt=1, H=4, Dk=128, Ds=64,
             Dv=128, scale=1.0, causal=1, ws=P, wsb=BIG, s=None)
    a.update(kw)
    return rda.lib.rda_latent_prefill(*a.values())


def backward(**kw):
    a = dict(q=P, qs=P, k=P, ks=P, v=P, out=P, lse=P, d_out=P, cu_q=P, cu_k=P, n=2, tq=10, tk=10, dq=P, dqs=P, dk=P,
             dks=P, dv=P, dt=1, H=4, Dk=128, Ds=64, Dv=128, scale=1.0, causal=1, ws=P, wsb=BIG, s=None)
    a.update(kw)
    return rda.lib.rda_latent_backward(*a.values())


def decode(**kw):
    a = dict(q=P, qs=P, pages=P, table=P, lens=P, out=P, lse=P, dt=1, B=2, T=1, H=4, Dl=512, Ds=64, np=8, ps=64, w=4,
             scale=1.0, ws=P, wsb=BIG, s=None)
    a.update(kw)
    return rda.lib.rda_latent_decode(*a.values())


def verify(**kw):
    a = dict(x=P, q=P, p=P, u=P, n=P, tok=P, acc=P, B=2, T=3, V=100, ws=P, wsb=BIG, s=None)
    a.update(kw)
    return rda.lib.rda_verify_drafts(*a.values())


@pytest.mark.parametrize("call", [prefill, backward])
def test_packed_refusals(call):
    assert call(dt=2) == UNSUPPORTED
    for kw in (dict(Dk=96), dict(Ds=32), dict(Dv=256), dict(H=1025)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(n=-1), dict(tq=-1), dict(tk=-1), dict(H=0), dict(q=None), dict(k=None), dict(v=None), dict(cu_q=None),
               dict(cu_k=None), dict(qs=None), dict(ks=None), dict(Ds=0), dict(tq=1 << 25, H=64), dict(out=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(q=P + 8), dict(qs=P + 2), dict(k=P + 4), dict(ks=P + 8), dict(v=P + 2), dict(out=P + 8),
               dict(lse=P + 2), dict(cu_q=P + 1), dict(cu_k=P + 2), dict(ws=P + 16)):
        assert call(**kw) == MISALIGNED, kw
    assert call(ws=None) == WORKSPACE and call(wsb=255) == WORKSPACE
    # nothing to do: nothing is launched
    assert call(n=0) == OK and call(tq=0, tk=0, q=None, qs=None, k=None, ks=None, v=None, out=None) == OK


def test_backward_refusals():
    for kw in (dict(dq=None), dict(dqs=None), dict(dk=None), dict(dks=None), dict(dv=None), dict(d_out=None), dict(lse=None)):
        assert backward(**kw) == INVALID, kw
    for name in ("dq", "dqs", "dk", "dks", "dv", "d_out"):
        assert backward(**{name: P + 8}) == MISALIGNED, name
    need = rda.rda_latent_backward_workspace_bytes(10, 10, 4, 128, 64, 128, 2)
    assert need >= 256 + 4 * 10 * 4 + 4 * 10 * 4 * 64 and backward(wsb=need - 1) == WORKSPACE


def test_decode_refusals():
    assert decode(dt=7) == UNSUPPORTED
    for kw in (dict(T=9), dict(B=65536), dict(Dl=64), dict(Dl=640), dict(Ds=32), dict(ps=24), dict(H=1025)):
        assert decode(**kw) == UNSUPPORTED, kw
    for kw in (dict(B=-1), dict(T=-1), dict(H=0), dict(np=-1), dict(ps=0), dict(w=-1), dict(q=None), dict(qs=None),
               dict(Ds=0), dict(lens=None), dict(out=None), dict(table=None), dict(pages=None),
               dict(np=1 << 26, ps=64), dict(w=1 << 26, ps=64), dict(B=60000, T=8, H=64)):
        assert decode(**kw) == INVALID, kw
    for kw in (dict(q=P + 8), dict(qs=P + 8), dict(pages=P + 8), dict(out=P + 4), dict(lse=P + 2), dict(table=P + 2),
               dict(lens=P + 1), dict(ws=P + 128)):
        assert decode(**kw) == MISALIGNED, kw
    assert decode(ws=None) == WORKSPACE
    assert decode(wsb=rda.rda_latent_decode_workspace_bytes(2, 1, 4, 512, 64) - 1) == WORKSPACE
    assert decode(B=0) == OK and decode(T=0) == OK


def test_verify_refusals():
    for kw in (dict(T=33), dict(B=65536)):
        assert verify(**kw) == UNSUPPORTED, kw
    for kw in (dict(B=-1), dict(T=-1), dict(V=0), dict(x=None), dict(p=None), dict(u=None), dict(tok=None), dict(acc=None)):
        assert verify(**kw) == INVALID, kw
    for name in ("x", "q", "p", "u", "n", "tok", "acc"):
        assert verify(**{name: P + 2}) == MISALIGNED, name
    assert verify(ws=None) == WORKSPACE and verify(wsb=256) == WORKSPACE and verify(B=0) == OK


def test_workspace_queries():
    assert rda.rda_latent_prefill_workspace_bytes(10, 10, 4, 128, 64, 128, 2) >= 256
    assert rda.rda_latent_prefill_workspace_bytes(10, 10, 4, 96, 64, 128, 2) == 0
    assert rda.rda_latent_backward_workspace_bytes(-1, 10, 4, 128, 64, 128, 2) == 0
    assert rda.rda_latent_decode_workspace_bytes(1, 9, 4, 512, 64) == 0
    assert rda.rda_latent_decode_workspace_bytes(0, 1, 4, 512, 64) >= 256
    assert rda.rda_verify_drafts_workspace_bytes(2, 3, 0) == 0
    assert rda.rda_verify_drafts_workspace_bytes(2, 33, 10) == 0
    assert rda.rda_verify_drafts_workspace_bytes(2, 3, 5000) >= 256 + 2 * 5 * 8


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        rda.rda_latent_prefill(x, x, x, torch.tensor([0, 4], dtype=torch.int32), scale=1.0)
    with pytest.raises(ValueError):
        rda.rda_verify_drafts(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2, 5), torch.zeros(1, 2))
    with pytest.raises(ValueError):
        rda.rda_latent_decode(torch.zeros(1, 1, 2, 128), torch.zeros(2, 16, 128), torch.zeros(1, 2, dtype=torch.int32),
                              torch.zeros(1, dtype=torch.int32), scale=1.0)


def test_sizes_that_pass_32_bits_are_refused():
    for call in (prefill, backward):
        assert call(n=(1 << 31) - 1) == INVALID and call(n=1 << 21, H=1024) == INVALID
    assert decode(w=(1 << 25) - 1, ps=64) == INVALID          # rounding the length up to tiles would pass 2^31
    assert decode(w=(1 << 31) - 1, ps=1 << 30) == INVALID
