"""The device-side timeout of the latent-attention kernels, made to run out on purpose through the test-only
fault injection: some tiles are never filled and waits are bounded at 20 ms.  Each kernel records
RDA_ERR_TIMEOUT and returns; the context stays usable, and the next call has the same bits as before."""
import pytest
import torch

import gated_delta_rule_rda_b200 as rda
from latent_util import packed, paged

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def off():
    yield
    rda.rda_debug_set_wait_fault()


def _calls():
    x = {n: t.cuda() if isinstance(t, torch.Tensor) else t
         for n, t in packed([500, 70], [500, 300], 2, 128, 64, 128, BF16, seed=1).items()}
    d = {n: t.cuda() if isinstance(t, torch.Tensor) else t
         for n, t in paged([40000, 90], 2, 16, 512, 64, 64, BF16, seed=2).items()}
    shared = dict(scale=x["scale"], q_shared=x["q_shared"], k_shared=x["k_shared"])
    out, lse = rda.rda_latent_prefill(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], return_lse=True, **shared)

    def prefill(ws):
        return rda.rda_latent_prefill(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], return_lse=True, workspace=ws, **shared)

    def backward(ws):
        g = rda.rda_latent_backward(x["q"], x["k"], x["v"], out, lse, x["d_out"], x["cu_q"], x["cu_k"], workspace=ws, **shared)
        return [g[n] for n in sorted(g)]

    def decode(ws):
        return rda.rda_latent_decode(d["q"], d["pages"], d["table"], d["lens"], scale=d["scale"], q_shared=d["q_shared"],
                                     return_lse=True, workspace=ws)

    return dict(prefill=prefill, backward=backward, decode=decode)


@pytest.mark.parametrize("tile", [0, 1, 3])
@pytest.mark.parametrize("name", ["prefill", "backward", "decode"])
def test_wait_runs_out_and_context_stays_usable(cuda_device, name, tile):
    call = _calls()[name]
    ws = rda.new_workspace(1 << 26, "cuda")
    ref = [t.clone() for t in call(ws)]
    assert rda.rda_read_device_error(ws) == 0
    rda.rda_debug_set_wait_fault(drop_chunk=tile, wait_limit_ns=20_000_000)
    call(ws)
    torch.cuda.synchronize()
    rda.rda_debug_set_wait_fault()
    assert rda.rda_read_device_error(ws) == 6
    again = call(ws)
    torch.cuda.synchronize()
    assert rda.rda_read_device_error(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(ref, again))
