"""Edges of the layer's epilogue and of a quantized head's log probabilities:
output counts and token counts that split warps, rows whose activations the
integer kernels cannot hold, the activations' far tails, and calls without a
workspace.  Tolerances as derived in test_gpu_epilogue.py, or beside the test.
"""
import math

import pytest
import torch

import weight_only_quantized_02_b200 as wq
from test_gpu_epilogue import ACTS, check, make_weight, operands, ws_for
from wqtest_helpers import dev, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_table():
    wq.wq_clear_tuning()
    yield
    wq.wq_clear_tuning()
    wq.wq_set_workspace(None)


# ---------------------------------------------------------------------------
# warps whose lanes go different ways
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("with_ws", [True, False])
@pytest.mark.parametrize("bits,K", [(8, 160), (4, 256)])
@pytest.mark.parametrize("N,M", [(16, 131), (1040, 1003), (2224, 389), (48, 3001), (912, 207)])
def test_ragged_outputs_split_warps(bits, K, N, M, with_ws):
    """Output counts that end 16 channels into a panel and token counts that end
    inside a 16-token chunk: the lanes of a warp part at every chunk of every tile
    (several tiles a pair of SMs among them), and the tensor-memory loads behind
    them are the whole warp's."""
    pw, w = make_weight(bits, 128 if bits == 4 else 0, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    ws = ws_for(M, K, N) if with_ws else None
    for _ in range(2):
        y = wq.wq_linear_epilogue(x, pw, bias=bias, act=wq.WQ_ACT_SILU, mul=mul, residual=res, ws=ws)
        check(y, x, w, bias, "silu", mul, res, torch.bfloat16)
    x16, bias16, mul16, res16 = operands(M, K, N, torch.float16)
    y = wq.wq_linear_epilogue_f16(x16, pw, bias=bias16, act=wq.WQ_ACT_RELU, mul=mul16, residual=res16)
    check(y, x16, w, bias16, "relu", mul16, res16, torch.float16)
    assert wq.wq_device_error() == 0


@pytest.mark.parametrize("bits,K", [(8, 160), (4, 256)])
@pytest.mark.parametrize("N,M", [(16, 131), (1040, 203), (2224, 389), (912, 64), (656, 40)])
def test_ragged_head_splits_warps(bits, K, N, M):
    """The same where the logits go out in fp32: their log probabilities are those
    of binary64 logits."""
    pw, w = make_weight(bits, 128 if bits == 4 else 0, K, N)
    x = operands(M, K, N, torch.bfloat16, 0, False, False, False)[0] * 2
    t = torch.arange(M, dtype=torch.int32, device=dev()) % N
    scratch = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, N), dtype=torch.uint8, device=dev())
    lp, H, _, _ = wq.wq_linear_logprobs(x, pw, t, 0, scratch, ws=workspace(M, K, N, 8))
    x64 = x.double()
    logp = torch.log_softmax(x64 @ w.t(), 1)
    dv = float((K * 2.0 ** -23 * (x64.abs() @ w.abs().t()) +
                2.0 ** -22 * x64.abs().amax(1, keepdim=True) * w.abs().sum(1).unsqueeze(0)).max())
    ref = logp.gather(1, t.long().unsqueeze(1)).squeeze(1)
    assert float((lp.double() - ref).abs().max()) <= 2 * dv + 2.0 ** -17 + 2.0 ** -22 * float(ref.abs().max())
    rH = -(logp.exp() * logp).sum(1)
    assert float((H.double() - rH).abs().max()) <= 2 * dv * (1 + float(rH.max())) + 2.0 ** -17 * (2 + float(rH.max()))
    assert wq.wq_device_error() == 0
