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


# ---------------------------------------------------------------------------
# rows with an element far above the others
# ---------------------------------------------------------------------------

def zero_channel_weight(bits, K, N, channel):
    """(packed weight, dequantized binary64 [N][K]) with w[:, channel] = 0; INT4 of
    groups of 128 with zero points of 8."""
    g = torch.Generator(device=dev()).manual_seed(11)
    if bits == 8:
        q = torch.randint(-127, 128, (N, K), generator=g, device=dev(), dtype=torch.int8)
        q[:, channel] = 0
        s = ((0.5 + torch.rand(N, generator=g, device=dev())) / (73 * math.sqrt(K))).bfloat16()
        return wq.wq_pack_int8(q, s.view(torch.int16)), q.double() * s.double().unsqueeze(1)
    q = torch.randint(0, 16, (N, K), generator=g, device=dev(), dtype=torch.int32)
    q[:, channel] = 8
    G = K // 128
    s = ((0.5 + torch.rand((N, G), generator=g, device=dev())) / (5 * math.sqrt(K))).bfloat16()
    words = sum(q[:, j::8] << (4 * j) for j in range(8)).to(torch.int32)
    zeros = torch.full((N, -(-G // 8)), -0x77777778, dtype=torch.int32, device=dev())  # 0x88888888
    w = (q - 8).double().view(N, G, 128) * s.double().unsqueeze(2)
    return wq.wq_pack_int4(words.contiguous(), s.view(torch.int16), zeros, 128), w.view(N, K)


def outlier_case(bits, M, K, N, outlier, seed=0):
    """A weight whose channel 5 is 0 in every row, N(0, 1) activations with an
    outlier there: no output sees the outlier, and the fixed point form of the
    integer kernels has its unit all the same."""
    pw, w = zero_channel_weight(bits, K, N, 5)
    x = operands(M, K, N, torch.bfloat16, seed, False, False, False)[0]
    x[:, 5] = outlier
    return pw, w, x


def rounded_sum(x):
    """R: the row sums of what rounding to the integer kernels' units leaves over, in units."""
    x = x.double()
    unit = torch.exp2(torch.floor(torch.log2(x.abs().amax(1, keepdim=True))) - 21)
    return (x / unit - torch.round(x / unit)).abs().sum(1)


@pytest.mark.parametrize("bits,variant,M", [(8, 5, 1), (8, 5, 5), (8, 4, 16), (4, 5, 3), (4, 4, 9), (8, 4, 40)])
def test_fp32_logits_of_outlier_rows(bits, variant, M):
    """The head's logits are off by 2^-21 of their values at most in rows that the
    fixed point form cannot hold, as sums in fp32 would be."""
    K, N, k = 5120, 1040, 64
    pw, w, x = outlier_case(bits, M, K, N, 2.0 ** 10)
    assert float(rounded_sum(x).min()) > max(4, K // 1024)
    wq.wq_set_choice(M, K, N, bits, 128 if bits == 4 else 0, variant, 1)
    scratch = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, N), dtype=torch.uint8, device=dev())
    wq.wq_linear_logprobs(x, pw, None, k, scratch, ws=workspace(M, K, N, 8))
    v = x.double() @ w.t()
    logits = scratch.view(torch.float32).view(M, N).double()
    # the rounding to fp32 is 2^-24 of the value; INT4's group sums are added in
    # fp32 where the guard accepted them, which it does for none of these rows
    tol = (2.0 ** -21 + 2.0 ** -23) * v.abs() + 2.0 ** -40
    assert bool(((logits - v).abs() <= tol).all()), float(((logits - v).abs() / tol).max())
    assert wq.wq_device_error() == 0


@pytest.mark.parametrize("bits,variant,M", [(8, 5, 1), (8, 5, 5), (8, 4, 16), (4, 5, 3), (4, 4, 9)])
def test_multiplied_outputs_of_outlier_rows(bits, variant, M):
    """An error of the sum that is accepted for its own size is multiplied with
    the sum: y is off by 2^-9 of the product and its own rounding, however small
    the sum."""
    K, N = 5120, 2064
    pw, w, x = outlier_case(bits, M, K, N, 2.0 ** 10, 1)
    assert float(rounded_sum(x).min()) > max(4, K // 1024)
    mul = operands(M, K, N, torch.bfloat16, 1, False, True, False)[2] * 2.0 ** 12
    wq.wq_set_choice(M, K, N, bits, 128 if bits == 4 else 0, variant, 1)
    y = wq.wq_linear_epilogue(x, pw, mul=mul, ws=ws_for(M, K, N))
    ref = (x.double() @ w.t()) * mul.double()
    # 2^-9 of the accepted sum, 2^-23 for fp32's sum and product, then bf16's half step of 2^-8
    tol = (2.0 ** -9 + 2.0 ** -23) * ref.abs() + 2.0 ** -8 * (1 + 2.0 ** -8) * ref.abs() + 1e-30
    assert bool(((y.double() - ref).abs() <= tol).all()), float(((y.double() - ref).abs() / tol).max())
    assert wq.wq_device_error() == 0


@pytest.mark.parametrize("bits,variant,M", [(8, 5, 3), (8, 4, 16), (4, 5, 3), (4, 4, 9)])
def test_fp32_logits_of_tiny_rows(bits, variant, M):
    """Rows around 2^-116, whose unit is held at 2^-127 (10 bits below the largest)."""
    K, N, k = 512, 400, 20
    pw, w = make_weight(bits, 128 if bits == 4 else 0, K, N)
    x = (operands(M, K, N, torch.float32, 2, False, False, False)[0] * 2.0 ** -118).bfloat16()
    wq.wq_set_choice(M, K, N, bits, 128 if bits == 4 else 0, variant, 1)
    scratch = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, N), dtype=torch.uint8, device=dev())
    wq.wq_linear_logprobs(x, pw, None, k, scratch, ws=workspace(M, K, N, 8))
    v = x.double() @ w.t()
    logits = scratch.view(torch.float32).view(M, N).double()
    # as above; fp32's own roundings of values around 2^-120 are its subnormals' step, 2^-149
    tol = (2.0 ** -21 + 2.0 ** -23) * v.abs() + 2.0 ** -149
    assert bool(((logits - v).abs() <= tol).all()), float(((logits - v).abs() / tol).max())


# ---------------------------------------------------------------------------
# activations that are not finite
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bits,variant,split,M", [(8, 0, 3, 5), (8, 2, 4, 5), (8, 4, 1, 5), (8, 4, 1, 40), (8, 5, 1, 5),
                                                  (8, 5, 2, 3), (8, None, 0, 200), (4, 0, 3, 5), (4, 2, 4, 5),
                                                  (4, 4, 1, 20), (4, 5, 1, 5), (4, 6, 1, 40), (4, None, 0, 200)])
def test_infinities_and_nan_in_a_row(bits, variant, split, M):
    """A token with a NaN or an infinity has the outputs of binary64 arithmetic: NaN,
    or an infinity of the weight's sign.  The other tokens' outputs are as without it."""
    K, N = 640, 272
    group = 128 if bits == 4 else 0
    pw, w = make_weight(bits, group, K, N)
    x, bias, _, res = operands(M, K, N, torch.bfloat16, 0, True, False, True)
    if variant is not None:
        wq.wq_set_choice(M, K, N, bits, group, variant, split)
    clean = wq.wq_linear_epilogue(x, pw, bias=bias, residual=res, ws=ws_for(M, K, N))
    check(clean, x, w, bias, "none", None, res, torch.bfloat16)
    x[0, 3] = math.nan
    x[1, 600] = math.inf
    x[2, 0] = -math.inf
    y = wq.wq_linear_epilogue(x, pw, bias=bias, residual=res, ws=ws_for(M, K, N))
    assert torch.equal(y[3:], clean[3:])
    assert bool(y[0].isnan().all())
    for m, k, sign in ((1, 600, 1), (2, 0, -1)):
        want = sign * torch.sign(w[:, k]) * math.inf  # 0 * inf: NaN
        assert torch.equal(y[m].double().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
    scratch = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, N), dtype=torch.uint8, device=dev())
    lp, H, top, _ = wq.wq_linear_logprobs(x, pw, torch.zeros(M, dtype=torch.int32, device=dev()), 3, scratch,
                                          ws=workspace(M, K, N, 8))
    assert bool(lp[:3].isnan().all()) and bool(H[:3].isnan().all()) and bool(top[:3].isnan().all())
    assert bool(lp[3:].isfinite().all()) and bool(H[3:].isfinite().all()) and bool(top[3:].isfinite().all())
    assert wq.wq_device_error() == 0
