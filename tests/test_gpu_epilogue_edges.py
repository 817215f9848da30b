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


def unit_of(x):
    """The integer kernels' unit of every row (include/wq.h), binary64 [M][1]."""
    E = torch.floor(torch.log2(x.double().abs().amax(1, keepdim=True)))
    return torch.exp2(-torch.clamp(21 - E, max=127))


def needs_more(x):
    """Rows that the integer kernels' form does not hold well enough as it is: R, what rounding
    to their units leaves over, is above max(4, K / 1024), or the unit is held at 2^-127."""
    q = x.double() / unit_of(x)
    R = (q - torch.round(q)).abs().sum(1)
    return (R > max(4, x.shape[1] // 1024)) | (unit_of(x)[:, 0] <= 2.0 ** -127)


def group_sum_rounding(x, w, group=128):
    """What INT4's fp32 sums over the groups may lose.  Every partial sum of a kernel is
    within B = sum_i 256^i S_i units, S_i twice the largest prefix sum over the groups of
    the i-th digits' products; it makes at most three roundings a group (two to
    put the digits together, one to scale and add) and one for each of at most G
    contributors, 2^-24 B each."""
    M, K = x.shape
    N, G = w.shape[0], K // group
    X = torch.round(x.double() / unit_of(x))
    B = torch.zeros((M, N), dtype=torch.float64, device=x.device)
    for i in range(3):
        d = torch.remainder(X + 128, 256) - 128
        X = (X - d) / 256
        t = torch.einsum("mgk,ngk->mng", d.view(M, G, group), w.view(N, G, group))
        B += 256.0 ** i * 2 * t.cumsum(2).abs().amax(2)
    return (4 * G + 8) * 2.0 ** -24 * B * unit_of(x)


def check_fp32_logits(x, pw, w, bits, variant, ws_bytes=None):
    """The logits that wq_linear_logprobs leaves in its scratch, against binary64:
    2^-21 of their values (rows accepted whole: as many units of their largest as the
    header allows), the rounding to fp32, and INT4's group sums."""
    M, K = x.shape
    N = w.shape[0]
    wq.wq_set_choice(M, K, N, bits, 128 if bits == 4 else 0, variant, 1)
    scratch = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, N), dtype=torch.uint8, device=dev())
    ws = workspace(M, K, N, 8)
    if ws_bytes is not None:
        ws = ws[:ws_bytes]
    t = torch.arange(M, dtype=torch.int32, device=dev())
    v = x.double() @ w.t()
    tol = (2.0 ** -21 + 2.0 ** -23) * v.abs() + 2.0 ** -149
    # w's bound: 128 s where the codes reach 127 s, 8 s of 7.5 s at least
    wmax = w.abs().amax(1) * 1.02 if bits == 8 else w.abs().max() * 1.1
    tol = tol + (~needs_more(x)).double().unsqueeze(1) * max(4, K // 1024) * unit_of(x) * wmax
    if bits == 4:
        tol = tol + group_sum_rounding(x, w) * 1.01
    first = None
    for tokens, k in ((None, min(64, N)), (t, 0), (t, 3)):  # the flags' place differs
        out = wq.wq_linear_logprobs(x, pw, tokens, k, scratch, ws=ws)
        logits = scratch.view(torch.float32).view(M, N)
        bad = ~((logits.double() - v).abs() <= tol)
        assert not bad.any(), float(((logits.double() - v).abs() / tol).max())
        first = logits.clone() if first is None else first
        assert torch.equal(logits, first)
        logp = torch.log_softmax(first.double(), 1)
        if tokens is not None:
            assert float((out[0].double() - logp.gather(1, t.long().unsqueeze(1)).squeeze(1)).abs().max()) <= 2.0 ** -16
        assert float((out[1].double() + (logp.exp() * logp).sum(1)).abs().max()) <= 2.0 ** -17 * 12
    assert int(ws[:262912].max()) == 0  # every counter back at zero
    assert wq.wq_device_error() == 0


@pytest.mark.parametrize("bits,variant,M,K,outlier", [(8, 5, 1, 5120, 10), (8, 5, 5, 5120, 10), (8, 5, 5, 5120, 13),
                                                      (8, 4, 16, 5120, 10), (8, 4, 40, 5120, 10), (8, 4, 64, 1056, 20),
                                                      (4, 5, 3, 512, 11), (4, 5, 8, 512, 11), (4, 4, 9, 512, 11),
                                                      (4, 4, 32, 512, 11), (4, 4, 1, 512, 14)])
def test_fp32_logits_of_outlier_rows(bits, variant, M, K, outlier):
    """The head's logits are off by 2^-21 of their values at most in rows that the
    fixed point form cannot hold, in whichever kernel."""
    pw, w, x = outlier_case(bits, M, K, 1040, 2.0 ** outlier)
    if M > 2:
        x[1, 5] = 1.0  # a row that is accepted whole, among the others
    assert needs_more(x).tolist() == [m != 1 or M <= 2 for m in range(M)]
    check_fp32_logits(x, pw, w, bits, variant)


def test_fp32_logits_without_room_for_a_second_pass():
    """A workspace that holds the integer GEMV's partial sums and no more: its
    outputs are recomputed one by one."""
    pw, w, x = outlier_case(8, 2, 512, 1040, 2.0 ** 12)
    assert bool(needs_more(x).all())
    check_fp32_logits(x, pw, w, 8, 5, 262912 + 448 * 8 * 2 * 16 * 8 * 4)


@pytest.mark.parametrize("bits,variant,M,k", [(8, 5, 3, 3), (8, 4, 20, 64), (4, 4, 9, 7)])
def test_second_pass_with_alternatives_alone(bits, variant, M, k):
    """Neither tokens nor entropy asked for: the rows' flags stand among the alternatives."""
    K, N = 512, 1040
    pw, w, x = outlier_case(bits, M, K, N, 2.0 ** 12)
    x[1, 5] = 1.0
    wq.wq_set_choice(M, K, N, bits, pw.group, variant, 1)
    nbytes = wq.wq_linear_logprobs_workspace_bytes(M, N)
    scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev())
    ws = workspace(M, K, N, 8)
    want = wq.wq_linear_logprobs(x, pw, None, k, scratch, ws=ws)
    logits = scratch.view(torch.float32).view(M, N).clone()
    scratch.zero_()
    top = torch.full((M + 1, k), 7.0, device=dev())
    idx = torch.full((M + 1, k), 7, dtype=torch.int32, device=dev())
    zeros = None if pw.zeros is None else pw.zeros.data_ptr()
    rc = wq.lib.wq_linear_logprobs(x.data_ptr(), M, K, pw.wq.data_ptr(), pw.scales.data_ptr(), zeros, pw.group, N, None,
                                   k, None, None, top.data_ptr(), idx.data_ptr(), scratch.data_ptr(), nbytes,
                                   ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(scratch.view(torch.float32).view(M, N), logits)
    assert torch.equal(top[:M], want[2]) and torch.equal(idx[:M], want[3])
    assert bool((top[M] == 7).all()) and bool((idx[M] == 7).all())


def test_second_pass_in_a_graph():
    """Captured once, replayed with rows that need the second pass and rows that do not."""
    K, N, M = 1024, 1040, 4
    pw, w, x = outlier_case(8, M, K, N, 2.0 ** 12)
    scratch = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, N), dtype=torch.uint8, device=dev())
    ws = workspace(M, K, N, 8)
    t = torch.arange(M, dtype=torch.int32, device=dev())
    plain = x.clone()
    plain[:, 5] = 0.5
    want = [[o.clone() for o in wq.wq_linear_logprobs(v, pw, t, 5, scratch, ws=ws)] for v in (x, plain)]
    held = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = wq.wq_linear_logprobs(held, pw, t, 5, scratch, ws=ws)
    torch.cuda.synchronize()
    for i in (1, 0, 0, 1, 0):
        held.copy_((x, plain)[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    assert int(ws[:262912].max()) == 0


def test_a_row_does_not_depend_on_the_others():
    """A row's logits are the same bits beside rows that need the second pass."""
    K, N, M = 1024, 1040, 9
    pw, w, x = outlier_case(8, M, K, N, 2.0 ** 12)
    x[::2, 5] = 0.5
    wq.wq_set_choice(M, K, N, 8, 0, 4, 1)
    scratch = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, N), dtype=torch.uint8, device=dev())
    ws = workspace(M, K, N, 8)
    wq.wq_linear_logprobs(x, pw, None, 1, scratch, ws=ws)
    both = scratch.view(torch.float32).view(M, N).clone()
    x[1::2, 5] = 0.5
    wq.wq_linear_logprobs(x, pw, None, 1, scratch, ws=ws)
    assert torch.equal(scratch.view(torch.float32).view(M, N)[::2], both[::2])


@pytest.mark.parametrize("bits,variant,M", [(8, 5, 1), (8, 5, 5), (8, 4, 16), (4, 5, 3), (4, 4, 9)])
def test_multiplied_outputs_of_outlier_rows(bits, variant, M):
    """An error of the sum that is accepted for its own size is multiplied with
    the sum: y is off by 2^-9 of the product and its own rounding, however small
    the sum."""
    K, N = 5120, 2064
    pw, w, x = outlier_case(bits, M, K, N, 2.0 ** 10, 1)
    assert bool(needs_more(x).all())
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
    K, N = 512, 400
    pw, w = make_weight(bits, 128 if bits == 4 else 0, K, N)
    x = (operands(M, K, N, torch.float32, 2, False, False, False)[0] * 2.0 ** -118).bfloat16()
    check_fp32_logits(x, pw, w, bits, variant)


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


# ---------------------------------------------------------------------------
# the activations' far tails
# ---------------------------------------------------------------------------

def activation64(v, act):
    """The formulas in binary64, and the relative error of the kernels' evaluation: erf
    GELU (2 + 1.4 a^2) 2^-22 at a = |v| / sqrt 2, whose own relative error of 0.36 2^-22
    counts 2 a^2 = v^2 times, with two more products below (4 + 1.1 v^2) 2^-22; the
    logistic forms' exponential (1 + 0.58 |u|) 2^-22, its sum, quotient and products,
    and for tanh the five roundings of u, 1.25 2^-22 of |u|, below (4 + 2 |u|) 2^-22."""
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2)), (4 + 1.1 * v * v) * 2.0 ** -22
    u = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    return v * torch.sigmoid(u), (4 + 2 * u.abs()) * 2.0 ** -22


@pytest.mark.parametrize("act,far", [("gelu", 12.5), ("gelu_tanh", 8.5), ("silu", 92.0)])
@pytest.mark.parametrize("bits,group,M,dtype", [(8, 0, 2, torch.bfloat16), (8, 0, 150, torch.bfloat16), (4, 128, 40, torch.bfloat16),
                                                (4, 64, 3, torch.bfloat16), (8, 0, 9, torch.float16), (4, 32, 3, torch.float16)])
def test_activations_keep_their_relative_accuracy(bits, group, M, dtype, act, far):
    """Through zero and both tails, as long as the answer is a normal number of the
    output's type: no error but the evaluation's, relative to the answer itself, and
    its one rounding."""
    K, N = 128, 4096
    pw, _ = make_weight(bits, group, K, N)
    x = torch.zeros((M, K), dtype=dtype, device=dev())
    bias = torch.cat([torch.linspace(-far, far, N - 1024, device=dev()),
                      torch.logspace(-3, math.log10(far), 1024, device=dev()) * -1]).to(dtype)
    if dtype == torch.bfloat16:
        y = wq.wq_linear_epilogue(x, pw, bias=bias, act=ACTS[act], ws=ws_for(M, K, N))
    else:
        y = wq.wq_linear_epilogue_f16(x, pw, bias=bias, act=ACTS[act])
    ref, rel = activation64(bias.double(), act)
    half = torch.finfo(dtype).eps / 2
    normal = ref.abs() >= torch.finfo(dtype).smallest_normal * (1 + 2 * half)
    tol = torch.where(normal, (rel + half * (1 + rel)) * ref.abs(), torch.finfo(dtype).smallest_normal * (1 + half))
    assert bool((y.double() - ref <= tol).all()) and bool((ref - y.double() <= tol).all())
    assert int(((bias < 0) & normal).sum()) > 900


# ---------------------------------------------------------------------------
# calls without a workspace
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bits,M,K,N", [(8, 9, 4096, 272), (8, 16, 8192, 144), (8, 32, 2048, 1040), (4, 9, 4096, 272),
                                        (4, 32, 8192, 144), (8, 8, 4096, 272)])
def test_long_k_and_few_channels_without_a_workspace(bits, M, K, N):
    """Few tiles and nowhere to put partial sums: the row-block GEMV, which uses every SM, by
    its bits (fp32 logits, so that another order of the sums would show); with a
    workspace, and with a kernel chosen, the call is as before."""
    group = 128 if bits == 4 else 0
    pw, w = make_weight(bits, group, K, N)
    x, bias, _, _ = operands(M, K, N, torch.bfloat16, 0, True, False, False)
    scratch = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, N), dtype=torch.uint8, device=dev())

    def logits(ws=None):
        wq.wq_linear_logprobs(x, pw, None, 1, scratch, ws=ws)
        return scratch.view(torch.float32).view(M, N).clone()

    auto = logits()
    by_split = []
    for split in (1, 2, 4, 8):
        wq.wq_set_choice(M, K, N, bits, group, wq.WQ_VARIANT_GEMV_RB, split)
        by_split.append(torch.equal(auto, logits()))
    assert any(by_split)
    wq.wq_set_choice(M, K, N, bits, group, wq.WQ_VARIANT_GEMM, 1)
    assert not torch.equal(auto, logits())
    wq.wq_clear_tuning()
    assert not torch.equal(auto, logits(workspace(M, K, N, 8)))
    y = wq.wq_linear_epilogue(x, pw, bias=bias)
    check(y, x, w, bias, "none", None, None, torch.bfloat16)
    assert wq.wq_device_error() == 0
