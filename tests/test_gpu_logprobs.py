"""Log probabilities of given tokens, entropy and alternatives (wq_logprobs,
wq_linear_logprobs) against the definition in binary64.

Tolerances.  A log probability x - lse is off by the roundings of x - max,
of log S and of the difference (2^-23 of each), and by S's relative error: each
term's exponential 2^-21 (its argument's rounding, 2 2^-24 |x - max| times the
term's weight, stays below that), and some 60 additions on the way from a
thread's first term to the row's sum, 2^-24 each: under 2^-17 in all.  The
entropy has log S and W / S, whose relative error is S's and W's: under
2^-17 (2 + entropy).  Indices are exact.
"""
import math

import pytest
import torch

import weight_only_quantized_02_b200 as wq
from test_gpu_epilogue import make_weight
from wqtest_helpers import dev, workspace

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def reference(x, tokens, k):
    x = x.double()
    d = x - x.max(1, keepdim=True).values  # about the maximum: x itself swallows log S where it is 1e38
    logp = d - d.exp().sum(1, keepdim=True).log()
    p = logp.exp()
    H = -(p * torch.where(p > 0, logp, torch.zeros_like(logp))).sum(1)
    lp = None if tokens is None else logp.gather(1, tokens.long().clamp(0, x.shape[1] - 1).unsqueeze(1)).squeeze(1)
    idx = torch.argsort(-x, dim=1, stable=True)[:, :k]
    return lp, H, logp.gather(1, idx), idx.int()


def close(a, ref, scale):
    both_nan = a.isnan() & ref.isnan()
    same_inf = (a == ref.float()) & ref.float().isinf()  # past fp32's 3.4e38 the rounded answer is infinite
    ok = (a.double() - ref).abs() <= 2.0 ** -17 * scale + 2.0 ** -22 * ref.abs()
    assert bool((ok | both_nan | same_inf).all()), (a, ref)


def check(x, tokens, k, out):
    lp, H, top, idx = out
    rl, rH, rt, ri = reference(x, tokens, k)
    if tokens is None:
        assert lp is None
    else:
        close(lp, rl, 1.0)
    close(H, rH, 2 + rH.abs())
    if k == 0:
        assert top is None and idx is None
        return
    assert torch.equal(idx, ri)
    close(top, rt, 1.0)


def rows(M, N, dtype, seed=0, scale=2.5):
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = (torch.randn((M, N), generator=g, device=dev()) * scale).to(dtype)
    return x, torch.randint(0, N, (M,), generator=g, device=dev(), dtype=torch.int32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,k", [(1, 1, 1), (1, 1, 0), (3, 2, 2), (2, 7, 3), (5, 64, 64), (4, 65, 64), (2, 127, 5),
                                   (1, 1000, 20), (7, 4097, 33), (300, 513, 1), (1, 20011, 64), (2, 40000, 20),
                                   (3, 152064, 64), (1, 152064, 1), (9, 152063, 20), (40, 50001, 8),
                                   (700, 9000, 64), (1, 1 << 20, 64)])
def test_against_the_definition(dtype, M, N, k):
    x, t = rows(M, N, dtype, M + N + k)
    check(x, t, k, wq.wq_logprobs(x, t, k))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,pad", [(1, 0), (3, 2), (5, 8), (0, 1), (7, 13)])
@pytest.mark.parametrize("M,N", [(5, 1003), (1, 33000), (2, 8), (6, 20001)])
def test_strides_and_alignment(dtype, offset, pad, M, N):
    """Rows that start anywhere, with NaN all around them that must not be read into the answer."""
    x, t = rows(M, N, dtype, 3)
    buf = torch.full((M * (N + pad) + offset + 16,), math.nan, dtype=dtype, device=dev())
    view = buf[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    view.copy_(x)
    check(x, t, min(5, N), wq.wq_logprobs(view, t, min(5, N)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [64, 5000, 70001])
def test_order_of_the_row(dtype, N):
    """Rising, falling, constant and two-valued rows: bounds that pass everything, and ties."""
    ramp = torch.linspace(-20, 20, N, device=dev())
    x = torch.stack([ramp, ramp.flip(0), torch.zeros(N, device=dev()), (torch.arange(N, device=dev()) % 3 == 1).float(),
                     torch.full((N,), -torch.finfo(dtype).max, device=dev()),
                     torch.cat([ramp[: N // 2], ramp[: N - N // 2].flip(0)])]).to(dtype)
    t = torch.tensor([0, N - 1, N // 2, 1, 3, 2], dtype=torch.int32, device=dev())
    check(x, t, min(64, N), wq.wq_logprobs(x, t, min(64, N)))
    for r in range(x.shape[0]):  # one row alone: spread over a cluster
        check(x[r:r + 1], t[r:r + 1], 20, wq.wq_logprobs(x[r:r + 1], t[r:r + 1], 20))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(12, 3001), (1, 50001), (12, 200)])
def test_masked_rows(dtype, M, N):
    x, t = rows(M, N, dtype, 8)
    g = torch.Generator(device=dev()).manual_seed(4)
    x[torch.rand(x.shape, generator=g, device=dev()) < 0.95] = -math.inf
    t[0] = int(torch.nonzero(x[0] > -math.inf)[0])
    check(x, t, 64, wq.wq_logprobs(x, t, 64))  # fewer than 64 allowed in the short rows: -inf alternatives, lowest index first
    x[0] = -math.inf
    x[0, N - 1] = 0.0  # a single allowed token
    t[0] = N - 1
    lp, H, top, idx = wq.wq_logprobs(x, t, 2)
    assert float(lp[0]) == 0.0 and float(H[0]) == 0.0 and idx[0].tolist() == [N - 1, 0] and float(top[0, 1]) == -math.inf


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,k", [(9, 50001, 20), (1, 152064, 64), (3, 9000, 64)])
@pytest.mark.parametrize("mask", [-math.inf, "lowest"])
def test_fewer_logits_left_than_alternatives(dtype, M, N, k, mask):
    """Row m keeps m + 1 logits; the alternatives behind them are the first masked ones."""
    x, t = rows(M, N, dtype, 5)
    keep = torch.zeros((M, N), dtype=torch.bool, device=dev())
    for m in range(M):
        keep[m, (torch.arange(m + 1) * 7919 + 13 * m + 40) % N] = True
    x[~keep] = torch.finfo(dtype).min if mask == "lowest" else mask
    lp, H, top, idx = wq.wq_logprobs(x, t, k)
    rl, rH, rt, ri = reference(x, t, k)
    assert torch.equal(idx, ri)
    close(H, rH, 2 + rH.abs())
    same = (lp.double() == rl) | ((lp.double() - rl).abs() <= 2.0 ** -17 + 2.0 ** -22 * rl.abs())
    assert bool(same.all())
    same = (top.double() == rt) | ((top.double() - rt).abs() <= 2.0 ** -17 + 2.0 ** -22 * rt.abs()) | \
        (top.isinf() & (rt < -3.4e38))
    assert bool(same.all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,k", [(4, 50001, 64), (1, 152064, 20), (700, 12000, 5), (200, 40000, 33)])
@pytest.mark.parametrize("above", [3, 40, 1500, 6000])
def test_many_equal_logits_below_some(dtype, M, N, k, above):
    """Most logits equal, `above` of them (anywhere in the row) of a few larger
    values, one row of them all of one value: the k-th largest is the common value,
    among the larger ones, or one of many equal larger ones."""
    g = torch.Generator(device=dev()).manual_seed(above)
    x = torch.full((M, N), -2.0, device=dev())
    at = torch.randint(0, N, (M, above), generator=g, device=dev())
    x.scatter_(1, at, torch.randint(0, 4000, (M, above), generator=g, device=dev()).float() / 500)
    x[0].clamp_(max=-1.0)
    x = x.to(dtype)
    t = at[:, 0].int().contiguous()
    check(x, t, k, wq.wq_logprobs(x, t, k))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [100, 40000])
def test_rows_without_a_distribution(dtype, N):
    x, t = rows(5, N, dtype, 2)
    x[0] = -math.inf
    x[1, 7] = math.nan
    x[2, 9] = math.inf
    x[3, [11, 50]] = math.nan
    x[3, 20] = math.inf
    lp, H, top, idx = wq.wq_logprobs(x, t, 4)
    assert bool(lp[:4].isnan().all()) and bool(H[:4].isnan().all()) and bool(top[:4].isnan().all())
    assert idx[0].tolist() == [0, 1, 2, 3]
    assert int(idx[1, 0]) == 7 and int(idx[2, 0]) == 9 and idx[3, :3].tolist() == [11, 50, 20]
    check(x[4:], t[4:], 4, (lp[4:], H[4:], top[4:], idx[4:]))


def test_extreme_values():
    """Logits at the ends of fp32: differences that overflow are far below, not NaN."""
    x = torch.zeros(3, 5000, device=dev())
    x[0, ::2] = -3.4e38
    x[1] = -3.4e38
    x[1, 4] = 3.4e38
    x[2] = 1e30
    x[2, 1] = -0.0
    t = torch.tensor([1, 4, 0], dtype=torch.int32, device=dev())
    check(x, t, 3, wq.wq_logprobs(x, t, 3))


@pytest.mark.parametrize("dtype", DTYPES)
def test_maxima_far_from_zero(dtype):
    """Maxima so large that 200 below them is the same 16-bit value, and so low
    that nothing but -inf is below them."""
    big, low = (6e4, -65504.0) if dtype == torch.float16 else (1e30, torch.finfo(dtype).min)
    x = torch.zeros(6, 9000, dtype=dtype, device=dev())
    x[0, 5] = big
    x[1] = -math.inf
    x[1, ::3] = low
    x[2] = -big
    x[2, 7] = -0.9 * big
    x[3] = torch.linspace(1000, 1100, 9000, device=dev()).to(dtype)
    x[4] = torch.linspace(-1100, -1000, 9000, device=dev()).to(dtype)
    x[5] = low
    x[5, 8000] = 0.97 * low
    t = torch.tensor([5, 3, 7, 8999, 8999, 8000], dtype=torch.int32, device=dev())
    check(x, t, 5, wq.wq_logprobs(x, t, 5))


def test_zeros_of_both_signs_are_equal():
    x = torch.full((1, 300), -1.0, device=dev())
    x[0, 5], x[0, 9], x[0, 200] = -0.0, 0.0, -0.0
    assert wq.wq_logprobs(x, None, 3)[3][0].tolist() == [5, 9, 200]


def test_tokens_outside_the_row_have_no_log_probability():
    x, _ = rows(4, 900, torch.bfloat16)
    t = torch.tensor([-1, 900, 3, -100], dtype=torch.int32, device=dev())
    lp, H, _, _ = wq.wq_logprobs(x, t)
    assert lp.isnan().tolist() == [True, True, False, True] and not bool(H.isnan().any())


def test_without_tokens_and_repeatable():
    x, t = rows(20, 30000, torch.bfloat16, 5)
    a = wq.wq_logprobs(x, None, 8)
    assert a[0] is None
    first = wq.wq_logprobs(x, t, 8)
    for _ in range(5):
        again = wq.wq_logprobs(x, t, 8)
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_rows_behind_the_last_stay():
    """Outputs given through the C entry: what lies behind the last row is left alone."""
    x, t = rows(3, 700, torch.bfloat16)
    lp = torch.full((5,), 9.0, device=dev())
    top = torch.full((5, 4), 9.0, device=dev())
    idx = torch.full((5, 4), 9, dtype=torch.int32, device=dev())
    rc = wq.lib.wq_logprobs(x.data_ptr(), 0, 3, 700, 700, t.data_ptr(), 4, lp.data_ptr(), None, top.data_ptr(),
                            idx.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert lp[3:].tolist() == [9.0, 9.0] and bool((top[3:] == 9.0).all()) and bool((idx[3:] == 9).all())
    assert bool((lp[:3] < 0).all())


def test_large_offsets():
    """A row that starts past 2^31 elements."""
    N, ld = 1001, 1 << 20
    M = (1 << 31) // ld + 3
    x = torch.empty((M, ld), dtype=torch.bfloat16, device=dev())
    r, t = rows(M, N, torch.bfloat16, 1)
    x[:, :N] = r
    check(r, t, 3, wq.wq_logprobs(x[:, :N], t, 3))


def test_other_stream_and_graph():
    x, t = rows(33, 12345, torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = wq.wq_logprobs(x, t, 5, stream=s)
    s.synchronize()
    check(x, t, 5, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = wq.wq_logprobs(x, t, 5)
    for i in range(3):
        y, u = rows(33, 12345, torch.bfloat16, 50 + i)
        x.copy_(y)
        t.copy_(u)
        g.replay()
        torch.cuda.synchronize()
        check(y, u, 5, out)


# ---------------------------------------------------------------------------
# from the activations of a quantized head
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bits,group", [(8, 0), (4, 128), (4, 64)])
@pytest.mark.parametrize("M", [1, 4, 16, 40, 100, 200, 600])
def test_head(bits, group, M):
    K, N, k = 512, 2064, 8
    pw, w = make_weight(bits, group, K, N)
    g = torch.Generator(device=dev()).manual_seed(M)
    x = (torch.randn((M, K), generator=g, device=dev()) * 2.5).bfloat16()
    t = torch.randint(0, N, (M,), generator=g, device=dev(), dtype=torch.int32)
    scratch = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, N), dtype=torch.uint8, device=dev())
    lp, H, top, idx = wq.wq_linear_logprobs(x, pw, t, k, scratch, ws=workspace(M, K, N, 1))
    x64 = x.double()
    logits = x64 @ w.t()
    # the logits' own error (see the epilogue's tests), no rounding to 16 bits
    dv = float((K * 2.0 ** -23 * (x64.abs() @ w.abs().t()) +
                2.0 ** -22 * x64.abs().amax(1, keepdim=True) * w.abs().sum(1).unsqueeze(0)).max())
    rl, rH, rt, _ = reference(logits, t, k)
    assert float((lp.double() - rl).abs().max()) <= 2 * dv + 2.0 ** -17 + 2.0 ** -22 * float(rl.abs().max())
    # dH = -sum p (log p + H) dx: at most dv sum p |log p + H| <= 2 dv (1 + H)
    assert float((H.double() - rH).abs().max()) <= 2 * dv * (1 + float(rH.max())) + 2.0 ** -17 * (2 + float(rH.max()))
    assert float((top.double() - rt).abs().max()) <= 3 * dv + 2.0 ** -17 + 2.0 ** -22 * float(rt.abs().max())
    # every alternative's log probability is its index's
    at = (logits - torch.logsumexp(logits, 1, keepdim=True)).gather(1, idx.long())
    assert float((top.double() - at).abs().max()) <= 2 * dv + 2.0 ** -17 + 2.0 ** -22 * float(rt.abs().max())
    assert wq.wq_device_error() == 0
