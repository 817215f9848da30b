"""The layer with its epilogue (wq_linear_epilogue, wq_linear_epilogue_f16)
against the same formula in binary64:

    y = act(x . W^T + bias) * mul + residual

on every kernel the dispatcher can pick (forced through the dispatcher table),
both weight formats, every INT4 group, token counts from one to a ragged
prompt, ragged output counts, strided and aliased operands, other streams and
captured graphs.

Tolerance.  With a = sum_k |x w| and A = max|x|, the kernels' sum v is off by
at most K 2^-23 a (fp32 accumulation in any order, one rounding of 2^-24
relative per product and per sum, doubled for the tensor cores' truncating
adders) plus 2^-22 A sum_k |w| (the integer kernels' activations are integers
of 22 bits below the row's largest).  An activation's slope is at most 1.13;
its own evaluation is off by at most (4 + v^2) 2^-22 of its value (a few
roundings, and erfc's or exp's argument rounded at 2^-24 relative).  The
output's rounding is eps / 2 of its value, and the epilogue's fp32 product and
sum 2^-23 of theirs.
"""
import math

import numpy as np
import pytest
import torch

import weight_only_quantized_02_b200 as wq
from wqtest_helpers import dev, pack_canonical_int8, to_dev, workspace

pytestmark = pytest.mark.gpu

ACTS = {"none": wq.WQ_ACT_NONE, "relu": wq.WQ_ACT_RELU, "gelu": wq.WQ_ACT_GELU, "gelu_tanh": wq.WQ_ACT_GELU_TANH,
        "silu": wq.WQ_ACT_SILU}


def make_weight(bits, group, K, N, seed=0):
    """(packed weight, dequantized binary64 [N][K] on the device) from random canonical codes."""
    rng = np.random.default_rng(seed)
    if bits == 8:
        q = rng.integers(-127, 128, (N, K), dtype=np.int8)
        s = (rng.uniform(0.5, 1.5, N) / (73 * math.sqrt(K))).astype(np.float32)
        sb = torch.from_numpy(s).bfloat16()
        pw = pack_canonical_int8(q, sb.view(torch.int16).numpy())
        return pw, to_dev(q).double() * sb.double().to(dev()).unsqueeze(1)
    G = K // group
    q = rng.integers(0, 16, (N, K), dtype=np.uint8)
    z = rng.integers(0, 16, (N, G), dtype=np.uint8)
    sb = torch.from_numpy((rng.uniform(0.5, 1.5, (N, G)) / (6 * math.sqrt(K))).astype(np.float32)).bfloat16()

    def words(v):
        v = np.pad(v, ((0, 0), (0, -v.shape[1] % 8))).astype(np.uint32)
        w = np.zeros((N, v.shape[1] // 8), np.uint32)
        for j in range(8):
            w |= v[:, j::8] << np.uint32(4 * j)
        return w
    pw = wq.wq_pack_int4(to_dev(words(q)), to_dev(sb.view(torch.int16).numpy()), to_dev(words(z)), group)
    w = (to_dev(q).double().view(N, G, group) - to_dev(z).double().unsqueeze(2)) * sb.double().to(dev()).unsqueeze(2)
    return pw, w.view(N, K)


def operands(M, K, N, dtype, seed=0, bias=True, mul=True, residual=True):
    g = torch.Generator(device=dev()).manual_seed(1000 + seed)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev()).to(dtype)  # noqa: E731
    return (rnd(M, K), rnd(N) if bias else None, rnd(M, N) if mul else None, rnd(M, N) if residual else None)


def act64(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "silu":
        return v * torch.sigmoid(v)
    return v


def check(y, x, w, bias, act, mul, residual, dtype):
    x64 = x.double()
    v = x64 @ w.t()
    K = x.shape[1]
    dv = K * 2.0 ** -23 * (x64.abs() @ w.abs().t()) + \
        2.0 ** -22 * x64.abs().amax(1, keepdim=True) * w.abs().sum(1).unsqueeze(0)
    if bias is not None:
        v = v + bias.double()
    a = act64(v, act)
    da = dv if act == "none" else 1.13 * dv + (4 + v * v) * 2.0 ** -22 * a.abs()
    da = da + 2.0 ** -23 * v.abs()
    mm = torch.ones_like(v) if mul is None else mul.double()
    rr = torch.zeros_like(v) if residual is None else residual.double()
    ref = a * mm + rr
    tol = da * mm.abs() + 2.0 ** -23 * ((a * mm).abs() + rr.abs())
    tol = tol * (1 + 2.0 ** -8) + torch.finfo(dtype).eps / 2 * ref.abs() + torch.finfo(dtype).smallest_normal
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol).max()))


def ws_for(M, K, N):
    return workspace(M, K, N, 8)


@pytest.fixture(autouse=True)
def _clean_table():
    wq.wq_clear_tuning()
    yield
    wq.wq_clear_tuning()
    wq.wq_set_workspace(None)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("bits,group", [(8, 0), (4, 128)])
def test_activations(bits, group, act):
    M, K, N = 5, 512, 400
    pw, w = make_weight(bits, group, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    x = x * 3  # pre-activations out to where erfc and the logistic function are far below 1
    y = wq.wq_linear_epilogue(x, pw, bias=bias, act=ACTS[act], mul=mul, residual=res, ws=ws_for(M, K, N))
    check(y, x, w, bias, act, mul, res, torch.bfloat16)


@pytest.mark.parametrize("parts", range(8))
def test_every_subset_of_the_parts(parts):
    M, K, N = 3, 256, 144
    pw, w = make_weight(8, 0, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16, 0, parts & 1, parts & 2, parts & 4)
    y = wq.wq_linear_epilogue(x, pw, bias=bias, mul=mul, residual=res, ws=ws_for(M, K, N))
    check(y, x, w, bias, "none", mul, res, torch.bfloat16)
    if parts == 0:  # nothing after the product: the layer's own bits
        wq.wq_set_workspace(ws_for(M, K, N))
        assert torch.equal(y, wq.wq_linear(x, pw))


# every (variant, split) the dispatcher's table can hold, on a ragged shape whose
# panels are split between CTAs and whose last panel is ragged
VARIANTS8 = [(0, 3, 5), (0, 1, 17), (0, 2, 32), (1, 1, 9), (1, 4, 50), (1, 2, 128), (2, 1, 8), (2, 8, 3), (2, 4, 31),
             (3, 2, 16), (3, 1, 33), (3, 2, 100), (4, 1, 1), (4, 1, 16), (4, 1, 40), (4, 1, 64), (5, 1, 1), (5, 2, 5),
             (5, 1, 8)]
VARIANTS4 = [(0, 3, 5), (0, 1, 17), (1, 1, 9), (1, 4, 70), (2, 2, 8), (2, 4, 31), (3, 2, 16), (3, 1, 100), (4, 1, 2),
             (4, 1, 16), (4, 1, 32), (5, 1, 1), (5, 2, 5), (5, 1, 8), (6, 1, 1), (6, 1, 20), (6, 1, 64), (6, 1, 127)]


@pytest.mark.parametrize("bits,variant,split,M", [(8,) + v for v in VARIANTS8] + [(4,) + v for v in VARIANTS4])
@pytest.mark.parametrize("K,N", [(1152, 1488), (384, 16)])
def test_every_kernel(bits, variant, split, M, K, N):
    group = 128 if bits == 4 else 0
    if variant == 1:
        split = min(split, K // 128)
    pw, w = make_weight(bits, group, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16, variant)
    ws = workspace(M, K, N, 8)
    wq.wq_set_choice(M, K, N, bits, group, variant, split)
    for _ in range(2):  # the second call finds the counters as the first left them
        y = wq.wq_linear_epilogue(x, pw, bias=bias, act=wq.WQ_ACT_SILU, mul=mul, residual=res, ws=ws)
        check(y, x, w, bias, "silu", mul, res, torch.bfloat16)
    assert int(ws[:262912].max()) == 0
    assert wq.wq_device_error() == 0


@pytest.mark.parametrize("M", [1, 7, 33, 64])
@pytest.mark.parametrize("bits,group", [(4, 32), (4, 64), (4, 768)])
def test_int4_groups(bits, group, M):
    K, N = 768, 272
    pw, w = make_weight(bits, group, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    y = wq.wq_linear_epilogue(x, pw, bias=bias, act=wq.WQ_ACT_GELU, residual=res, ws=ws_for(M, K, N))
    check(y, x, w, bias, "gelu", None, res, torch.bfloat16)


@pytest.mark.parametrize("M", [1, 3, 16, 17, 45, 150, 500])
@pytest.mark.parametrize("bits,group", [(8, 0), (4, 32), (4, 64), (4, 128), (4, 640)])
def test_f16(bits, group, M):
    K, N = 640, 336
    pw, w = make_weight(bits, group, K, N)
    x, bias, mul, res = operands(M, K, N, torch.float16)
    y = wq.wq_linear_epilogue_f16(x, pw, bias=bias, act=wq.WQ_ACT_GELU_TANH, mul=mul, residual=res)
    assert y.dtype == torch.float16
    check(y, x, w, bias, "gelu_tanh", mul, res, torch.float16)


@pytest.mark.parametrize("M", [9, 11, 16, 33, 65, 128, 129, 200, 256, 300, 777])
@pytest.mark.parametrize("bits,group,K,N", [(8, 0, 1056, 656), (8, 0, 96, 2064), (4, 128, 1024, 656), (4, 128, 256, 2064)])
def test_prompts(bits, group, K, N, M):
    pw, w = make_weight(bits, group, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    y = wq.wq_linear_epilogue(x, pw, bias=bias, act=wq.WQ_ACT_SILU, mul=mul, residual=res, ws=ws_for(M, K, N))
    check(y, x, w, bias, "silu", mul, res, torch.bfloat16)
    # without a workspace
    y = wq.wq_linear_epilogue(x, pw, bias=bias, act=wq.WQ_ACT_SILU, mul=mul, residual=res)
    check(y, x, w, bias, "silu", mul, res, torch.bfloat16)
    assert wq.wq_device_error() == 0


@pytest.mark.parametrize("bits,group,K,N,M", [(8, 0, 4128, 528, 364), (8, 0, 8192, 144, 150), (4, 128, 4096, 528, 364),
                                              (4, 128, 8192, 16, 400), (4, 128, 8192, 272, 70), (8, 0, 64, 3008, 385),
                                              (8, 0, 6144, 16, 16), (4, 128, 128, 16, 193), (8, 0, 32, 16, 2000)])
def test_prompts_of_few_panels(bits, group, K, N, M):
    """Tiles cut between many pairs of CTAs, the parts summed by the last to
    come; the same bits every time, from a workspace used over and over."""
    pw, w = make_weight(bits, group, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    ws = ws_for(M, K, N)
    first = None
    for _ in range(3):
        y = wq.wq_linear_epilogue(x, pw, bias=bias, act=wq.WQ_ACT_GELU, mul=mul, residual=res, ws=ws)
        check(y, x, w, bias, "gelu", mul, res, torch.bfloat16)
        first = y if first is None else first
        assert torch.equal(y, first)
    assert int(ws[:262912].max()) == 0
    assert wq.wq_device_error() == 0


@pytest.mark.parametrize("bits,group,M", [(8, 0, 200), (4, 128, 200), (8, 0, 40)])
def test_prompt_workspace_edges(bits, group, M):
    """A workspace too small for any partial sum, and canaries behind one that
    holds them exactly."""
    K, N = 4096, 400
    pw, w = make_weight(bits, group, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    small = torch.zeros(262912, dtype=torch.uint8, device=dev())
    y = wq.wq_linear_epilogue(x, pw, residual=res, ws=small)
    check(y, x, w, None, "none", None, res, torch.bfloat16)
    plan = wq.wq_prompt_plan(bits, M, K, N, torch.cuda.get_device_properties(0).multi_processor_count // 2, 1 << 30)
    need = 262912 + plan["G"] * 4 * plan["nsub"] * plan["n"] * 128 * 4
    buf = torch.zeros(need + 4096, dtype=torch.uint8, device=dev())
    buf[need:] = 0xA5
    y = wq.wq_linear_epilogue(x, pw, residual=res, ws=buf[:need])
    check(y, x, w, None, "none", None, res, torch.bfloat16)
    assert bool((buf[need:] == 0xA5).all())


@pytest.mark.parametrize("M", [1, 4, 64, 150])
def test_strided_and_unaligned_operands(M):
    K, N = 512, 208
    pw, w = make_weight(4, 128, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    wide = torch.full((M, 2 * N + 3), float("nan"), dtype=torch.bfloat16, device=dev())
    wide[:, 1:N + 1] = mul
    wide[:, N + 1:2 * N + 1] = res
    b = torch.empty(N + 1, dtype=torch.bfloat16, device=dev())
    b[1:] = bias
    y = wq.wq_linear_epilogue(x, pw, bias=b[1:], act=wq.WQ_ACT_RELU, mul=wide[:, 1:N + 1],
                              residual=wide[:, N + 1:2 * N + 1], ws=ws_for(M, K, N))
    check(y, x, w, bias, "relu", mul, res, torch.bfloat16)


@pytest.mark.parametrize("M", [1, 8, 100, 300])
@pytest.mark.parametrize("bits,group", [(8, 0), (4, 128)])
def test_in_place(bits, group, M):
    """y is the residual buffer, then the mul buffer; rows behind M stay as they were."""
    K, N = 1024, 400
    pw, w = make_weight(bits, group, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    ws = ws_for(M, K, N)
    buf = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=dev())
    buf[:M] = res
    y = wq.wq_linear_epilogue(x, pw, bias=bias, mul=mul, residual=buf[:M], ws=ws, y=buf[:M])
    assert y.data_ptr() == buf.data_ptr()
    check(y, x, w, bias, "none", mul, res, torch.bfloat16)
    assert bool((buf[M:] == 7.0).all())
    buf[:M] = mul
    y = wq.wq_linear_epilogue(x, pw, bias=bias, mul=buf[:M], residual=res, ws=ws, y=buf[:M])
    check(y, x, w, bias, "none", mul, res, torch.bfloat16)


def test_outlier_rows_through_the_recompute():
    """Rows whose outputs the integer kernels' guard recomputes in binary64 go
    through the epilogue as the others do."""
    M, K, N = 4, 1024, 272
    for bits, group, variant in ((8, 0, 5), (8, 0, 4), (4, 128, 5), (4, 128, 4)):
        pw, w = make_weight(bits, group, K, N)
        x, bias, mul, res = operands(M, K, N, torch.bfloat16)
        x[:, 5] = torch.tensor([2.0 ** 12, -2.0 ** 14, 2.0 ** 15, 2.0 ** 16], device=dev())
        wq.wq_set_choice(M, K, N, bits, group, variant, 1)
        y = wq.wq_linear_epilogue(x, pw, bias=bias, mul=mul, residual=res, ws=ws_for(M, K, N))
        # every sum is within 2^-9 max(|v|, 1) of the exact one where the guard
        # accepted it (the layer's contract), and the output rounded once: bf16
        # has 8 significant bits, so by up to 2^-8 of its value (1 + 2^-8 lies
        # halfway between 1 and 1 + 2^-7)
        v = x.double() @ w.t()
        ref = (v + bias.double()) * mul.double() + res.double()
        tol = 2.0 ** -9 * v.abs().clamp(min=1) * mul.double().abs() + 2.0 ** -8 * ref.abs() + \
            2.0 ** -22 * (v.abs() + 1) * mul.double().abs() + 2.0 ** -22 * res.double().abs()
        assert bool(((y.double() - ref).abs() <= tol * 1.01).all())


def test_other_stream_and_graph():
    """On a side stream, and captured into a graph beside a second one that
    shares the workspace, replayed in turn with new inputs."""
    M, K, N = 6, 1024, 528
    pw, w = make_weight(4, 128, K, N)
    pw2, w2 = make_weight(8, 0, 512, 256)
    ws = ws_for(16, 1024, 528)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    x2, bias2, mul2, res2 = operands(M, 512, 256, torch.bfloat16, 5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = wq.wq_linear_epilogue(x, pw, bias=bias, residual=res, ws=ws, stream=s)
    s.synchronize()
    check(y, x, w, bias, "none", None, res, torch.bfloat16)
    graphs = []
    for args in ((x, pw, bias, mul, res), (x2, pw2, bias2, mul2, res2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = wq.wq_linear_epilogue(args[0], args[1], bias=args[2], act=wq.WQ_ACT_SILU, mul=args[3],
                                        residual=args[4], ws=ws)
        graphs.append((g, out))
    for i in range(3):
        x.copy_(operands(M, K, N, torch.bfloat16, 10 + i)[0])
        x2.copy_(operands(M, 512, 256, torch.bfloat16, 20 + i)[0])
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        check(graphs[0][1], x, w, bias, "silu", mul, res, torch.bfloat16)
        check(graphs[1][1], x2, w2, bias2, "silu", mul2, res2, torch.bfloat16)


def test_feed_forward_run():
    """A gated feed-forward layer as a decode step runs it: gate (silu), up
    times gate, down plus the residual stream in place, on one workspace."""
    M, D, H = 8, 512, 1024
    gate, wg = make_weight(4, 128, D, H, 1)
    up, wu = make_weight(4, 128, D, H, 2)
    down, wd = make_weight(8, 0, H, D, 3)
    ws = ws_for(M, H, H)
    x, _, _, _ = operands(M, D, H, torch.bfloat16)
    stream = operands(M, D, D, torch.bfloat16, 9)[3]
    before = stream.clone()
    g = wq.wq_linear_epilogue(x, gate, act=wq.WQ_ACT_SILU, ws=ws)
    h = wq.wq_linear_epilogue(x, up, mul=g, ws=ws)
    out = wq.wq_linear_epilogue(h, down, residual=stream, ws=ws, y=stream)
    check(g, x, wg, None, "silu", None, None, torch.bfloat16)
    check(h, x, wu, None, "none", g, None, torch.bfloat16)
    check(out, h, wd, None, "none", None, before, torch.bfloat16)


@pytest.mark.parametrize("bits,group,M", [(8, 0, 4000), (4, 128, 3000), (8, 0, 6000)])
def test_many_tiles_a_pair(bits, group, M):
    """Every pair of CTAs writes several tiles out, each behind the next one's products."""
    K, N = 256, 2064
    pw, w = make_weight(bits, group, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    for ws in (ws_for(M, K, N), None):
        y = wq.wq_linear_epilogue(x, pw, bias=bias, act=wq.WQ_ACT_RELU, mul=mul, residual=res, ws=ws)
        check(y, x, w, bias, "relu", mul, res, torch.bfloat16)
    assert wq.wq_device_error() == 0


def test_prompts_and_decode_steps_in_graphs_that_share_a_workspace():
    K, N = 2048, 528
    pw8, w8 = make_weight(8, 0, K, N)
    pw4, w4 = make_weight(4, 128, K, N)
    ws = ws_for(300, K, N)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    runs = []
    for i, (pw, w, M) in enumerate([(pw8, w8, 300), (pw4, w4, 5), (pw4, w4, 300), (pw8, w8, 1), (pw4, w4, 64)]):
        x, bias, mul, res = operands(M, K, N, torch.bfloat16, i)
        wq.wq_linear_epilogue(x, pw, residual=res, ws=ws, stream=s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y = wq.wq_linear_epilogue(x, pw, bias=bias, mul=mul, residual=res, ws=ws)
        runs.append((g, y, x, w, bias, mul, res))
    for order in ((0, 1, 2, 3, 4), (4, 2, 0, 1, 3), (2, 2, 0, 0, 4)):
        for i in order:
            runs[i][2].copy_(torch.roll(runs[i][2], 1, 0))
            runs[i][0].replay()
        torch.cuda.synchronize()
        for i in set(order):
            _, y, x, w, bias, mul, res = runs[i]
            check(y, x, w, bias, "none", mul, res, torch.bfloat16)
    assert int(ws[:262912].max()) == 0
    assert wq.wq_device_error() == 0


@pytest.mark.parametrize("M", [4, 200])
def test_two_calls_at_once(M):
    """On two streams, each with its own workspace."""
    K, N = 2048, 1040
    pw, w = make_weight(4, 128, K, N)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [(operands(M, K, N, torch.bfloat16, i), ws_for(M, K, N)) for i in range(2)]
    torch.cuda.synchronize()
    out = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            (x, bias, mul, res), ws = sets[i]
            out[i].append(wq.wq_linear_epilogue(x, pw, bias=bias, mul=mul, residual=res, ws=ws, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        (x, bias, mul, res), _ = sets[i]
        for y in out[i]:
            check(y, x, w, bias, "none", mul, res, torch.bfloat16)


def test_a_tuned_table_and_a_chosen_kernel():
    """wq_tune's entry (the plain layer's fastest kernel) and wq_set_choice's are
    both good for calls with an epilogue."""
    M, K, N = 32, 1024, 528
    pw, w = make_weight(8, 0, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    ws = ws_for(M, K, N)
    wq.wq_set_workspace(ws)
    try:
        wq.wq_tune(x, pw, torch.empty((M, N), dtype=torch.bfloat16, device=dev()), warmup=1, iters=2)
        y = wq.wq_linear_epilogue(x, pw, bias=bias, residual=res)
        check(y, x, w, bias, "none", None, res, torch.bfloat16)
        wq.wq_set_choice(M, K, N, 8, 0, wq.WQ_VARIANT_GEMV_RB, 4)
        y = wq.wq_linear_epilogue(x, pw, bias=bias, residual=res)
        check(y, x, w, bias, "none", None, res, torch.bfloat16)
    finally:
        wq.wq_clear_tuning()
        wq.wq_set_workspace(None)


@pytest.mark.parametrize("M", [1, 6, 150])
def test_decode_step_to_log_probabilities(M):
    """The layers of a step and the vocabulary head's log probabilities behind
    them, captured together and replayed with another input; the same bits as the
    calls one by one."""
    D, H, V, k = 512, 1024, 3088, 5
    gate, up = make_weight(4, 128, D, H, 1)[0], make_weight(4, 128, D, H, 2)[0]
    down, head = make_weight(8, 0, H, D, 3)[0], make_weight(8, 0, D, V, 4)[0]
    ws = ws_for(max(M, 64), H, V)
    scratch = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, V), dtype=torch.uint8, device=dev())
    x = operands(M, D, H, torch.bfloat16)[0]
    t = torch.arange(M, dtype=torch.int32, device=dev()) * 7 % V

    def step():
        g = wq.wq_linear_epilogue(x, gate, act=wq.WQ_ACT_SILU, ws=ws)
        h = wq.wq_linear_epilogue(x, up, mul=g, ws=ws)
        y = wq.wq_linear_epilogue(h, down, residual=x, ws=ws)
        return (y, *wq.wq_linear_logprobs(y, head, t, k, scratch, ws=ws))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        captured = step()
    for seed in (11, 12):
        x.copy_(operands(M, D, H, torch.bfloat16, seed)[0])
        g.replay()
        torch.cuda.synchronize()
        once = step()
        torch.cuda.synchronize()
        for a, b in zip(captured, once):
            assert torch.equal(a, b)
        y, lp, ent, top, idx = once
        assert bool((top[:, 1:] <= top[:, :-1]).all()) and bool((top <= 0).all()) and bool((lp <= top[:, 0]).all())
        assert bool((ent >= 0).all()) and bool((ent <= math.log(V) + 2 ** -17 * (2 + math.log(V))).all())
        # the alternatives' own log probabilities, asked for as tokens
        again = wq.wq_linear_logprobs(y, head, idx[:, 1].contiguous(), 0, scratch, ws=ws)[0]
        assert torch.equal(again, top[:, 1])
    assert wq.wq_device_error() == 0


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits,group,M", [(8, 0, 2), (4, 128, 40), (8, 0, 150)])
def test_activations_over_their_range(bits, group, M, dtype, act):
    """No product: the bias alone goes through the activation, from -12.5 (where
    erfc is 7e-36) to 12.5, and the largest finite values on both sides, where the
    answer is 0 or the value itself."""
    K, N = 128, 4096
    pw, w = make_weight(bits, group, K, N)
    x = torch.zeros((M, K), dtype=dtype, device=dev())
    bias = torch.linspace(-12.5, 12.5, N, device=dev()).to(dtype)
    bias[:2] = torch.tensor([-torch.finfo(dtype).max, torch.finfo(dtype).max], dtype=dtype)
    if dtype == torch.bfloat16:
        y = wq.wq_linear_epilogue(x, pw, bias=bias, act=ACTS[act], ws=ws_for(M, K, N))
    else:
        y = wq.wq_linear_epilogue_f16(x, pw, bias=bias, act=ACTS[act])
    ends = [0.0 if act != "none" else -torch.finfo(dtype).max, torch.finfo(dtype).max]
    assert torch.equal(y[:, :2].double(), torch.tensor([ends] * M, dtype=torch.float64, device=dev()))
    check(y[:, 2:], x, w[2:], bias[2:], act, None, None, dtype)


@pytest.mark.parametrize("bits,group,K,N,M", [(8, 0, 32, 1 << 20, 130), (4, 128, 128, 1 << 20, 3), (8, 0, 32, 16, 65536),
                                              (4, 128, 128, 16, 65536), (4, 64, 128, 16, 65536)])
def test_largest_sizes(bits, group, K, N, M):
    """The most output channels and the most tokens; the corners are looked at, and
    the rows around y stay as they were."""
    pw, w = make_weight(bits, group, K, N)
    x, bias, mul, res = operands(M, K, N, torch.bfloat16)
    buf = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=dev())
    y = wq.wq_linear_epilogue(x, pw, bias=bias, act=wq.WQ_ACT_SILU, mul=mul, residual=res, ws=ws_for(128, K, N),
                              y=buf[1:M + 1])
    for n in (slice(0, 300), slice(max(0, N - 300), N)):
        for m in (slice(0, 300), slice(max(0, M - 300), M)):
            check(y[m, n], x[m], w[n], bias[n], "silu", mul[m, n], res[m, n], torch.bfloat16)
    assert bool((buf[0] == 7).all()) and bool((buf[M + 1] == 7).all())
    assert wq.wq_device_error() == 0
