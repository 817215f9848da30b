"""Operators of the quantized layer and its vocabulary head, as they are timed.

Three operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and as the calls a user of
``weight_only_quantized_02_b200`` makes:

  linear_epilogue   y = act(x . dequant(W)^T + bias) * mul + residual, one
                    rounding to the activations' type, for W8A16 and W4A16
                    weights (``wq_linear_epilogue``, ``wq_linear_epilogue_f16``)
  logprobs          log probabilities of given tokens, the entropy and the k
                    most likely alternatives of rows of logits
                    (``wq_logprobs``)
  head_logprobs     the same straight from the activations of a quantized
                    vocabulary head, whose logits are never rounded to 16 bits
                    (``wq_linear_logprobs``)

``own`` selects which of the two ``run`` calls.
"""
import math
import os

import torch

own = False

BF16, F16, F32 = "bf16", "f16", "f32"
DTYPES = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _linear(name, bits, group, K, N, M, act="none", bias=False, mul=False, residual=False, dtype=BF16):
    return dict(name=name, op="linear_epilogue", bits=bits, group=group, K=K, N=N, M=M, act=act, bias=bias, mul=mul,
                residual=residual, dtype=dtype)


def _logprobs(name, M, N, k, dtype=BF16, pad=0, masked=0.0):
    return dict(name=name, op="logprobs", M=M, N=N, k=k, dtype=dtype, pad=pad, masked=masked)


def _head(name, bits, group, K, N, M):
    return dict(name=name, op="head_logprobs", bits=bits, group=group, K=K, N=N, M=M)


def listed():
    return [
        # the smallest layer of the benchmark, one token: launch and latency
        _linear("w8_1024x1024_m1_bias_residual", 8, 0, 1024, 1024, 1, bias=True, residual=True),
        # an up projection of a decode batch with its activation
        _linear("w8_5120x17408_m4_bias_gelu", 8, 0, 5120, 17408, 4, act="gelu", bias=True),
        # the gated half of a feed-forward layer, eight sequences
        _linear("w4g128_5120x25600_m8_mul", 4, 128, 5120, 25600, 8, mul=True),
        # a down projection that adds the residual stream, a full decode batch
        _linear("w4g128_17408x5120_m64_residual", 4, 128, 17408, 5120, 64, residual=True),
        # the same layer over a prompt
        _linear("w4g128_17408x5120_m2048_residual", 4, 128, 17408, 5120, 2048, residual=True),
        # a ragged prompt chunk through an INT8 up projection
        _linear("w8_5120x17408_m333_bias_silu", 8, 0, 5120, 17408, 333, act="silu", bias=True),
        # fp16 activations, a fine-grained group, an output count that ends inside a panel
        _linear("f16_w4g64_5120x5136_m3_bias_relu", 4, 64, 5120, 5136, 3, act="relu", bias=True, dtype=F16),
        # one decode step's log probabilities with alternatives
        _logprobs("logprobs_152064_m1_k20", 1, 152064, 20),
        # scoring a prompt against its own tokens
        _logprobs("logprobs_152064_m2048_k5", 2048, 152064, 5),
        # constrained decoding: fp32 logits, nine in ten masked out, odd vocabulary in padded rows
        _logprobs("logprobs_50001_m77_k64_f32_masked", 77, 50001, 64, dtype=F32, pad=7, masked=0.9),
        # a decode batch scored at the INT8 vocabulary head
        _head("head_w8_5120x152064_m16", 8, 0, 5120, 152064, 16),
        # a prompt scored at the INT4 vocabulary head
        _head("head_w4g128_5120x152064_m200", 4, 128, 5120, 152064, 200),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear_epilogue", "linear_epilogue", "logprobs", "logprobs", "head_logprobs"))
    if op == "logprobs":
        N = _log_uniform(rng, 1000, 152064)
        dtype = rng.choice((BF16, BF16, F16, F32))
        size = 4 if dtype == F32 else 2
        M = _log_uniform(rng, 1, min(2048, 2048 * 152064 * 2 // (N * size)))
        masked = rng.choice((0.0, 0.0, 0.5, 0.9))
        c = _logprobs("", M, N, rng.choice((0, 1, 5, 20, 64)), dtype, rng.choice((0, 0, 1, 8)), masked)
    elif op == "head_logprobs":
        bits = rng.choice((8, 4))
        K = 128 * rng.randint(4, 40)
        N = 16 * _log_uniform(rng, 1000, 9504)
        c = _head("", bits, 128 if bits == 4 else 0, K, N, _log_uniform(rng, 1, 200))
    else:
        dtype = rng.choice((BF16, BF16, BF16, F16))
        bits = rng.choice((8, 4))
        K = 128 * _log_uniform(rng, 4, 136)
        N = 16 * _log_uniform(rng, 32, 1600)
        group = 0 if bits == 8 else rng.choice((128, 128, 128, 32, 64, K))
        # fp16 activations and groups of 32 and 64 are decode formats
        hi = 64 if dtype == F16 or group in (32, 64) else 2048
        hi = max(1, min(hi, 2048 * 17408 * 5120 // (K * N)))
        c = _linear("", bits, group, K, N, _log_uniform(rng, 1, hi), rng.choice(ACTS), rng.random() < 0.5,
                    rng.random() < 0.3, rng.random() < 0.5, dtype)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _bf16_scales(shape, base, g):
    s = base * (0.75 + 0.5 * torch.rand(shape, generator=g, device="cuda"))
    return s.to(torch.bfloat16)


def _weights(case, g):
    """Codes of normally distributed weights of variance 1/K: INT8 with the
    row's largest at 127, INT4 with the group's range over 15 steps."""
    bits, group, K, N = case["bits"], case["group"], case["K"], case["N"]
    out = {}
    q = torch.empty((N, K), dtype=torch.int8, device="cuda")
    rows = max(1, (1 << 28) // K)
    for r0 in range(0, N, rows):  # in row blocks, so that no 32-bit copy of a whole vocabulary head is held
        w = torch.randn((min(rows, N - r0), K), generator=g, device="cuda")
        if bits == 8:
            q[r0:r0 + rows] = (w * 30.0).round_().clamp_(-127, 127).to(torch.int8)
        else:
            q[r0:r0 + rows] = (w * 2.8 + 7.5).round_().clamp_(0, 15).to(torch.int8)
    out["q"] = q
    if bits == 8:
        out["scale"] = _bf16_scales((N,), 1.0 / (30.0 * math.sqrt(K)), g)
    else:
        out["scale"] = _bf16_scales((N, K // group), 1.0 / (2.8 * math.sqrt(K)), g)
        out["zero"] = torch.randint(6, 10, (N, K // group), generator=g, device="cuda").to(torch.int8)
    return out


def _inputs(case, seed):
    g = _generator(seed)
    M, N = case["M"], case["N"]
    dt = DTYPES[case.get("dtype", BF16)]
    if case["op"] == "logprobs":
        buf = torch.randn((M, N + case["pad"]), generator=g, device="cuda").mul_(2.5)
        if case["masked"]:
            buf[torch.rand(buf.shape, generator=g, device="cuda") < case["masked"]] = -math.inf
        tokens = torch.randint(0, N, (M,), generator=g, device="cuda", dtype=torch.int32)
        # the given token is an allowed one, as likely as a sampled token is
        buf.scatter_(1, tokens.long().unsqueeze(1), 3.0 + 4.0 * torch.rand((M, 1), generator=g, device="cuda"))
        return {"logits": buf.to(dt)[:, :N], "tokens": tokens}
    out = _weights(case, g)
    x = torch.randn((M, case["K"]), generator=g, device="cuda")
    if case["op"] == "head_logprobs":
        out["x"] = (x * 2.5).to(torch.bfloat16)
        out["tokens"] = torch.randint(0, N, (M,), generator=g, device="cuda", dtype=torch.int32)
        return out
    out["x"] = x.to(dt)
    for name, shape in (("bias", (N,)), ("mul", (M, N)), ("residual", (M, N))):
        if case[name]:
            out[name] = torch.randn(shape, generator=g, device="cuda").to(dt)
    return out


def _pack_words(v):
    """4-bit values [..., 8 n] as 32-bit words, low nibble first."""
    w = torch.zeros(v.shape[:-1] + (v.shape[-1] // 8,), dtype=torch.int32, device=v.device)
    for j in range(8):
        w |= v[..., j::8].to(torch.int32) << (4 * j)
    return w


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if not own:
        return state
    import weight_only_quantized_02_b200 as wq
    if case["op"] == "logprobs":
        return state
    table = os.path.join(os.path.dirname(wq.LIB_PATH), "tuning_b200.txt")
    if wq.wq_load_tuning(table) != 0:
        raise RuntimeError("unreadable " + table)
    M, K, N, group = case["M"], case["K"], case["N"], case["group"]
    q, scale = state.pop("q"), state.pop("scale").view(torch.int16)
    if case["bits"] == 8:
        state["packed"] = wq.wq_pack_int8(q, scale)
    else:
        zero = state.pop("zero")
        zero = torch.nn.functional.pad(zero, (0, -zero.shape[1] % 8))
        state["packed"] = wq.wq_pack_int4(_pack_words(q), scale, _pack_words(zero), group)
    state["workspace"] = torch.zeros(wq.wq_workspace_bytes(M, K, N, 1), dtype=torch.uint8, device="cuda")
    if case["op"] == "head_logprobs":
        state["scratch"] = torch.empty(wq.wq_linear_logprobs_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _dequant(state):
    q, s = state["q"].float(), state["scale"].float()
    if "zero" not in state:
        return q.mul_(s.unsqueeze(1))
    N, K = q.shape
    q = q.view(N, s.shape[1], -1)
    return q.sub_(state["zero"].float().unsqueeze(2)).mul_(s.unsqueeze(2)).view(N, K)


def _activation(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _plain_linear(state):
    v = state["x"].float() @ _dequant(state).t()
    if "bias" in state:
        v = v + state["bias"].float()
    v = _activation(v, state["case"]["act"])
    if "mul" in state:
        v = v * state["mul"].float()
    if "residual" in state:
        v = v + state["residual"].float()
    return v.to(state["x"].dtype)


def _plain_logprobs(logits, tokens, k):
    x = logits.float()
    shifted = x - x.max(dim=1, keepdim=True).values
    e = torch.exp(shifted)
    total = e.sum(dim=1)
    log_total = torch.log(total)
    # a masked logit has probability zero and adds nothing
    entropy = log_total - torch.where(e > 0, e * shifted, torch.zeros_like(e)).sum(dim=1) / total
    token = torch.gather(shifted, 1, tokens.long().unsqueeze(1)).squeeze(1) - log_total
    if k == 0:
        return token, entropy
    # a stable sort leaves equal logits in index order
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    top = torch.gather(shifted, 1, order) - log_total.unsqueeze(1)
    return token, entropy, top, order.to(torch.int32)


def run(state):
    case = state["case"]
    if own:
        import weight_only_quantized_02_b200 as wq
        if case["op"] == "logprobs":
            token, entropy, top, index = wq.wq_logprobs(state["logits"], state["tokens"], case["k"])
            return (token, entropy) if case["k"] == 0 else (token, entropy, top, index)
        if case["op"] == "head_logprobs":
            token, entropy, _, _ = wq.wq_linear_logprobs(state["x"], state["packed"], state["tokens"], 0,
                                                         state["scratch"], ws=state["workspace"])
            return token, entropy
        call = wq.wq_linear_epilogue_f16 if case["dtype"] == F16 else wq.wq_linear_epilogue
        return call(state["x"], state["packed"], bias=state.get("bias"), act=getattr(wq, "WQ_ACT_" + case["act"].upper()),
                    mul=state.get("mul"), residual=state.get("residual"), ws=state["workspace"])
    if case["op"] == "logprobs":
        return _plain_logprobs(state["logits"], state["tokens"], case["k"])
    if case["op"] == "head_logprobs":
        return _plain_logprobs(state["x"].float() @ _dequant(state).t(), state["tokens"], 0)
    return _plain_linear(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    M, N = case["M"], case["N"]
    if case["op"] == "logprobs":
        size = 4 if case["dtype"] == F32 else 2
        # per logit: the maximum, a difference, an exponential, two sums and a product
        return {"bytes": M * N * size + M * (12 + 8 * case["k"]), "flops": 6 * M * N}
    K = case["K"]
    if case["bits"] == 8:
        nbytes = N * K + 2 * N
    else:
        nbytes = N * K // 2 + (5 * N * (K // case["group"]) + 1) // 2
    nbytes += 2 * M * K
    if case["op"] == "head_logprobs":
        nbytes += 12 * M
    else:
        nbytes += 2 * M * N * (1 + case["mul"] + case["residual"]) + 2 * N * case["bias"]
    return {"bytes": nbytes, "flops": 2 * M * N * K}


def _exact_logits(inp):
    """sum over the groups of scale * (codes - zero) . x, every product and
    sum in 64 bits, in blocks of output channels."""
    x, q, s = inp["x"].double(), inp["q"], inp["scale"].double()
    N, K = q.shape
    out = torch.empty((x.shape[0], N), dtype=torch.float64, device=x.device)
    rows = max(1, (1 << 27) // K)
    for r0 in range(0, N, rows):
        r = slice(r0, min(N, r0 + rows))
        if "zero" in inp:
            reps = K // s.shape[1]
            w = q[r].double() - inp["zero"][r].double().repeat_interleave(reps, dim=1)
            w *= s[r].repeat_interleave(reps, dim=1)
            out[:, r] = torch.matmul(x, w.t())
        else:
            out[:, r] = torch.matmul(x, q[r].double().t()) * s[r]
    return out


def _exact_logprobs(x, tokens, k):
    x = x.double()
    logp = x - torch.logsumexp(x, dim=1, keepdim=True)
    p = logp.exp()
    entropy = -(p * logp.masked_fill(p == 0, 0.0)).sum(dim=1)
    rows = torch.arange(x.shape[0], device=x.device)
    token = logp[rows, tokens.long()]
    if k == 0:
        return token, entropy
    # the k largest by value, then by lowest index
    top = torch.argsort(-x, dim=1, stable=True)[:, :k]
    return token, entropy, logp.gather(1, top), top.to(torch.int32)


def exact(case, seed):
    inp = _inputs(case, seed)
    if case["op"] == "logprobs":
        parts = []
        for r in range(0, case["M"], 64):
            parts.append(_exact_logprobs(inp["logits"][r:r + 64], inp["tokens"][r:r + 64], case["k"]))
        return tuple(torch.cat(p) for p in zip(*parts))
    if case["op"] == "head_logprobs":
        return _exact_logprobs(_exact_logits(inp), inp["tokens"], 0)
    v = _exact_logits(inp)
    if "bias" in inp:
        v += inp["bias"].double()
    act = case["act"]
    if act == "relu":
        v = v.clamp(min=0.0)
    elif act == "gelu":
        v = v * torch.special.ndtr(v)
    elif act == "gelu_tanh":
        # 0.5 (1 + tanh u) is the logistic function of 2 u
        v = v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v.pow(3)))
    elif act == "silu":
        v = v * torch.sigmoid(v)
    if "mul" in inp:
        v = v * inp["mul"].double()
    if "residual" in inp:
        v = v + inp["residual"].double()
    return v
