"""Refusals of the layer's epilogue and of the log probabilities, on the CPU:
every argument the C entries turn away before any device work, and what the
binding turns away before it."""
import ctypes

import pytest
import torch

import weight_only_quantized_02_b200 as wq

P = ctypes.c_void_p(1 << 20)   # aligned, never dereferenced: the checks come first
ODD = ctypes.c_void_p((1 << 20) + 1)
NULL, SHAPE, ALIGN, GROUP, WORKSPACE, EPILOGUE, DTYPE = -1, -2, -3, -4, -6, -12, -13


def epi(bias=None, mul=None, residual=None, ld_mul=0, ld_residual=0, act=0):
    return wq._Epilogue(bias=bias, mul=mul, residual=residual, ld_mul=ld_mul, ld_residual=ld_residual, act=act)


def linear(e, x=P, M=4, K=256, w=P, s=P, z=P, group=128, N=64, y=P, f16=False):
    ep = None if e is None else ctypes.byref(e)
    if f16:
        return wq.lib.wq_linear_epilogue_f16(x, M, K, w, s, z, group, N, ep, y, None)
    return wq.lib.wq_linear_epilogue(x, M, K, w, s, z, group, N, ep, y, None, 0, None)


@pytest.mark.parametrize("f16", [False, True])
def test_linear_epilogue_refusals(f16):
    ok = epi()
    assert linear(None, f16=f16) == NULL
    for name in ("x", "w", "s", "z", "y"):
        assert linear(ok, f16=f16, **{name: None}) == NULL, name
    for act in (-1, 5, 1000):
        assert linear(epi(act=act), f16=f16) == EPILOGUE
    assert linear(epi(mul=P, ld_mul=63), f16=f16) == EPILOGUE
    assert linear(epi(residual=P, ld_residual=0), f16=f16) == EPILOGUE
    assert linear(epi(residual=P, ld_residual=-64), f16=f16) == EPILOGUE
    for part in ("bias", "mul", "residual"):
        assert linear(epi(ld_mul=64, ld_residual=64, **{part: ODD}), f16=f16) == ALIGN, part
    assert linear(ok, f16=f16, M=0) == SHAPE and linear(ok, f16=f16, M=65537) == SHAPE
    assert linear(ok, f16=f16, N=40) == SHAPE and linear(ok, f16=f16, K=200) == SHAPE
    assert linear(ok, f16=f16, group=48) == GROUP
    assert linear(ok, f16=f16, x=ctypes.c_void_p((1 << 20) + 8)) == ALIGN
    assert linear(ok, f16=f16, y=ctypes.c_void_p((1 << 20) + 2)) == ALIGN


def logprobs(logits=P, dtype=0, M=4, N=100, ld=100, tokens=P, k=3, lp=P, H=P, top=P, idx=P):
    return wq.lib.wq_logprobs(logits, dtype, M, N, ld, tokens, k, lp, H, top, idx, None)


def test_logprobs_refusals():
    assert logprobs(logits=None) == NULL
    assert logprobs(dtype=3) == DTYPE and logprobs(dtype=-1) == DTYPE
    for M in (0, -1, 65537):
        assert logprobs(M=M) == SHAPE
    assert logprobs(N=0, ld=0) == SHAPE and logprobs(N=(1 << 20) + 1, ld=1 << 21) == SHAPE
    assert logprobs(ld=99) == SHAPE and logprobs(ld=-100) == SHAPE
    assert logprobs(k=-1) == SHAPE and logprobs(k=65) == SHAPE and logprobs(N=2, k=3) == SHAPE
    assert logprobs(tokens=None) == NULL and logprobs(lp=None) == NULL
    assert logprobs(top=None) == NULL and logprobs(idx=None) == NULL
    assert logprobs(tokens=None, lp=None, H=None, k=0) == NULL
    assert logprobs(logits=ODD) == ALIGN and logprobs(logits=ctypes.c_void_p((1 << 20) + 2), dtype=2) == ALIGN
    for name in ("tokens", "lp", "H", "top", "idx"):
        assert logprobs(**{name: ctypes.c_void_p((1 << 20) + 2)}) == ALIGN, name


def head(x=P, M=4, K=256, N=64, group=0, tokens=P, k=3, lp=P, H=P, top=P, idx=P, scratch=P, nbytes=4 * 64 * 4):
    return wq.lib.wq_linear_logprobs(x, M, K, P, P, None, group, N, tokens, k, lp, H, top, idx, scratch, nbytes, None, 0,
                                     None)


def test_linear_logprobs_refusals():
    assert head(x=None) == NULL and head(scratch=None) == NULL
    assert head(nbytes=4 * 64 * 4 - 1) == WORKSPACE
    assert head(scratch=ctypes.c_void_p((1 << 20) + 4)) == ALIGN
    assert head(k=65) == SHAPE and head(M=0) == SHAPE and head(tokens=None) == NULL
    assert wq.wq_linear_logprobs_workspace_bytes(4, 64) == 4 * 64 * 4
    # the logits of 512 tokens at most are held at once
    assert wq.wq_linear_logprobs_workspace_bytes(5000, 152064) == 512 * 152064 * 4
    assert wq.wq_linear_logprobs_workspace_bytes(0, 64) == 0 and wq.wq_linear_logprobs_workspace_bytes(4, 0) == 0
    assert wq.wq_linear_logprobs_workspace_bytes(65537, 64) == 0


def weight(K=256, N=64):
    return wq.PackedWeight(torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int16), None, 8, K, N, 0)


def refused(status, call, *args, **kw):
    with pytest.raises(wq.WQError) as e:
        call(*args, **kw)
    assert e.value.status == status


def test_binding_refuses_before_the_library():
    pw = weight()
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    refused(DTYPE, wq.wq_linear_epilogue, x.half(), pw)
    refused(DTYPE, wq.wq_linear_epilogue_f16, x, pw)
    refused(SHAPE, wq.wq_linear_epilogue, x[:, :128], pw)
    refused(SHAPE, wq.wq_linear_epilogue, torch.zeros(256, 4, dtype=torch.bfloat16).t(), pw)
    refused(SHAPE, wq.wq_linear_epilogue, x, pw)  # tensors on the CPU
    refused(DTYPE, wq.wq_logprobs, torch.zeros(4, 10, dtype=torch.float64))
    refused(SHAPE, wq.wq_logprobs, torch.zeros(10))
    refused(SHAPE, wq.wq_logprobs, torch.zeros(10, 4).t())
    refused(SHAPE, wq.wq_logprobs, torch.zeros(4, 10))
    refused(DTYPE, wq.wq_linear_logprobs, x.float(), pw, None, 0, torch.zeros(1))


def test_binding_checks_the_operands():
    M, N, dt, cpu = 4, 64, torch.bfloat16, -1
    good = torch.zeros(M, N, dtype=dt)
    assert wq._rows(good, (M, N), dt, cpu, "t") == N
    assert wq._rows(torch.zeros(M, 2 * N, dtype=dt)[:, 3:N + 3], (M, N), dt, cpu, "t") == 2 * N
    refused(DTYPE, wq._rows, good.float(), (M, N), dt, cpu, "t")
    refused(SHAPE, wq._rows, good[:, :60], (M, N), dt, cpu, "t")
    refused(SHAPE, wq._rows, torch.zeros(N, M, dtype=dt).t(), (M, N), dt, cpu, "t")
    refused(SHAPE, wq._rows, good, (M, N), dt, 1, "t")
    refused(DTYPE, wq._vector, torch.zeros(4, dtype=torch.int64), 4, torch.int32, cpu, "t")
    refused(SHAPE, wq._vector, torch.zeros(8, dtype=torch.int32)[::2], 4, torch.int32, cpu, "t")
    refused(SHAPE, wq._vector, torch.zeros(4, dtype=torch.int32), 4, torch.int32, 0, "t")
    refused(SHAPE, wq._logprob_outputs, good, 4, None, -1, cpu, "t")
    refused(SHAPE, wq._scratch, torch.zeros(8), 0, "t")


def test_new_statuses_have_names():
    assert wq.STATUS[EPILOGUE] == "WQ_ERR_EPILOGUE" and wq.STATUS[DTYPE] == "WQ_ERR_DTYPE"
    assert "epilogue" in wq.strerror(EPILOGUE) and "logits" in wq.strerror(DTYPE)
