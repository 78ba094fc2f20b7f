"""Refusals of the operators with which the router and the weights learn: the
C ABI's argument checks and the binding's (no GPU needed: both come before any
CUDA call)."""
import ctypes

import numpy as np
import pytest
import torch

from mixture_experts_layer_28_b200 import build as mb
from mixture_experts_layer_28_b200 import moe_zc as mz

F = 1 << 20   # an aligned, never-dereferenced address


@pytest.fixture(scope="module")
def L():
    mb.build()
    return mz.lib()


def test_limits_match_header():
    text = open(mz.HEADER).read()
    assert f"#define MOE_ZC_ADAMW_BLOCK {mz.ADAMW_BLOCK}" in text
    assert f"enum {{ MOE_ZC_F32 = {mz.F32}, MOE_ZC_BF16 = {mz.BF16} }};" in text
    assert mz._ADAMW_TENSOR.itemsize == 64 and ctypes.sizeof(mz.AdamwArgs) == 56


def workspace(L, T, S, E):
    n = ctypes.c_int64(0)
    return L.moe_zc_balance_workspace(T, S, E, ctypes.byref(n)), n.value


def test_workspace_holds_a_slot_for_every_block_and_sequence(L):
    for T in (0, 1, 8, 9, 2368, 2369, 16384, 100000):
        for S in (0, 1, 7, 3000):
            st, n = workspace(L, T, S, 20)
            # one wave (three blocks on each of 148 multiprocessors) of at least 8 tokens,
            # of 16 where there are more than one wave of 8
            chunk = max(8, -(-T // 444))
            chunk = 16 if 8 < chunk < 16 else chunk
            slots = -(-T // chunk) + S
            assert st == mz.OK and n >= slots * (20 * 8 + 4)
    assert L.moe_zc_balance_workspace(4, 1, 4, None) == mz.ERR_INVALID_ARG
    assert workspace(L, -1, 1, 4)[0] == mz.ERR_INVALID_ARG
    assert workspace(L, 1, -1, 4)[0] == mz.ERR_INVALID_ARG
    assert workspace(L, 1, 1, 1025)[0] == mz.ERR_UNSUPPORTED


def _balance(L, **kw):
    a = dict(logits=F, off=None, idx=F, mask=None, seq=None, weight=None, T=16, S=1, E=12, K=2, loss=F, counts=F, prob=F, coef=F, ws=F, bytes=1 << 30)
    a.update(kw)
    return L.moe_zc_balance_loss(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), mz.ERR_INVALID_ARG), (dict(idx=None), mz.ERR_INVALID_ARG), (dict(loss=None), mz.ERR_INVALID_ARG), (dict(counts=None), mz.ERR_INVALID_ARG),
    (dict(prob=None), mz.ERR_INVALID_ARG), (dict(coef=None), mz.ERR_INVALID_ARG), (dict(ws=None), mz.ERR_INVALID_ARG), (dict(bytes=100), mz.ERR_INVALID_ARG),
    (dict(T=-1), mz.ERR_INVALID_ARG), (dict(S=-1, seq=F), mz.ERR_INVALID_ARG), (dict(S=2), mz.ERR_INVALID_ARG), (dict(S=0), mz.ERR_INVALID_ARG),
    (dict(E=0, K=1), mz.ERR_INVALID_ARG), (dict(K=0), mz.ERR_INVALID_ARG), (dict(K=13), mz.ERR_INVALID_ARG), (dict(E=1025), mz.ERR_UNSUPPORTED),
    (dict(E=40, K=33), mz.ERR_UNSUPPORTED), (dict(T=1 << 31, bytes=1 << 50), mz.ERR_UNSUPPORTED),
    (dict(logits=F + 4), mz.ERR_UNSUPPORTED), (dict(off=F + 8), mz.ERR_UNSUPPORTED), (dict(coef=F + 4), mz.ERR_UNSUPPORTED), (dict(ws=F + 4), mz.ERR_UNSUPPORTED),
    (dict(idx=F + 2), mz.ERR_UNSUPPORTED), (dict(seq=F + 1), mz.ERR_UNSUPPORTED), (dict(counts=F + 2), mz.ERR_UNSUPPORTED), (dict(weight=F + 1), mz.ERR_UNSUPPORTED),
])
def test_balance_loss_refusals(L, kw, status):
    assert _balance(L, **kw) == status


def test_no_sequences_is_no_work(L):
    assert _balance(L, S=0, seq=F, loss=None, counts=None, prob=None, coef=None, ws=None, bytes=0) == mz.OK


def _route(L, **kw):
    a = dict(logits=F, off=None, idx=F, dgate=F, mask=None, seq=None, coef=F, dloss=F, T=16, S=1, E=12, K=2, out=F, dtype=mz.F32)
    a.update(kw)
    return L.moe_zc_route_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), mz.ERR_INVALID_ARG), (dict(idx=None), mz.ERR_INVALID_ARG), (dict(dloss=None), mz.ERR_INVALID_ARG), (dict(out=None), mz.ERR_INVALID_ARG),
    (dict(S=2), mz.ERR_INVALID_ARG), (dict(dtype=2), mz.ERR_INVALID_ARG), (dict(T=-1), mz.ERR_INVALID_ARG), (dict(K=0), mz.ERR_INVALID_ARG),
    (dict(E=1025), mz.ERR_UNSUPPORTED), (dict(E=40, K=33), mz.ERR_UNSUPPORTED), (dict(out=F + 4), mz.ERR_UNSUPPORTED), (dict(coef=F + 8), mz.ERR_UNSUPPORTED),
    (dict(dgate=F + 2), mz.ERR_UNSUPPORTED), (dict(dloss=F + 1), mz.ERR_UNSUPPORTED),
])
def test_route_backward_refusals(L, kw, status):
    assert _route(L, **kw) == status


def test_no_tokens_is_no_work(L):
    assert _route(L, T=0, logits=None, idx=None, out=None, dgate=None, coef=None, dloss=None) == mz.OK
    assert _combine(L, T=0, dout=None, x=None, y=None, slot=None, gate=None, dgate=None, dy=None) == mz.OK


def _combine(L, **kw):
    a = dict(dout=F, x=F, y=F, slot=F, gate=F, T=16, d=128, K=2, rows=32, dgate=F, dy=F)
    a.update(kw)
    return L.moe_zc_combine_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dout=None), mz.ERR_INVALID_ARG), (dict(x=None), mz.ERR_INVALID_ARG), (dict(y=None), mz.ERR_INVALID_ARG), (dict(slot=None), mz.ERR_INVALID_ARG),
    (dict(gate=None), mz.ERR_INVALID_ARG), (dict(dgate=None), mz.ERR_INVALID_ARG), (dict(T=-1), mz.ERR_INVALID_ARG), (dict(d=0), mz.ERR_INVALID_ARG),
    (dict(K=0), mz.ERR_INVALID_ARG), (dict(rows=-1), mz.ERR_INVALID_ARG), (dict(K=33), mz.ERR_UNSUPPORTED), (dict(d=100), mz.ERR_UNSUPPORTED),
    (dict(T=1 << 31), mz.ERR_UNSUPPORTED), (dict(dout=F + 8), mz.ERR_UNSUPPORTED), (dict(y=F + 2), mz.ERR_UNSUPPORTED), (dict(dy=F + 4), mz.ERR_UNSUPPORTED),
    (dict(slot=F + 2), mz.ERR_UNSUPPORTED),
])
def test_combine_backward_refusals(L, kw, status):
    assert _combine(L, **kw) == status


def _adamw(L, n=1, tensor=None, step=F, **kw):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, param_type=mz.F32, grad_type=mz.F32, state_bits=32, master=0)
    a.update(kw)
    t = np.zeros(max(n, 1), dtype=mz._ADAMW_TENSOR)
    whole = dict(param=F, grad=F, exp_avg=F, exp_avg_sq=F, exp_avg_scale=F, exp_avg_sq_scale=F, master=F, n=100)
    for k, v in {**whole, **(tensor or {})}.items():
        t[k] = v
    return L.moe_zc_adamw(t.ctypes.data, n, ctypes.byref(mz.AdamwArgs(*a.values())), step, None, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), mz.ERR_INVALID_ARG), (dict(step=None), mz.ERR_INVALID_ARG), (dict(step=F + 2), mz.ERR_UNSUPPORTED),
    (dict(beta1=1.0), mz.ERR_INVALID_ARG), (dict(beta2=-0.1), mz.ERR_INVALID_ARG), (dict(beta2=float("nan")), mz.ERR_INVALID_ARG), (dict(eps=0.0), mz.ERR_INVALID_ARG),
    (dict(eps=float("nan")), mz.ERR_INVALID_ARG), (dict(eps=1e-60), mz.ERR_INVALID_ARG), (dict(lr=float("inf")), mz.ERR_INVALID_ARG), (dict(weight_decay=float("nan")), mz.ERR_INVALID_ARG),
    (dict(param_type=2), mz.ERR_INVALID_ARG), (dict(grad_type=-1), mz.ERR_INVALID_ARG), (dict(state_bits=16), mz.ERR_INVALID_ARG), (dict(master=1), mz.ERR_INVALID_ARG),
    (dict(master=2, param_type=mz.BF16), mz.ERR_INVALID_ARG),
])
def test_adamw_refusals(L, kw, status):
    assert _adamw(L, **kw) == status


@pytest.mark.parametrize("tensor,kw,status", [
    (dict(param=0), {}, mz.ERR_INVALID_ARG), (dict(grad=0), {}, mz.ERR_INVALID_ARG), (dict(exp_avg=0), {}, mz.ERR_INVALID_ARG), (dict(exp_avg_sq=0), {}, mz.ERR_INVALID_ARG),
    (dict(exp_avg_scale=0), dict(state_bits=8), mz.ERR_INVALID_ARG), (dict(master=0), dict(master=1, param_type=mz.BF16), mz.ERR_INVALID_ARG), (dict(n=-1), {}, mz.ERR_INVALID_ARG),
    (dict(n=1 << 41), {}, mz.ERR_UNSUPPORTED), (dict(param=F + 8), {}, mz.ERR_UNSUPPORTED), (dict(grad=F + 2), {}, mz.ERR_UNSUPPORTED),
    (dict(exp_avg_sq_scale=F + 2), dict(state_bits=8), mz.ERR_UNSUPPORTED),
])
def test_adamw_tensor_refusals(L, tensor, kw, status):
    assert _adamw(L, tensor=tensor, **kw) == status


def test_route_logits_refusals(L):
    r = lambda **kw: L.moe_zc_route_logits(F, F, F, None, 16, kw.get("d", 128), 4, 2, 2, kw.get("logits", F), F, F, F, kw.get("counts", F), None)
    assert r(logits=None) == mz.ERR_INVALID_ARG
    assert r(logits=F + 4) == mz.ERR_UNSUPPORTED
    assert r(d=96) == mz.ERR_UNSUPPORTED
    assert r(counts=None) == mz.ERR_INVALID_ARG


def test_binding_refuses_host_tensors_and_wrong_types():
    t, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        mz.balance_loss(t, i)
    with pytest.raises(ValueError, match="logits must be"):
        mz.balance_loss(t.double(), i)
    with pytest.raises(ValueError, match="mask must be"):
        mz.balance_loss(t, i, mask=torch.zeros(4))
    with pytest.raises(ValueError, match="seq_start"):
        mz.balance_loss(t, i, seq_start=torch.zeros(0, dtype=torch.int32))
    with pytest.raises(ValueError, match="go together"):
        mz.route_backward(t, i, coef=torch.zeros(1, 8))
    with pytest.raises(ValueError, match="needs idx"):
        mz.route_backward(t, dgate=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="dtype"):
        mz.route_backward(t, i, dgate=torch.zeros(4, 2), dtype=torch.float16)
    b = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dout must be"):
        mz.combine_backward(t, b, b, i, torch.zeros(4, 2))


def test_adamw_refuses_at_construction():
    p = torch.zeros(4)
    with pytest.raises(ValueError, match="empty"):
        mz.AdamW([], 1e-3)
    with pytest.raises(ValueError, match="state_bits"):
        mz.AdamW([p], 1e-3, state_bits=4)
    with pytest.raises(ValueError, match="params must be"):
        mz.AdamW([p.half()], 1e-3)
    with pytest.raises(ValueError, match="master"):
        mz.AdamW([p], 1e-3, master=True)
    with pytest.raises(ValueError, match="one entry per parameter"):
        mz.AdamW([p], 1e-3, exp_avg=[p, p])
    with pytest.raises(ValueError, match="count"):
        mz.AdamW([p], 1e-3, step=-1)
    with pytest.raises(ValueError, match="CUDA device"):
        mz.AdamW([p], 1e-3)


def test_adamw_names_the_tensor():
    with pytest.raises(ValueError, match=r"^params\[0\] must be on the current CUDA device$"):
        mz.AdamW([torch.zeros(4)], 1e-3)
