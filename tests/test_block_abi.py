"""Refusals of the gated block, the e4m3 products and the AdamW step (no GPU: every
call here fails validation, or has nothing to do, before any launch)."""
import ctypes

import pytest
import torch

L = pytest.importorskip("sparse_mixture_experts_04_amd._lib")
lib = L.lib
P = ctypes.c_void_p(0x1000)      # never dereferenced
ODD = ctypes.c_void_p(0x1001)    # aligned to nothing
EIGHT = ctypes.c_void_p(0x1008)  # not 16-byte aligned
ref = ctypes.byref


def size_of(fn, d, *more):
    n = ctypes.c_size_t(0)
    return fn(ref(d) if d is not None else None, *more, ref(n)), n.value


# ------------------------------------------------------------ gated block

def gated(**kw):
    return L.GatedFfDesc(**{**dict(M=40, d=64, F=32, E=2, act=L.BF16), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 2), (dict(d=0), 2), (dict(F=0), 2), (dict(E=0), 2), (dict(act=L.MXFP4), 3),
    (dict(act=7), 3), (dict(d=131073), 5), (dict(F=131073), 5), (dict(E=257), 5),
    (dict(M=(1 << 31) - 1023, d=1, F=1), 5), (dict(M=(1 << 31) - 1024, d=1024, F=1), 5),
    (dict(M=(1 << 31) - 1024, d=256, F=1), 0), (dict(M=1 << 23, F=1 << 16), 5),
    (dict(E=256, d=131072, F=32768), 5), (dict(M=0), 0), (dict(), 0),
    (dict(E=256, d=131072, F=32767), 0),
])
def test_gated_desc(kw, code):
    assert size_of(lib.moe_gated_ff_workspace_size, gated(**kw), 1, 1)[0] == code


def test_gated_workspace_sizes():
    size = lib.moe_gated_ff_workspace_size
    assert size(ref(gated()), 0, 1, None) == 1
    assert size_of(size, None, 0, 1)[0] == 1
    fwd, back, again = (size_of(size, gated(), *a)[1] for a in ((0, 1), (1, 1), (1, 0)))
    assert fwd <= back < again
    assert back >= 40 * 64 * 2 and again >= back + 40 * 64 * 4
    # slices of K: only one group's
    assert size_of(size, gated(E=1, M=256, d=7168, F=2048), 0, 1)[1] > 0
    assert size_of(size, gated(E=2, M=256, d=7168, F=2048), 0, 1)[1] == 0


def forward_args(**kw):
    a = dict(x=P, w_gate=P, w_up=P, offsets=P, h=P, pre=None)
    a.update(kw)
    return [a[n] for n in ("x", "w_gate", "w_up", "offsets", "h", "pre")]


def test_gated_forward_checks():
    f = lib.moe_gated_ff
    d, one = gated(), gated(E=1, M=256, d=7168, F=2048)
    need = size_of(lib.moe_gated_ff_workspace_size, one, 0, 1)[1]
    assert f(None, *forward_args(), P, 1 << 20, None) == 1
    for hole in ("x", "w_gate", "w_up", "h", "offsets"):
        assert f(ref(d), *forward_args(**{hole: None}), P, 1 << 20, None) == 1, hole
    for bad in ("x", "w_gate", "w_up", "h", "offsets", "pre"):
        assert f(ref(d), *forward_args(**{bad: ODD}), P, 1 << 20, None) == 5, bad
    assert f(ref(one), *forward_args(offsets=None), P, need - 1, None) == 4
    assert f(ref(one), *forward_args(offsets=None), None, need, None) == 4
    assert f(ref(one), *forward_args(offsets=None), EIGHT, need, None) == 5
    assert f(ref(gated(act=9)), *forward_args(), P, 1 << 20, None) == 3
    nothing = gated(M=0, E=1)
    assert f(ref(nothing), *[None] * 6, None, 0, None) == 0


def backward_args(**kw):
    a = dict(x=P, w_gate=P, w_up=P, offsets=P, dh=P, pre=P, dx=P, dw_gate=P, dw_up=P)
    a.update(kw)
    return [a[n] for n in ("x", "w_gate", "w_up", "offsets", "dh", "pre", "dx", "dw_gate", "dw_up")]


def test_gated_backward_checks():
    f = lib.moe_gated_ff_backward
    d = gated()
    need = size_of(lib.moe_gated_ff_workspace_size, d, 1, 1)[1]
    again = size_of(lib.moe_gated_ff_workspace_size, d, 1, 0)[1]
    assert f(None, *backward_args(), P, need, None) == 1
    for hole in ("x", "w_gate", "w_up", "dh", "offsets", "dw_gate", "dw_up"):
        assert f(ref(d), *backward_args(**{hole: None}), P, need, None) == 1, hole
    for bad in ("x", "w_gate", "w_up", "dh", "offsets", "pre", "dx", "dw_gate", "dw_up"):
        assert f(ref(d), *backward_args(**{bad: ODD}), P, need, None) == 5, bad
    assert f(ref(d), *backward_args(), P, need - 1, None) == 4
    assert f(ref(d), *backward_args(), None, need, None) == 4
    assert f(ref(d), *backward_args(), EIGHT, need, None) == 5
    assert f(ref(d), *backward_args(pre=None), P, again - 1, None) == 4
    assert f(ref(gated(M=-1)), *backward_args(), P, need, None) == 2


# -------------------------------------------------------------- e4m3 products

def test_quantize_fp8_checks():
    q = lib.moe_quantize_fp8
    assert q(-1, 64, L.F32, P, P, P, None) == 2
    assert q(4, 0, L.F32, P, P, P, None) == 2
    assert q(4, 64, L.MXFP4, P, P, P, None) == 3
    assert q(4, 131073, L.F32, P, P, P, None) == 5
    assert q((1 << 31) - 1023, 64, L.F32, P, P, P, None) == 5
    for hole in range(3):
        a = [P, P, P]
        a[hole] = None
        assert q(4, 64, L.F32, *a, None) == 1
    assert q(4, 64, L.BF16, P, EIGHT, P, None) == 5
    assert q(4, 64, L.BF16, ODD, P, P, None) == 5
    assert q(4, 64, L.BF16, P, P, ODD, None) == 5
    assert q(0, 64, L.BF16, None, None, None, None) == 0


def test_quantize_fp8_weights_checks():
    q = lib.moe_quantize_fp8_weights
    assert q(-1, 8, 64, L.F32, P, P, P, None) == 2
    assert q(1, -1, 64, L.F32, P, P, P, None) == 2
    assert q(1, 8, 0, L.F32, P, P, P, None) == 2
    assert q(1, 8, 64, 5, P, P, P, None) == 3
    assert q(1, 8, 131073, L.F32, P, P, P, None) == 5
    assert q(65536, 8, 64, L.F32, P, P, P, None) == 5
    assert q(1, 65535 * 128 + 1, 64, L.F32, P, P, P, None) == 5
    assert q(65535, 65535 * 128, 131072, L.F32, P, P, P, None) == 5
    for hole in range(3):
        a = [P, P, P]
        a[hole] = None
        assert q(1, 8, 64, L.F32, *a, None) == 1
    assert q(1, 8, 64, L.F32, P, EIGHT, P, None) == 5
    assert q(0, 8, 64, L.F32, None, None, None, None) == 0
    assert q(1, 0, 64, L.F32, None, None, None, None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 2), (dict(N=-1), 2), (dict(K=0), 2), (dict(E=0), 2), (dict(out=2), 3),
    (dict(K=131073), 5), (dict(E=257), 5), (dict(E=256, N=1 << 24, K=1 << 14), 5),
    (dict(M=1 << 30, K=1 << 11), 5), (dict(M=(1 << 31) - 1023), 5), (dict(N=(1 << 31) - 1023), 5),
    (dict(M=(1 << 31) - 1024), 0), (dict(), 0), (dict(M=0), 0), (dict(K=131072), 0),
])
def test_gemm_fp8_desc(kw, code):
    d = L.GemmFp8Desc(**{**dict(M=4, N=8, K=100, E=1, out=L.BF16), **kw})
    assert size_of(lib.moe_gemm_fp8_workspace_size, d)[0] == code


def test_gemm_fp8_checks():
    g = lib.moe_gemm_fp8
    d = L.GemmFp8Desc(4, 8, 100, 1, L.BF16)
    assert g(None, P, P, P, P, None, P, P, 0, None) == 1
    for hole in range(4):
        a = [P, P, P, P]
        a[hole] = None
        assert g(ref(d), *a, None, P, P, 0, None) == 1
    assert g(ref(d), P, P, P, P, None, None, P, 0, None) == 1
    assert g(ref(d), EIGHT, P, P, P, None, P, P, 0, None) == 5
    assert g(ref(d), P, ODD, P, P, None, P, P, 0, None) == 5
    assert g(ref(d), P, P, EIGHT, P, None, P, P, 0, None) == 5
    assert g(ref(d), P, P, P, ODD, None, P, P, 0, None) == 5
    assert g(ref(d), P, P, P, P, ODD, P, P, 0, None) == 5
    assert g(ref(d), P, P, P, P, None, EIGHT, P, 0, None) == 5
    grouped = L.GemmFp8Desc(4, 8, 100, 2, L.BF16)
    assert g(ref(grouped), P, P, P, P, None, P, P, 0, None) == 1    # offsets missing
    sliced = L.GemmFp8Desc(1024, 2048, 7168, 1, L.BF16)
    need = size_of(lib.moe_gemm_fp8_workspace_size, sliced)[1]
    assert need >= 2 * 1024 * 2048 * 4 and need % (1024 * 2048 * 4) == 0
    assert g(ref(sliced), P, P, P, P, None, P, P, need - 1, None) == 4
    assert g(ref(sliced), P, P, P, P, None, P, None, need, None) == 4
    assert g(ref(sliced), P, P, P, P, None, P, EIGHT, need, None) == 5
    assert g(ref(L.GemmFp8Desc(0, 8, 100, 1, L.BF16)), None, None, None, None, None, None, None, 0,
             None) == 0
    assert lib.moe_gemm_fp8_workspace_size(ref(d), None) == 1


# -------------------------------------------------------------------- AdamW

def adamw(**kw):
    return L.AdamwDesc(**{**dict(count=1, param=L.F32, grad=L.F32, state_bits=32), **kw})


def tensor(**kw):
    t = L.AdamwTensor(p=0x1000, g=0x1000, m=0x1000, v=0x1000, n=10)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), 2), (dict(param=2), 3), (dict(grad=5), 3), (dict(state_bits=16), 3),
    (dict(count=(1 << 20) + 1), 5), (dict(), 0), (dict(count=0), 0), (dict(count=1 << 20), 0),
    (dict(param=L.BF16, grad=L.F32, state_bits=8), 0),
])
def test_adamw_desc(kw, code):
    st, n = size_of(lib.moe_adamw_table_size, adamw(**kw))
    assert st == code and (code != 0 or n >= 80 * kw.get("count", 1))


@pytest.mark.parametrize("dk,tk,code", [
    ({}, dict(n=-1), 2), ({}, dict(n=(1 << 40) + 1), 5), ({}, dict(p=None), 1),
    ({}, dict(g=None), 1), ({}, dict(m=None), 1), ({}, dict(v=None), 1),
    (dict(state_bits=8), {}, 1), (dict(state_bits=8), dict(m_scale=0x1000), 1),
    (dict(state_bits=8), dict(m_scale=0x1000, v_scale=0x1000, m_values=0x1000), 1),
    (dict(param=L.BF16), dict(copy=0x1000), 3),
    ({}, dict(p=0x1002), 5), (dict(param=L.BF16), dict(p=0x1001), 5), ({}, dict(g=0x1002), 5),
    (dict(grad=L.BF16), dict(g=0x1001), 5), ({}, dict(m=0x1002), 5), ({}, dict(v=0x1001), 5),
    ({}, dict(copy=0x1001), 5),
    (dict(state_bits=8), dict(m_scale=0x1001, v_scale=0x1000), 5),
])
def test_adamw_tensors(dk, tk, code):
    n = ctypes.c_int64(0)
    t = (L.AdamwTensor * 1)(tensor(**tk))
    assert lib.moe_adamw_prepare(ref(adamw(**dk)), t, ref(n), P, 1 << 20, None) == code


def test_adamw_prepare_checks():
    f, n = lib.moe_adamw_prepare, ctypes.c_int64(0)
    t, need = (L.AdamwTensor * 1)(tensor()), size_of(lib.moe_adamw_table_size, adamw())[1]
    assert f(None, t, ref(n), P, need, None) == 1
    assert f(ref(adamw()), None, ref(n), P, need, None) == 1
    assert f(ref(adamw()), t, None, P, need, None) == 1
    assert f(ref(adamw()), t, ref(n), P, need - 1, None) == 4
    assert f(ref(adamw()), t, ref(n), None, need, None) == 4
    assert f(ref(adamw()), t, ref(n), EIGHT, need, None) == 5
    many = (L.AdamwTensor * 2)(tensor(n=1 << 40), tensor(n=1))
    assert f(ref(adamw(count=2)), many, ref(n), P, 1 << 20, None) == 5
    assert f(ref(adamw(count=0)), None, ref(n), P, 1 << 20, None) == 0 and n.value == 0


@pytest.mark.parametrize("first,second", [
    (dict(p=0x1000, n=100), dict(p=0x1000, n=100)), (dict(p=0x1000, n=100), dict(p=0x118c, n=1)),
    (dict(p=0x2000, n=10), dict(p=0x1000, n=1025)),
])
def test_parameters_that_overlap_are_refused(first, second):
    n = ctypes.c_int64(0)
    t = (L.AdamwTensor * 3)(tensor(**first), tensor(n=0), tensor(**second))
    assert lib.moe_adamw_prepare(ref(adamw(count=3)), t, ref(n), P, 1 << 20, None) == 5


@pytest.mark.parametrize("kw,code", [
    (dict(step=0), 2), (dict(beta1=1.0), 2), (dict(beta1=-0.1), 2), (dict(beta2=1.0), 2),
    (dict(beta2=float("nan")), 2), (dict(eps=-1e-8), 2), (dict(eps=float("inf")), 2),
    (dict(weight_decay=float("nan")), 2), (dict(lr=float("inf")), 2),
    (dict(lr_dev=0x1002), 5), (dict(step_dev=0x1004), 5), (dict(grad_scale_dev=0x1001), 5),
])
def test_adamw_step_checks(kw, code):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1)
    s = L.AdamwStep(**{**base, **kw})
    assert lib.moe_adamw(ref(adamw()), ref(s), 1, P, None) == code
    ok = L.AdamwStep(**base)
    assert lib.moe_adamw(ref(adamw()), None, 1, P, None) == 1
    assert lib.moe_adamw(ref(adamw()), ref(ok), -1, P, None) == 2
    assert lib.moe_adamw(ref(adamw()), ref(ok), 1, None, None) == 1
    assert lib.moe_adamw(ref(adamw()), ref(ok), 1, EIGHT, None) == 5
    assert lib.moe_adamw(ref(adamw()), ref(ok), 0, None, None) == 0
    assert lib.moe_adamw(ref(adamw(count=0)), ref(ok), 0, None, None) == 0


def test_adamw_values_checks():
    f = lib.moe_adamw_state_values
    assert f(ref(adamw()), 1, P, None) == 3           # fp32 states have none
    eight = adamw(state_bits=8)
    assert f(None, 1, P, None) == 1
    assert f(ref(eight), -1, P, None) == 2
    assert f(ref(eight), 1, None, None) == 1
    assert f(ref(eight), 1, EIGHT, None) == 5
    assert f(ref(eight), 0, None, None) == 0


# ------------------------------------------------------------------ binding

def test_tensors_not_on_a_gpu_are_refused():
    x, w, h = torch.zeros(4, 8), torch.zeros(1, 16, 8), torch.zeros(4, 16)
    with pytest.raises(ValueError):
        L.gated_ff(x, w, w, h)
    with pytest.raises(ValueError):
        L.gated_ff_backward(x, w, w, h, None, None, None)
    with pytest.raises(ValueError):
        L.quantize_fp8(x)
    with pytest.raises(ValueError):
        L.quantize_fp8_weights(w)
    with pytest.raises(ValueError):
        L.gemm_fp8(x, x, w, w, h)
    with pytest.raises(ValueError):
        L.adamw_plan([x], [x], [x], [x])


def test_plan_lists():
    x = torch.zeros(4)
    with pytest.raises(ValueError):
        L.adamw_plan([], [], [], [])
    with pytest.raises(ValueError):
        L.adamw_plan([x, x], [x], [x, x], [x, x])
    with pytest.raises(TypeError):
        L.adamw_plan([3], [x], [x], [x])
