"""Refusals of the INT8 calls: every argument error is a status from the
host, before any HIP call (no GPU needed), and the binding refuses what it can
see."""
import pytest
import torch

import quantized_moe_grouped_route_amd as mq
from tests.test_abi_lora import L, at  # noqa: F401  (L: the library, a fixture)


def _quant(L, **kw):
    a = dict(x=at(0), dt=mq.BF16, rows=4, K=64, q=at(1), s=at(2))
    a.update(kw)
    return L.moe_quantize_int8(a["x"], a["dt"], a["rows"], a["K"], a["q"], a["s"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), mq.EINVAL), (dict(rows=2 ** 31), mq.EINVAL), (dict(K=0), mq.EINVAL), (dict(K=2 ** 24 + 16), mq.EINVAL),
    (dict(K=72), mq.EALIGN), (dict(dt=mq.I32), mq.EUNSUPPORTED), (dict(dt=mq.U8), mq.EUNSUPPORTED),
    (dict(x=None), mq.EINVAL), (dict(q=None), mq.EINVAL), (dict(s=None), mq.EINVAL), (dict(x=at(0) + 8), mq.EALIGN),
    (dict(q=at(1) + 8), mq.EALIGN), (dict(s=at(2) + 2), mq.EALIGN), (dict(q=at(0)), mq.EINVAL),
    (dict(q=at(0) + 4 * 64 * 2 - 16), mq.EINVAL), (dict(q=at(0) - 4 * 64 + 16), mq.EINVAL), (dict(s=at(0) + 508), mq.EINVAL),
    (dict(s=at(1) + 252), mq.EINVAL),
])
def test_quantize_rejects(L, kw, status):
    assert _quant(L, **kw) == status
    assert b"moe_quantize_int8" in L.moeq_last_error()


def _gemm(L, **kw):
    a = dict(a=at(0), sa=at(1), rows=8, arow=0, w=at(2), sw=at(3), off=at(4), srt=at(5), P=16, topk=2, E=4, N=64, K=128,
             act=0, od=mq.F16, out=at(6), sched=0)
    a.update(kw)
    return L.grouped_gemm_qint8(a["a"], a["sa"], a["rows"], a["arow"], a["w"], a["sw"], a["off"], a["srt"], a["P"],
                                a["topk"], a["E"], a["N"], a["K"], a["act"], a["od"], a["out"], a["sched"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), mq.EINVAL), (dict(E=1025), mq.EINVAL), (dict(topk=0), mq.EINVAL), (dict(topk=65), mq.EINVAL),
    (dict(P=-1), mq.EINVAL), (dict(P=2 ** 31), mq.EINVAL), (dict(rows=0), mq.EINVAL), (dict(rows=2 ** 31), mq.EINVAL),
    (dict(N=0), mq.EINVAL), (dict(N=48), mq.EALIGN), (dict(K=64), mq.EALIGN), (dict(K=192), mq.EALIGN),
    (dict(K=131072), mq.EINVAL), (dict(N=2 ** 20 + 32), mq.EINVAL), (dict(arow=2), mq.EINVAL),
    (dict(a=None), mq.EINVAL), (dict(w=None), mq.EINVAL), (dict(off=None), mq.EINVAL), (dict(out=None), mq.EINVAL),
    (dict(sa=None), mq.EINVAL), (dict(sw=None), mq.EINVAL), (dict(a=at(0) + 4), mq.EALIGN), (dict(sa=at(1) + 2), mq.EALIGN),
    (dict(srt=at(5) + 1), mq.EALIGN), (dict(out=at(6) + 8), mq.EALIGN), (dict(act=2), mq.EUNSUPPORTED),
    (dict(od=mq.U8), mq.EUNSUPPORTED), (dict(od=mq.I32, act=1), mq.EUNSUPPORTED), (dict(srt=None), mq.EINVAL),
    (dict(sched=3), mq.EINVAL), (dict(sched=-1), mq.EINVAL), (dict(P=2 ** 30, N=2 ** 20, rows=2 ** 30), mq.EINVAL),
    (dict(rows=7), mq.EINVAL), (dict(arow=1, rows=15), mq.EINVAL), (dict(arow=1, rows=15, srt=None), mq.EINVAL),
    (dict(out=at(0)), mq.EINVAL), (dict(out=at(1)), mq.EINVAL), (dict(out=at(2) + 4 * 64 * 128 - 16), mq.EINVAL),
    (dict(out=at(3)), mq.EINVAL), (dict(out=at(4)), mq.EINVAL), (dict(out=at(5)), mq.EINVAL),
    (dict(out=at(5) - 16 * 64 * 2 + 16), mq.EINVAL), (dict(out=at(5) - 16 * 64 * 4 + 16, od=mq.I32), mq.EINVAL),
    (dict(out=at(5) - 16 * 32 * 4 + 16, od=mq.F32, act=1), mq.EINVAL),
])
def test_gemm_rejects(L, kw, status):
    assert _gemm(L, **kw) == status
    assert b"grouped_gemm_qint8" in L.moeq_last_error()


def test_gemm_without_rows_takes_null_rows(L):
    assert _gemm(L, P=0, rows=0, a=None, sa=None, out=None, srt=None) == mq.OK
    assert _gemm(L, P=0, rows=0, a=None, sa=None, out=None, srt=None, w=None) == mq.EINVAL


def _grad(L, **kw):
    a = dict(dy=at(0), dt=mq.BF16, w=at(1), sw=at(2), off=at(3), P=16, E=4, N=64, K=128, base=at(4), dx=at(5), ws=at(6),
             wsb=1 << 30)
    a.update(kw)
    return L.grouped_gemm_qint8_backward(a["dy"], a["dt"], a["w"], a["sw"], a["off"], a["P"], a["E"], a["N"], a["K"],
                                         a["base"], a["dx"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=mq.F32), mq.EUNSUPPORTED), (dict(dt=0), mq.EUNSUPPORTED), (dict(E=0), mq.EINVAL), (dict(E=1025), mq.EINVAL),
    (dict(P=-1), mq.EINVAL), (dict(P=2 ** 31), mq.EINVAL), (dict(N=0), mq.EINVAL), (dict(N=131072), mq.EINVAL),
    (dict(N=48), mq.EALIGN), (dict(K=64), mq.EALIGN), (dict(K=131072 + 128), mq.EINVAL), (dict(dy=None), mq.EINVAL),
    (dict(w=None), mq.EINVAL), (dict(sw=None), mq.EINVAL), (dict(off=None), mq.EINVAL), (dict(dx=None), mq.EINVAL),
    (dict(ws=None), mq.EINVAL), (dict(wsb=16 * (2 * 128 + 4) - 1), mq.EINVAL), (dict(dy=at(0) + 8), mq.EALIGN),
    (dict(base=at(4) + 8), mq.EALIGN), (dict(dx=at(5) + 2), mq.EALIGN), (dict(ws=at(6) + 4), mq.EALIGN),
    (dict(sw=at(2) + 2), mq.EALIGN), (dict(off=at(3) + 2), mq.EALIGN), (dict(dx=at(0)), mq.EINVAL),
    (dict(dx=at(1)), mq.EINVAL), (dict(dx=at(2)), mq.EINVAL), (dict(dx=at(3)), mq.EINVAL),
    (dict(dx=at(4) + 16), mq.EINVAL), (dict(dx=at(4) - 16), mq.EINVAL), (dict(ws=at(0)), mq.EINVAL),
    (dict(ws=at(3)), mq.EINVAL), (dict(ws=at(4)), mq.EINVAL), (dict(ws=at(5)), mq.EINVAL),
    (dict(ws=at(5) - 16 * (2 * 128 + 4) + 16), mq.EINVAL), (dict(P=2 ** 31 - 1, K=131072, wsb=1 << 60), mq.EINVAL),
])
def test_gemm_backward_rejects(L, kw, status):
    assert _grad(L, **kw) == status
    assert b"grouped_gemm_qint8_backward" in L.moeq_last_error()


def test_gemm_backward_workspace_bytes(L):
    f = L.grouped_gemm_qint8_backward_workspace_bytes
    assert f(16, 4, 64, 128) == 16 * (2 * 128 + 4)      # rows of whole 128-value stages
    assert f(16, 4, 128, 128) == 16 * (2 * 128 + 4)
    assert f(16, 4, 160, 128) == 16 * (2 * 256 + 4)
    assert f(0, 4, 64, 128) == 0
    for bad in ((-1, 4, 64, 128), (2 ** 31, 4, 64, 128), (16, 0, 64, 128), (16, 1025, 64, 128), (16, 4, 48, 128),
                (16, 4, 131072, 128), (16, 4, 64, 64), (16, 4, 64, 131072 + 128), (2 ** 31 - 1, 4, 64, 131072)):
        assert f(*bad) == 0
    # no rows: nothing to check but the weights and the table, and nothing to do
    assert _grad(L, P=0, dy=None, dx=None, ws=None, wsb=0, base=None) == mq.OK


def _silu(L, **kw):
    a = dict(gu=at(0), dt=mq.BF16, off=at(1), E=4, P=16, I=136, h=at(2), ck=at(3), cs=at(4))
    a.update(kw)
    return L.moe_silu_mul(a["gu"], a["dt"], a["off"], a["E"], a["P"], a["I"], a["h"], a["ck"], a["cs"], None)


SILU_BAD = [
    (dict(dt=mq.I32), mq.EUNSUPPORTED), (dict(dt=mq.U8), mq.EUNSUPPORTED), (dict(E=0), mq.EINVAL), (dict(E=1025), mq.EINVAL),
    (dict(P=-1), mq.EINVAL), (dict(P=2 ** 31), mq.EINVAL), (dict(I=0), mq.EINVAL), (dict(I=2 ** 20 + 8), mq.EINVAL),
    (dict(I=132), mq.EALIGN), (dict(off=at(1) + 2), mq.EALIGN), (dict(ck=at(3) + 8), mq.EALIGN), (dict(cs=at(4) + 2), mq.EALIGN),
    (dict(ck=None), mq.EINVAL), (dict(cs=None), mq.EINVAL),
]


@pytest.mark.parametrize("kw,status", SILU_BAD + [
    (dict(gu=None), mq.EINVAL), (dict(h=None), mq.EINVAL), (dict(gu=at(0) + 8), mq.EALIGN), (dict(h=at(2) + 8), mq.EALIGN),
    (dict(h=at(0)), mq.EINVAL), (dict(h=at(0) + 16 * 272 * 2 - 16), mq.EINVAL), (dict(h=at(1)), mq.EINVAL),
    (dict(ck=at(0)), mq.EINVAL), (dict(ck=at(2)), mq.EINVAL), (dict(cs=at(3) + 16 * 272 - 4), mq.EINVAL),
    (dict(cs=at(2) - 16 * 4 * 4 + 4), mq.EINVAL), (dict(cs=at(1)), mq.EINVAL),
])
def test_silu_rejects(L, kw, status):
    assert _silu(L, **kw) == status
    assert b"moe_silu_mul" in L.moeq_last_error()


def _silu_bwd(L, **kw):
    a = dict(dh=at(0), dt=mq.BF16, gu=None, ck=at(3), cs=at(4), off=at(1), E=4, P=16, I=136, dgu=at(2), h=at(5))
    a.update(kw)
    return L.moe_silu_mul_backward(a["dh"], a["dt"], a["gu"], a["ck"], a["cs"], a["off"], a["E"], a["P"], a["I"],
                                   a["dgu"], a["h"], None)


@pytest.mark.parametrize("kw,status", SILU_BAD + [
    (dict(dh=None), mq.EINVAL), (dict(dgu=None), mq.EINVAL), (dict(dh=None, dgu=None, h=None), mq.EINVAL),
    (dict(dh=None, dgu=None, ck=None, cs=None), mq.EINVAL), (dict(gu=at(6)), mq.EINVAL),
    (dict(ck=None, cs=None), mq.EINVAL), (dict(dh=at(0) + 8), mq.EALIGN), (dict(dgu=at(2) + 8), mq.EALIGN),
    (dict(h=at(5) + 8), mq.EALIGN), (dict(gu=at(6) + 8, ck=None, cs=None), mq.EALIGN), (dict(dgu=at(0)), mq.EINVAL),
    (dict(dgu=at(3)), mq.EINVAL), (dict(dgu=at(4)), mq.EINVAL), (dict(dgu=at(1)), mq.EINVAL), (dict(h=at(0)), mq.EINVAL),
    (dict(h=at(2) + 16 * 272 * 2 - 16), mq.EINVAL), (dict(h=at(3)), mq.EINVAL), (dict(h=at(1)), mq.EINVAL),
    (dict(gu=at(2) + 16, ck=None, cs=None), mq.EINVAL), (dict(gu=at(5), ck=None, cs=None), mq.EINVAL),
])
def test_silu_backward_rejects(L, kw, status):
    assert _silu_bwd(L, **kw) == status
    assert b"moe_silu_mul_backward" in L.moeq_last_error()


def test_silu_without_rows_takes_null_pointers(L):
    assert _silu(L, P=0, gu=None, h=None, ck=None, cs=None) == mq.OK
    assert _silu_bwd(L, P=0, dh=None, dgu=None, ck=None, cs=None, h=None) == mq.OK
    assert _silu(L, P=0, off=None, E=0, gu=None, h=None, ck=None, cs=None) == mq.OK     # E is read with offsets only


# ---------------------------------------------------------------- binding
def _t(*s, dt=torch.bfloat16):
    return torch.zeros(*s, dtype=dt)


I8, F4, I4 = torch.int8, torch.float32, torch.int32


@pytest.mark.parametrize("call,error,text", [
    (lambda: mq.quantize_int8_rows(_t(4, 64)), ValueError, "x must be on the GPU"),
    (lambda: mq.quantize_int8_rows(_t(4, 64, dt=I8)), TypeError, "x has dtype"),
    (lambda: mq.quantize_int8_rows(_t(4, 64).T), ValueError, "contiguous"),
    (lambda: mq.quantize_int8_rows(_t(4, 64), q=_t(4, 32, dt=I8)), ValueError, "q must be"),
    (lambda: mq.quantize_int8_rows(_t(4, 64), scale=_t(3, dt=F4)), ValueError, "scale must be"),
])
def test_binding_refuses_quantize(L, call, error, text):
    with pytest.raises(error, match=text):
        call()


def _bg(a=None, sa=None, w=None, sw=None, off=None, srt=None, **kw):
    pick = lambda v, d: d if v is None else v
    return mq.grouped_gemm_qint8(pick(a, _t(4, 128, dt=I8)), pick(sa, _t(4, dt=F4)), pick(w, _t(3, 64, 128, dt=I8)),
                                 pick(sw, _t(3, 64, dt=F4)), pick(off, _t(4, dt=I4)), pick(srt, _t(8, dt=I4)), 2, **kw)


@pytest.mark.parametrize("kw,error,text", [
    (dict(), ValueError, "a must be on the GPU"), (dict(a=_t(4, 128, dt=torch.uint8)), TypeError, "a has dtype"),
    (dict(a=_t(4, 64, dt=I8)), ValueError, "operand shapes"), (dict(sa=_t(5, dt=F4)), ValueError, "operand shapes"),
    (dict(sw=_t(3, 32, dt=F4)), ValueError, "weight shapes"), (dict(off=_t(5, dt=I4)), ValueError, "weight shapes"),
    (dict(out_dtype=torch.int64), TypeError, "out_dtype"), (dict(out=_t(8, 32, dt=torch.float16)), ValueError, "out must be"),
    (dict(out=_t(8, 64)), TypeError, "out has dtype"), (dict(P=9), ValueError, "sorted_pair_ids needs"),
    (dict(srt=_t(8, dt=torch.int64)), TypeError, "sorted_pair_ids has dtype"),
    (dict(act="silu_mul", out=_t(8, 64, dt=torch.float16)), ValueError, "out must be"),
])
def test_binding_refuses_gemm(L, kw, error, text):
    with pytest.raises(error, match=text):
        _bg(**kw)


def _bb(dy=None, w=None, sw=None, off=None, **kw):
    pick = lambda v, d: d if v is None else v
    return mq.grouped_gemm_qint8_backward(pick(dy, _t(8, 64)), pick(w, _t(3, 64, 128, dt=I8)), pick(sw, _t(3, 64, dt=F4)),
                                          pick(off, _t(4, dt=I4)), **kw)


@pytest.mark.parametrize("kw,error,text", [
    (dict(), ValueError, "dy must be on the GPU"), (dict(dy=_t(8, 64, dt=F4)), TypeError, "dy has dtype"),
    (dict(dy=_t(8, 32)), ValueError, "dy must be"), (dict(base=_t(8, 64)), ValueError, "base must be"),
    (dict(base=_t(8, 128, dt=torch.float16)), TypeError, "base has dtype"), (dict(dx=_t(7, 128)), ValueError, "dx must be"),
    (dict(off=_t(3, dt=I4)), ValueError, "weight shapes"), (dict(workspace=[1]), TypeError, "workspace"),
])
def test_binding_refuses_gemm_backward(L, kw, error, text):
    with pytest.raises(error, match=text):
        _bb(**kw)


@pytest.mark.parametrize("call,error,text", [
    (lambda: mq.moe_silu_mul(_t(4, 16)), ValueError, "gu must be on the GPU"),
    (lambda: mq.moe_silu_mul(_t(4, 15)), ValueError, "even number"),
    (lambda: mq.moe_silu_mul(_t(4, 16, dt=I8)), TypeError, "gu has dtype"),
    (lambda: mq.moe_silu_mul(_t(4, 16), ck=_t(4, 16, dt=I8)), ValueError, "checkpoint is false"),
    (lambda: mq.moe_silu_mul(_t(4, 16), cs=_t(4, 2, dt=F4)), ValueError, "checkpoint is false"),
    (lambda: mq.moe_silu_mul(_t(4, 16), checkpoint=True, ck=_t(4, 8, dt=I8)), ValueError, "ck must be"),
    (lambda: mq.moe_silu_mul(_t(4, 272), checkpoint=True, cs=_t(4, 2, dt=F4)), ValueError, "cs must be"),
    (lambda: mq.moe_silu_mul(_t(4, 16), _t(3, dt=torch.int64)), TypeError, "expert_offsets has dtype"),
    (lambda: mq.moe_silu_mul(_t(4, 16), _t(0, dt=I4)), ValueError, "E\\+1 entries"),
    (lambda: mq.moe_silu_mul_backward(_t(4, 8), _t(1, dt=I4), gu=_t(4, 16)), ValueError, "E\\+1 entries"),
    (lambda: mq.moe_silu_mul_backward(_t(4, 8)), ValueError, "give gu"),
    (lambda: mq.moe_silu_mul_backward(_t(4, 8), gu=_t(4, 16), ck=_t(4, 16, dt=I8), cs=_t(4, 2, dt=F4)), ValueError, "give gu"),
    (lambda: mq.moe_silu_mul_backward(_t(4, 8), ck=_t(4, 16, dt=I8)), ValueError, "give gu"),
    (lambda: mq.moe_silu_mul_backward(_t(4, 8), gu=_t(4, 16, dt=F4)), TypeError, "gu has dtype"),
    (lambda: mq.moe_silu_mul_backward(_t(4, 8), gu=_t(4, 24)), ValueError, "gu must be"),
    (lambda: mq.moe_silu_mul_backward(_t(4, 8), gu=_t(4, 16), h=_t(4, 8)), ValueError, "need_h is false"),
    (lambda: mq.moe_silu_mul_backward(_t(4, 8), gu=_t(4, 16)), ValueError, "dh must be on the GPU"),
    (lambda: mq.moe_silu_mul_again(_t(4, 16, dt=I8), _t(4, 2, dt=F4)), ValueError, "ck must be on the GPU"),
    (lambda: mq.moe_silu_mul_again(_t(4, 16), _t(4, 2, dt=F4)), TypeError, "ck has dtype"),
    (lambda: mq.moe_silu_mul_again(_t(4, 16, dt=I8), _t(4, 4, dt=F4)), ValueError, "cs must be"),
    (lambda: mq.moe_silu_mul_again(_t(4, 16, dt=I8), _t(4, 2, dt=F4), dtype=I8), TypeError, "floating type"),
    (lambda: mq.moe_silu_mul_again(_t(4, 16, dt=I8), _t(4, 2, dt=F4), h=_t(4, 8, dt=F4)), TypeError, "h has dtype"),
])
def test_binding_refuses_silu(L, call, error, text):
    with pytest.raises(error, match=text):
        call()
