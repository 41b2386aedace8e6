"""Refusals of the permutation, combine-gradient and adapter calls: every
argument error is a status from the host, before any HIP call (no GPU
needed), and the binding refuses what it can see."""
import os

import pytest
import torch

import quantized_moe_grouped_route_amd as mq

# Fake device addresses, far apart: only their values are inspected.
STEP = 1 << 44


def at(i):
    return (i + 1) * STEP


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mq.LIB_PATH):
        pytest.skip("libmoeq.so not built")
    return mq.lib()


def _permute(L, **kw):
    a = dict(x=at(0), dt=mq.BF16, p2s=at(1), T=4, topk=2, N=64, xs=at(2))
    a.update(kw)
    return L.moe_permute(a["x"], a["dt"], a["p2s"], a["T"], a["topk"], a["N"], a["xs"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), mq.EINVAL), (dict(T=2 ** 31), mq.EINVAL), (dict(T=2 ** 62, topk=4), mq.EINVAL),
    (dict(T=2 ** 30, topk=2), mq.EINVAL), (dict(topk=0), mq.EINVAL), (dict(topk=65), mq.EINVAL),
    (dict(N=0), mq.EINVAL), (dict(N=2 ** 24 + 8), mq.EINVAL), (dict(N=12), mq.EALIGN),
    (dict(dt=mq.U8, N=24), mq.EALIGN), (dict(dt=mq.I32), mq.EUNSUPPORTED), (dict(dt=0), mq.EUNSUPPORTED),
    (dict(x=None), mq.EINVAL), (dict(p2s=None), mq.EINVAL), (dict(xs=None), mq.EINVAL),
    (dict(x=at(0) + 8), mq.EALIGN), (dict(xs=at(2) + 2), mq.EALIGN), (dict(p2s=at(1) + 2), mq.EALIGN),
    (dict(xs=at(0)), mq.EINVAL), (dict(xs=at(0) + 4 * 64 * 2 - 16), mq.EINVAL),
    (dict(xs=at(0) - 8 * 64 * 2 + 16), mq.EINVAL),
])
def test_permute_rejects(L, kw, status):
    assert _permute(L, **kw) == status
    assert b"moe_permute" in L.moeq_last_error()


def _permute_bwd(L, **kw):
    a = dict(d=at(0), dd=mq.BF16, p2s=at(1), T=4, topk=2, N=64, xd=mq.F32, dx=at(2))
    a.update(kw)
    return L.moe_permute_backward(a["d"], a["dd"], a["p2s"], a["T"], a["topk"], a["N"], a["xd"], a["dx"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), mq.EINVAL), (dict(topk=65), mq.EINVAL), (dict(N=4), mq.EALIGN), (dict(dd=mq.U8), mq.EUNSUPPORTED),
    (dict(xd=mq.U8), mq.EUNSUPPORTED), (dict(xd=mq.I32), mq.EUNSUPPORTED), (dict(d=None), mq.EINVAL),
    (dict(dx=None), mq.EINVAL), (dict(p2s=None), mq.EINVAL), (dict(d=at(0) + 4), mq.EALIGN),
    (dict(dx=at(0)), mq.EINVAL), (dict(dx=at(0) + 8 * 64 * 2 - 16), mq.EINVAL),
])
def test_permute_backward_rejects(L, kw, status):
    assert _permute_bwd(L, **kw) == status


def _combine_bwd(L, **kw):
    a = dict(d=at(0), dd=mq.BF16, y=at(1), yd=mq.F16, p2s=at(2), w=at(3), T=4, topk=2, N=64, dy=at(4), dw=at(5))
    a.update(kw)
    return L.moe_scatter_combine_backward(a["d"], a["dd"], a["y"], a["yd"], a["p2s"], a["w"], a["T"], a["topk"],
                                          a["N"], a["dy"], a["dw"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), mq.EINVAL), (dict(topk=0), mq.EINVAL), (dict(N=20), mq.EALIGN), (dict(dd=mq.I32), mq.EUNSUPPORTED),
    (dict(yd=mq.U8), mq.EUNSUPPORTED), (dict(w=None), mq.EINVAL), (dict(dy=None), mq.EINVAL),
    (dict(dw=None), mq.EINVAL), (dict(y=None), mq.EINVAL), (dict(dw=at(5) + 2), mq.EALIGN),
    (dict(dy=at(4) + 8), mq.EALIGN), (dict(dy=at(1)), mq.EINVAL), (dict(dy=at(0)), mq.EINVAL),
    (dict(dw=at(3)), mq.EINVAL), (dict(dw=at(4) + 64), mq.EINVAL),
])
def test_combine_backward_rejects(L, kw, status):
    assert _combine_bwd(L, **kw) == status


def _lora(L, **kw):
    # (K long enough to need a workspace)
    a = dict(x=at(0), dt=mq.BF16, rows=8, arow=0, a=at(1), b=at(2), sc=at(3), off=at(4), srt=at(5), p2s=None, P=16,
             topk=2, E=4, N=64, K=8192, R=16, base=at(6), orow=0, out=at(7), h=None, ws=at(8), wsb=1 << 30)
    a.update(kw)
    return L.grouped_lora(a["x"], a["dt"], a["rows"], a["arow"], a["a"], a["b"], a["sc"], a["off"], a["srt"],
                          a["p2s"], a["P"], a["topk"], a["E"], a["N"], a["K"], a["R"], a["base"], a["orow"],
                          a["out"], a["h"], a["ws"], a["wsb"], None)


LORA_SHARED = [
    (dict(dt=mq.F32), mq.EUNSUPPORTED), (dict(dt=mq.U8), mq.EUNSUPPORTED), (dict(E=0), mq.EINVAL),
    (dict(E=1025), mq.EINVAL), (dict(topk=0), mq.EINVAL), (dict(topk=65), mq.EINVAL), (dict(P=-1), mq.EINVAL),
    (dict(P=2 ** 31, rows=2 ** 30), mq.EINVAL), (dict(N=0), mq.EINVAL), (dict(K=2 ** 20 + 8), mq.EINVAL),
    (dict(N=60), mq.EALIGN), (dict(K=100), mq.EALIGN), (dict(R=12), mq.EALIGN), (dict(R=0), mq.EINVAL),
    (dict(R=264), mq.EINVAL), (dict(arow=2), mq.EINVAL), (dict(orow=2), mq.EINVAL), (dict(rows=7), mq.EINVAL),
    (dict(rows=15, arow=1), mq.EINVAL), (dict(rows=-1), mq.EINVAL), (dict(rows=2 ** 31), mq.EINVAL),
    (dict(x=None), mq.EINVAL), (dict(a=None), mq.EINVAL),
    (dict(b=None), mq.EINVAL), (dict(off=None), mq.EINVAL), (dict(srt=None), mq.EINVAL),
    (dict(srt=None, arow=1, rows=16, orow=1), mq.EINVAL),
    (dict(x=at(0) + 8), mq.EALIGN), (dict(a=at(1) + 2), mq.EALIGN), (dict(b=at(2) + 4), mq.EALIGN),
    (dict(sc=at(3) + 2), mq.EALIGN), (dict(ws=at(8) + 4), mq.EALIGN), (dict(wsb=0), mq.EINVAL),
    (dict(ws=None), mq.EINVAL), (dict(ws=at(0)), mq.EINVAL),
]


@pytest.mark.parametrize("kw,status", LORA_SHARED + [
    (dict(out=None), mq.EINVAL), (dict(out=at(7) + 8), mq.EALIGN), (dict(base=at(6) + 8), mq.EALIGN),
    (dict(h=at(9) + 4), mq.EALIGN), (dict(orow=1), mq.EINVAL), (dict(orow=1, base=None), mq.EINVAL),
    (dict(out=at(0)), mq.EINVAL), (dict(out=at(6) + 16), mq.EINVAL), (dict(out=at(1)), mq.EINVAL),
    (dict(h=at(7)), mq.EINVAL), (dict(ws=at(7)), mq.EINVAL), (dict(h=at(8)), mq.EINVAL),
    (dict(h=at(1)), mq.EINVAL), (dict(h=at(2) + 16), mq.EINVAL), (dict(ws=at(1)), mq.EINVAL),
    (dict(ws=at(2)), mq.EINVAL),
])
def test_lora_rejects(L, kw, status):
    assert _lora(L, **kw) == status
    assert b"grouped_lora" in L.moeq_last_error()


def _lora_bwd(L, **kw):
    a = dict(dy=at(0), dt=mq.BF16, orow=0, x=at(1), rows=8, arow=0, a=at(2), b=at(3), sc=at(4), h=at(5), off=at(6),
             srt=at(7), P=16, topk=2, E=4, N=64, K=128, R=16, dx=at(9), da=at(10), db=at(11), ws=at(8), wsb=1 << 30)
    a.update(kw)
    return L.grouped_lora_backward(a["dy"], a["dt"], a["orow"], a["x"], a["rows"], a["arow"], a["a"], a["b"],
                                   a["sc"], a["h"], a["off"], a["srt"], a["P"], a["topk"], a["E"], a["N"], a["K"],
                                   a["R"], a["dx"], a["da"], a["db"], a["ws"], a["wsb"], None)


BWD_AT = dict(x=at(1) + 8, a=at(2) + 2, b=at(3) + 4, sc=at(4) + 2)


@pytest.mark.parametrize("kw,status", [({n: BWD_AT.get(n, v) if st == mq.EALIGN and n in BWD_AT else v
                                         for n, v in kw.items()}, st) for kw, st in LORA_SHARED] + [
    (dict(dy=None), mq.EINVAL), (dict(h=None), mq.EINVAL), (dict(da=None), mq.EINVAL), (dict(db=None), mq.EINVAL),
    (dict(dy=at(0) + 2), mq.EALIGN), (dict(dx=at(9) + 8), mq.EALIGN), (dict(dx=at(1)), mq.EINVAL),
    (dict(da=at(2)), mq.EINVAL), (dict(db=at(10) + 16), mq.EINVAL), (dict(ws=at(11)), mq.EINVAL),
    (dict(dx=at(0)), mq.EINVAL), (dict(db=at(5)), mq.EINVAL),
])
def test_lora_backward_rejects(L, kw, status):
    assert _lora_bwd(L, **kw) == status


# More workgroups than one launch holds: rows, columns and ranks near their
# limits together; fewer rows of the same are taken.
@pytest.mark.parametrize("P,E,N,K,R", [(2 ** 31 - 1, 1, 2 ** 20, 8, 256), (2 ** 30, 1, 64, 2 ** 20, 256)])
def test_lora_refuses_what_one_launch_cannot_hold(L, P, E, N, K, R):
    kw = dict(P=P, E=E, N=N, K=K, R=R, rows=P, arow=1, topk=1, wsb=1 << 62)
    assert _lora(L, **kw) == mq.EINVAL
    assert b"too large for one launch" in L.moeq_last_error()
    assert _lora_bwd(L, **kw) == mq.EINVAL
    assert b"too large for one launch" in L.moeq_last_error()
    for f in (L.grouped_lora_workspace_bytes, L.grouped_lora_backward_workspace_bytes):
        assert f(P, E, N, K, R) == 0
        assert f(P >> 12, E, N, K, R) > 0


def test_lora_of_few_rows_needs_no_workspace(L):
    assert L.grouped_lora_workspace_bytes(16, 4, 64, 128, 16) == 0
    assert _lora(L, K=128, ws=None, wsb=0, out=None) == mq.EINVAL      # refused for out, not for the workspace
    assert b"null pointer" in L.moeq_last_error()
    assert L.grouped_lora_backward_workspace_bytes(16, 4, 64, 128, 16) > 0


def test_lora_workspace_sizes_of_refused_arguments_are_zero(L):
    for f in (L.grouped_lora_workspace_bytes, L.grouped_lora_backward_workspace_bytes):
        assert f(16, 4, 64, 8192, 16) > 0
        for bad in ((-1, 4, 64, 128, 16), (2 ** 31, 4, 64, 128, 16), (16, 0, 64, 128, 16), (16, 1025, 64, 128, 16),
                    (16, 4, 60, 128, 16), (16, 4, 64, 100, 16), (16, 4, 64, 128, 12), (16, 4, 64, 128, 264),
                    (16, 4, 2 ** 20 + 8, 128, 16)):
            assert f(*bad) == 0


def test_binding_refuses_before_the_library():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    x, a, b, off, srt = bf(8, 128), bf(4, 16, 128), bf(4, 64, 16), i32(5), i32(16)
    with pytest.raises(ValueError, match="GPU"):
        mq.moe_permute(bf(4, 64), i32(8), 2)
    with pytest.raises(ValueError, match="T\\*topk"):
        mq.moe_permute(bf(4, 64), i32(7), 2)
    with pytest.raises(ValueError, match="T\\*topk"):
        mq.moe_permute(bf(4, 64), i32(8), 0)
    with pytest.raises(ValueError, match="rows"):
        mq.moe_permute(bf(5, 64), i32(8), 2)
    with pytest.raises(ValueError, match="contiguous"):
        mq.moe_permute(bf(64, 4).t(), i32(8), 2)
    with pytest.raises(TypeError):
        mq.moe_permute(torch.zeros(4, 64, dtype=torch.float64), i32(8), 2)
    with pytest.raises(ValueError, match="out must be"):
        mq.moe_permute(bf(4, 64), i32(8), 2, out=bf(7, 64))
    with pytest.raises(TypeError, match="out_dtype"):
        mq.moe_permute_backward(bf(8, 64), i32(8), 2, out_dtype=torch.uint8)
    with pytest.raises(ValueError, match="dxs"):
        mq.moe_permute_backward(bf(7, 64), i32(8), 2)
    w = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="dout"):
        mq.moe_scatter_combine_backward(bf(3, 64), bf(8, 64), i32(8), w)
    with pytest.raises(ValueError, match="rows"):
        mq.moe_scatter_combine_backward(bf(4, 64), bf(9, 64), i32(8), w)
    with pytest.raises(ValueError, match="GPU"):
        mq.moe_scatter_combine_backward(bf(4, 64), bf(8, 64), i32(8), w)
    with pytest.raises(ValueError, match="GPU"):
        mq.grouped_lora(x, a, b, off, srt, 2)
    with pytest.raises(TypeError):
        mq.grouped_lora(x, a.half(), b, off, srt, 2)
    with pytest.raises(TypeError):
        mq.grouped_lora(x.float(), a.float(), b.float(), off, srt, 2)
    with pytest.raises(ValueError, match="adapter shapes"):
        mq.grouped_lora(x, a, bf(4, 64, 8), off, srt, 2)
    with pytest.raises(ValueError, match="adapter shapes"):
        mq.grouped_lora(x, a, b, i32(4), srt, 2)
    with pytest.raises(ValueError, match="scale"):
        mq.grouped_lora(x, a, b, off, srt, 2, scale=torch.ones(3))
    with pytest.raises(ValueError, match="base"):
        mq.grouped_lora(x, a, b, off, srt, 2, base=bf(15, 64))
    with pytest.raises(ValueError, match="pair_to_sorted"):
        mq.grouped_lora(x, a, b, off, srt, 2, pair_to_sorted=i32(15))
    with pytest.raises(TypeError, match="h has dtype"):
        mq.grouped_lora(x, a, b, off, srt, 2, h=bf(16, 16))
    h, dy = torch.zeros(16, 16), bf(16, 64)
    with pytest.raises(ValueError, match="GPU"):
        mq.grouped_lora_backward(dy, x, a, b, h, off, srt, 2)
    with pytest.raises(ValueError, match="need_dx"):
        mq.grouped_lora_backward(dy, x, a, b, h, off, srt, 2, need_dx=False, dx=bf(16, 128))
    with pytest.raises(ValueError, match="dy"):
        mq.grouped_lora_backward(bf(15, 64), x, a, b, h, off, srt, 2)
    with pytest.raises(TypeError, match="dy"):
        mq.grouped_lora_backward(None, x, a, b, h, off, srt, 2)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The kernels run on the current device; a tensor elsewhere is refused by
    name.  Device placement is faked: this needs no GPU."""
    class Fake(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1

    t = torch.zeros(4).as_subclass(Fake)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="y is on cuda:1"):
        mq._here("x y", None, t)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    mq._here("y absent", t, None)
