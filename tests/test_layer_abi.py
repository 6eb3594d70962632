"""Refusals of the operators around the attention, on the host: every call here fails a check before
any CUDA call, so the made-up addresses are never used."""

import ctypes

import pytest
import torch

import block_sparse_masked_segment_b200 as opr

INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 4
BF16, FP32, FP16 = 0, 1, 2


def at(mib):
    return ctypes.c_void_p(mib << 20)


@pytest.fixture(scope="module")
def lib():
    return opr.load_library()


def rotary(lib, **kw):
    a = dict(x=at(16), xt=BF16, xs=256, y=at(64), yt=FP16, ys=256, pos=at(1), freq=at(2), rot=64, inter=0, scale=1.0,
             inv=0, row_map=None, total=10, heads=2, d=128, st=None)
    assert set(kw) <= set(a)
    return lib.opr_rotary(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(total=-1), INVALID), (dict(total=1 << 31), INVALID), (dict(heads=-1), INVALID),
    (dict(heads=65537, xs=1 << 30, ys=1 << 30), INVALID),
    (dict(d=257, xs=514, ys=514), INVALID), (dict(rot=63), INVALID), (dict(rot=0), INVALID),
    (dict(rot=130), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(xs=255), INVALID), (dict(ys=255), INVALID), (dict(xt=3), UNSUPPORTED), (dict(yt=-1), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID),
    (dict(x=ctypes.c_void_p((16 << 20) + 1)), INVALID),                # not on an element
    (dict(y=at(16)), INVALID),                                         # in place, two types
    (dict(y=at(16), yt=BF16, row_map=at(3)), INVALID),                 # in place, rows sent elsewhere
    (dict(y=at(16), yt=BF16, ys=512), INVALID),                        # in place, two strides
    (dict(y=ctypes.c_void_p((16 << 20) + 2), yt=BF16), INVALID),       # shifted by an element
    (dict(xs=512, ys=512, yt=BF16, y=ctypes.c_void_p((16 << 20) + 510)), INVALID),  # one element shared with the next head
    (dict(total=0, x=None, y=None), 0), (dict(heads=0, xs=0, ys=0), 0),
])
def test_rotary_refusals(lib, kw, want):
    assert rotary(lib, **kw) == want


@pytest.mark.parametrize("args,want", [
    ((63, 1e4, 0, 1.0, 0.0, 1.0, 32.0), INVALID), ((0, 1e4, 0, 1.0, 0.0, 1.0, 32.0), INVALID),
    ((258, 1e4, 0, 1.0, 0.0, 1.0, 32.0), INVALID), ((64, 1.0, 0, 1.0, 0.0, 1.0, 32.0), INVALID),
    ((64, 1e4, 5, 1.0, 0.0, 1.0, 32.0), UNSUPPORTED), ((64, 1e4, -1, 1.0, 0.0, 1.0, 32.0), UNSUPPORTED),
    ((64, 1e4, 1, 0.5, 0.0, 1.0, 32.0), INVALID), ((64, 1e4, 1, float("nan"), 0.0, 1.0, 32.0), INVALID),
    ((64, 1e4, 3, 4.0, 0.0, 1.0, 32.0), INVALID), ((64, 1e4, 3, 4.0, 8192.0, 32.0, 32.0), INVALID),
    ((64, 1e4, 4, 4.0, 8192.0, 0.0, 4.0), INVALID), ((64, 1e4, 4, 4.0, -1.0, 1.0, 4.0), INVALID),
])
def test_frequency_refusals(lib, args, want):
    out, s = (ctypes.c_double * 128)(), ctypes.c_double()
    assert lib.opr_rotary_frequencies(*args, ctypes.cast(out, ctypes.c_void_p), ctypes.byref(s)) == want
    assert lib.opr_rotary_frequencies(64, 1e4, 0, 1.0, 0.0, 1.0, 32.0, None, ctypes.byref(s)) == INVALID


def qk(lib, **kw):
    a = dict(q=at(16), qs=1024, k=at(32), ks=256, v=at(48), vs=256, xt=BF16, qw=at(1), kw=at(2), wt=BF16, eps=1e-6,
             pos=at(3), freq=at(4), rot=128, inter=0, scale=1.0, row_map=None, total=10, hq=8, hkv=2, d=128, qo=at(64),
             ko=at(80), vo=at(96), yt=FP16, st=None)
    assert set(kw) <= set(a)
    return lib.opr_qk_norm_rope(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(total=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=-1), INVALID), (dict(d=258), INVALID),
    (dict(rot=129), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(qs=1023), INVALID), (dict(ks=255), INVALID), (dict(vs=255), INVALID), (dict(xt=9), UNSUPPORTED),
    (dict(yt=9), UNSUPPORTED), (dict(wt=9), UNSUPPORTED), (dict(v=None), INVALID), (dict(vo=None), INVALID),
    (dict(q=None), INVALID), (dict(qw=None), INVALID), (dict(kw=None), INVALID), (dict(pos=None), INVALID),
    (dict(freq=None), INVALID), (dict(ko=None), INVALID),
    (dict(qo=at(80)), INVALID),             # two outputs in one place
    (dict(qo=at(32), yt=BF16), INVALID),    # q over k
    (dict(qo=at(16)), INVALID),             # over its own input, in another type
    (dict(qo=at(16), yt=BF16, row_map=at(5)), INVALID),
    (dict(ko=at(1)), INVALID),              # over a weight
    (dict(total=0, q=None), 0),
])
def test_qk_norm_refusals(lib, kw, want):
    assert qk(lib, **kw) == want


def qk_bwd(lib, **kw):
    a = dict(dq=at(16), dk=at(32), dv=at(48), gt=FP32, q=at(64), qs=1024, k=at(80), ks=256, xt=BF16, qw=at(1),
             kw=at(2), wt=BF16, eps=1e-6, pos=at(3), freq=at(4), rot=128, inter=0, scale=1.0, row_map=None, total=10,
             hq=8, hkv=2, d=128, dqo=at(96), dqs=1024, dko=at(112), dks=256, dvo=at(128), dvs=256, ot=BF16, dqw=at(5),
             dkw=at(6), ws=at(144), wsb=1 << 20, st=None)
    assert set(kw) <= set(a)
    return lib.opr_qk_norm_rope_bwd(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(total=-1), INVALID), (dict(hq=0), INVALID), (dict(eps=0.0), INVALID), (dict(rot=0), INVALID),
    (dict(gt=7), UNSUPPORTED), (dict(xt=7), UNSUPPORTED), (dict(ot=7), UNSUPPORTED), (dict(wt=7), UNSUPPORTED),
    (dict(qs=1), INVALID), (dict(dqs=1023), INVALID), (dict(dks=255), INVALID), (dict(dvs=255), INVALID),
    (dict(dv=None), INVALID), (dict(dvo=None), INVALID), (dict(dq=None), INVALID), (dict(dqo=None), INVALID),
    (dict(qw=None), INVALID), (dict(dqw=None), INVALID), (dict(dkw=None), INVALID), (dict(ws=None), INVALID),
    (dict(wsb=16), TOO_SMALL), (dict(ws=ctypes.c_void_p((144 << 20) + 8)), INVALID),
    (dict(dqo=at(16)), INVALID),                              # over dq in another type
    (dict(dqo=at(16), ot=FP32, row_map=at(7)), INVALID),      # over dq, whose rows are read elsewhere
    (dict(dqo=at(80)), INVALID), (dict(dqo=at(112)), INVALID), (dict(dqw=at(6)), INVALID),
    (dict(ws=at(16)), INVALID),
])
def test_qk_norm_gradient_refusals(lib, kw, want):
    assert qk_bwd(lib, **kw) == want


def test_qk_norm_gradient_workspace(lib):
    f = lib.opr_qk_norm_rope_bwd_workspace_bytes
    assert f(0, 8, 2, 128) >= 2 * 4 * 128 and f(65536, 64, 8, 128) % 256 == 0
    assert f(-1, 8, 2, 128) == 0 and f(10, 0, 2, 128) == 0 and f(10, 8, 2, 258) == 0


def lin(lib, **kw):
    a = dict(x=at(16), ldx=64, w=at(32), ldw=64, t=BF16, bias=at(1), bt=BF16, act=0, res=at(48), ldr=96, rt=BF16,
             y=at(64), ldy=96, yt=BF16, z=at(80), ldz=96, m=10, n=96, k=64, ws=None, wsb=0, st=at(2))
    assert set(kw) <= set(a)
    return lib.opr_linear(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(m=(1 << 31) - 511), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID),
    (dict(n=(1 << 31) - 511, ldy=1 << 31, ldr=1 << 31, ldz=1 << 31), INVALID), (dict(ldx=63), INVALID), (dict(ldw=63), INVALID), (dict(ldy=95), INVALID), (dict(ldr=95), INVALID),
    (dict(ldz=95), INVALID), (dict(act=4), UNSUPPORTED), (dict(act=-1), UNSUPPORTED), (dict(t=FP32), UNSUPPORTED),
    (dict(yt=5), UNSUPPORTED), (dict(bt=5), UNSUPPORTED), (dict(rt=5), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(st=None), INVALID),
    (dict(y=at(16)), INVALID), (dict(y=at(80)), INVALID), (dict(z=at(48)), INVALID),
    (dict(y=at(48), yt=FP32), INVALID),              # over the residual in another type
    (dict(y=at(48), ldy=128), INVALID),              # ... with another row length
    (dict(ldx=65), TOO_SMALL),                       # rows off the 16-byte grid go through the workspace
    (dict(x=ctypes.c_void_p((16 << 20) + 2)), TOO_SMALL),
    (dict(ldx=65, wsb=1 << 20), INVALID), (dict(ldx=65, wsb=1 << 20, ws=at(64)), INVALID),
    (dict(m=0, x=None, y=None), 0),
])
def test_linear_refusals(lib, kw, want):
    assert lin(lib, **kw) == want


def test_linear_workspace(lib):
    f = lib.opr_linear_workspace_bytes
    assert f(at(1), 64, at(2), 64, 10, 96, 64) == 0
    assert f(at(1), 65, at(2), 64, 10, 96, 64) >= 10 * 64 * 2
    assert f(at(1), 64, ctypes.c_void_p((2 << 20) + 8), 64, 10, 96, 61) >= 96 * 64 * 2
    assert f(at(1), 63, at(2), 64, 10, 96, 64) == 0  # sizes the call refuses


def lin_bwd(lib, **kw):
    a = dict(dy=at(16), ldy=96, x=at(32), ldx=64, w=at(48), ldw=64, t=BF16, z=at(64), ldz=96, act=1, res=at(80), ldr=64,
             rt=BF16, dx=at(96), ldxo=64, dxt=BF16, dw=at(112), ldwo=64, dwt=BF16, db=at(1), m=10, n=96, k=64,
             ws=at(128), wsb=1 << 20, st=at(2))
    assert set(kw) <= set(a)
    return lib.opr_linear_bwd(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(ldy=95), INVALID),
    (dict(ldx=63), INVALID), (dict(ldz=95), INVALID), (dict(ldxo=63), INVALID), (dict(ldwo=63), INVALID),
    (dict(ldr=63), INVALID), (dict(act=9), UNSUPPORTED), (dict(t=FP32), UNSUPPORTED), (dict(dxt=9), UNSUPPORTED),
    (dict(dwt=9), UNSUPPORTED), (dict(rt=9), UNSUPPORTED), (dict(z=None), INVALID), (dict(dy=None), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(st=None), INVALID), (dict(dx=None), INVALID),
    (dict(wsb=16), TOO_SMALL), (dict(ws=None), INVALID), (dict(dx=at(16)), INVALID), (dict(dw=at(96)), INVALID),
    (dict(dx=at(80), dxt=FP32), INVALID), (dict(ws=at(48)), INVALID),
    (dict(dx=None, dw=None, db=None, res=None), 0),
])
def test_linear_gradient_refusals(lib, kw, want):
    assert lin_bwd(lib, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(y=at(1)), dict(y=at(2)), dict(y=at(3), row_map=at(3)), dict(y=at(1), pos=ctypes.c_void_p((1 << 20) + 5080)),
    dict(y=ctypes.c_void_p((2 << 20) + 248), yt=FP32, ys=256),             # the table's last entry
    dict(y=at(1), ys=512, pos=ctypes.c_void_p((1 << 20) + 1000)),          # positions that reach into the second row
])
def test_rotary_refuses_outputs_over_positions_table_and_map(lib, kw):
    assert rotary(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(qo=at(3)), dict(ko=at(4)), dict(vo=at(5), row_map=at(5)), dict(qo=at(4)),
                                dict(ko=at(5), row_map=at(5))])
def test_qk_norm_refuses_outputs_over_positions_table_and_map(lib, kw):
    assert qk(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dqo=at(3)), dict(dko=at(4)), dict(dvo=at(7), row_map=at(7)), dict(dqw=at(4)),
                                dict(dkw=at(3)), dict(ws=at(4)), dict(ws=at(7), row_map=at(7))])
def test_qk_norm_gradient_refuses_outputs_over_positions_table_and_map(lib, kw):
    assert qk_bwd(lib, **kw) == INVALID


def off(mib, by):
    return ctypes.c_void_p((mib << 20) + by)


@pytest.mark.parametrize("kw", [dict(pos=off(1, 2)), dict(freq=off(2, 4)), dict(row_map=off(3, 1)), dict(st=off(4, 2))])
def test_head_calls_refuse_arrays_off_their_elements(lib, kw):
    """An address inside an element would end the process on the device."""
    assert rotary(lib, **kw) == INVALID
    kw = {k: off(v.value >> 20 << 3, v.value & 15) for k, v in kw.items()}  # elsewhere: apart from the weights
    assert qk(lib, **kw) == INVALID and qk_bwd(lib, **kw) == INVALID


@pytest.mark.parametrize("by", [1, 2])
def test_products_refuse_a_status_word_off_its_element(lib, by):
    assert lin(lib, st=off(2, by)) == INVALID and lin_bwd(lib, st=off(2, by)) == INVALID


def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(4, 2, 64)
    pos, freq = torch.zeros(4, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    with pytest.raises(opr.OprError):
        opr.opr_rotary(x, pos, freq)
    with pytest.raises(opr.OprError):
        opr.opr_qk_norm_rope(x, x, torch.ones(64), torch.ones(64), pos, freq)
    m = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(opr.OprError):
        opr.opr_linear(m, m)
    with pytest.raises(opr.OprError):
        opr.opr_rotary_frequencies(64, 1e4, "other", device="cpu")
