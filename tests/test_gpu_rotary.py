"""opr_rotary, opr_qk_norm_rope and its gradient on the GPU against the fp64 oracle."""

import numpy as np
import pytest
import torch

import block_sparse_masked_segment_b200 as opr
from block_sparse_masked_segment_b200 import _abi
from layer_helpers import TYPES, heads, to64, within
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

EPS = 1e-6


def positions(rng, total, far=1 << 20):
    return torch.from_numpy(rng.integers(-far, far, size=total).astype(np.int32)).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def rotary_bound(x, rot, interleaved, scale):
    """cos and sin are within 2^-22 (a few fp32 steps of a value up to 1), the two products and their
    sum within 3 * 2^-24 of their terms: 2^-21 of scale (|a| + |b|)."""
    ia, ib = lo.pair_indices(rot, interleaved)
    b = np.zeros_like(x)
    b[..., ia] = b[..., ib] = abs(scale) * (np.abs(x[..., ia]) + np.abs(x[..., ib])) * 2.0 ** -21
    return b


# total, heads, d, rot: one token, odd counts, pairs off the grid of eight, whole and part of the head
SHAPES = [(1, 1, 64, 64), (1, 32, 128, 128), (3, 2, 128, 64), (37, 5, 80, 20), (129, 3, 256, 256), (65, 1, 96, 48),
          (17, 7, 6, 2), (260, 8, 128, 32), (33, 2, 72, 64), (40, 2, 200, 16),
          (700, 3, 80, 80), (450, 1, 48, 16), (300, 40, 128, 128), (50, 3, 16, 16), (33, 2, 32, 16)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("types", ["bf16-fp16", "fp32-fp32", "fp16-bf16"])
def test_rotary_matches_oracle(shape, types, interleaved):
    total, n, d, rot = shape
    xt, yt = types.split("-")
    rng = np.random.default_rng(total * 1000 + d)
    for inverse, mapped in ((False, False), (True, True)):
        x, pos = heads(rng, total, n, d, xt), positions(rng, total)
        freq, scale = opr.opr_rotary_frequencies(rot, 1e4, "yarn", 4.0, 4096.0)
        row_map = torch.randperm(total, device="cuda").int() if mapped else None
        st = status()
        out = torch.empty(x.shape, dtype=TYPES[yt], device="cuda")
        got = opr.opr_rotary(x, pos, freq, interleaved, scale, inverse, out=out, row_map=row_map, dev_status=st)
        assert got is out and opr.read_status(st) == []
        if mapped:
            got = got[row_map.long()]
        ref = lo.rotate(to64(x), to64(pos), to64(freq), interleaved, scale, inverse)
        within(got, ref, rotary_bound(to64(x), rot, interleaved, scale), yt, f"{shape} {types}")


@pytest.mark.parametrize("wide,offset", [(64, 0), (64, 32), (3, 1), (8, 4)])
def test_rotary_reads_and_writes_parts_of_wider_rows(wide, offset):
    rng = np.random.default_rng(5)
    total, n, d, rot = 50, 3, 64, 32
    x = heads(rng, total, n, d, "bf16", wide, offset)
    whole = torch.full((total, n * d + wide), 7.0, dtype=torch.float16, device="cuda")
    out = whole[:, offset:offset + n * d].unflatten(1, (n, d))
    pos = positions(rng, total)
    freq, _ = opr.opr_rotary_frequencies(rot, 1e4)
    opr.opr_rotary(x, pos, freq, out=out)
    ref = lo.rotate(to64(x), to64(pos), to64(freq))
    within(out, ref, rotary_bound(to64(x), rot, False, 1.0), "fp16")
    assert (whole[:, :offset] == 7).all() and (whole[:, offset + n * d:] == 7).all()
    # in place, on a part of rows whose other part keeps its values
    keep = x.clone()
    base = x._base.clone()
    opr.opr_rotary(x, pos, freq)
    within(x, ref, rotary_bound(to64(keep), rot, False, 1.0), "bf16")
    other = torch.ones(base.shape, dtype=torch.bool, device="cuda").view(total, -1)
    other[:, offset:offset + n * d] = False
    assert torch.equal(x._base.view(total, -1)[other], base.view(total, -1)[other])


def test_rotary_angles_at_the_ends_of_the_position_range():
    """Positions up to the ends of int32.  Both sides round pos * freq (up to 2^31) to 53 bits: 2^-22 rad
    each, and the reduction of the product by whole turns adds nothing: 2^-20 with the arithmetic."""
    pos = torch.tensor([2**31 - 1, -2**31, 2**31 - 12345, 1 << 30, 0, 1, -1], dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(6)
    freq, _ = opr.opr_rotary_frequencies(64, 1e6)
    for n in (1, 8):
        x = heads(rng, 7, n, 64, "fp32")
        out = torch.empty_like(x)
        opr.opr_rotary(x, pos, freq, out=out)
        ref = lo.rotate(to64(x), to64(pos), to64(freq))
        within(out, ref, 2 * rotary_bound(to64(x), 64, False, 1.0), "fp32")


def test_rotary_is_opr_rope_for_whole_heads():
    """Both round the same fp32 expression of cos and sin that differ by a step or two."""
    rng = np.random.default_rng(7)
    x, pos = heads(rng, 333, 8, 128, "bf16"), positions(rng, 333, 65536)
    freq, _ = opr.opr_rotary_frequencies(128, 1e6)
    pos = pos.abs()
    a = opr.opr_rope(x, pos, 1e6, out=torch.empty(x.shape, dtype=torch.float32, device="cuda"))
    b = opr.opr_rotary(x, pos, freq, out=torch.empty_like(a))
    within(b, to64(a), 2 * rotary_bound(to64(x), 128, False, 1.0), "fp32")


@pytest.mark.parametrize("d,rot", [(128, 128), (128, 32), (18, 6)])
def test_rotary_inverse_is_the_gradient(d, rot):
    """sum(R x * y) = sum(x * R^T y) for fp32 outputs: each side's terms are off by 2^-21 of their sizes."""
    rng = np.random.default_rng(8)
    x, y = heads(rng, 30, 2, d, "fp32"), heads(rng, 30, 2, d, "fp32")
    pos = positions(rng, 30)
    freq, _ = opr.opr_rotary_frequencies(rot, 1e4)
    rx = opr.opr_rotary(x, pos, freq, True, 1.5, out=torch.empty_like(x))
    ty = opr.opr_rotary(y, pos, freq, True, 1.5, inverse=True, out=torch.empty_like(y))
    a, b = (rx.double() * y.double()).sum(), (x.double() * ty.double()).sum()
    assert abs(a - b) <= 2 * 2.0 ** -21 * 4 * 1.5 * x.double().norm() * y.double().norm()


@pytest.mark.parametrize("d", [64, 18])
def test_rotary_flags(d):
    """An fp16 overflow and a row map out of range are reported; the named rows are written, no others."""
    rng = np.random.default_rng(9)
    x, pos = heads(rng, 6, 2, d, "fp32"), positions(rng, 6)
    freq, _ = opr.opr_rotary_frequencies(16 if d == 64 else 6, 1e4)
    st = status()
    row_map = torch.tensor([5, -1, 3, 6, 1, 0], dtype=torch.int32, device="cuda")
    out = torch.full((6, 2, d), 9.0, dtype=torch.float16, device="cuda")
    opr.opr_rotary(x, pos, freq, out=out, row_map=row_map, dev_status=st)
    assert opr.read_status(st) == [_abi.DEV_BITS[1]]
    ref = lo.rotate(to64(x), to64(pos), to64(freq))
    for t, r in enumerate([5, None, 3, None, 1, 0]):
        if r is not None:
            within(out[r], ref[t], 1e-5, "fp16")
    assert (out[2] == 9).all() and (out[4] == 9).all()
    x[3, 1, d - 1] = 70000.0
    opr.opr_rotary(x, pos, freq, out=out, dev_status=st.zero_())
    assert opr.read_status(st) == [_abi.DEV_BITS[16]]
    x[3, 1, d - 1] = float("nan")
    opr.opr_rotary(x, pos, freq, out=out, dev_status=st.zero_())
    assert opr.read_status(st) == [_abi.DEV_BITS[16]]
    assert out.isnan().sum() == 1 and out[3, 1, d - 1].isnan()


def test_rotary_empty_and_refused_tensors():
    freq, _ = opr.opr_rotary_frequencies(64, 1e4)
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 4, 64, device="cuda")
    assert opr.opr_rotary(x, pos, freq).shape == (0, 4, 64)
    x, pos = torch.zeros(4, 2, 64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(pos_id=pos[:3]), dict(pos_id=pos.long()), dict(freq=freq.float()), dict(freq=freq.repeat(2)),
                dict(x=x.double()), dict(x=x[0]), dict(x=x.transpose(0, 1)), dict(out=x[:3]), dict(row_map=pos),
                dict(row_map=pos[:2], out=x.clone()), dict(out=x.half().view(4, 2, 64)[:, :, :32])):
        with pytest.raises(opr.OprError):
            opr.opr_rotary(**{**dict(x=x, pos_id=pos, freq=freq), **bad})


# ------------------------------------------------------------------ norm with rotation
def norm_bound(x, w, rot, interleaved, scale):
    """The mean of d <= 256 squares, the root and the division lose at most 32 fp32 half steps of the
    normed value, the rotation as above: 2^-18 of the terms' sizes."""
    n = np.abs(lo.norm(x, EPS) * w)
    return n * 2.0 ** -18 + 8 * rotary_bound(n, rot, interleaved, scale)


def qkv(rng, total, hq, hkv, d, dtype, packed, scale=2.0):
    if packed:
        x = heads(rng, total, hq + 2 * hkv, d, dtype, scale=scale)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return tuple(heads(rng, total, h, d, dtype, scale=scale) for h in (hq, hkv, hkv))


def weights(rng, d, dtype):
    return tuple((1 + 0.2 * torch.from_numpy(rng.standard_normal(d).astype(np.float32))).to("cuda", TYPES[dtype])
                 for _ in range(2))


QK_SHAPES = [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (5, 3, 1, 128, 64), (67, 8, 2, 64, 32), (130, 4, 4, 256, 256),
             (19, 2, 1, 80, 20), (300, 5, 1, 128, 128), (12, 2, 2, 6, 4), (21, 3, 3, 72, 64), (40, 1, 1, 200, 16),
             (700, 2, 1, 80, 80), (450, 1, 1, 48, 16), (310, 20, 2, 128, 96), (900, 1, 5, 256, 64), (50, 3, 1, 16, 16), (33, 2, 2, 32, 16)]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", QK_SHAPES, ids=str)
@pytest.mark.parametrize("types", ["bf16-fp16", "fp32-fp32", "fp16-bf16"])
def test_qk_norm_matches_oracle(shape, types, interleaved, packed):
    total, hq, hkv, d, rot = shape
    xt, yt = types.split("-")
    rng = np.random.default_rng(total + d)
    q, k, v = qkv(rng, total, hq, hkv, d, xt, packed)
    qw, kw = weights(rng, d, "bf16" if xt == "fp32" else xt)
    pos = positions(rng, total)
    freq, scale = opr.opr_rotary_frequencies(rot, 1e6, "linear", 2.0)
    row_map = torch.randperm(total, device="cuda").int() if packed else None
    st = status()
    out = opr.opr_qk_norm_rope(q, k, qw, kw, pos, freq, EPS, interleaved, scale, v=v, out_dtype=TYPES[yt],
                               row_map=row_map, dev_status=st)
    assert opr.read_status(st) == []
    if packed:
        out = [o[row_map.long()] for o in out]
    for got, x, w in ((out[0], q, qw), (out[1], k, kw)):
        ref = lo.norm_rotate(to64(x), to64(w), to64(pos), to64(freq), EPS, interleaved, scale)
        within(got, ref, norm_bound(to64(x), to64(w), rot, interleaved, scale), yt)
    within(out[2], to64(v), 0.0, yt)
    # without v: the same q and k, bit for bit
    two = opr.opr_qk_norm_rope(q, k, qw, kw, pos, freq, EPS, interleaved, scale, out_dtype=TYPES[yt], row_map=row_map)
    assert len(two) == 2
    for a, b in zip(two, out):
        assert torch.equal(a if row_map is None else a[row_map.long()], b)


def test_qk_norm_of_tiny_huge_and_zero_rows():
    """eps carries a row of zeros (and of values whose squares vanish next to it); a row of 2^60 does not
    overflow the sum of squares in fp32."""
    rng = np.random.default_rng(11)
    q, k, _ = qkv(rng, 4, 2, 1, 128, "bf16", False)
    q[0] = 0
    q[1] *= 2.0 ** -60
    q[2] *= 2.0 ** 55
    qw, kw = weights(rng, 128, "bf16")
    pos = positions(rng, 4)
    freq, _ = opr.opr_rotary_frequencies(128, 1e4)
    out, _ = opr.opr_qk_norm_rope(q, k, qw, kw, pos, freq, EPS, out_dtype=torch.float32)
    ref = lo.norm_rotate(to64(q), to64(qw), to64(pos), to64(freq), EPS)
    within(out, ref, norm_bound(to64(q), to64(qw), 128, False, 1.0), "fp32")
    assert (out[0] == 0).all()


def test_qk_norm_in_place_and_into_given_buffers():
    rng = np.random.default_rng(12)
    q, k, v = qkv(rng, 33, 4, 2, 64, "bf16", False)
    qw, kw = weights(rng, 64, "fp32")
    pos = positions(rng, 33)
    freq, _ = opr.opr_rotary_frequencies(64, 1e4)
    want = opr.opr_qk_norm_rope(q, k, qw, kw, pos, freq, v=v, out_dtype=torch.bfloat16)
    buf = tuple(torch.empty_like(t) for t in (q, k, v))
    got = opr.opr_qk_norm_rope(q, k, qw, kw, pos, freq, v=v, out=buf)
    assert all(g is b and torch.equal(g, w) for g, b, w in zip(got, buf, want))
    opr.opr_qk_norm_rope(q, k, qw, kw, pos, freq, v=v, out=(q, k, v))
    assert all(torch.equal(g, w) for g, w in zip((q, k, v), want))
    with pytest.raises(opr.OprError):
        opr.opr_qk_norm_rope(q, k, qw, kw, pos, freq, out=(k, q))
    with pytest.raises(opr.OprError):
        opr.opr_qk_norm_rope(q, k.float(), qw, kw, pos, freq)
    with pytest.raises(opr.OprError):
        opr.opr_qk_norm_rope(q, k, qw[:32], kw, pos, freq)
    with pytest.raises(opr.OprError):
        opr.opr_qk_norm_rope(q, k, qw, kw, pos, freq, eps=0.0)


# ------------------------------------------------------------------ its gradient
def grad_bounds(dy, x, w, pos, freq, interleaved, scale):
    """Bounds of dx and dw from the sizes of the terms that are added.  dx = rs (u - xh mean(u xh)): up to
    32 fp32 half steps (2^-19) of rs (|u| + |xh| mean |u xh|).  dw: the sum over the rows goes through
    at most 1024 additions in a chain (2^-14 of the sum of sizes), the terms within 2^-18."""
    ia, ib = lo.pair_indices(2 * len(freq), interleaved)
    g = np.abs(dy)
    both = abs(scale) * (g[..., ia] + g[..., ib])
    g[..., ia] = both
    g[..., ib] = both
    xh = np.abs(lo.norm(x, EPS))
    rs = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    u = g * np.abs(w)
    return (rs * (u + xh * (u * xh).mean(-1, keepdims=True)) * 2.0 ** -18,
            (g * xh).sum((0, 1)) * (2.0 ** -14 + 2.0 ** -18))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", QK_SHAPES, ids=str)
@pytest.mark.parametrize("types", ["bf16-fp32-bf16", "fp32-fp32-fp32", "fp16-bf16-fp16", "bf16-bf16-fp32"])
def test_qk_norm_gradient_matches_oracle(shape, types, interleaved, packed):
    total, hq, hkv, d, rot = shape
    xt, gt, ot = types.split("-")
    rng = np.random.default_rng(3 * total + d)
    q, k, _ = qkv(rng, total, hq, hkv, d, xt, packed)
    dq, dk, dv = (heads(rng, total, h, d, gt, scale=0.1) for h in (hq, hkv, hkv))
    qw, kw = weights(rng, d, "bf16" if xt == "fp32" else xt)
    pos = positions(rng, total)
    freq, scale = opr.opr_rotary_frequencies(rot, 1e4, "yarn", 2.0, 4096.0)
    row_map = torch.randperm(total, device="cuda").int() if packed else None
    out = whole = None
    if packed:  # into the parts of one projection's gradient
        whole = torch.full((total, hq + 2 * hkv + 1, d), 3.0, dtype=TYPES[ot], device="cuda")
        out = (whole[:, :hq], whole[:, hq:hq + hkv], whole[:, hq + hkv:hq + 2 * hkv])
    st = status()
    args = (q, k, qw, kw, pos, freq, EPS, interleaved, scale)
    gq, gk, gv, gqw, gkw = opr.opr_qk_norm_rope_bwd(dq, dk, *args, dv=dv, out=out, out_dtype=TYPES[ot],
                                                    row_map=row_map, dev_status=st)
    assert opr.read_status(st) == []
    for got, gw, dy, x, w in ((gq, gqw, dq, q, qw), (gk, gkw, dk, k, kw)):
        dy64 = to64(dy if row_map is None else dy[row_map.long()])
        rx, rw = lo.norm_rotate_bwd(dy64, to64(x), to64(w), to64(pos), to64(freq), EPS, interleaved, scale)
        bx, bw = grad_bounds(dy64, to64(x), to64(w), to64(pos), to64(freq), interleaved, scale)
        within(got, rx, bx, ot)
        within(gw, rw, bw, "fp32")
    within(gv, to64(dv if row_map is None else dv[row_map.long()]), 0.0, ot)
    if packed:
        assert (whole[:, -1] == 3).all()
    # a second call, without dv, gives the same bits
    again = opr.opr_qk_norm_rope_bwd(dq, dk, *args, out_dtype=TYPES[ot], row_map=row_map)
    for a, b in zip(again, (gq, gk, gqw, gkw)):
        assert torch.equal(a, b)


def test_qk_norm_gradient_of_many_rows():
    """More rows than the pass has warps, so that each block sums several: closed form.  With x = 1 and
    w = 1 the normed heads are 1 / sqrt(1 + eps), and dw is the sum of the rotated-back gradients."""
    total, hq, hkv, d = 9001, 6, 2, 64
    rng = np.random.default_rng(14)
    dq, dk = heads(rng, total, hq, d, "fp32"), heads(rng, total, hkv, d, "fp32")
    q, k = torch.ones(total, hq, d, device="cuda"), torch.ones(total, hkv, d, device="cuda")
    w = torch.ones(d, device="cuda")
    pos = positions(rng, total)
    freq, _ = opr.opr_rotary_frequencies(d, 1e4)
    *_, gq, gk = opr.opr_qk_norm_rope_bwd(dq, dk, q, k, w, w, pos, freq, EPS)
    for got, dy in ((gq, dq), (gk, dk)):
        ref = lo.rotate(to64(dy), to64(pos), to64(freq), inverse=True) / np.sqrt(1 + EPS)
        within(got, ref.sum((0, 1)), np.abs(ref).sum((0, 1)) * 2.0 ** -14, "fp32")


def test_qk_norm_gradient_of_many_tokens_of_one_wide_head():
    """The largest tables that a block holds: 32 tokens of 128 pairs.  Closed form as above."""
    total, d = 9700, 256
    rng = np.random.default_rng(24)
    dq, dk = heads(rng, total, 1, d, "fp32"), heads(rng, total, 1, d, "fp32")
    one, w = torch.ones(total, 1, d, device="cuda"), torch.ones(d, device="cuda")
    pos = positions(rng, total)
    freq, _ = opr.opr_rotary_frequencies(d, 1e4)
    *_, gq, gk = opr.opr_qk_norm_rope_bwd(dq, dk, one, one, w, w, pos, freq, EPS)
    for got, dy in ((gq, dq), (gk, dk)):
        ref = lo.rotate(to64(dy), to64(pos), to64(freq), inverse=True) / np.sqrt(1 + EPS)
        within(got, ref.sum((0, 1)), np.abs(ref).sum((0, 1)) * 2.0 ** -14, "fp32")


def test_rows_past_two_to_the_31_entries():
    """More than 2^31 entries in one tensor: the last tokens of the rotation, of the norm (in place) and of
    its gradient (one projection's packed rows)."""
    total, hq, hkv, d = 140000, 104, 8, 128
    x = torch.zeros(total, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(3)
    tail = slice(total - 3, total)
    x[tail] = torch.randn(3, hq + 2 * hkv, d, device="cuda", generator=g).bfloat16()
    keep = x[tail].clone()
    pos = torch.arange(total, dtype=torch.int32, device="cuda")
    freq, _ = opr.opr_rotary_frequencies(d, 1e6)
    w = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    y = opr.opr_rotary(x, pos, freq, out=torch.empty_like(x))
    K = to64(keep)
    P, F, W = to64(pos[tail]), to64(freq), to64(w)
    within(y[tail], lo.rotate(K, P, F), rotary_bound(K, d, False, 1.0), "bf16")
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    dq, dk, dv = (torch.zeros(total, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    for t in (dq, dk, dv):
        t[tail] = torch.randn(3, t.shape[1], d, device="cuda", generator=g).bfloat16()
    out = (y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:])
    y[:-3] = 0
    *_, gqw, _ = opr.opr_qk_norm_rope_bwd(dq, dk, q, k, w, w, pos, freq, EPS, dv=dv, out=out)
    for got, dy, a in ((out[0], dq, K[:, :hq]), (out[1], dk, K[:, hq:hq + hkv])):
        rx, rw = lo.norm_rotate_bwd(to64(dy[tail]), a, W, P, F, EPS)
        bx, bw = grad_bounds(to64(dy[tail]), a, W, P, F, False, 1.0)
        within(got[tail], rx, bx, "bf16")
        if dy is dq:
            within(gqw, rw, bw, "fp32")
    assert torch.equal(out[2][tail], dv[tail]) and not y[:-3].any()


def test_qk_norm_gradient_of_no_tokens_is_zero():
    z = torch.empty(0, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    freq, _ = opr.opr_rotary_frequencies(64, 1e4)
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    dq, dk, gq, gk = opr.opr_qk_norm_rope_bwd(z, z, z, z, w, w, pos, freq)
    assert dq.shape == (0, 2, 64) and (gq == 0).all() and (gk == 0).all()


def test_qk_norm_gradient_in_place():
    rng = np.random.default_rng(15)
    q, k, _ = qkv(rng, 70, 3, 1, 128, "bf16", False)
    dq, dk, dv = (heads(rng, 70, h, 128, "fp32", scale=0.1) for h in (3, 1, 1))
    qw, kw = weights(rng, 128, "bf16")
    pos = positions(rng, 70)
    freq, _ = opr.opr_rotary_frequencies(128, 1e4)
    want = opr.opr_qk_norm_rope_bwd(dq, dk, q, k, qw, kw, pos, freq, dv=dv, out_dtype=torch.float32)
    got = opr.opr_qk_norm_rope_bwd(dq, dk, q, k, qw, kw, pos, freq, dv=dv, out=(dq, dk, dv))
    assert got[0] is dq and all(torch.equal(a, b) for a, b in zip(got, want))


def test_heads_calls_on_a_side_stream_and_in_a_graph():
    """Captured and replayed on new inputs in the same buffers, next to eager calls on another stream."""
    rng = np.random.default_rng(16)
    q, k, v = qkv(rng, 200, 8, 2, 128, "bf16", True)
    qw, kw = weights(rng, 128, "bf16")
    pos = positions(rng, 200)
    freq, _ = opr.opr_rotary_frequencies(128, 1e4)
    dq, dk = heads(rng, 200, 8, 128, "fp32"), heads(rng, 200, 2, 128, "fp32")

    def step():
        out = opr.opr_qk_norm_rope(q, k, qw, kw, pos, freq, v=v)
        grads = opr.opr_qk_norm_rope_bwd(dq, dk, q, k, qw, kw, pos, freq)
        return (*out, *grads, opr.opr_rotary(dq, pos, freq, True, out=torch.empty_like(dq)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))
    q.copy_(torch.randn_like(q))
    dq.copy_(torch.randn_like(dq))
    graph.replay()
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, held))


def test_rotary_of_more_heads_than_a_grid_has_blocks():
    """2^34 heads and more, eight to a block of the form for odd sizes, would take more blocks than a grid
    has; the last token's heads are rotated too (in place, 69 GB)."""
    total, n, d = 2 ** 18 + 1, 65536, 2
    if torch.cuda.mem_get_info()[0] < 80 * 2 ** 30:
        torch.cuda.empty_cache()
        if torch.cuda.mem_get_info()[0] < 80 * 2 ** 30:
            pytest.skip("needs 80 GB of device memory")
    x = torch.zeros(total, n, d, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, total // 2, total - 2, total - 1]
    rng = np.random.default_rng(30)
    for r in rows:
        x[r] = heads(rng, 1, n, d, "bf16")[0]
    keep = to64(x[rows])
    pos = torch.arange(5, 5 + total, dtype=torch.int32, device="cuda")
    freq = torch.ones(1, dtype=torch.float64, device="cuda")
    st = status()
    opr.opr_rotary(x, pos, freq, dev_status=st)
    assert opr.read_status(st) == []
    within(x[rows], lo.rotate(keep, to64(pos[rows]), to64(freq)), rotary_bound(keep, d, False, 1.0), "bf16")
    assert not x[2:total // 2:9973].any()
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d,rot", [(80, 20), (72, 64), (18, 6), (200, 104)])
def test_weight_gradients_of_odd_sizes_repeat(d, rot):
    """In the form for odd sizes the lane that adds to an entry's sum is another than the one that clears it
    (interleaved pairs): blocks of one head or a few, whose sums follow the clearing at once, many times;
    against the formula, and the same bits each time."""
    rng = np.random.default_rng(50)
    for total in (1, 40):
        q, k, _ = qkv(rng, total, 3, 1, d, "bf16", False)
        dq, dk = heads(rng, total, 3, d, "fp32"), heads(rng, total, 1, d, "fp32")
        qw, kw = weights(rng, d, "bf16")
        pos = positions(rng, total)
        freq, _ = opr.opr_rotary_frequencies(rot, 1e4)
        first = opr.opr_qk_norm_rope_bwd(dq, dk, q, k, qw, kw, pos, freq, EPS, True)
        for got, dy, x, w in ((first[2], dq, q, qw), (first[3], dk, k, kw)):
            _, rw = lo.norm_rotate_bwd(to64(dy), to64(x), to64(w), to64(pos), to64(freq), EPS, True)
            within(got, rw, grad_bounds(to64(dy), to64(x), to64(w), to64(pos), to64(freq), True, 1.0)[1], "fp32")
        for _ in range(100):
            again = opr.opr_qk_norm_rope_bwd(dq, dk, q, k, qw, kw, pos, freq, EPS, True)
            assert all(torch.equal(a, b) for a, b in zip(again, first))


def test_positions_between_the_rows_of_an_output():
    """What lies between the rows of a wider buffer is no part of the output: positions and table there are
    taken, and keep their values."""
    rng = np.random.default_rng(51)
    total, n, d = 6, 2, 64
    buf = torch.zeros(total, 512, device="cuda")
    x, out = heads(rng, total, n, d, "fp32"), buf[:, :n * d].unflatten(1, (n, d))
    pos, freq = buf[0, 200:200 + total].view(torch.int32), buf[1, 256:256 + d].view(torch.float64)
    p, f = positions(rng, total), opr.opr_rotary_frequencies(d, 1e4)[0]
    pos.copy_(p), freq.copy_(f)
    opr.opr_rotary(x, pos, freq, out=out)
    within(out, lo.rotate(to64(x), to64(p), to64(f)), rotary_bound(to64(x), d, False, 1.0), "fp32")
    assert torch.equal(pos, p) and torch.equal(freq, f)


@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32), (80, 20), (18, 6)])
@pytest.mark.parametrize("packed", [False, True])
def test_qk_norm_gradient_over_its_inputs(d, rot, packed):
    """dq and dk written over q and k themselves (one type, one stride), v's gradient beside them where the
    three are parts of one projection: as into buffers of their own."""
    rng = np.random.default_rng(52)
    total, hq, hkv = 300, 4, 2
    q, k, v = qkv(rng, total, hq, hkv, d, "bf16", packed)
    dq, dk, dv = (heads(rng, total, h, d, "fp32", scale=0.1) for h in (hq, hkv, hkv))
    qw, kw = weights(rng, d, "bf16")
    pos = positions(rng, total)
    freq, _ = opr.opr_rotary_frequencies(rot, 1e4)
    args = (qw, kw, pos, freq, EPS, True)
    want = opr.opr_qk_norm_rope_bwd(dq, dk, q, k, *args, dv=dv)
    got = opr.opr_qk_norm_rope_bwd(dq, dk, q, k, *args, dv=dv, out=(q, k, v))
    assert got[0] is q and all(torch.equal(a, b) for a, b in zip(got, want))
