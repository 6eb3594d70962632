"""opr_linear and opr_linear_bwd on the GPU against the fp64 oracle."""

import numpy as np
import pytest
import torch

import block_sparse_masked_segment_b200 as opr
from block_sparse_masked_segment_b200 import _abi
from layer_helpers import TYPES, half_step, matrix, to64, within
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def sum_bound(a, b, k):
    """Of a sum of k exact products: the tensor cores add sixteen at a time and may drop up to two of the
    running sum's last bits (2^-22) each time; the running sum is at most the sum of the sizes."""
    return (np.abs(a) @ np.abs(b).T) * (k / 16 + 8) * 2.0 ** -22


# |act'| <= 1.13 for all three; the functions themselves within 2^-20 of |z| + 1
def act_bound(z, bz, activation):
    return bz if activation is None else 1.13 * bz + (np.abs(z) + 1) * 2.0 ** -20


SHAPES = [(1, 8, 8), (1, 1, 1), (2, 130, 64), (1, 256, 1000), (7, 3, 5), (16, 512, 513), (33, 64, 96), (64, 300, 40),
          (127, 129, 65), (128, 128, 64), (129, 257, 72), (130, 200, 136), (257, 511, 320), (300, 1000, 24),
          (513, 40, 130), (700, 96, 33), (1, 777, 2050), (5, 2048, 4096), (1030, 264, 512)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_matches_oracle(shape, dtype):
    m, n, k = shape
    rng = np.random.default_rng(m * 7 + n)
    x, w = matrix(rng, m, k, dtype), matrix(rng, n, k, dtype, scale=k ** -0.5)
    b = matrix(rng, 1, n, dtype)[0]
    st = status()
    bz = sum_bound(to64(x), to64(w), k)
    plain = opr.opr_linear(x, w, dev_status=st)
    assert opr.read_status(st) == []
    within(plain, to64(x) @ to64(w).T, bz, dtype, f"{shape}")
    # bias, activation, residual and z together, fp32 out
    r = matrix(rng, m, n, "fp32")
    y, z = opr.opr_linear(x, w, b, "silu", r, out_dtype=torch.float32, save_z=True, dev_status=st)
    assert opr.read_status(st) == []
    ry, rz = lo.linear(to64(x), to64(w), to64(b), "silu", to64(r))
    bz = bz + (np.abs(rz) + 1) * 2.0 ** -23
    within(z, rz, bz, dtype, f"z {shape}")
    within(y, ry, act_bound(rz, bz, "silu") + (np.abs(ry) + np.abs(to64(r))) * 2.0 ** -23, "fp32", f"y {shape}")


@pytest.mark.parametrize("activation", [None, "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16", "bf16"), ("fp16", "fp32", "bf16", "fp16"),
                                   ("bf16", "fp16", "fp32", "fp32"), ("fp16", None, "fp16", "bf16"),
                                   ("bf16", "bf16", None, "fp16")])
def test_linear_epilogues(types, activation):
    dtype, bt, rt, yt = types
    rng = np.random.default_rng(3)
    for m, n, k in ((37, 100, 80), (200, 264, 128)):
        x, w = matrix(rng, m, k, dtype), matrix(rng, n, k, dtype, scale=2 * k ** -0.5)
        b = matrix(rng, 1, n, bt)[0] if bt else None
        r = matrix(rng, m, n, rt) if rt else None
        y = opr.opr_linear(x, w, b, activation, r, out_dtype=TYPES[yt])
        ry, rz = lo.linear(to64(x), to64(w), 0 if b is None else to64(b), activation, None if r is None else to64(r))
        bz = sum_bound(to64(x), to64(w), k) + (np.abs(rz) + 2) * 2.0 ** -23
        within(y, ry, act_bound(rz, bz, activation) + (np.abs(ry) + 4) * 2.0 ** -23, yt, f"{m, n, k}")


@pytest.mark.parametrize("activation", ["silu", "gelu", "gelu_tanh"])
def test_activations_over_their_whole_range(activation):
    """Every exponent of z, both signs, the ends and NaN, through a product by one: forward within 2^-20 of
    |z| + 1, slope (the gradient of y for dy = 1) within 2^-19; far out they are 0 or z, 0 or 1."""
    e = np.arange(-40, 41)
    z = np.concatenate([s * m * 2.0 ** e for s in (1, -1) for m in (1, 1.25, 1.5, 1.75)] + [[0.0], np.linspace(-9, 9, 511)])
    z = torch.from_numpy(z.astype(np.float32)).to("cuda", torch.bfloat16)
    one = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    one[0, 0] = 1
    x = torch.zeros(len(z), 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = z
    y = opr.opr_linear(x, one, activation=activation, out_dtype=torch.float32)[:, 0]
    Z = to64(z)
    with np.errstate(over="ignore"):
        ref, slope = lo.act(Z, activation), lo.act_slope(Z, activation)
    big = np.abs(Z) > 1e6  # z^3 overflows in the plain formula: the limits
    ref[big], slope[big] = np.where(Z[big] > 0, Z[big], 0), np.where(Z[big] > 0, 1, 0)
    within(y, ref, (np.abs(Z) + 1) * 2.0 ** -20 * np.where(np.abs(Z) > 64, 0.25, 1), "fp32")
    dy = torch.ones(len(z), 1, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    dz, _, _ = opr.opr_linear_bwd(dy, x, w, z[:, None], activation, need_dw=False, dx_dtype=torch.float32)
    within(dz[:, 0], slope, 2.0 ** -19 + half_step("bf16") * np.abs(slope), "fp32")
    for v in (float("nan"), float("inf"), float("-inf")):
        x[0, 0] = v
        got = opr.opr_linear(x, one, activation=activation, out_dtype=torch.float32)[0, 0]
        want = torch.nn.functional.silu(torch.tensor(v)) if v != float("inf") else torch.tensor(v)
        assert torch.isnan(got) == torch.isnan(want) and (v != float("inf") or got == v)


@pytest.mark.parametrize("wide,offset", [(8, 0), (8, 8), (64, 16), (3, 0), (8, 1)])
def test_linear_on_parts_of_wider_rows(wide, offset):
    """Operands, residual and result inside wider rows, on and off the 16-byte grid; nothing else is written,
    and what lies next to the operands does not reach the sums (it is NaN here)."""
    rng = np.random.default_rng(4)
    m, n, k = 150, 72, 104

    def inside(rows, cols, dtype):
        t = torch.full((rows + 2, cols + wide), float("nan"), dtype=TYPES[dtype], device="cuda")
        v = t[1:rows + 1, offset:offset + cols]
        v.copy_(matrix(rng, rows, cols, dtype))
        return t, v

    (_, x), (_, w), (_, r) = inside(m, k, "bf16"), inside(n, k, "bf16"), inside(m, n, "bf16")
    ty, y = inside(m, n, "bf16")
    ty.fill_(5.0)
    got = opr.opr_linear(x, w, residual=r, out=y)
    ref = to64(x) @ to64(w).T + to64(r)
    within(got, ref, sum_bound(to64(x), to64(w), k) + np.abs(ref) * 2.0 ** -23, "bf16")
    rest = torch.ones_like(ty, dtype=torch.bool)
    rest[1:m + 1, offset:offset + n] = False
    assert (ty[rest] == 5).all()
    # gradients of the same views, into views
    dy = matrix(rng, m, n, "bf16")
    (tdx, dx), (tdw, dw) = inside(m, k, "bf16"), inside(n, k, "bf16")
    tdx.fill_(5.0), tdw.fill_(5.0)
    opr.opr_linear_bwd(dy, x, w, out=(dx, dw))
    within(dx, to64(dy) @ to64(w), sum_bound(to64(dy), to64(w).T, n), "bf16")
    within(dw, to64(dy).T @ to64(x), sum_bound(to64(dy).T, to64(x).T, m), "bf16")
    for t, rows, cols in ((tdx, m, k), (tdw, n, k)):
        rest = torch.ones_like(t, dtype=torch.bool)
        rest[1:rows + 1, offset:offset + cols] = False
        assert (t[rest] == 5).all()


@pytest.mark.parametrize("n,k", [(72, 101), (71, 100), (70, 99), (69, 98), (68, 97), (65, 66)])
@pytest.mark.parametrize("m", [5, 150, 2400])
def test_linear_rows_that_end_inside_sixteen_bytes(m, n, k):
    """Rows that start on the 16-byte grid (and so are read in place) but end off it, NaN right behind them
    in every operand: nothing of it reaches a sum, and nothing is written behind the results' ends."""
    rng = np.random.default_rng(18)
    if m == 2400:
        n += 2296  # many tiles: the CTA pairs

    def inside(rows, cols, dtype, fill=float("nan")):
        t = torch.full((rows, (cols + 7) // 8 * 8 + 8), fill, dtype=TYPES[dtype], device="cuda")
        v = t[:, :cols]
        v.copy_(matrix(rng, rows, cols, dtype))
        return t, v

    (_, x), (_, w), (_, r), (_, dy) = (inside(*a, "bf16") for a in ((m, k), (n, k), (m, n), (m, n)))
    ty, y = inside(m, n, "bf16", 5.0)
    opr.opr_linear(x, w, residual=r, out=y)
    ref = to64(x) @ to64(w).T + to64(r)
    within(y, ref, sum_bound(to64(x), to64(w), k) + np.abs(ref) * 2.0 ** -23, "bf16")
    (tdx, dx), (tdw, dw) = inside(m, k, "bf16", 5.0), inside(n, k, "bf16", 5.0)
    _, _, db = opr.opr_linear_bwd(dy, x, w, bias=True, out=(dx, dw))
    within(dx, to64(dy) @ to64(w), sum_bound(to64(dy), to64(w).T, n), "bf16")
    within(dw, to64(dy).T @ to64(x), sum_bound(to64(dy).T, to64(x).T, m), "bf16")
    within(db, to64(dy).sum(0), np.abs(to64(dy)).sum(0) * 2.0 ** -14, "fp32")
    for t, v in ((ty, y), (tdx, dx), (tdw, dw)):
        assert (t[:, v.shape[1]:] == 5).all()


def test_linear_into_its_residual():
    rng = np.random.default_rng(5)
    x, w, r = matrix(rng, 300, 128, "bf16"), matrix(rng, 200, 128, "bf16"), matrix(rng, 300, 200, "fp32")
    want = opr.opr_linear(x, w, residual=r, out_dtype=torch.float32)
    got = opr.opr_linear(x, w, residual=r, out=r)
    assert got is r and torch.equal(got, want)
    dy, add = matrix(rng, 300, 200, "bf16"), matrix(rng, 300, 128, "bf16")
    want, _, _ = opr.opr_linear_bwd(dy, x, w, dx_residual=add, need_dw=False)
    got, dw, db = opr.opr_linear_bwd(dy, x, w, dx_residual=add, need_dw=False, out=(add, None))
    assert got is add and dw is None and db is None and torch.equal(got, want)


def test_large_products_into_their_residual():
    rng = np.random.default_rng(17)
    x, w, r = matrix(rng, 2500, 64, "bf16"), matrix(rng, 2304, 64, "bf16"), matrix(rng, 2500, 2304, "bf16")
    want = opr.opr_linear(x, w, residual=r)
    assert torch.equal(opr.opr_linear(x, w, residual=r, out=r), want)
    r32 = matrix(rng, 2500, 2304, "fp32")
    want = opr.opr_linear(x, w, residual=r32, out_dtype=torch.float32)
    assert torch.equal(opr.opr_linear(x, w, residual=r32, out=r32), want)


@pytest.mark.parametrize("m", [2, 100])
def test_linear_with_very_many_columns(m):
    """More tiles along n than a grid has rows; offsets of y and w past 2^31 bytes."""
    n, k = 64 * 65535 * (8 if m == 2 else 3) + 200, 8 if m == 100 else 40
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, k, device="cuda", dtype=torch.bfloat16, generator=g)
    w = torch.randn(n, k, device="cuda", dtype=torch.bfloat16, generator=g)
    y = opr.opr_linear(x, w)
    for cols in (slice(0, 1000), slice(n // 2, n // 2 + 1000), slice(n - 1000, n)):
        X, W = to64(x), to64(w[cols])
        within(y[:, cols], X @ W.T, sum_bound(X, W, k), "bf16")


def test_linear_keeps_infinities_and_nan_in_their_rows():
    rng = np.random.default_rng(6)
    x, w = matrix(rng, 140, 64, "bf16"), matrix(rng, 96, 64, "bf16")
    clean = opr.opr_linear(x, w)
    x[3, 5], x[139, 0] = float("inf"), float("nan")
    y = opr.opr_linear(x, w)
    rows = torch.ones(140, dtype=torch.bool, device="cuda")
    rows[[3, 139]] = False
    assert torch.equal(y[rows], clean[rows]) and y[139].isnan().all() and not y[3].isfinite().any()


def test_linear_flags_fp16_overflow():
    st = status()
    x, w = torch.full((4, 64), 64.0, dtype=torch.float16, device="cuda"), torch.ones(8, 64, dtype=torch.float16, device="cuda")
    opr.opr_linear(x, w, dev_status=st)
    assert opr.read_status(st) == []
    opr.opr_linear(x, w * 16, dev_status=st)  # 65536
    assert opr.read_status(st) == [_abi.DEV_BITS[16]]
    y = opr.opr_linear(x, w * 16, out_dtype=torch.float32, dev_status=st.zero_())
    assert opr.read_status(st) == [] and (y == 65536).all()


BWD_SHAPES = [(1, 8, 8), (1, 1, 1), (3, 130, 7), (64, 64, 64), (129, 72, 200), (300, 257, 96), (1000, 40, 264),
              (2500, 96, 128), (130, 513, 33), (17, 2000, 1024), (5000, 136, 72)]


@pytest.mark.parametrize("activation", [None, "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", BWD_SHAPES, ids=str)
def test_linear_gradients_match_oracle(shape, dtype, activation):
    """With an activation dz is rounded for the products: half a step of each |dz|, times the other factor,
    summed (the worst case), and the whole dx and dw within one step (two independent half steps) in norm."""
    m, n, k = shape
    rng = np.random.default_rng(m + 3 * n)
    x, w, dy = matrix(rng, m, k, dtype), matrix(rng, n, k, dtype, scale=k ** -0.5), matrix(rng, m, n, dtype)
    z = matrix(rng, m, n, dtype, scale=2.0) if activation else None
    add = matrix(rng, m, k, dtype)
    st = status()
    dx, dw, db = opr.opr_linear_bwd(dy, x, w, z, activation, dx_residual=add, bias=True, dev_status=st)
    assert opr.read_status(st) == []
    X, W = to64(x), to64(w)
    rx, rw, rb, dz = lo.linear_bwd(to64(dy), X, W, to64(z) if activation else None, activation, to64(add))
    # the slope in fp32 within 2^-19 (its terms are at most a few units), dz rounded to the operands' type
    slip = 0 * dz if activation is None else np.abs(to64(dy)) * 2.0 ** -19
    off = slip if activation is None else slip + half_step(dtype) * (np.abs(dz) + slip) + (2.0 ** -25 if dtype == "fp16" else 0)
    within(dx, rx, sum_bound(dz, W.T, n) + off @ np.abs(W) + np.abs(rx) * 2.0 ** -23, dtype, f"dx {shape}")
    within(dw, rw, sum_bound(dz.T, X.T, m) + off.T @ np.abs(X), dtype, f"dw {shape}")
    # db: a chain of at most 1024 fp32 additions
    within(db, rb, np.abs(dz).sum(0) * 2.0 ** -14 + slip.sum(0), "fp32", f"db {shape}")
    eps = torch.finfo(TYPES[dtype]).eps
    for got, ref in ((dx, rx), (dw, rw)):
        assert np.linalg.norm(to64(got) - ref) <= eps * np.linalg.norm(ref)
    # each result asked for alone is the same, bit for bit
    a, none, no = opr.opr_linear_bwd(dy, x, w, z, activation, dx_residual=add, need_dw=False)
    assert none is None and no is None and torch.equal(a, dx)
    _, b, _ = opr.opr_linear_bwd(dy, x, w, z, activation, need_dx=False)
    _, _, c = opr.opr_linear_bwd(dy, x, w, z, activation, bias=True, need_dx=False, need_dw=False)
    assert torch.equal(b, dw) and torch.equal(c, db)


def test_linear_gradients_in_fp32():
    rng = np.random.default_rng(8)
    m, n, k = 3000, 136, 200
    x, w, dy = matrix(rng, m, k, "bf16"), matrix(rng, n, k, "bf16"), matrix(rng, m, n, "bf16")
    dx, dw, _ = opr.opr_linear_bwd(dy, x, w, dx_dtype=torch.float32, dw_dtype=torch.float32)
    within(dx, to64(dy) @ to64(w), sum_bound(to64(dy), to64(w).T, n), "fp32")
    within(dw, to64(dy).T @ to64(x), sum_bound(to64(dy).T, to64(x).T, m), "fp32")


@pytest.mark.parametrize("n,k", [(40, 64), (3, 7), (1, 1)])
def test_linear_of_no_rows(n, k):
    x, w = torch.empty(0, k, dtype=torch.bfloat16, device="cuda"), torch.ones(n, k, dtype=torch.bfloat16, device="cuda")
    assert opr.opr_linear(x, w).shape == (0, n)
    dy = torch.empty(0, n, dtype=torch.bfloat16, device="cuda")
    for z, act in ((None, None), (dy, "silu")):
        dx, dw, db = opr.opr_linear_bwd(dy, x, w, z, act, bias=True)
        assert dx.shape == (0, k) and (dw == 0).all() and (db == 0).all() and dw.shape == (n, k)


@pytest.mark.parametrize("m,n", [(5, 128), (64, 72), (33, 65), (300, 320), (16384, 256)])
def test_each_product_sees_the_one_before(m, n):
    """A chain of products with a permutation matrix, each on the last one's result, in buffers that take
    turns: exact, so that any product that started on unfinished rows shows."""
    g = torch.Generator(device="cuda").manual_seed(m)
    perm = torch.randperm(n, device="cuda", generator=g)
    w = torch.zeros(n, n, dtype=torch.bfloat16, device="cuda")
    w[torch.arange(n, device="cuda"), perm] = 1  # (x w^T)[:, j] = x[:, perm[j]]
    x = torch.randn(m, n, device="cuda", generator=g).bfloat16()
    want, st = x, status()
    bufs = [x.clone(), torch.empty_like(x)]
    torch.cuda.synchronize()
    for i in range(60):
        opr.opr_linear(bufs[i % 2], w, out=bufs[1 - i % 2], dev_status=st)
    for i in range(60):  # and back, through the gradient of x
        opr.opr_linear_bwd(bufs[i % 2], bufs[i % 2], w, need_dw=False, out=(bufs[1 - i % 2], None), dev_status=st)
    assert torch.equal(bufs[0], want) and opr.read_status(st) == []


def test_linear_refusals_of_tensors():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(x=x.float()), dict(w=w.half()), dict(w=w[:, :32]), dict(x=x.t()), dict(bias=x[0]),
                dict(activation="relu6"), dict(residual=x), dict(out=torch.zeros(4, 9, device="cuda")),
                dict(out_dtype=torch.float64), dict(dev_status=torch.zeros(1, device="cuda")), dict(out=x[:, :8])):
        with pytest.raises(opr.OprError):
            opr.opr_linear(**{**dict(x=x, w=w), **bad})
    dy = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(dy=dy.float()), dict(dy=dy[:3]), dict(activation="silu"), dict(need_dx=False, dx_residual=x),
                dict(out=(x, None)), dict(out=(None, w)), dict(dw_dtype=torch.int32)):
        with pytest.raises(opr.OprError):
            opr.opr_linear_bwd(**{**dict(dy=dy, x=x, w=w), **bad})


@pytest.mark.parametrize("sizes", [(150, 136, 264), (37, 65, 33), (1, 1024, 512)], ids=str)
def test_linear_on_a_side_stream_and_in_a_graph(sizes):
    m, n, k = sizes
    rng = np.random.default_rng(9)
    x, w, dy = matrix(rng, m, k, "bf16"), matrix(rng, n, k, "bf16"), matrix(rng, m, n, "bf16")

    def step():
        y, z = opr.opr_linear(x, w, activation="gelu_tanh", save_z=True)
        return (y, z, *opr.opr_linear_bwd(dy, x, w, z, "gelu_tanh", bias=True))

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
    x.copy_(matrix(rng, m, k, "bf16"))
    graph.replay()
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, held))


@pytest.mark.parametrize("sizes", [(257, 264, 128), (2300, 2304, 200), (2200, 2056, 72), (6000, 1001, 136),
                                   (2600, 2068, 64), (4100, 1500, 640)], ids=str)
def test_large_products_match_oracle(sizes):
    """Enough 256 x 256 tiles for every pair of SMs to take more than one, with ends inside tiles in each
    direction."""
    m, n, k = sizes
    rng = np.random.default_rng(m)
    x, w, r = matrix(rng, m, k, "bf16"), matrix(rng, n, k, "bf16", scale=k ** -0.5), matrix(rng, m, n, "bf16")
    b = matrix(rng, 1, n, "bf16")[0]
    y = opr.opr_linear(x, w, b, "silu", r)
    X, W = to64(x), to64(w)
    ry, rz = lo.linear(X, W, to64(b), "silu", to64(r))
    bz = sum_bound(X, W, k) + (np.abs(rz) + 2) * 2.0 ** -23
    within(y, ry, act_bound(rz, bz, "silu") + (np.abs(ry) + 4) * 2.0 ** -23, "bf16")
    dy = matrix(rng, m, n, "bf16", scale=0.1)
    dx, dw, _ = opr.opr_linear_bwd(dy, x, w)
    within(dx, to64(dy) @ W, sum_bound(to64(dy), W.T, n), "bf16")
    within(dw, to64(dy).T @ X, sum_bound(to64(dy).T, X.T, m), "bf16")
    # the transposed problem has the same dw, transposed: other operands, other tiles
    _, dwt, _ = opr.opr_linear_bwd(x, dy, torch.zeros(k, n, dtype=torch.bfloat16, device="cuda"), need_dx=False)
    within(dwt, to64(x).T @ to64(dy), sum_bound(to64(x).T, to64(dy).T, m), "bf16")


@pytest.mark.parametrize("activation", [None, "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16", "bf16"), ("fp16", "fp32", "bf16", "fp16"),
                                   ("bf16", "fp16", "fp32", "fp32"), ("fp16", None, "fp16", "bf16"),
                                   ("bf16", "bf16", None, "fp16")])
def test_large_epilogues(types, activation):
    """As test_linear_epilogues with z kept, where the products go through the CTA pairs; n ends inside a
    block of 32 columns, and inside eight entries of it."""
    dtype, bt, rt, yt = types
    rng = np.random.default_rng(13)
    for m, n, k in ((2500, 2075, 64), (2311, 2304, 72)):
        x, w = matrix(rng, m, k, dtype), matrix(rng, n, k, dtype, scale=2 * k ** -0.5)
        b = matrix(rng, 1, n, bt)[0] if bt else None
        ld = (n + 7) // 8 * 8
        r = matrix(rng, m, n, rt, wide=ld - n) if rt else None
        out = torch.full((m, ld), 5.0, dtype=TYPES[yt], device="cuda")
        y = opr.opr_linear(x, w, b, activation, r, out=out[:, :n])
        z = opr.opr_linear(x, w, b, activation, r, save_z=True)[1]
        assert (out[:, n:] == 5).all()
        ry, rz = lo.linear(to64(x), to64(w), 0 if b is None else to64(b), activation, None if r is None else to64(r))
        bz = sum_bound(to64(x), to64(w), k) + (np.abs(rz) + 2) * 2.0 ** -23
        within(z, rz, bz, dtype, f"z {m, n, k}")
        within(y, ry, act_bound(rz, bz, activation) + (np.abs(ry) + 4) * 2.0 ** -23, yt, f"{m, n, k}")


@pytest.mark.parametrize("sizes", [(3, 64, 4096), (300, 300, 4096), (6000, 1024, 512)], ids=str)
def test_linear_reports_a_pipeline_timeout(sizes):
    """With a wait limit of 0 every wait that is not already done gives up: the call reports it, the kernel
    ends, and the next call with the usual limit is right.  (A wait may be done already: not every try trips.)"""
    m, n, k = sizes
    rng = np.random.default_rng(1)
    x, w = matrix(rng, m, k, "bf16"), matrix(rng, n, k, "bf16")
    want = opr.opr_linear(x, w)
    torch.cuda.synchronize()
    lib, st = opr.load_library(), status()
    prev = lib.opr_testing_set_wait_limit_ns(0)
    try:
        opr.opr_linear(x, w, dev_status=st)
        torch.cuda.synchronize()
    finally:
        lib.opr_testing_set_wait_limit_ns(prev)
    assert opr.read_status(st) == [_abi.DEV_BITS[8]]
    assert torch.equal(opr.opr_linear(x, w, dev_status=st.zero_()), want) and opr.read_status(st) == []


@pytest.mark.parametrize("k", [2 ** 30 - 7, 2 ** 30 + 9])
def test_linear_copies_rows_whose_bytes_pass_32_bits(k):
    """One row each of x and w off the 16-byte grid, about 2^31 bytes long: every piece of them reaches the
    copies (the workspace is NaN before).  Ones in a few places, so the sum is exact."""
    at = [0, 7, 2 ** 29 - 1, 2 ** 29, 2 ** 29 + 300, k - 513, k - 256, k - 9, k - 8, k - 2, k - 1]
    x = torch.zeros(k + 1, dtype=torch.bfloat16, device="cuda")[1:].view(1, k)
    w = torch.zeros(k + 3, dtype=torch.bfloat16, device="cuda")[3:].view(1, k)
    x[0, at], w[0, at] = 1, 1
    x[0, [1, 2 ** 29 + 1, k - 3]] = 1  # against zeros of w
    ws = torch.full((opr.opr_linear_workspace_bytes(x, w) // 4,), float("nan"), device="cuda")
    st = status()
    y = opr.opr_linear(x, w, out_dtype=torch.float32, workspace=ws, dev_status=st)
    assert opr.read_status(st) == [] and y.item() == len(at)


@pytest.mark.parametrize("activation", ["silu", "gelu", "gelu_tanh"])
def test_activations_of_every_bf16_exponent(activation):
    """z from the smallest normal bf16 to the largest, both signs, as above; the slope at the infinities is
    its limit, 0 or 1, and NaN stays NaN.  (In fp64 the formulas reach these limits without overflow.)"""
    e = np.arange(-126, 128)
    z = np.concatenate([s * m * 2.0 ** e for s in (1, -1) for m in (1, 1.25, 1.5, 1.75)])
    z = torch.from_numpy(z).to("cuda", torch.bfloat16)
    one = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    one[0, 0] = 1
    x = torch.zeros(len(z), 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = z
    y = opr.opr_linear(x, one, activation=activation, out_dtype=torch.float32)[:, 0]
    Z = to64(z)
    with np.errstate(over="ignore"):
        ref, slope = lo.act(Z, activation), lo.act_slope(Z, activation)
    within(y, ref, (np.abs(Z) + 1) * 2.0 ** -20 * np.where(np.abs(Z) > 64, 0.25, 1), "fp32")
    z = torch.cat((z, torch.tensor([float("inf"), float("-inf"), float("nan")], device="cuda").bfloat16()))
    slope = np.concatenate((slope, [1, 0]))
    for n in (1, 8):  # entry by entry, and in 16-byte accesses
        dy, zn = torch.ones(len(z), n, dtype=torch.bfloat16, device="cuda"), z[:, None].expand(-1, n).contiguous()
        w = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
        w[n - 1] = 1
        x = torch.zeros(len(z), 8, dtype=torch.bfloat16, device="cuda")
        dz, _, db = opr.opr_linear_bwd(dy, x, w, zn, activation, need_dw=False, bias=True, dx_dtype=torch.float32)
        within(dz[:-1, 0], slope, 2.0 ** -19 + half_step("bf16") * np.abs(slope), "fp32")
        assert dz[-1].isnan().all() and db.isnan().all()
        _, _, db = opr.opr_linear_bwd(dy[:-1], x[:-1], w, zn[:-1], activation, need_dx=False, need_dw=False, bias=True)
        within(db, np.full(n, slope.sum()), np.full(n, len(slope) * (2.0 ** -19 + 2.0 ** -14)), "fp32")


def test_results_keep_the_status_word_of_a_call_that_was_given_none():
    """A timeout and an fp16 overflow are there to read on the results, each call with a word of its own."""
    rng = np.random.default_rng(31)
    x, w, dy = matrix(rng, 300, 4096, "bf16"), matrix(rng, 300, 4096, "bf16"), matrix(rng, 300, 300, "bf16")
    good, z = opr.opr_linear(x, w, save_z=True)
    assert opr.read_status(good) == [] and opr.read_status(z) == []
    lib = opr.load_library()
    torch.cuda.synchronize()
    prev = lib.opr_testing_set_wait_limit_ns(0)
    try:
        y, z = opr.opr_linear(x, w, save_z=True)
        grads = opr.opr_linear_bwd(dy, x, w, bias=True)
        torch.cuda.synchronize()
    finally:
        lib.opr_testing_set_wait_limit_ns(prev)
    for t in (y, z, *grads):
        assert opr.read_status(t) == [_abi.DEV_BITS[8]]
    assert opr.read_status(good) == []
    x, w = torch.full((4, 64), 64.0, dtype=torch.float16, device="cuda"), torch.full((8, 64), 16.0, dtype=torch.float16, device="cuda")
    assert opr.read_status(opr.opr_linear(x, w)) == [_abi.DEV_BITS[16]]
    out = torch.empty(4, 8, device="cuda")
    assert opr.read_status(opr.opr_linear(x, w, out=out)) == []
    # a word that the caller gives is the results' too
    st = status()
    assert opr.read_status(opr.opr_linear(x, w, dev_status=st)) == opr.read_status(st) == [_abi.DEV_BITS[16]]


# sums of 64 products by one: 65504 with 1023.5 each, the largest below fp16's overflow, the first that overflows
NEAR = {65511.5: {0: 1031.0}, 65519.5: {0: 1039.0}, 65520.0: {0: 1039.0, 1: 1024.0}}


@pytest.mark.parametrize("m,n", [(4, 16), (4, 13), (200, 72), (200, 65), (2500, 2304), (2500, 2075)])
@pytest.mark.parametrize("value", NEAR)
def test_fp16_overflow_is_that_of_the_stored_value(m, n, value):
    """Sums up to 65520 round to 65504, which is no overflow; 65520 itself is stored as an infinity."""
    x, w = torch.ones(m, 64, dtype=torch.float16, device="cuda"), torch.full((n, 64), 1023.5, dtype=torch.float16, device="cuda")
    for i, v in NEAR[value].items():
        w[n - 1, i] = v
    over = value >= 65520
    for kw in (dict(), dict(save_z=True, out_dtype=torch.float32)):
        st = status()
        got = opr.opr_linear(x, w, dev_status=st, **kw)
        got = got[1] if kw else got
        assert (got[:, :-1] == 65504).all() and (got[:, -1] == (float("inf") if over else 65504)).all()
        assert opr.read_status(st) == ([_abi.DEV_BITS[16]] if over else [])


@pytest.mark.parametrize("n", [8, 3])
def test_fp16_overflow_of_a_gradient_behind_an_activation(n):
    """dz = dy act'(z), silu: entries between 65504 and 65520 by a margin above the slope's error, and past
    65520."""
    z = torch.arange(1.0, 4.0, 2.0 ** -9, device="cuda").half()
    slope = torch.from_numpy(lo.act_slope(to64(z), "silu"))
    dy = torch.arange(57344.0, 65504.0, 32.0)
    prod = dy.double()[:, None] * slope
    x, w = torch.zeros(5, 8, dtype=torch.float16, device="cuda"), torch.zeros(n, 8, dtype=torch.float16, device="cuda")
    for a, b, over in ((65506, 65518, False), (65522, 65530, True)):
        i, j = ((prod > a) & (prod < b)).nonzero()[0].tolist()
        g, zz = torch.zeros(5, n, dtype=torch.float16, device="cuda"), torch.zeros(5, n, dtype=torch.float16, device="cuda")
        g[4, n - 1], zz[4, n - 1] = dy[i].item(), z[j]
        st = status()
        opr.opr_linear_bwd(g, x, w, zz, "silu", dev_status=st)
        assert opr.read_status(st) == ([_abi.DEV_BITS[16]] if over else [])


@pytest.mark.parametrize("n,m", [(18945, 32768), (151552, 8192)], ids=["entry by entry", "sixteen bytes"])
def test_column_sums_of_many_rows_under_wide_outputs(n, m):
    """So many columns that all rows could be one block's, eight threads to them: 2^8 in each thread's first
    row, then 2^-17, which a running fp32 sum would drop every time.  At most 256 entries are added to one fp32
    sum (each addition off by at most 2^-24 of the sum so far), the parts in fp64, and the eight threads'
    results in fp32: (256 + 8) 2^-24 of the sum of sizes."""
    dy = torch.full((m, n), 2.0 ** -17, dtype=torch.bfloat16, device="cuda")
    dy[:8] = 2.0 ** 8
    x, w = torch.zeros(m, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    _, _, db = opr.opr_linear_bwd(dy, x, w, bias=True, need_dx=False, need_dw=False)
    want = 8 * 2.0 ** 8 + (m - 8) * 2.0 ** -17
    within(db, np.full(n, want), np.full(n, 264 * 2.0 ** -24 * want), "fp32")


@pytest.mark.parametrize("n", [3, 8])
def test_column_sums_of_more_row_blocks_than_a_grid_is_high(n):
    """2048 rows at most to a block, 2^15 blocks to each z of the grid: ones, which sum exactly up to the
    result's rounding; the last rows, which lie in the second z, count 3."""
    m = 2 ** 26 + 4099
    dy = torch.ones(m, n, dtype=torch.bfloat16, device="cuda")
    dy[-4000:] = 3
    x, w = torch.zeros(m, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    _, _, db = opr.opr_linear_bwd(dy, x, w, bias=True, need_dx=False, need_dw=False)
    within(db, np.full(n, m + 2.0 * 4000), np.zeros(n), "fp32")
