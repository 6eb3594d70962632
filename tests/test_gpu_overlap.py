"""Kernels of the layer start while the kernel before them ends: nothing that runs behind them, however
early it starts, may meet unfinished work of what ran before them."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import block_sparse_masked_segment_b200 as opr
from layer_helpers import heads, matrix, to64, within
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


@pytest.fixture(scope="module")
def probes():
    if not os.path.exists(NVCC) and shutil.which("nvcc") is None:
        pytest.skip("needs nvcc")
    out_dir = os.path.join(ROOT, ".pytest_cache", "early_reader")  # git-ignored
    os.makedirs(out_dir, exist_ok=True)
    lib = os.path.join(out_dir, "libearly_reader.so")
    r = subprocess.run([NVCC if os.path.exists(NVCC) else "nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                        "-Xcompiler", "-fPIC", "-std=c++17", "-o", lib,
                        os.path.join(ROOT, "tests", "c", "early_reader.cu"), "-lcudart"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(lib)
    P = ctypes.c_void_p
    lib.write_late.argtypes = [P, ctypes.c_int32, ctypes.c_uint32, P]
    lib.read_early.argtypes = [P, P, P]
    return lib


def calls():
    """(name, call) with the inputs on the device: one call or more of each kernel that starts early."""
    rng = np.random.default_rng(40)
    x, k3 = heads(rng, 64, 8, 128, "bf16"), heads(rng, 64, 2, 128, "bf16")
    odd = heads(rng, 64, 2, 18, "bf16")
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    freq, freq6 = opr.opr_rotary_frequencies(128, 1e4)[0], opr.opr_rotary_frequencies(6, 1e4)[0]
    qw = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def product(m, n, k, **kw):
        a, b = matrix(rng, m, k, "bf16"), matrix(rng, n, k, "bf16")
        out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(opr.opr_linear_workspace_bytes(a, b), 16), dtype=torch.uint8, device="cuda")
        return lambda: opr.opr_linear(a, b, out=out, workspace=ws, dev_status=st, **kw)

    def sums(activation):
        a, b = matrix(rng, 200, 64, "bf16"), matrix(rng, 72, 64, "bf16")
        dy, z = matrix(rng, 200, 72, "bf16"), matrix(rng, 200, 72, "bf16")
        return lambda: opr.opr_linear_bwd(dy, a, b, z, activation, bias=True, need_dx=False, need_dw=False, dev_status=st)

    out, out_odd = torch.empty_like(x), torch.empty_like(odd)
    norm = (torch.empty_like(x), torch.empty_like(k3))
    return [("rotary", lambda: opr.opr_rotary(x, pos, freq, out=out)),
            ("rotary, odd sizes", lambda: opr.opr_rotary(odd, pos, freq6, out=out_odd)),
            ("norm", lambda: opr.opr_qk_norm_rope(x, k3, qw, qw, pos, freq, out=norm)),
            ("few rows", product(3, 256, 512)), ("tiles", product(130, 200, 64)), ("depth split", product(128, 128, 4096)),
            ("pairs", product(2600, 2304, 64)), ("row copies", product(65, 130, 67)), ("column sums", sums("silu"))]


@pytest.mark.parametrize("i", range(9))
def test_what_starts_early_finds_all_but_the_last_kernel_complete(probes, i):
    """A word is written late by the kernel before the call and read by one behind it before that waits for
    the call: the reader may start early, but not before the writer is complete."""
    name, call = calls()[i]
    word, seen = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(32, dtype=torch.int32, device="cuda")
    call()
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    for j in range(32):
        assert probes.write_late(word.data_ptr(), j + 1, 200_000, stream) == 0
        call()
        assert probes.read_early(word.data_ptr(), seen[j:].data_ptr(), stream) == 0
    assert seen.tolist() == list(range(1, 33)), name


@pytest.mark.parametrize("d", [64, 18])
def test_each_rotation_sees_the_one_before(d):
    """Sixty rotations in place and the sixty transposed ones, each on the last one's result: an entry that a
    rotation missed is off by a rotation.  Each step rounds fp32: 120 times the bound of one."""
    rng = np.random.default_rng(41)
    x = heads(rng, 3000, 3, d, "fp32")
    keep = to64(x)
    pos = torch.arange(1, 3001, dtype=torch.int32, device="cuda")
    freq, _ = opr.opr_rotary_frequencies(16 if d == 64 else 6, 1e4)
    rot = 2 * freq.numel()
    for inverse in (False, True):
        for _ in range(60):
            opr.opr_rotary(x, pos, freq, inverse=inverse)
        if not inverse:
            ref = lo.rotate(keep, 60 * to64(pos), to64(freq))
            size = np.zeros_like(keep)  # of the pairs, which rotations keep
            a, b = keep[..., :rot // 2], keep[..., rot // 2:rot]
            size[..., :rot // 2] = size[..., rot // 2:rot] = np.sqrt(a * a + b * b)
            within(x, ref, 60 * size * 2.0 ** -20, "fp32")
    within(x, keep, 120 * size * 2.0 ** -20, "fp32")


def test_rotation_and_norm_see_the_product_before():
    """A product with a permutation matrix (exact), its heads rotated behind it, the norm on the same heads,
    and a product of the rotated heads, in buffers that take turns: each call as if it ran alone."""
    rng = np.random.default_rng(42)
    m, h, d = 700, 2, 64
    n = h * d
    w = torch.zeros(n, n, dtype=torch.bfloat16, device="cuda")
    w[torch.arange(n, device="cuda"), torch.randperm(n, device="cuda", generator=torch.Generator("cuda").manual_seed(1))] = 1
    pos = torch.arange(m, dtype=torch.int32, device="cuda")
    freq, _ = opr.opr_rotary_frequencies(d, 1e4)
    qw = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    bufs = [torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    norm = tuple(torch.empty(m, h // 2, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i in range(20):
        x = matrix(rng, m, n, "bf16")
        results = []
        for apart in (True, False):
            for b in (*bufs, *norm):
                b.fill_(float("nan"))
            pause = torch.cuda.synchronize if apart else (lambda: None)
            pause()
            opr.opr_linear(x, w, out=bufs[0])
            pause()
            opr.opr_rotary(bufs[0].view(m, h, d), pos, freq, out=bufs[1].view(m, h, d))
            pause()
            heads3 = bufs[1].view(m, h, d)
            opr.opr_qk_norm_rope(heads3[:, :1], heads3[:, 1:], qw, qw, pos, freq, out=norm)
            pause()
            opr.opr_linear(bufs[1], w, out=bufs[2])
            results.append([b.clone() for b in (*bufs, *norm)])
        assert all(torch.equal(a, b) for a, b in zip(*results))
