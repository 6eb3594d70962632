"""The attention layer end to end (OnePassAttentionLayer): projections, norm with rotation, masked
attention, output projection and residual, forward and backward, against the layer in fp64."""

import ctypes

import numpy as np
import pytest
import torch

import block_sparse_masked_segment_b200 as opr
import synth
from layer_helpers import matrix, to64
from oracle import layer_oracle as lo
from oracle import opr_oracle as orc

pytestmark = pytest.mark.gpu


def layer64(x, wqkv, wo, qw, kw, bqkv, bo, res, w, lay, freq, scale, interleaved, dy):
    """The layer and its gradients in fp64."""
    T, hq, hkv, d = len(x), w.hq, w.hkv, w.d
    proj = (x @ wqkv.T + bqkv).reshape(T, hq + 2 * hkv, d)
    q, k, v = proj[:, :hq], proj[:, hq:hq + hkv], proj[:, hq + hkv:]
    pos = lay.pos_id
    qr = lo.norm_rotate(q, qw, pos, freq, 1e-6, interleaved, scale)
    kr = lo.norm_rotate(k, kw, pos, freq, 1e-6, interleaved, scale)
    o, lse = orc.attention_fwd(qr, kr, v, lay)
    y = o.reshape(T, -1) @ wo.T + bo + res
    do = (dy @ wo).reshape(T, hq, d)
    dqr, dkr, dv = orc.attention_bwd(qr, kr, v, o, do, lse, lay)
    dq, dqw = lo.norm_rotate_bwd(dqr, q, qw, pos, freq, 1e-6, interleaved, scale)
    dk, dkw = lo.norm_rotate_bwd(dkr, k, kw, pos, freq, 1e-6, interleaved, scale)
    dp = np.concatenate([dq, dk, dv], 1).reshape(T, -1)
    return y, dict(x=dp @ wqkv, w_qkv=dp.T @ x, w_o=dy.T @ o.reshape(T, -1), q_weight=dqw, k_weight=dkw,
                   b_qkv=dp.sum(0), b_o=dy.sum(0))


@pytest.mark.parametrize("interleaved,rot,biased", [(False, 128, True), (True, 64, False)])
def test_layer_forward_and_backward(interleaved, rot, biased):
    """Every intermediate (q, k, v, o, do, dq, dk, dv) is rounded to 16 bits on the way, P and dS too:
    about a dozen roundings of up to 2^-9, 2^-9 * sqrt(12) = 7e-3 of each result in norm where they are
    independent; the bound is twice that."""
    w = synth.make_custom_workload([[[(9, 40, 21), (5, 33, 30)], [(12, 20, 7)]], [[(30, 64, 50)]]], hq=4, hkv=2, d=128,
                                   base=1e4)
    T, width = w.total_tokens, 200
    lay = orc.build_layout(w.turn_lens, w.conv_turn_ptr, w.seq_conv_ptr)
    freq, scale = opr.opr_rotary_frequencies(rot, 1e4, "yarn", 4.0, 64.0)
    layer = opr.OnePassAttentionLayer(w.turn_lens, w.conv_turn_ptr, w.seq_conv_ptr, w.hq, w.hkv, w.d, freq, scale,
                                      interleaved)
    rng = np.random.default_rng(21)
    rows = (w.hq + 2 * w.hkv) * w.d
    x, res, dy = (matrix(rng, T, width, "bf16") for _ in range(3))
    wqkv, wo = matrix(rng, rows, width, "bf16", scale=width ** -0.5), matrix(rng, width, w.hq * w.d, "bf16", scale=0.05)
    bqkv, bo = (matrix(rng, 1, n, "bf16", scale=0.3)[0] for n in (rows, width)) if biased else (None, None)
    qw, kw = (1 + 0.2 * matrix(rng, 1, w.d, "bf16")[0] for _ in range(2))
    y, saved = layer.forward(x, wqkv, wo, qw, kw, bqkv, bo, residual=res)
    grads = layer.backward(dy, saved)
    torch.cuda.synchronize()
    assert opr.read_status(layer.layout.dev_status) == []
    zero = np.zeros(1)
    ry, ref = layer64(to64(x), to64(wqkv), to64(wo), to64(qw), to64(kw), to64(bqkv) if biased else zero,
                      to64(bo) if biased else zero, to64(res), w, lay, to64(freq), scale, interleaved, to64(dy))
    bound = 2 * 12 ** 0.5 * 2.0 ** -9
    assert np.linalg.norm(to64(y) - ry) <= bound * np.linalg.norm(ry)
    for name, r in ref.items():
        if not biased and name.startswith("b_"):
            assert grads[name] is None
            continue
        off = np.linalg.norm(to64(grads[name]).reshape(r.shape) - r) / np.linalg.norm(r)
        assert off <= bound, f"{name}: {off:.3e}"


def test_layer_gradient_is_the_slope_of_the_layer():
    """Along x's gradient direction the fp64 layer's change is the gradient's length: the library's dx gives
    the slope of sum(y dy) to within the layer's rounding."""
    w = synth.make_custom_workload([[[(6, 20, 9), (4, 11, 8)]]], hq=2, hkv=1, d=64, base=1e4)
    T, width = w.total_tokens, 64
    lay = orc.build_layout(w.turn_lens, w.conv_turn_ptr, w.seq_conv_ptr)
    freq, scale = opr.opr_rotary_frequencies(64, 1e4)
    layer = opr.OnePassAttentionLayer(w.turn_lens, w.conv_turn_ptr, w.seq_conv_ptr, w.hq, w.hkv, w.d, freq, scale)
    rng = np.random.default_rng(22)
    x, dy = matrix(rng, T, width, "bf16"), matrix(rng, T, width, "bf16")
    wqkv, wo = matrix(rng, 4 * 64, width, "bf16", scale=0.1), matrix(rng, width, 128, "bf16", scale=0.1)
    qw, kw = (1 + 0.2 * matrix(rng, 1, 64, "bf16")[0] for _ in range(2))
    _, saved = layer.forward(x, wqkv, wo, qw, kw)
    dx = to64(layer.backward(dy, saved)["x"])

    def value(xv):
        y, _ = layer64(xv, to64(wqkv), to64(wo), to64(qw), to64(kw), np.zeros(1), np.zeros(1), 0.0, w, lay, to64(freq),
                       scale, False, to64(dy))
        return (y * to64(dy)).sum()

    h = 1e-5
    slope = (value(to64(x) + h * dx) - value(to64(x) - h * dx)) / (2 * h)
    assert slope == pytest.approx((dx * dx).sum(), rel=2 * 12 ** 0.5 * 2.0 ** -9)


def test_layer_step_in_a_graph():
    w = synth.make_custom_workload([[[(20, 70, 40), (9, 80, 33)]]], hq=4, hkv=2, d=128, base=1e4)
    T, width = w.total_tokens, 256
    freq, scale = opr.opr_rotary_frequencies(128, 1e4)
    layer = opr.OnePassAttentionLayer(w.turn_lens, w.conv_turn_ptr, w.seq_conv_ptr, 4, 2, 128, freq, scale)
    rng = np.random.default_rng(23)
    x, dy = matrix(rng, T, width, "bf16"), matrix(rng, T, width, "bf16")
    wqkv, wo = matrix(rng, 8 * 128, width, "bf16", scale=0.1), matrix(rng, width, 512, "bf16", scale=0.1)
    qw, kw = (torch.ones(128, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        y, saved = layer.forward(x, wqkv, wo, qw, kw, residual=x)
        return [y] + [g for g in layer.backward(dy, saved).values() if g is not None]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.copy_(matrix(rng, T, width, "bf16"))
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_layer_refuses_other_shapes_and_types():
    w = synth.make_custom_workload([[[(6, 20, 9)]]], hq=2, hkv=1, d=64, base=1e4)
    freq, _ = opr.opr_rotary_frequencies(64, 1e4)
    layer = opr.OnePassAttentionLayer(w.turn_lens, w.conv_turn_ptr, w.seq_conv_ptr, 2, 1, 64, freq)
    x = torch.zeros(w.total_tokens, 64, dtype=torch.bfloat16, device="cuda")
    wqkv, wo = torch.zeros(256, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(64, 128, dtype=torch.bfloat16, device="cuda")
    qw = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(x=x[:-1]), dict(x=x.half()), dict(w_qkv=wqkv[:255]), dict(w_o=wo[:, :64])):
        with pytest.raises(opr.OprError):
            layer.forward(**{**dict(x=x, w_qkv=wqkv, w_o=wo, q_weight=qw, k_weight=qw), **bad})


def test_a_reported_cuda_error_is_not_left_behind():
    """A launch that fails on the host (into a capture that was ended by a call it forbids) is reported as
    OPR_CUDA_ERROR; the caller's next check of the runtime's last error, such as torch makes at each of its
    launches, does not find it again."""
    lib, runtime = opr.load_library(), ctypes.CDLL("libcudart.so.12")  # the runtime that both use
    x, y = torch.ones(4, 2, 64, device="cuda"), torch.empty(4, 2, 64, device="cuda")
    pos, freq = torch.arange(4, dtype=torch.int32, device="cuda"), torch.ones(32, dtype=torch.float64, device="cuda")
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert runtime.cudaStreamCreate(ctypes.byref(stream)) == 0
    assert runtime.cudaStreamBeginCapture(stream, 0) == 0
    assert runtime.cudaStreamSynchronize(stream) != 0  # forbidden: the capture is invalid from here
    runtime.cudaGetLastError()
    st = lib.opr_rotary(x.data_ptr(), 1, 128, y.data_ptr(), 1, 128, pos.data_ptr(), freq.data_ptr(), 64, 0, 1.0, 0, None,
                        4, 2, 64, None, stream)
    left = runtime.cudaGetLastError()
    runtime.cudaStreamEndCapture(stream, ctypes.byref(graph))
    runtime.cudaGetLastError()
    runtime.cudaStreamDestroy(stream)
    assert st == 3 and b"captur" in lib.opr_last_error() and left == 0
    assert opr.opr_rotary(x, pos, freq, out=y) is y and (y.isfinite()).all()
