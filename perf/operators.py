"""The measured cases of the layer operators around the one-pass attention: rotary positions
(``opr_rotary``), the norm of each head of q and k with the rotation in the same pass
(``opr_qk_norm_rope`` and its gradient), and the matrix product with bias, activation and residual
(``opr_linear`` and its gradients).

``run`` computes them in elementary torch operations in 32 bits, or, with ``own`` set, through the
package's calls.  ``exact`` computes the same outputs in 64 bits from the definitions.
"""

import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token's q heads of the 32q model shape, rotated in place of a longer call: pure latency
        dict(name="rotary one token", op="rotary", tokens=1, heads=32, d=128, rot=128, interleaved=True, inverse=False,
             rule="none", base=1e4, far=32768, x="bf16", y="bf16", mapped=False),
        # q of a 16K batch (32 heads of 128), half of each head rotated, frequencies stretched for a long
        # context, positions up to a million, written in the attention order as fp16
        dict(name="rotary long context", op="rotary", tokens=16384, heads=32, d=128, rot=64, interleaved=False,
             inverse=False, rule="yarn", base=1e6, far=1 << 20, x="bf16", y="fp16", mapped=True),
        # the fp32 gradient of k (8 heads) of an odd-sized batch rotated back
        dict(name="rotary gradient", op="rotary", tokens=32749, heads=8, d=128, rot=128, interleaved=True,
             inverse=True, rule="linear", base=1e6, far=65536, x="fp32", y="fp32", mapped=False),
        # one token, 32q/8kv heads: latency of the fused pass
        dict(name="qk norm one token", op="qknorm", tokens=1, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             rule="none", base=1e6, far=32768, x="bf16", y="fp16", mapped=False, packed=True),
        # the 16K packed batch of the 32q/8kv shape, q, k, v of one projection into the attention order
        dict(name="qk norm 16K", op="qknorm", tokens=16384, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             rule="none", base=1e6, far=4096, x="bf16", y="fp16", mapped=True, packed=True),
        # gradients of the 64K batch of the 64q/8kv shape, as the attention's backward leaves them (fp32)
        dict(name="qk norm gradient 64K", op="qknorm_bwd", tokens=65536, hq=64, hkv=8, d=128, rot=128,
             interleaved=False, rule="none", base=1e6, far=32768, x="bf16", dy="fp32", packed=True),
        # an odd-sized small batch with 64-wide heads, part of the head rotated, interleaved pairs
        dict(name="qk norm gradient ragged", op="qknorm_bwd", tokens=2377, hq=8, hkv=2, d=64, rot=32,
             interleaved=True, rule="linear", base=1e4, far=8192, x="fp16", dy="fp32", packed=False),
        # one row through the q, k, v projection of the 32q/8kv shape: bound by reading the weight
        dict(name="linear one row", op="linear", m=1, n=6144, k=4096, x="bf16", y="bf16", bias=True,
             act=None, residual=False, keep_z=False),
        # the q, k, v projection of the 16K batch
        dict(name="linear 16K", op="linear", m=16384, n=6144, k=4096, x="bf16", y="bf16", bias=True, act=None,
             residual=False, keep_z=False),
        # odd sizes everywhere (no row is a multiple of 16 bytes), activation, residual and the kept z
        dict(name="linear ragged", op="linear", m=777, n=1003, k=1111, x="fp16", y="fp16", bias=True,
             act="gelu", residual=True, keep_z=True),
        # the gradients of the output projection of the 16K batch
        dict(name="linear gradient 16K", op="linear_bwd", m=16384, n=4096, k=4096, x="bf16", act=None, bias=False,
             add=False),
        # a ragged batch through an activation: gradients of x (with the residual's), w and bias
        dict(name="linear gradient ragged", op="linear_bwd", m=2377, n=4096, k=1024, x="bf16", act="silu", bias=True,
             add=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A matrix width: any size half of the time, else a multiple of 64."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.5 else max(lo, n // 64 * 64)


def draw(rng):
    op = rng.choice(["rotary", "qknorm", "qknorm_bwd", "linear", "linear_bwd"])
    if op in ("rotary", "qknorm", "qknorm_bwd"):
        d = rng.choice([64, 128, 128, 80, 256])
        rot = rng.choice([d, d, d // 2, d // 4])
        common = dict(op=op, tokens=_log_int(rng, 1, 32768), d=d, rot=rot, interleaved=rng.random() < 0.5,
                      rule=rng.choice(["none", "linear", "yarn"]), base=rng.choice([1e4, 1e6]),
                      far=_log_int(rng, 4096, 1 << 20))
        if op == "rotary":
            return dict(common, heads=rng.choice([1, 2, 3, 8, 32]), inverse=rng.random() < 0.4,
                        x=rng.choice(["bf16", "fp16", "fp32"]), y=rng.choice(["bf16", "fp16", "fp32"]),
                        mapped=rng.random() < 0.5)
        hkv = rng.choice([1, 2, 8])
        common.update(hkv=hkv, hq=hkv * rng.choice([1, 2, 5]), x=rng.choice(["bf16", "fp16", "fp32"]),
                      packed=rng.random() < 0.5)
        if op == "qknorm":
            return dict(common, y=rng.choice(["bf16", "fp16", "fp32"]), mapped=rng.random() < 0.5)
        return dict(common, dy=rng.choice(["fp32", "bf16"]))
    m, n, k = _log_int(rng, 1, 16384), _width(rng, 8, 6144), _width(rng, 8, 4096)
    x = rng.choice(["bf16", "fp16"])
    act = rng.choice([None, None, "silu", "gelu", "gelu_tanh"])
    if op == "linear":
        return dict(op=op, m=m, n=n, k=k, x=x, y=x, bias=rng.random() < 0.5, act=act, residual=rng.random() < 0.5,
                    keep_z=act is not None and rng.random() < 0.5)
    return dict(op=op, m=m, n=n, k=k, x=x, act=act, bias=rng.random() < 0.5, add=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _frequencies(rot, rule, base):
    """(frequency of each pair, factor on the rotated values) for contexts stretched four times from 8192."""
    j = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * j / rot)
    if rule == "linear":
        return f / 4.0, 1.0
    if rule == "yarn":
        def index(turns):
            return rot * math.log(8192 / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), rot - 1)
        ramp = np.clip((j - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f * (1.0 - ramp) + f / 4.0 * ramp, 0.1 * math.log(4.0) + 1.0
    return f, 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype="fp32", scale=1.0):
        # drawn in the type itself: a 64K batch's fp32 copy would only be thrown away
        return torch.randn(*shape, device=dev, generator=g, dtype=_TYPES[dtype]).mul_(scale)

    s = dict(case=case, status=torch.zeros(1, dtype=torch.int32, device=dev))
    op = case["op"]
    if op in ("rotary", "qknorm", "qknorm_bwd"):
        t, d = case["tokens"], case["d"]
        f, s["scale"] = _frequencies(case["rot"], case["rule"], case["base"])
        s["freq"] = torch.from_numpy(f).to(dev)
        s["pos"] = torch.randint(0, case["far"], (t,), device=dev, generator=g, dtype=torch.int32)
        s["map"] = torch.randperm(t, device=dev, generator=g).int() if case.get("mapped") else None
    if op == "rotary":
        s["x"] = normal(t, case["heads"], d, dtype=case["x"])
    elif op in ("qknorm", "qknorm_bwd"):
        hq, hkv = case["hq"], case["hkv"]
        if case["packed"]:  # one projection's output: rows of q, k and v heads side by side
            qkv = normal(t, hq + 2 * hkv, d, dtype=case["x"], scale=2.0)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = (normal(t, h, d, dtype=case["x"], scale=2.0) for h in (hq, hkv, hkv))
        wt = "bf16" if case["x"] == "fp32" else case["x"]
        s["wq"], s["wk"] = (normal(d, dtype=wt, scale=0.2).add_(1.0) for _ in range(2))
        if op == "qknorm_bwd":
            s["dq"], s["dk"], s["dv"] = (normal(t, h, d, dtype=case["dy"], scale=1e-2) for h in (hq, hkv, hkv))
    else:
        m, n, k, x = case["m"], case["n"], case["k"], case["x"]
        s["x"], s["w"] = normal(m, k, dtype=x), normal(n, k, dtype=x, scale=k ** -0.5)
        if op == "linear":
            s["bias"] = normal(n, dtype=x, scale=0.1) if case["bias"] else None
            s["residual"] = normal(m, n, dtype=x) if case["residual"] else None
        else:
            s["dy"] = normal(m, n, dtype=x, scale=1e-2)
            s["z"] = normal(m, n, dtype=x) if case["act"] else None  # kept by the forward pass
            s["add"] = normal(m, k, dtype=x, scale=1e-2) if case["add"] else None
    return s


# ------------------------------------------------------------------ plain forms, in 32 bits
def _cos_sin(s):
    angle = s["pos"].double()[:, None] * s["freq"]
    return (torch.cos(angle) * s["scale"]).float()[:, None], (torch.sin(angle) * s["scale"]).float()[:, None]


def _rotate(x, s, inverse):
    c, sn = _cos_sin(s)
    sn = -sn if inverse else sn
    r = s["case"]["rot"]
    y = x.clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if s["case"]["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    y[..., a] = x[..., a] * c - x[..., b] * sn
    y[..., b] = x[..., b] * c + x[..., a] * sn
    return y


def _placed(y, s, dtype):
    y = y.to(_TYPES[dtype])
    if s["map"] is None:
        return y
    out = torch.empty_like(y)
    out[s["map"].long()] = y
    return out


def _normed(h):
    h = h.float()
    rs = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    return h * rs, rs


def _head_gradient(dy, h, w, s):
    """(dh, dw) of rotate(normed(h) * w)."""
    g = _rotate(dy.float(), s, True)
    xh, rs = _normed(h)
    dw = (g * xh).sum((0, 1))
    u = g * w.float()
    return (rs * (u - xh * (u * xh).mean(-1, keepdim=True))).to(h.dtype), dw


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "silu":
        sg = torch.sigmoid(z)
        return sg * (1.0 + z * (1.0 - sg))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rotary":
        return _placed(_rotate(s["x"].float(), s, case["inverse"]), s, case["y"])
    if op == "qknorm":
        q, k = (_rotate(_normed(h)[0] * w.float(), s, False) for h, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
        return {"q": _placed(q, s, case["y"]), "k": _placed(k, s, case["y"]),
                "v": _placed(s["v"].float(), s, case["y"])}
    if op == "qknorm_bwd":
        dq, dwq = _head_gradient(s["dq"], s["q"], s["wq"], s)
        dk, dwk = _head_gradient(s["dk"], s["k"], s["wk"], s)
        return {"dq": dq, "dk": dk, "dv": s["dv"].to(s["v"].dtype), "dwq": dwq, "dwk": dwk}
    x, w = s["x"].float(), s["w"].float()
    t = s["x"].dtype
    if op == "linear":
        z = x @ w.T
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(_TYPES[case["y"]]), "z": z.to(t)} if case["keep_z"] else {"y": y.to(_TYPES[case["y"]])}
    dz = s["dy"].float()
    if case["act"]:
        dz = dz * _act_slope(s["z"].float(), case["act"])
    dx = dz @ w
    if s["add"] is not None:
        dx = dx + s["add"].float()
    out = {"dx": dx.to(t), "dw": (dz.T @ x).to(t)}
    if case["bias"]:
        out["db"] = dz.sum(0)
    return out


# ------------------------------------------------------------------ the package's calls
def _calls(s):
    import block_sparse_masked_segment_b200 as opr

    case = s["case"]
    op = case["op"]
    if op == "rotary":
        out = torch.empty(s["x"].shape, dtype=_TYPES[case["y"]], device=s["x"].device)
        return opr.opr_rotary(s["x"], s["pos"], s["freq"], interleaved=case["interleaved"], scale=s["scale"],
                              inverse=case["inverse"], out=out, row_map=s["map"], dev_status=s["status"])
    if op == "qknorm":
        q, k, v = opr.opr_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], eps=EPS,
                                       interleaved=case["interleaved"], scale=s["scale"], v=s["v"],
                                       out_dtype=_TYPES[case["y"]], row_map=s["map"], dev_status=s["status"])
        return {"q": q, "k": k, "v": v}
    if op == "qknorm_bwd":
        dq, dk, dv, dwq, dwk = opr.opr_qk_norm_rope_bwd(
            s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], eps=EPS,
            interleaved=case["interleaved"], scale=s["scale"], dv=s["dv"], dev_status=s["status"])
        return {"dq": dq, "dk": dk, "dv": dv, "dwq": dwq, "dwk": dwk}
    if op == "linear":
        y = opr.opr_linear(s["x"], s["w"], s["bias"], activation=case["act"], residual=s["residual"],
                           out_dtype=_TYPES[case["y"]], save_z=case["keep_z"], dev_status=s["status"])
        return {"y": y[0], "z": y[1]} if case["keep_z"] else {"y": y}
    dx, dw, db = opr.opr_linear_bwd(s["dy"], s["x"], s["w"], z=s["z"], activation=case["act"], dx_residual=s["add"],
                                    bias=case["bias"], dev_status=s["status"])
    return {"dx": dx, "dw": dw, "db": db} if case["bias"] else {"dx": dx, "dw": dw}


def run(state):
    return _calls(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op == "rotary":
        n = case["tokens"] * case["heads"] * case["d"]
        return {"bytes": n * (_SIZE[case["x"]] + _SIZE[case["y"]]) + case["tokens"] * (8 if case["mapped"] else 4),
                "flops": 3.0 * n * case["rot"] / case["d"]}
    if op in ("qknorm", "qknorm_bwd"):
        t, d = case["tokens"], case["d"]
        heads = case["hq"] + case["hkv"]
        n, nv = t * heads * d, t * case["hkv"] * d
        if op == "qknorm":
            return {"bytes": (n + nv) * (_SIZE[case["x"]] + _SIZE[case["y"]]) + t * (8 if case["mapped"] else 4) + 4 * d,
                    "flops": 7.0 * n}
        return {"bytes": n * (2 * _SIZE[case["x"]] + _SIZE[case["dy"]]) + nv * (_SIZE[case["x"]] + _SIZE[case["dy"]])
                + 4 * t + 12 * d, "flops": 14.0 * n}
    m, n, k, e = case["m"], case["n"], case["k"], _SIZE[case["x"]]
    if op == "linear":
        return {"bytes": e * (m * k + n * k + (n if case["bias"] else 0) + (m * n if case["residual"] else 0)
                              + (m * n if case["keep_z"] else 0)) + _SIZE[case["y"]] * m * n,
                "flops": 2.0 * m * n * k}
    return {"bytes": e * (m * n * (2 if case["act"] else 1) + 2 * m * k + 2 * n * k + (m * k if case["add"] else 0))
            + (4 * n if case["bias"] else 0), "flops": 4.0 * m * n * k}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _turned(x, s, inverse):
    """The rotation as a product of complex numbers."""
    r = s["case"]["rot"]
    turn = torch.polar(torch.full_like(s["freq"], s["scale"]).expand(len(s["pos"]), -1),
                       torch.outer(s["pos"].double(), -s["freq"] if inverse else s["freq"]))[:, None]
    lead = x[..., :r]
    if s["case"]["interleaved"]:
        got = torch.view_as_real(torch.view_as_complex(lead.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
    else:
        got = torch.complex(*lead.chunk(2, -1)) * turn
        got = torch.cat((got.real, got.imag), -1)
    return torch.cat((got, x[..., r:]), -1)


def _in_order(y, s):
    return y if s["map"] is None else y[torch.argsort(s["map"].long())]


def _function(z, act):
    return {None: lambda: z, "silu": lambda: torch.nn.functional.silu(z), "gelu": lambda: torch.nn.functional.gelu(z),
            "gelu_tanh": lambda: torch.nn.functional.gelu(z, approximate="tanh")}[act]()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return _in_order(_turned(s["x"].double(), s, case["inverse"]), s)

    def head(h, w):
        return _turned(h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * w, s, False)

    if op == "qknorm":
        return {"q": _in_order(head(s["q"].double(), s["wq"].double()), s),
                "k": _in_order(head(s["k"].double(), s["wk"].double()), s), "v": _in_order(s["v"].double(), s)}
    if op == "qknorm_bwd":
        out = {}
        for name in ("q", "k"):  # some heads at a time: the graph of the largest case in 64 bits is big
            w = s["w" + name].double().requires_grad_()
            parts = []
            for heads, dy in zip(s[name].split(8, 1), s["d" + name].split(8, 1)):
                h = heads.double().requires_grad_()
                head(h, w).backward(dy.double())
                parts.append(h.grad)
            out["d" + name], out["dw" + name] = torch.cat(parts, 1), w.grad
        return {"dq": out["dq"], "dk": out["dk"], "dv": s["dv"].double(), "dwq": out["dwq"], "dwk": out["dwk"]}
    x, w = s["x"].double(), s["w"].double()
    if op == "linear":
        z = torch.nn.functional.linear(x, w, None if s["bias"] is None else s["bias"].double())
        y = _function(z, case["act"])
        y = y if s["residual"] is None else y + s["residual"].double()
        return {"y": y, "z": z} if case["keep_z"] else {"y": y}
    dz = s["dy"].double()
    if case["act"]:
        z = s["z"].double().requires_grad_()
        dz, = torch.autograd.grad(_function(z, case["act"]), z, dz)
    out = {"dx": torch.einsum("mn,nk->mk", dz, w), "dw": torch.einsum("mn,mk->nk", dz, x)}
    if s["add"] is not None:
        out["dx"] = out["dx"] + s["add"].double()
    if case["bias"]:
        out["db"] = dz.sum(0)
    return out
