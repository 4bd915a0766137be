"""Cases of the grouped product of 16-bit rows (forward, gradient of the rows, gradient of the weights) and of
activations held in 8 bits for the backward pass (quantise and back, SwiGLU that keeps its inputs so, the weights'
gradient from rows held so): inputs, the plain torch form, the framework's calls, and the results in 64 bits.

Rows are in expert order, rows [offsets[e], offsets[e + 1]) expert e's, in a caller's buffer with some rows more; a
product's expert counts are drawn from a Zipf law of exponent `skew`.  8 bits are MXFP8: e4m3 codes in blocks of 32 along
a row, and one power of two a block."""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
SLACK = 96  # rows a caller's row buffers hold past the routed ones


def listed():
    """The shapes are the repository's configurations and their pieces, and odd ones beside them."""
    return [
        # decoding: the first product of 64 routed rows over eight experts, bound by the weights
        dict(name="product decode", op="product", type="bf16", rows=64, experts=8, n=4096, k=7168, skew=0.0),
        # a small odd model, one token's rows: latency
        dict(name="product few rows", op="product", type="fp16", rows=4, experts=12, n=1000, k=520, skew=0.0),
        # the second product of a skewed share: experts from a few dozen rows to thousands
        dict(name="product skewed share", op="product", type="fp16", rows=3777, experts=8, n=7168, k=2048, skew=1.2),
        # the first product (gate and up side by side) of a training step's even share
        dict(name="product share", op="product", type="bf16", rows=16384, experts=8, n=4096, k=7168, skew=0.0),
        # gradient of that share's routed rows
        dict(name="rows gradient share", op="rows", type="bf16", rows=16384, experts=8, n=4096, k=7168, skew=0.0),
        # the same for a small odd model with many experts
        dict(name="rows gradient ragged", op="rows", type="fp16", rows=2777, experts=33, n=1000, k=1048, skew=0.6),
        # gradient of the share's first weights, float32 as the layer's own
        dict(name="weights gradient share", op="weights", held=16, type="bf16", into="fp32", rows=16384, experts=8, n=4096, k=7168, skew=0.0),
        # gradient of the second weights of a skewed share, from activations held in 8 bits
        dict(name="weights gradient from 8 bits", op="weights", held=8, type="bf16", into="bf16", rows=16384, experts=8, n=7168, k=2048, skew=0.8),
        # a batch's activations put away in 8 bits and read back
        dict(name="hold and read activations", op="hold", type="fp16", rows=777, cols=2080, spread=1.0),
        # a share's routed rows put away and read back
        dict(name="hold and read share", op="hold", type="bf16", rows=16384, cols=7168, spread=1.0),
        # activation of a share, forward and backward, its inputs held in 8 bits between
        dict(name="swiglu step share", op="step", type="bf16", rows=16384, inner=2048, spread=1.0),
        # activation's backward pass of a small odd model: its gradients and the activation again
        dict(name="swiglu backward ragged", op="backward", type="fp32", rows=2777, inner=1056, spread=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "rows", "weights", "weights", "hold", "step", "backward"])
    while True:
        if op == "hold":
            c = dict(op=op, type=rng.choice(["bf16", "fp16", "fp32"]), rows=_log(rng, 1, 20000), cols=32 * _log(rng, 1, 256), spread=rng.choice([0.02, 1.0, 30.0]))
        elif op in ("step", "backward"):
            c = dict(op=op, type=rng.choice(["bf16", "fp16", "fp32"]), rows=_log(rng, 1, 20000), inner=32 * _log(rng, 1, 128), spread=rng.choice([0.1, 1.0, 4.0]))
        else:
            c = dict(op=op, type=rng.choice(["bf16", "fp16"]), rows=_log(rng, 1, 16384), experts=rng.choice([1, 2, 4, 8, 8, 13, 16, 32]), n=8 * _log(rng, 8, 1024), k=8 * _log(rng, 8, 1024), skew=rng.choice([0.0, 0.6, 1.2]))
            if op == "weights":
                c["held"] = rng.choice([8, 16])
                c["into"] = rng.choice(["fp32", c["type"]])
                if c["held"] == 8:
                    c["k"] = 32 * ((c["k"] + 31) // 32)
        w = work(c)
        if w["bytes"] < 1.0e9 and w["flops"] < 0.9e12 and c.get("experts", 1) * c.get("n", 1) * c.get("k", 1) < 0.23e9:
            return c


# ------------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------------
def _experts_with_rows(c):
    """Experts that have rows, in expectation."""
    p = [(e + 1.0) ** (-c["skew"]) for e in range(c["experts"])]
    return sum(1.0 - (1.0 - x / sum(p)) ** c["rows"] for x in p)


def _blocks(x):
    return x.reshape(*x.shape[:-1], -1, 32)


def _hold(x):
    """Codes and exponents of float32 rows: the smallest n with amax 2^-n <= 448, codes to the nearest, ties to even."""
    b = _blocks(x)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    n = e - 9 + (2 * m > 1.75)
    n = torch.where(m == 0, -127, n).clamp(-127, 127)
    return torch.ldexp(b, -n).to(torch.float8_e4m3fn), n


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def empty(*shape, dtype):
        return torch.zeros(*shape, dtype=dtype, device=dev)

    def held(x):
        codes, n = _hold(x)
        return codes.view(torch.uint8).reshape(x.shape), (n + 127).to(torch.uint8).reshape(x.shape[0], -1)

    s = dict(case)
    dt = DTYPE[case["type"]]
    op = case["op"]
    if op == "hold":
        r, c = case["rows"], case["cols"]
        s["src"] = (normal(r, c) * case["spread"]).to(dt)
        s["codes"], s["scales"] = empty(r, c, dtype=torch.uint8), empty(r, c // 32, dtype=torch.uint8)
        s["out"] = torch.zeros_like(s["src"])
        return s
    if op in ("step", "backward"):
        # the rows of a caller's buffer that are routed; their number is on the device
        r, i = case["rows"], case["inner"]
        s["offsets"] = torch.tensor([0, r // 2, r], dtype=torch.int32, device=dev)
        ab = (normal(r + SLACK, 2 * i) * case["spread"]).to(dt)
        s["dh"] = normal(r + SLACK, i).to(dt)
        s["h"], s["d_ab"] = empty(r + SLACK, i, dtype=dt), empty(r + SLACK, 2 * i, dtype=dt)
        if op == "backward":
            s["codes"], s["scales"] = held(ab.float())
        else:
            s["ab"], s["h_again"] = ab, torch.zeros_like(s["h"])
            s["codes"], s["scales"] = empty(r + SLACK, 2 * i, dtype=torch.uint8), empty(r + SLACK, i // 16, dtype=torch.uint8)
        return s
    r, e, n, k = (case[x] for x in ("rows", "experts", "n", "k"))
    p = (torch.arange(e, device=dev, dtype=torch.float32) + 1) ** (-case["skew"])
    counts = torch.bincount(torch.multinomial(p, r, replacement=True, generator=g), minlength=e)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["bounds"] = s["offsets"].tolist()  # the plain form's plan
    if op != "rows":
        a = normal(r + SLACK, k)
        if case.get("held") == 8:
            s["a"], s["a_scales"] = held(a)
        else:
            s["a"] = a.to(dt)
    if op != "product":
        s["d_out"] = normal(r + SLACK, n).to(dt)
    if op != "weights":
        s["b"] = torch.stack([(normal(n, k) * 0.02).to(dt) for _ in range(e)])
    s["out"] = empty(e, n, k, dtype=DTYPE[case["into"]]) if op == "weights" else empty(r + SLACK, n if op == "product" else k, dtype=dt)
    return s


# ------------------------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------------------------
def _values(codes, scales):
    """Float32 values of codes and scales."""
    v = codes.view(torch.float8_e4m3fn).float()
    return torch.ldexp(_blocks(v), scales.unsqueeze(-1).int() - 127).reshape(v.shape)


def _there(s, new, old):
    """`new` in the routed rows, the others as they were."""
    at = torch.arange(old.shape[0], device=old.device) < s["offsets"][-1]
    return torch.where(at.unsqueeze(1), new.to(old.dtype), old)


def _swiglu(x):
    a, b = x.chunk(2, dim=1)
    return a * torch.sigmoid(a) * b


def _swiglu_backward(x, dh):
    a, b = x.chunk(2, dim=1)
    s = torch.sigmoid(a)
    return torch.cat([dh * b * s * (1 + a * (1 - s)), dh * a * s], 1)


def _plain(s):
    op = s["op"]
    if op == "hold":
        codes, n = _hold(s["src"].float())
        return torch.ldexp(codes.float(), n).reshape(s["out"].shape).to(s["out"].dtype)
    if op in ("step", "backward"):
        if op == "step":
            x = s["ab"].float()
            codes, n = _hold(x)
            back = torch.ldexp(codes.float(), n).reshape(x.shape)
        else:
            back = _values(s["codes"], s["scales"])
        d_ab = _there(s, _swiglu_backward(back, s["dh"].float()), s["d_ab"])
        again = _there(s, _swiglu(back), s["h"])
        return (_there(s, _swiglu(x), s["h"]), d_ab, again) if op == "step" else (d_ab, again)
    at = s["bounds"]
    if op == "weights":
        a = _values(s["a"], s["a_scales"]) if s["held"] == 8 else s["a"].float()
        return torch.stack([(s["d_out"][i:j].float().t() @ a[i:j]).to(s["out"].dtype) for i, j in zip(at, at[1:])])
    out = s["out"].clone()
    for e, (i, j) in enumerate(zip(at, at[1:])):
        if j > i:
            w = s["b"][e].float()
            out[i:j] = (s["a"][i:j].float() @ w.t() if op == "product" else s["d_out"][i:j].float() @ w).to(out.dtype)
    return out


def run(state):
    s = state
    if not own:
        return _plain(s)
    from mixture_experts_layer_mok_amd import ops

    op = s["op"]
    if op == "product":
        return ops.grouped_mm(s["a"], s["offsets"], s["b"], out=s["out"])
    if op == "rows":
        return ops.grouped_mm_backward_rows(s["d_out"], s["offsets"], s["b"], out=s["out"])
    if op == "weights":
        return ops.grouped_mm_backward_weights(s["d_out"], s["a"], s["offsets"], a_scales=s.get("a_scales"), out=s["out"])
    if op == "hold":
        ops.quantize_mx8(s["src"], codes=s["codes"], scales=s["scales"])
        return ops.dequantize_mx8(s["codes"], s["scales"], out=s["out"])
    if op == "step":
        ops.swiglu_mx8(s["ab"], offsets=s["offsets"], h=s["h"], codes=s["codes"], scales=s["scales"])
        ops.swiglu_mx8_backward(s["dh"], s["codes"], s["scales"], offsets=s["offsets"], d_ab=s["d_ab"], h=s["h_again"])
        return s["h"], s["d_ab"], s["h_again"]
    return ops.swiglu_mx8_backward(s["dh"], s["codes"], s["scales"], offsets=s["offsets"], d_ab=s["d_ab"], h=s["h"])


def work(case):
    op, b = case["op"], SIZE[case["type"]]
    if op == "hold":
        v = case["rows"] * case["cols"]
        return {"bytes": 2.0 * v * b, "flops": 4.0 * v}
    if op in ("step", "backward"):
        v = float(case["rows"] * case["inner"])
        held = 2 * (1 + 1 / 32)  # both inputs of an element
        if op == "step":  # the inputs and dh in, both activations and the gradients out, what is held written and read
            return {"bytes": v * (2 * b + b + 2 * b + 2 * b + 2 * held), "flops": 40.0 * v}
        return {"bytes": v * (held + b + 2 * b + b), "flops": 25.0 * v}
    r, n, k = case["rows"], case["n"], case["k"]
    flops = 2.0 * r * n * k
    if op == "weights":
        a = k * (33 / 32 if case["held"] == 8 else b)
        return {"bytes": r * a + r * n * b + case["experts"] * n * k * float(SIZE[case["into"]]), "flops": flops}
    return {"bytes": r * k * b + _experts_with_rows(case) * n * k * b + r * n * b, "flops": flops}


# ------------------------------------------------------------------------------------------------------------------
# 64 bits
# ------------------------------------------------------------------------------------------------------------------
def _held64(x):
    """The values that 8 bits hold of double rows."""
    v = x.unflatten(1, (-1, 32))
    amax = v.abs().amax(2, keepdim=True)
    # the scale by comparison with the powers of two around the largest magnitude
    p = torch.exp2(torch.floor(torch.log2(amax.clamp(min=1e-300))) - 9)
    for _ in range(3):
        p = torch.where(amax > 448 * p, 2 * p, p)
    p = p.clamp(min=2.0**-127)
    u = v.abs() / p
    # e4m3: steps of an eighth of the power of two below, 2^-9 from 2^-6 down
    step = torch.exp2(torch.floor(torch.log2(u.clamp(min=2.0**-6)))) / 8
    return (torch.sign(v) * torch.round(u / step) * step * p).flatten(1)


def _decode64(codes, scales):
    """Values of codes from their bits: sign, exponent and mantissa fields, times 2 ** (scale - 127)."""
    c = codes.to(torch.int64)
    ef, m = c >> 3 & 15, (c & 7).double() / 8
    mag = torch.where(ef == 0, m * 2.0**-6, (1 + m) * torch.exp2((ef - 7).double()))
    return torch.where(c >= 128, -mag, mag) * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "hold":
        return torch.cat([_held64(x.double()) for x in s["src"].split(2048)])
    if op in ("step", "backward"):
        r, i = case["rows"], case["inner"]
        h, d_ab, again = s["h"].double(), s["d_ab"].double(), s["h"].double()
        for lo in range(0, r, 2048):
            at = slice(lo, min(lo + 2048, r))
            back = _held64(s["ab"][at].double()) if op == "step" else _decode64(s["codes"][at], s["scales"][at])
            a, b, dh = back[:, :i], back[:, i:], s["dh"][at].double()
            sig = 1 / (1 + torch.exp(-a))
            again[at] = a * sig * b
            d_ab[at, :i] = dh * b * (sig + a * sig * torch.exp(-a) * sig)
            d_ab[at, i:] = dh * a * sig
            if op == "step":
                x = s["ab"][at].double()
                h[at] = x[:, :i] / (1 + torch.exp(-x[:, :i])) * x[:, i:]
        return (h, d_ab, again) if op == "step" else (d_ab, again)
    off = s["offsets"].tolist()
    out = s["out"].double()
    for e in range(case["experts"]):
        at = slice(off[e], off[e + 1])
        if off[e + 1] == off[e]:
            continue
        if op == "weights":
            a = _decode64(s["a"][at], s["a_scales"][at]) if case["held"] == 8 else s["a"][at].double()
            out[e] = torch.matmul(s["d_out"][at].double().t().contiguous(), a)
        elif op == "product":
            out[at] = torch.matmul(s["a"][at].double(), s["b"][e].double().t().contiguous())
        else:
            out[at] = torch.matmul(s["d_out"][at].double(), s["b"][e].double())
    return out
