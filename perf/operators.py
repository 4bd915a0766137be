"""Cases of the row operators (permute, unpermute and their gradients) and of the microscaled 4-bit operators (quantise
and back, grouped product): inputs, the plain torch form, the framework's calls, and the results in 64 bits.

A case's routing is drawn as the layer's inputs are: the k largest of E normal logits a token (with ln p_e added for a
Zipf share, ranks permuted over the experts when `shuffled`), softmax gates over them, a share `masked` of the slots
set to -1, and the rows of the first `local` experts placed in (expert, token, slot) order."""
import math

import numpy as np
import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
SLACK = 96  # rows a caller's row buffers hold past the expected ones


def listed():
    """The shapes are the repository's configurations and their pieces, and odd ones beside them."""
    return [
        # dispatch of one decoded token to eight experts: latency
        dict(name="permute one token", op="permute", type="bf16", tokens=1, hidden=7168, experts=8, local=8, k=8, zipf=0.0, shuffled=False, masked=0.0),
        # dispatch of one GPU's share: a pool of 16384 tokens, 8 of 64 experts local
        dict(name="permute share", op="permute", type="bf16", tokens=16384, hidden=7168, experts=64, local=8, k=8, zipf=0.0, shuffled=False, masked=0.0),
        # gradient of a dispatch where every expert is local: every token sums four rows
        dict(name="permute backward", op="permute_backward", type="fp16", tokens=4096, hidden=2048, experts=16, local=16, k=4, zipf=0.0, shuffled=False, masked=0.0),
        # combine of a decoding batch
        dict(name="unpermute decode", op="unpermute", type="bf16", tokens=64, hidden=7168, experts=64, local=64, k=8, zipf=0.0, shuffled=False, masked=0.0),
        # combine of a skewed share: this GPU holds the eight hottest experts, about five rows a token
        dict(name="unpermute skewed share", op="unpermute", type="bf16", tokens=16384, hidden=7168, experts=64, local=8, k=8, zipf=1.2, shuffled=False, masked=0.0),
        # gradient of the combine of a training step's share
        dict(name="unpermute backward share", op="unpermute_backward", type="bf16", tokens=16384, hidden=7168, experts=64, local=8, k=8, zipf=0.0, shuffled=False, masked=0.0),
        # the same in fp32 for a small odd model, with slots dropped by a capacity limit
        dict(name="unpermute backward ragged", op="unpermute_backward", type="fp32", tokens=2777, hidden=1000, experts=12, local=7, k=6, zipf=0.5, shuffled=True, masked=0.3),
        # a batch's activations on their way to a 4-bit product
        dict(name="quantise activations", op="quantise", type="fp16", rows=777, cols=2080, spread=1.0),
        # one weight of a share's eight experts, [8 * 2048, 7168], when a model is loaded
        dict(name="quantise weights", op="quantise", type="bf16", rows=16384, cols=7168, spread=0.02),
        # decoding: 64 rows over eight experts, bound by the weights
        dict(name="product decode", op="product", left="e4m3", type="bf16", rows=64, experts=8, n=4096, k=7168, skew=0.0),
        # the second product of a skewed share: experts from a few dozen rows to thousands
        dict(name="product skewed share", op="product", left="e4m3", type="bf16", rows=3777, experts=8, n=7168, k=2048, skew=1.2),
        # the first product (gate and up side by side) of an even share
        dict(name="product share", op="product", left="e2m1", type="bf16", rows=16384, experts=8, n=4096, k=7168, skew=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "permute_backward", "unpermute", "unpermute_backward", "quantise", "product", "product"])
    while True:
        if op == "quantise":
            c = dict(op=op, type=rng.choice(["bf16", "fp16", "fp32"]), rows=_log(rng, 1, 20000), cols=32 * _log(rng, 1, 256), spread=rng.choice([0.02, 1.0, 30.0]))
        elif op == "product":
            c = dict(op=op, left=rng.choice(["e4m3", "e2m1"]), type=rng.choice(["bf16", "bf16", "fp32"]), rows=_log(rng, 1, 16384), experts=rng.choice([1, 2, 4, 8, 8, 13, 16, 32]), n=8 * _log(rng, 8, 1024), k=32 * _log(rng, 2, 256), skew=rng.choice([0.0, 0.6, 1.2]))
        else:
            experts = rng.choice([4, 8, 12, 16, 32, 64])
            c = dict(op=op, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), tokens=_log(rng, 1, 16384), hidden=8 * _log(rng, 8, 1024), experts=experts, local=rng.randint(1, experts), k=rng.randint(1, min(8, experts)), zipf=rng.choice([0.0, 0.0, 0.8]), shuffled=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.2]))
        w = work(c)
        if w["bytes"] < 1.0e9 and w["flops"] < 0.9e12 and c.get("experts", 1) * c.get("n", 1) * c.get("k", 1) < 0.3e9:
            return c


# ------------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------------
def _bias(c):
    """Added to every token's logits: the Zipf popularity of each expert."""
    e = c["experts"]
    p = (np.arange(e) + 1.0) ** (-c["zipf"])
    b = np.log(p / p.sum()) if c["zipf"] > 0 else np.zeros(e)
    return b[np.random.default_rng(1004).permutation(e)] if c["shuffled"] else b


def _share(c):
    """Routed rows per token, from a sample of tokens."""
    rng = np.random.default_rng(7)
    ids = np.argsort(-(rng.standard_normal((2048, c["experts"])) + _bias(c)), axis=1)[:, : c["k"]]
    return float((ids < c["local"]).sum(1).mean()) * (1.0 - c["masked"])


def _capacity(c):
    """Rows of the caller's row buffers: some past the expected ones, at most every pair's.  Pairs past them are dropped."""
    rows = c["tokens"] * _share(c)
    return min(c["tokens"] * c["k"], int(1.05 * rows + 6 * math.sqrt(rows))) + SLACK


def _weights_read(c):
    """Experts that have rows, in expectation."""
    p = (np.arange(c["experts"]) + 1.0) ** (-c["skew"])
    p /= p.sum()
    return float((1.0 - (1.0 - p) ** c["rows"]).sum())


def _pack4(v):
    """e2m1 codes of values on the grid, two a byte, the even element in the low half."""
    a = v.abs()
    i = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    i = i | (torch.signbit(v).to(torch.uint8) << 3)
    return (i[..., 0::2] | (i[..., 1::2] << 4)).contiguous()


def _blocks(x):
    return x.reshape(*x.shape[:-1], -1, 32)


def _exponent(b, emax, top):
    """The shared exponent of each block of 32: the smallest n with amax 2^-n <= top 2^emax; top in (1, 2)."""
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    n = e - 1 - emax + (2 * m > top)
    return torch.where(m == 0, -127, n).clamp(-127, 127)


def _e2m1(v):
    """To the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 in magnitude, ties to the even code."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(v / step) * step


def _quantise(x, fmt):
    """Codes and scales of float32 rows: what a user's program has of its operands before a product."""
    b = _blocks(x)
    n = _exponent(b, 2, 1.5) if fmt == "e2m1" else _exponent(b, 8, 1.75)
    v = torch.ldexp(b, -n)
    scales = (n + 127).squeeze(-1).to(torch.uint8).contiguous()
    codes = _pack4(_e2m1(v).reshape(x.shape)) if fmt == "e2m1" else v.reshape(x.shape).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scales


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case)
    if case["op"] == "quantise":
        r, c = case["rows"], case["cols"]
        s["src"] = (normal(r, c) * case["spread"]).to(DTYPE[case["type"]])
        s["codes"] = torch.zeros(r, c // 2, dtype=torch.uint8, device=dev)
        s["scales"] = torch.zeros(r, c // 32, dtype=torch.uint8, device=dev)
        s["out"] = torch.zeros_like(s["src"])
    elif case["op"] == "product":
        r, e, n, k = (case[x] for x in ("rows", "experts", "n", "k"))
        p = (torch.arange(e, device=dev, dtype=torch.float32) + 1) ** (-case["skew"])
        at = torch.multinomial(p, r, replacement=True, generator=g)
        counts = torch.bincount(at, minlength=e)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())
        s["a"], s["a_scales"] = _quantise(normal(r + SLACK, k), case["left"])
        w = [_quantise(normal(n, k) * 0.02, "e2m1") for _ in range(e)]
        s["b"], s["b_scales"] = (torch.stack([x[i] for x in w]) for i in (0, 1))
        s["out"] = torch.zeros(r + SLACK, n, dtype=DTYPE[case["type"]], device=dev)
    else:
        t, d, e, k = (case[x] for x in ("tokens", "hidden", "experts", "k"))
        dt = DTYPE[case["type"]]
        logits = normal(t, e) + torch.tensor(_bias(case), dtype=torch.float32, device=dev)
        top, ids = torch.topk(logits, k, dim=1)
        s["gates"] = torch.softmax(top, 1)
        ids = torch.where((ids < case["local"]) & (torch.rand(t, k, generator=g, device=dev) >= case["masked"]), ids, e).reshape(-1)
        order = torch.argsort(ids, stable=True)
        cap = _capacity(case)
        routed = min(int((ids < e).sum()), cap)
        pos = torch.full((t * k,), -1, dtype=torch.int32, device=dev)
        pos[order[:routed]] = torch.arange(routed, dtype=torch.int32, device=dev)
        s["pos"] = pos.reshape(t, k)
        if case["op"].startswith("permute"):
            s["x" if case["op"] == "permute" else "d_rows"] = normal(t if case["op"] == "permute" else cap, d).to(dt)
        else:
            s["rows"] = normal(cap, d).to(dt)
            if case["op"] == "unpermute_backward":
                s["dy"] = normal(t, d).to(dt)
                s["d_gates"] = torch.zeros(t, k, device=dev)
        # the caller's outputs: rows past the last routed one stay as they are
        s["out"] = torch.zeros(cap if case["op"] in ("permute", "unpermute_backward") else t, d, dtype=dt, device=dev)
    return s


# ------------------------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------------------------
def _placed(s, rows):
    """For each of `rows` rows the pair that goes there, and whether one does."""
    pos = s["pos"].reshape(-1).long()
    pair = torch.full((rows + 1,), -1, dtype=torch.long, device=pos.device)
    pair[torch.where(pos >= 0, pos, rows)] = torch.arange(pos.numel(), device=pos.device)
    return pair[:rows].clamp(min=0), (pair[:rows] >= 0).unsqueeze(1)


def _gathered(s, rows):
    """Every pair's row in float32, zeros for pairs without one: [T, k, D]."""
    pos = s["pos"].long()
    return torch.where(pos.unsqueeze(2) >= 0, rows[pos.clamp(min=0)].float(), 0.0)


def _values(codes, scales, fmt):
    """Float32 values of codes and scales."""
    if fmt == "e4m3":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
        v = grid[torch.stack([codes & 15, codes >> 4], -1).int()].reshape(*codes.shape[:-1], -1)
    return torch.ldexp(_blocks(v), scales.unsqueeze(-1).int() - 127).reshape(v.shape)


def _plain(s):
    op, out = s["op"], s["out"]
    if op == "permute":
        pair, there = _placed(s, out.shape[0])
        return torch.where(there, s["x"][pair // s["k"]], out)
    if op == "permute_backward":
        return _gathered(s, s["d_rows"]).sum(1).to(out.dtype)
    if op == "unpermute":
        return (_gathered(s, s["rows"]) * s["gates"].unsqueeze(2)).sum(1).to(out.dtype)
    if op == "unpermute_backward":
        pair, there = _placed(s, out.shape[0])
        d_rows = s["dy"][pair // s["k"]].float() * s["gates"].reshape(-1)[pair].unsqueeze(1)
        return torch.where(there, d_rows.to(out.dtype), out), (_gathered(s, s["rows"]) * s["dy"].float().unsqueeze(1)).sum(2)
    if op == "quantise":
        b = _blocks(s["src"].float())
        n = _exponent(b, 2, 1.5)
        return torch.ldexp(_e2m1(torch.ldexp(b, -n)), n).reshape(out.shape).to(out.dtype)
    # product: every expert's rows padded to the longest, one batched product
    a, b, off = _values(s["a"], s["a_scales"], s["left"]), _values(s["b"], s["b_scales"], "e2m1"), s["offsets"].long()
    at = off[:-1].unsqueeze(1) + torch.arange(s["most"], device=a.device)
    c = torch.bmm(a[at.clamp(max=a.shape[0] - 1)], b.transpose(1, 2).contiguous()).reshape(-1, b.shape[1])
    r = torch.arange(out.shape[0], device=a.device)
    e = (torch.searchsorted(off, r, right=True) - 1).clamp(0, b.shape[0] - 1)
    i = (e * s["most"] + r - off[e]).clamp(0, c.shape[0] - 1)
    return torch.where((r < off[-1]).unsqueeze(1), c[i].to(out.dtype), out)


def run(state):
    s = state
    if not own:
        return _plain(s)
    from mixture_experts_layer_mok_amd import ops

    op = s["op"]
    if op == "permute":
        return ops.permute(s["x"], s["pos"], s["out"])
    if op == "permute_backward":
        return ops.permute_backward(s["d_rows"], s["pos"], out=s["out"])
    if op == "unpermute":
        return ops.unpermute(s["rows"], s["pos"], s["gates"], out=s["out"])
    if op == "unpermute_backward":
        return ops.unpermute_backward(s["dy"], s["rows"], s["pos"], s["gates"], s["out"], d_weights=s["d_gates"])
    if op == "quantise":
        ops.quantize_mx4(s["src"], codes=s["codes"], scales=s["scales"])
        return ops.dequantize_mx4(s["codes"], s["scales"], out=s["out"])
    return ops.grouped_mx4(s["a"], s["a_scales"], s["offsets"], s["b"], s["b_scales"], out=s["out"])


def work(case):
    if case["op"] == "quantise":
        v = case["rows"] * case["cols"]
        return {"bytes": 2.0 * v * SIZE[case["type"]], "flops": 4.0 * v}
    if case["op"] == "product":
        r, n, k = case["rows"], case["n"], case["k"]
        a = k * (1.0 if case["left"] == "e4m3" else 0.5) + k / 32
        return {"bytes": r * a + _weights_read(case) * n * (k / 2 + k / 32) + r * n * SIZE[case["type"]], "flops": 2.0 * r * n * k}
    t, d, b = case["tokens"], case["hidden"], SIZE[case["type"]]
    rows = t * _share(case)
    moved = {"permute": 1, "permute_backward": 1, "unpermute": 1, "unpermute_backward": 2}[case["op"]] * rows * d * b + t * d * b
    flops = {"permute": 0, "permute_backward": 1, "unpermute": 2, "unpermute_backward": 3}[case["op"]] * rows * d
    return {"bytes": moved + 4.0 * t * case["k"] * (1 if case["op"].startswith("permute") else 2), "flops": float(flops)}


# ------------------------------------------------------------------------------------------------------------------
# 64 bits
# ------------------------------------------------------------------------------------------------------------------
def _decode64(codes, scales, fmt):
    """Values of codes from their bits: sign, exponent and mantissa fields, times 2 ** (scale - 127)."""
    if fmt == "e4m3":
        ebits, mbits, bias, c = 4, 3, 7, codes.to(torch.int64)
    else:
        ebits, mbits, bias = 2, 1, 1
        c = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.int64, device=codes.device)
        c[..., 0::2], c[..., 1::2] = codes % 16, codes // 16
    sign = 1.0 - 2.0 * (c >> (ebits + mbits) & 1).double()
    ef, m = c >> mbits & (2**ebits - 1), (c & (2**mbits - 1)).double() / 2**mbits
    mag = torch.where(ef == 0, m * 2.0 ** (1 - bias), (1 + m) * torch.exp2((ef - bias).double()))
    return sign * mag * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        out = []
        for x in s["src"].split(2048):
            v = x.double().unflatten(1, (-1, 32))
            amax = v.abs().amax(2, keepdim=True)
            # the scale by comparison with the powers of two around the largest magnitude
            p = torch.exp2(torch.floor(torch.log2(amax.clamp(min=1e-300))) - 3)
            p = torch.where(amax > 6 * p, 2 * p, p)
            p = torch.where(amax > 6 * p, 2 * p, p)
            p = torch.where(amax > 6 * p, 2 * p, p).clamp(min=2.0**-127)
            u = v.abs() / p
            mid = ((0.25, 0.0, 0.5), (0.75, 0.5, 1.0), (1.25, 1.0, 1.5), (1.75, 1.5, 2.0), (2.5, 2.0, 3.0), (3.5, 3.0, 4.0), (5.0, 4.0, 6.0))
            q = torch.zeros_like(u)
            for i, (m, lo, hi) in enumerate(mid):  # a tie goes to the neighbour whose code is even
                q = torch.where((u > m) | ((u == m) & (i % 2 == 1)), hi, q)
            out.append((torch.sign(v) * q * p).flatten(1))
        return torch.cat(out)
    if op == "product":
        off = s["offsets"].tolist()
        out = s["out"].double()
        for e in range(case["experts"]):
            i, j = off[e], off[e + 1]
            if j > i:
                w = _decode64(s["b"][e], s["b_scales"][e], "e2m1")
                out[i:j] = _decode64(s["a"][i:j], s["a_scales"][i:j], case["left"]) @ w.t().contiguous()
        return out
    pos, k = s["pos"].long(), case["k"]
    if op == "permute":
        out = s["out"].double()
        for j in range(k):
            at = pos[:, j] >= 0
            out[pos[at, j]] = s["x"][at].double()
        return out
    if op in ("permute_backward", "unpermute"):
        rows = s["d_rows" if op == "permute_backward" else "rows"]
        out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device=rows.device)
        for j in range(k):
            at = pos[:, j] >= 0
            out[at] += rows[pos[at, j]].double() * (1.0 if op == "permute_backward" else s["gates"][at, j].double().unsqueeze(1))
        return out
    d_rows, d_gates = s["out"].double(), torch.zeros(case["tokens"], k, dtype=torch.float64, device=pos.device)
    for j in range(k):
        at = pos[:, j] >= 0
        dy = s["dy"][at].double()
        d_rows[pos[at, j]] = dy * s["gates"][at, j].double().unsqueeze(1)
        d_gates[at, j] = (dy * s["rows"][pos[at, j]].double()).sum(1)
    return d_rows, d_gates
