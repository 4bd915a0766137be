"""A run of the operators as they are used: one layer's experts between the schedule's permute and
unpermute, in 16 bits, trained, with the activations between the passes held in 8 bits; forward and
every gradient against float64 of the same formulas on the same held values."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import ops
from mixture_experts_layer_mok_amd.layer import MoKLayer
from oracle import operators as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def f64(t):
    return t.detach().cpu().double().numpy()


def make(T=150, D=160, I=96, E=6, k=2, seed=0):
    g = torch.Generator().manual_seed(seed)

    def rnd(*s, scale=1.0):
        return (torch.randn(*s, generator=g) * scale).to(DEV, BF)

    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    ids[::11, 0] = -1  # masked slots
    ids[ids == E - 1] = 0  # an expert without rows (and pairs of one expert twice are not drawn)
    ids[:, 1][ids[:, 0] == ids[:, 1]] = -1
    w = torch.softmax(torch.randn(T, k, generator=g), 1).to(DEV)
    layer = MoKLayer(L.make_desc(T, 192, 64, E, k, M=64, S=2, comm_cus=8))
    layer.schedule(ids.to(DEV))
    return dict(layer=layer, ids=ids.numpy(), x=rnd(T, D), w=w, dy=rnd(T, D), w1=rnd(E, 2 * I, D, scale=0.1),
                w2=rnd(E, D, I, scale=0.1), max_rows=T * k)


def step(s):
    """Forward and backward; every tensor of the step by name."""
    layer, n = s["layer"], s["max_rows"]
    t = {}
    t["rows"] = layer.permute(s["x"], torch.zeros(n, s["x"].shape[1], dtype=BF, device=DEV))
    t["held"], t["held_s"] = ops.quantize_mx8(t["rows"])
    t["ab"] = layer.grouped_mm(t["rows"], s["w1"])
    t["h"], t["c"], t["cs"] = layer.swiglu_mx8(t["ab"])
    t["yr"] = layer.grouped_mm(t["h"], s["w2"])
    t["y"] = layer.unpermute(t["yr"], s["w"])
    t["dyr"], t["dw"] = layer.unpermute_backward(s["dy"], t["yr"], s["w"], torch.zeros_like(t["yr"]))
    t["dh"] = layer.grouped_mm_backward_rows(t["dyr"], s["w2"])
    t["dab"], t["h2"] = layer.swiglu_mx8_backward(t["dh"], t["c"], t["cs"])
    t["dw2"] = layer.grouped_mm_backward_weights(t["dyr"], t["h2"])
    t["dw1"] = layer.grouped_mm_backward_weights(t["dab"], t["held"], a_scales=t["held_s"])
    t["drows"] = layer.grouped_mm_backward_rows(t["dab"], s["w1"])
    t["dx"] = layer.permute_backward(t["drows"])
    return t


def close(got, want, mag, terms, what):
    """fp32 sums of `terms` terms and one rounding to got's type; the inputs are got's own."""
    eps = torch.finfo(got.dtype).eps / 2
    tol = terms * 2.0**-23 * mag
    tol = tol + eps * (np.abs(want) + tol) + 1e-37
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), (what, float((err / tol).max()))


def test_a_step_of_an_expert_function():
    s = make()
    t = step(s)
    tab = s["layer"].tables()
    off, R = tab["offsets"], tab["R"]
    assert R < s["max_rows"] and (np.diff(off) == 0).any()
    v = {n: f64(x) for n, x in t.items() if x.is_floating_point()}
    w1, w2 = f64(s["w1"]), f64(s["w2"])
    zero = lambda n: np.zeros((s["max_rows"], n))  # noqa: E731
    D, I = w2.shape[1], w2.shape[2]
    live = slice(0, R)
    # every operator on what it was given
    for what, got, (want, mag), terms in (
            ("ab", t["ab"], O.grouped_mm(v["rows"], off, w1, zero(2 * I)), D),
            ("yr", t["yr"], O.grouped_mm(v["h"], off, w2, zero(D)), I),
            ("dh", t["dh"], O.grouped_mm_backward_rows(v["dyr"], off, w2, zero(I)), D),
            ("drows", t["drows"], O.grouped_mm_backward_rows(v["dab"], off, w1, zero(D)), 2 * I)):
        close(got[live], want[live], mag[live], terms, what)
    held = O.values_mx8(t["held"].cpu().numpy(), t["held_s"].cpu().numpy())
    assert np.array_equal(*(a[live] for a in (O.quantize_mx8(v["rows"])[0], t["held"].cpu().numpy())))
    most = int(np.diff(off).max())
    close(t["dw2"], *O.grouped_mm_backward_weights(v["dyr"], v["h2"], off), most, "dw2")
    close(t["dw1"], *O.grouped_mm_backward_weights(v["dab"], held, off), most, "dw1")
    ab8 = O.values_mx8(t["c"].cpu().numpy(), t["cs"].cpu().numpy())[live]
    for what, got, ab in (("h", t["h"], v["ab"][live]), ("h2", t["h2"], ab8)):
        close(got[live], O.swiglu(ab), np.abs(O.swiglu(ab)) * 8, 1, what)
    want, terms = O.swiglu_backward(ab8, v["dh"][live])
    close(t["dab"][live], want, terms * 8, 1, "dab")


def test_the_step_against_autograd():
    """The whole step in float64 by autograd: what is left is bf16's rounding of each tensor between
    the operators (2^-8 of its size, six of them one after the other) and e4m3's of what is held (2^-4
    of its size in two of the gradients' factors, independent from element to element)."""
    s = make(seed=1)
    t = step(s)
    tab = s["layer"].tables()
    off, perm = tab["offsets"], torch.from_numpy(tab["perm"].astype(np.int64))
    k = s["ids"].shape[1]
    leaf = {n: torch.tensor(f64(s[n]), requires_grad=True) for n in ("x", "w", "w1", "w2")}
    rows = leaf["x"][perm // k]
    y = torch.zeros_like(leaf["x"])
    for e in range(len(off) - 1):
        at = slice(int(off[e]), int(off[e + 1]))
        a, b = (rows[at] @ leaf["w1"][e].t()).chunk(2, 1)
        out = (torch.nn.functional.silu(a) * b) @ leaf["w2"][e].t()
        y = y.index_add(0, perm[at] // k, out * leaf["w"].reshape(-1)[perm[at]].unsqueeze(1))
    (y * torch.tensor(f64(s["dy"]))).sum().backward()

    def off_by(got, want):
        want = want.detach().numpy()
        return float(np.linalg.norm(f64(got) - want) / np.linalg.norm(want))

    # in norm: six roundings of 2^-8 / sqrt(3) each, and 2^-4 / sqrt(3) twice where held values enter
    plain, with_held = 6 * 2.0**-8 / 3**0.5, (6 * 2.0**-8 + 2 * 2.0**-4) / 3**0.5
    assert off_by(t["y"], y) < plain
    assert off_by(t["dw"], leaf["w"].grad) < plain
    for n in ("x", "w1", "w2"):
        assert off_by(t["d" + n], leaf[n].grad) < with_held, n
    assert not t["dw1"][np.diff(off) == 0].any() and not t["dw2"][np.diff(off) == 0].any()


def test_the_step_captured_and_replayed():
    s = make(seed=2)
    eager = step(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t = step(s)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        R = s["layer"].tables()["R"]
        for n in t:
            rows = n not in ("y", "dw", "dx", "dw1", "dw2")
            a, b = (t[n][:R], eager[n][:R]) if rows else (t[n], eager[n])
            assert torch.equal(a, b), n
