"""The layer for a few tokens with 8- and 4-bit weights where a row of x, or of h, is tiny: fp16's inputs are brought up by
2^112 at most, so that a row whose largest is below 2^-98 no longer reaches fp16's upper end.

Tolerance: as plain64_block.mlp derives it, with an input's own error by its kind. An input stands in fp16 behind the row's
power of two: half of fp16's lowest step, 2^-25 there, is 2^-39 of a largest value of 2^14 or 2^-137 where the power is 2^112;
4-bit weights divide some inputs by 16 before, which makes 2^-35 and 2^-133. h's fp32 has half a lowest step of 2^-150, and its
product with the power of two is exact.

These bounds add worst cases up. In the 2-norm the outputs are off by their rounding, at most 2^-8 of each value, and by what
the inputs' errors make: a matrix of independent entries takes a vector of errors and a vector of values alike, so that a
relative error in x or h becomes one of u or out, and h, the product of two u, has twice that; 8 times the inputs' largest
error over their size leaves room."""
import numpy as np
import pytest
import torch

import plain64 as P
from plain64_block import U
from test_gpu_layer_few import DEV, M, make, run  # noqa: F401

pytestmark = pytest.mark.gpu
LOST = {"fp8": (2.0 ** -39, 2.0 ** -137), "w4": (2.0 ** -35, 2.0 ** -133)}


def mlp(x, up, down, inner, kind, up_mag, down_mag):
    def product(v, w, mag):
        K = w.shape[1]
        rel, least = LOST[kind]
        B = (K / 8 + K / 16 + 24) * U * (np.abs(v) @ np.abs(w).T)
        B = B + np.maximum(rel * np.abs(v).max(1, keepdims=True), least) * np.abs(w).sum(1)
        if mag is not None:
            B = B + 52 * U * (np.abs(v) @ mag.T)
        return v @ w.T, B
    r, B = product(x, up, up_mag)
    g, u, Bg, Bu = r[:, :inner], r[:, inner:], B[:, :inner], B[:, inner:]
    s = g / (1.0 + np.exp(-g))
    h = s * u
    reach = 1.1 * Bg * np.abs(u) + np.abs(s) * Bu + Bg * Bu + (2.0 ** -21 + 2.0 ** -11) * np.abs(h) + 2.0 ** -149
    out, Bo = product(h, down, down_mag)
    return out, Bo + reach @ np.abs(down).T


def check(s, out, size):
    """size: 2^-low, that of the tiny rows' values"""
    ri, ok, rw, _ = P.gate(s["logits"].double().cpu().numpy(), s["bias"].double().cpu().numpy(), s["k"], sigmoid=True, scale=1.5)
    x = s["x"].double().cpu().numpy()
    ref, bound = np.zeros((s["T"], s["H"])), np.zeros((s["T"], s["H"]))
    for e in range(s["E"] + s["shared"]):
        t, j = np.nonzero((ri == e) & ok) if e < s["E"] else (np.arange(s["T"]), None)
        if len(t) == 0:
            continue
        v, B = mlp(x[t], s["up"][2][e], s["down"][2][e], s["I"], s["kind"],
                   *(m[3][e] if m[3] is not None else None for m in (s["up"], s["down"])))
        by = rw[t, j][:, None] if j is not None else 1.0
        ref[t] += by * v
        bound[t] += np.abs(by) * (B + (2.0 ** -19 + 2.0 ** -20) * np.abs(v))
    o = out.double().cpu().numpy()
    assert np.isfinite(o).all() and np.abs(ref).min() > 0
    bar = bound + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
    assert (np.abs(o - ref) <= bar).all(), (np.abs(o - ref) / bar).max()
    assert np.linalg.norm(o - ref) <= (2.0 ** -8 + 2.0 ** -12 + 8 * LOST[s["kind"]][1] / size) * np.linalg.norm(ref)


def times(m, by):
    """Weights by a power of two, through their scales."""
    q, scale, v, mag = m
    return q, (scale.float() * by).to(scale.dtype), v * by, None if mag is None else mag * by


@pytest.mark.parametrize("kind,group", [("fp8", 128), ("w4", 32), ("w4", 64), ("w4", 128)])
@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("low", [60, 97, 99, 104, 112, 118])
def test_tiny_inputs(M, T, low, kind, group):
    s = make(M, T, 4, 2, 384, 256, kind, group, 1)
    s["x"] = (s["x"].float() * 2.0 ** -low).to(torch.bfloat16)
    s["up"] = times(s["up"], 2.0 ** low)
    check(s, run(M, s)[2], 2.0 ** -low)


@pytest.mark.parametrize("kind,group", [("fp8", 128), ("w4", 32), ("w4", 64), ("w4", 128)])
@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("low", [60, 96, 104, 112, 118])
def test_tiny_h(M, T, low, kind, group):
    """u of 2^(-low / 2), so that h = silu(u) u' is about 2^-low / 4, and the down product brings it up again."""
    s = make(M, T, 4, 2, 384, 256, kind, group, 1)
    s["up"] = times(s["up"], 2.0 ** (-low // 2))
    s["down"] = times(s["down"], 2.0 ** low)
    check(s, run(M, s)[2], 2.0 ** (-low - 2))
