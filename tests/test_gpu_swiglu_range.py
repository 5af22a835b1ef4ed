"""The gated activation and its backward pass over the gate's whole range,
against float64: silu(g) = g e^g / (1 + e^g) is a float down to g = -108, and
times a large u it is no small value.

Bars: the result's rounding (2^-8 or 2^-24 of the value, half the smallest
subnormal of the type), 2^-17 of the terms for the float evaluation, and for a
subnormal e^-|g|, whose error is absolute, two of its steps (2^-148) through
the factors that it meets."""
import numpy as np
import pytest

import synth
from helpers import bf16_from_dev, bf16_to_dev, log, to_dev
from oracle import train

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

UB = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
LEAST = {"bf16": 2.0 ** -134, "f32": 2.0 ** -150}
FLT, STEP = 2.0 ** -17, 2.0 ** -148
GATES = np.concatenate([np.arange(-112.0, 112.0, 0.5), [-1e3, -1e4, 1e3, 1e4, -2.0 ** -30, 2.0 ** -30]])


def _pair(v, kind):
    v = np.asarray(v, np.float32)
    if kind == "f32":
        return to_dev(v), v.astype(np.float64)
    bits = synth.f32_to_bf16_bits(v)
    return bf16_to_dev(bits), synth.as_f64(bits)


def _val(t):
    return synth.as_f64(bf16_from_dev(t)) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("u", [1.0, -3.0, 1e30])
def test_swiglu_over_the_range_of_the_gate(kind, u):
    import fp8_block_scaled_sigmoid_amd as moe
    I = len(GATES)
    a, a64 = _pair(np.concatenate([GATES, np.full(I, u)])[None, :], kind)
    dh, dh64 = _pair(np.full((1, I), 0.75), kind)
    w = np.array([0.5], np.float32)
    log(f"moe_swiglu over the gate's range, u={u}, {kind}")
    g, u64 = a64[:, :I], a64[:, I:]
    s = train.sigmoid(g)
    h = _val(moe.moe_swiglu(a))
    want = train.swiglu(a64)
    assert np.all(np.abs(h - want) <= (UB[kind] + FLT) * np.abs(want) + np.abs(g * u64) * STEP + LEAST[kind])
    da, dgate, hg = moe.moe_swiglu_backward(a, dh, to_dev(w))
    wda, wdg, whg, mag = train.swiglu_backward(a64, dh64, w)
    wd = np.abs(0.5 * dh64)
    tol_g = UB[kind] * np.abs(wda[:, :I]) + wd * np.abs(u64) * (
        FLT * (s + np.abs(g * s) * (1 - s)) + 2 * (1 + np.abs(g)) * STEP) + LEAST[kind]
    tol_u = (UB[kind] + FLT) * np.abs(wda[:, I:]) + wd * np.abs(g) * STEP + LEAST[kind]
    assert np.all(np.abs(_val(da) - wda) <= np.concatenate([tol_g, tol_u], 1))
    assert np.all(np.abs(_val(hg) - whg) <= (UB[kind] + FLT) * np.abs(whg)
                  + 0.5 * np.abs(g * u64) * STEP + LEAST[kind])
    assert np.all(np.abs(_val(dgate) - wdg) <= (FLT + I * 2.0 ** -24) * mag
                  + (np.abs(g * u64 * dh64)).sum(1) * STEP)
