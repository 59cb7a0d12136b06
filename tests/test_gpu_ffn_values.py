"""GPU tests of the feed-forward operators' values where only a relative bound
shows an error: the activations' tails and their slopes, which are far smaller
than the largest values of a call. Identity weights make a product return its
input, so each output is one activation (or slope) rounded to T."""
from __future__ import annotations

import math

import pytest
import torch

import hyper_connection_rank_amd as hc
from _ffn import F, T_OF, U, tiny

pytestmark = pytest.mark.gpu
N = 64


def grid(lo, hi, dt):
    """64 x 64 values from lo to hi, rounded to T."""
    return torch.linspace(lo, hi, N * N, dtype=torch.float64).to(dt).view(N, N).cuda()


def relative(got, exact, rel, label):
    """|got - exact| <= rel |exact| + one rounding of a value that far off (half a step of T's subnormal
    numbers where that is more)."""
    err = (got.double() - exact).abs()
    tol = rel * exact.abs() + U(got.dtype) * (1 + rel) * exact.abs() + tiny(got.dtype)
    bad = ~(err <= tol)
    if bad.any():
        i = int((err / tol).nan_to_num(nan=math.inf).argmax())
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} off; worst: got {got.flatten()[i].item()}, "
                             f"exact {exact.flatten()[i].item()}, error / allowed {(err / tol).flatten()[i].item():.2f}")


# 16-bit T: Phi's tail is off by at most 1.1e-6 (its polynomial) and its exponent a^2 / 2 log2(e), of at most 47 for
# a <= 8, is rounded three times: 3 * 47 * 2^-24 ln 2 = 5.8e-6; the remaining steps add less than 16 * 2^-24. In all
# below 2^-17. fp32: the argument x / sqrt 2 is rounded twice (the constant, the product), which moves erfc(y) by
# 2 y^2 = x^2 times that, 2 * 64 * 2^-24, and erfc itself and the steps after it are good to 16 * 2^-24.
GELU_REL = {"f32": 144 * F, "f16": 2.0 ** -17, "bf16": 2.0 ** -17}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gelu_keeps_its_relative_accuracy_in_the_tail(dtype):
    dt = T_OF[dtype]
    x, eye = grid(-8.0, -2.0, dt), torch.eye(N, dtype=dt, device="cuda")
    xd = x.double()
    exact = 0.5 * xd * torch.special.erfc(-xd * 0.5 ** 0.5)  # no cancellation, unlike 1 + erf
    rel = GELU_REL[dtype]
    relative(hc.linear(x, eye, activation="gelu"), exact, rel, ("linear", dtype))
    ones = torch.ones(N, dtype=dt, device="cuda")
    h = hc.glu(x, eye, torch.zeros_like(eye), None, ones, activation="gelu")  # u = 1
    relative(h, exact, rel, ("glu", dtype))
    # The slope Phi(x) + x phi(x): the terms have opposite signs, Phi at most 0.22 of the other for x <= -2, so
    # their sum is off by at most (1 + 0.22) / (1 - 0.22) < 1.6 times their own relative error.
    dx, _, _ = hc.linear_backward(x, eye, torch.ones_like(x), x, activation="gelu")
    slope = 0.5 * torch.special.erfc(-xd * 0.5 ** 0.5) + xd * torch.exp(-0.5 * xd * xd) / (2 * math.pi) ** 0.5
    # two roundings: dz to T, then dx (the same value, exact); the second adds nothing
    relative(dx, slope, 1.6 * rel, ("slope", dtype))


# With e = exp(-|x|), |x| <= 16: fp32's exponential (2 F), sum (F), quotient (F) and products (2 F) are off by 8 F
# at most; 16-bit T's exponent, of at most 23.1, is rounded twice (2 * 23.1 ln 2 F = 32 F), its exponential,
# reciprocal and products by 8 F more.
SIGMOID_REL = {"f32": 8 * F, "f16": 40 * F, "bf16": 40 * F}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_sigmoid_slope_keeps_its_relative_accuracy(dtype):
    """s (1 - s) of large x, where 1 - s is small."""
    dt = T_OF[dtype]
    x, eye = grid(-16.0, 16.0, dt), torch.eye(N, dtype=dt, device="cuda")
    e = torch.exp(-x.double().abs())
    exact = e / (1 + e) ** 2
    dx, _, _ = hc.linear_backward(x, eye, torch.ones_like(x), x, activation="sigmoid")
    relative(dx, exact, SIGMOID_REL[dtype], ("linear_backward", dtype))
    zero, one = torch.zeros_like(eye), torch.ones_like(x)
    dx = hc.glu_backward(x, eye, zero, x, one, one, activation="sigmoid")[0]  # u = dh = 1: dg Wg^T + du 0
    relative(dx, exact, SIGMOID_REL[dtype], ("glu_backward", dtype))


def test_slopes_of_large_preactivations_reach_one():
    """The slopes of silu and gelu_tanh hold a factor 1 - s that x (and its cube) multiply."""
    x, eye = grid(2.0, 12.0, torch.float32), torch.eye(N, device="cuda")
    xd = x.double()
    for act in ("silu", "gelu_tanh"):
        dx, _, _ = hc.linear_backward(x, eye, torch.ones_like(x), x, activation=act)
        if act == "silu":
            e = torch.exp(-xd)
            exact = (1 + xd * e / (1 + e)) / (1 + e)
        else:  # with t the tanh form's argument: s = sigmoid(2 t)
            c = (2 / math.pi) ** 0.5
            e = torch.exp(-2 * c * (xd + 0.044715 * xd ** 3))
            s = 1 / (1 + e)
            exact = s + 2 * xd * s * (e * s) * c * (1 + 3 * 0.044715 * xd * xd)
        # silu, s (1 + x c): x c <= 0.24 is off by 6 F of itself, the sum, s and the product by 5 F: 7 F in all.
        # gelu_tanh, s + term: 2 t is rounded seven times, term <= 0.11 and term times 2 t <= 0.41, so the term is
        # off by 7 * 0.41 F + 11 * 0.11 F, s by 3 F, the sum by F: 9 F in all.
        relative(dx, exact, 9 * F, act)
