"""Binary64 reference of the gated MLP and of the linear layer with bias, activation and residual,
and seeded problems for their tests.  The weight's elements come from the oracle's decoder; the
rest is written out here in numpy.

Tolerance of the bf16 outputs (gpu_util.assert_close: relative Frobenius error 4e-3, largest error
2e-2 of the largest magnitude): one bf16 rounding is off by at most 2^-8 of the value, uniformly
spread within its step, so at most 2^-8 / sqrt(3) = 2.3e-3 in Frobenius norm; no output passes more
than three independent roundings (an operand, a rank-r product, the output): sqrt(3) x 2.3e-3 =
3.9e-3.  binary32 accumulation adds less than 1e-5 at these sizes."""
import numpy as np
from scipy.special import erf, expit

from bit_quantized_base_b200 import synth
from oracle import oracle as O

ACTS = ("none", "silu", "gelu", "gelu_tanh")


def f64(bits):
    return synth.bf16_bits_to_f32(bits).astype(np.float64)


def decoded(p):
    """deq(W) [N, K] in binary64 (NVFP4: the exact block product times the tensor scale)."""
    kw = dict(scales2=p["scales2"]) if p["fmt"] == "nf4dq" else {}
    bits = O.dequant(p["fmt"], p["N"], p["K"], p["codes"], p["scales"], 1.0, **kw) if p["fmt"] != "nvfp4" else \
        O.dequant("nvfp4", p["N"], p["K"], p["codes"], p["scales"], p["tensor_scale"], with_tensor_scale=False)
    w = f64(bits)
    return w * float(p["tensor_scale"]) if p["fmt"] == "nvfp4" else w


def act(name, z):
    """(act(z), act'(z))."""
    if name == "none":
        return z, np.ones_like(z)
    if name == "silu":
        p = expit(z)
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        c = 0.5 * (1 + erf(z / np.sqrt(2)))
        return z * c, c + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    k = np.sqrt(2 / np.pi)
    t = np.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def layer(p, X, W=None):
    """(Z, T) of one LoRA layer."""
    T = X @ f64(p["A"]).T
    return X @ (decoded(p) if W is None else W).T + p["s"] * (T @ f64(p["B"]).T), T


def layer_grad(p, X, T, d, W=None):
    """(dX, dA, dB) of one LoRA layer for the output gradient d."""
    U = d @ f64(p["B"])
    return d @ (decoded(p) if W is None else W) + p["s"] * (U @ f64(p["A"])), p["s"] * (U.T @ X), p["s"] * (d.T @ T)


def problem(fmt, M, N, K, r, seed=0, s=2.0):
    """Gate and up projection of one gated MLP: two layers on one X (dX's gradient dH is the
    gate's dY), the up weight twice as large (NVFP4: another tensor scale), adapters large enough
    for the LoRA terms to weigh in every output."""
    pg = synth.small_layer(fmt, M, N, K, r, s=s, seed=100 + seed, b_std=0.05)
    pu = synth.small_layer(fmt, M, N, K, r, s=s, seed=200 + seed, b_std=0.05)
    if fmt == "nvfp4":
        pu["tensor_scale"] = float(np.float32(pu["tensor_scale"] * 2.5))
    pu["X"] = pg["X"]
    return pg, pu
