"""GPU parity of the linear layer with bias, activation and residual (qlora_linear_act_fwd / _bwd)
against binary64; the tolerance's derivation is in mlp_ref."""
import numpy as np
import pytest
import torch

import mlp_ref as R
from bit_quantized_base_b200 import synth
from gpu_util import assert_close, to_f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SHAPES = [(1, 16, 64, 8), (1, 272, 1856, 16), (3, 4096, 256, 64), (20, 208, 448, 64), (64, 336, 768, 8),
          (65, 400, 320, 16), (256, 528, 256, 64), (257, 272, 512, 32), (517, 1040, 576, 64), (1030, 528, 256, 16),
          (1, 2064, 2112, 64), (9, 144, 1088, 32), (16, 1296, 8256, 8), (40, 160, 448, 64), (5, 40000, 192, 8)]
FMTS = ("nf4", "mxfp4", "nvfp4", "nf4dq")


def nan(*shape):
    return torch.full(shape, float("nan"), dtype=BF, device="cuda")


class Linear:
    def __init__(self, fmt, M, N, K, r, seed=0):
        from bit_quantized_base_b200 import qlora as Q
        self.Q, self.M, self.N, self.K, self.r = Q, M, N, K, r
        self.p = p = synth.small_layer(fmt, M, N, K, r, seed=300 + seed, b_std=0.05)
        self.W = Q.weight_from_numpy(fmt, p["codes"], p["scales"], p["tensor_scale"], scales2=p.get("scales2"))
        self.X, self.A, self.B, self.dY = (Q.bf16_from_bits(p[k]) for k in ("X", "A", "B", "dY"))
        rng = np.random.default_rng(seed)
        self.bias = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).to(BF).cuda()
        self.res = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).to(BF).cuda()
        self.ws = Q.alloc_workspace(Q.OP_ACT_BWD, self.W, M, r)

    def fwd(self, act, bias=True, res=True, Y=None, save=True):
        Y = nan(self.M, self.N) if Y is None else Y
        Z, T = (nan(self.M, self.N), nan(self.M, self.r)) if save else (None, None)
        self.Q.qlora_linear_act_fwd(self.W, self.X, self.A, self.B, self.bias if bias else None, act,
                                    (self.res if res is True else res) if res is not False else None, Y, Z, T,
                                    self.M, self.r, self.p["s"], self.ws)
        return Y, Z, T

    def bwd(self, act, Z, T, bias=True, want_dx=True):
        dX = nan(self.M, self.K) if want_dx else None
        dA, dB, db = nan(self.r, self.K), nan(self.N, self.r), nan(self.N) if bias else None
        self.Q.qlora_linear_act_bwd(self.W, self.X, self.A, self.B, T, Z, act, self.dY, dX, dA, dB, db, self.M,
                                    self.r, self.p["s"], self.ws)
        return dX, dA, dB, db

    def ok(self):
        torch.cuda.synchronize()
        assert self.Q.qlora_get_device_status(self.ws) == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_parity(fmt, i, shape):
    k = i + FMTS.index(fmt)
    act, bias, res = R.ACTS[k % 4], k % 3 != 0, k % 5 != 0
    g = Linear(fmt, *shape, seed=i)
    Y, Z, T = g.fwd(act, bias, res)
    Y2, *_ = g.fwd(act, bias, res, save=False)
    g.ok()
    X, W = R.f64(g.p["X"]), R.decoded(g.p)
    Zr, Tr = R.layer(g.p, X, W)
    if bias:
        Zr = Zr + to_f64(g.bias)[None, :]
    Yr = R.act(act, Zr)[0] + (to_f64(g.res) if res else 0.0)
    assert_close(to_f64(Z), Zr, "Z")
    assert_close(to_f64(T), Tr, "T")
    assert_close(to_f64(Y), Yr, "Y")
    assert torch.equal(Y, Y2)
    outs = g.bwd(act, Z, T, bias)
    again = g.bwd(act, Z if act != "none" else None, None, bias)
    no_dx = g.bwd(act, Z, T, bias, want_dx=False)
    g.ok()
    d = R.f64(g.p["dY"]) * R.act(act, to_f64(Z))[1]
    refs = R.layer_grad(g.p, X, to_f64(T), d, W)
    for name, got, ref in zip(("dX", "dA", "dB"), outs, refs):
        assert_close(to_f64(got), ref, name)
    if bias:
        # one rounding, M binary32 additions, and the derivative's own absolute error: erff and the
        # exponential are within 2 ulp of values up to 1 (2^-22), the sums and products of the
        # formula add 2 more half ulp of values up to 1.13 -- below 2^-21, of every |dY|
        ref, mag = d.sum(axis=0), np.abs(d).sum(axis=0)
        slack = (shape[0] + 64) * 2.0 ** -23 * mag + 2.0 ** -21 * np.abs(R.f64(g.p["dY"])).sum(axis=0)
        err = np.abs(to_f64(outs[3]) - ref)
        assert np.all(err <= 2.0 ** -8 * np.abs(ref) + slack), (err / (2.0 ** -8 * np.abs(ref) + slack)).max()
    for x, y in zip(outs, again):
        assert x is None or torch.equal(x, y)
    for x, y in zip(outs[1:], no_dx[1:]):
        assert x is None or torch.equal(x, y)


def test_plain_call_is_the_layer():
    # no bias, activation or residual: the layer's own forward (another epilogue, the same sums) and
    # its own backward, bit for bit
    g = Linear("nf4", 300, 272, 320, 16)
    Y, _, T = g.fwd("none", bias=False, res=False)
    Y0, T0 = nan(300, 272), nan(300, 16)
    ws = g.Q.alloc_workspace(g.Q.OP_BWD, g.W, 300, 16)
    g.Q.qlora_linear_fwd(g.W, g.X, g.A, g.B, Y0, T0, 300, 16, g.p["s"], ws)
    dX, dA, dB, _ = g.bwd("none", None, T, bias=False)
    dX0, dA0, dB0 = nan(300, 320), nan(16, 320), nan(272, 16)
    g.Q.qlora_linear_bwd(g.W, g.X, g.A, g.B, T0, g.dY, dX0, dA0, dB0, 300, 16, g.p["s"], ws)
    g.ok()
    for x, y in ((Y, Y0), (T, T0), (dX, dX0), (dA, dA0), (dB, dB0)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("M", [1, 50, 200, 300])
def test_in_place_residual(M):
    g = Linear("nvfp4", M, 528, 320, 16)
    want, *_ = g.fwd("none", bias=True, res=True)
    buf = g.res.clone()
    g.fwd("none", bias=True, res=buf, Y=buf)
    g.ok()
    assert torch.equal(buf, want)


def test_extreme_preactivations():
    # a bias of +-1e4, +-100 and infinities: the activations saturate without a NaN of their own
    M, N, K, r = 4, 64, 64, 8
    g = Linear("mxfp4", M, N, K, r)
    g.bias[:6] = torch.tensor([1e4, -1e4, 100.0, -100.0, 3e38, -3e38], dtype=BF)
    for act in ("silu", "gelu", "gelu_tanh"):
        Y, Z, T = g.fwd(act, res=False)
        dX, dA, dB, db = g.bwd(act, Z, T)
        g.ok()
        y = to_f64(Y)
        z = to_f64(Z)
        assert np.all(np.isfinite(y)) and np.all(np.isfinite(to_f64(db)))
        big, small = z > 50, z < -50
        assert big.any() and small.any()
        assert np.all(np.abs(y[big] / z[big] - 1) <= 2.0 ** -7)     # Y and the saved Z, one rounding each
        assert np.all(np.abs(y[small]) <= 1e-18)


def test_no_rows():
    g = Linear("nf4", 4, 64, 128, 8)
    g.M = 0
    g.X, g.dY, g.res = g.X[:0], g.dY[:0], g.res[:0]
    Y, Z, T = g.fwd("silu")
    dX, dA, dB, db = g.bwd("silu", Z, T)
    g.ok()
    for o in (dA, dB, db):
        assert torch.count_nonzero(o) == 0


def test_mlp_block_forward_and_backward():
    """The block as it is used: norm with residual, gated MLP, down projection added to the residual
    stream, and the gradients back to the block's input, against the same chain in binary64.  Each
    stage reads the bf16 tensors of the stage before it, so the reference follows the library's
    stored tensors stage by stage."""
    from bit_quantized_base_b200 import qlora as Q
    M, D, F, r, eps = 150, 320, 576, 16, 1e-6
    rng = np.random.default_rng(11)
    pg, pu = R.problem("nvfp4", M, F, D, r, seed=5)
    pd = synth.small_layer("nf4", M, D, F, r, seed=6, b_std=0.05)
    bf = lambda a: torch.from_numpy(a.astype(np.float32)).to(BF).cuda()       # noqa: E731
    X, Res, gamma, dOut = (bf(rng.standard_normal(s)) for s in ((M, D), (M, D), (D,), (M, D)))
    Wg, Wu, Wd = (Q.weight_from_numpy(p["fmt"], p["codes"], p["scales"], p["tensor_scale"]) for p in (pg, pu, pd))
    ad = [Q.bf16_from_bits(p[k]) for p in (pg, pu) for k in ("A", "B")]
    Ad, Bd = Q.bf16_from_bits(pd["A"]), Q.bf16_from_bits(pd["B"])
    wsg, wsd = Q.alloc_workspace(Q.OP_GATED_MLP_BWD, Wg, M, r), Q.alloc_workspace(Q.OP_ACT_BWD, Wd, M, r)
    wsn = torch.empty(Q.qlora_rmsnorm_workspace_size(M, D), dtype=torch.uint8, device="cuda")
    S, Y, rstd, Out = nan(M, D), nan(M, D), torch.empty(M, device="cuda"), nan(M, D)
    H, G, U, T, Td = nan(M, F), nan(M, F), nan(M, F), nan(2, M, r), nan(M, r)
    Q.qlora_rmsnorm_fwd(X, Res, gamma, eps, S, Y, None, None, rstd, M, D)
    Q.qlora_gated_mlp_fwd(Wg, Wu, "silu", Y, *ad, H, G, U, T, M, r, 2.0, wsg)
    Q.qlora_linear_act_fwd(Wd, H, Ad, Bd, None, "none", S, Out, None, Td, M, r, 2.0, wsd)
    dH, dY, dS = nan(M, F), nan(M, D), nan(M, D)
    dAd, dBd, dAg, dBg, dAu, dBu, dgam = nan(r, F), nan(D, r), nan(r, D), nan(F, r), nan(r, D), nan(F, r), nan(D)
    Q.qlora_linear_act_bwd(Wd, H, Ad, Bd, Td, None, "none", dOut, dH, dAd, dBd, None, M, r, 2.0, wsd)
    Q.qlora_gated_mlp_bwd(Wg, Wu, "silu", Y, *ad, T, G, U, dH, dY, dAg, dBg, dAu, dBu, M, r, 2.0, wsg)
    Q.qlora_rmsnorm_bwd(S, rstd, gamma, eps, dY, dOut, dS, dgam, M, D, wsn)
    torch.cuda.synchronize()
    assert Q.qlora_get_device_status(wsg) == 0 and Q.qlora_get_device_status(wsd) == 0
    f = to_f64
    Sr = f(X) + f(Res)
    assert_close(f(S), Sr, "S")
    Yr = f(S) / np.sqrt((f(S) ** 2).mean(axis=1, keepdims=True) + eps) * f(gamma)
    assert_close(f(Y), Yr, "Y")
    Gr, Ur = R.layer(pg, f(Y))[0], R.layer(pu, f(Y))[0]
    assert_close(f(H), R.act("silu", Gr)[0] * Ur, "H")
    assert_close(f(Out), R.layer(pd, f(H))[0] + f(S), "Out")
    xd, ad_, bd_ = R.layer_grad(pd, f(H), f(Td), f(dOut))
    for name, a, b in (("dH", dH, xd), ("dAd", dAd, ad_), ("dBd", dBd, bd_)):
        assert_close(f(a), b, name)
    a, da = R.act("silu", f(G))
    xg, rAg, rBg = R.layer_grad(pg, f(Y), f(T)[0], f(dH) * f(U) * da)
    xu, rAu, rBu = R.layer_grad(pu, f(Y), f(T)[1], f(dH) * a)
    for name, got, ref in (("dY", dY, xg + xu), ("dAg", dAg, rAg), ("dBg", dBg, rBg), ("dAu", dAu, rAu), ("dBu", dBu, rBu)):
        assert_close(f(got), ref, name)
    v = f(dY) * f(gamma)
    r_ = f(rstd)[:, None]
    assert_close(f(dS), f(dOut) + r_ * (v - f(S) * r_ * r_ * (v * f(S)).mean(axis=1, keepdims=True)), "dS")
    assert_close(f(dgam), (f(dY) * f(S) * r_).sum(axis=0), "dgamma")
