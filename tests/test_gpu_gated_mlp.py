"""GPU parity of the gated MLP block (qlora_gated_mlp_fwd / _bwd) against binary64; the tolerance's
derivation is in mlp_ref."""
import numpy as np
import pytest
import torch

import mlp_ref as R
from gpu_util import assert_close, to_f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# rows from one to several tiles; columns and depth ragged against every tile (128, 256 and 64 wide)
SHAPES = [(1, 16, 64, 8), (1, 272, 192, 16), (2, 4096, 256, 64), (7, 208, 448, 64), (33, 512, 1024, 32),
          (64, 336, 768, 8), (65, 400, 320, 16), (256, 528, 256, 64), (257, 272, 512, 32), (517, 1040, 576, 64),
          (1030, 528, 256, 16), (600, 144, 4096, 64),
          (1, 2064, 2112, 64), (9, 144, 1088, 32), (16, 1296, 8256, 8), (24, 160, 448, 64), (5, 20000, 192, 8)]
FMTS = ("nf4", "mxfp4", "nvfp4", "nf4dq")


def cu(bits):
    from bit_quantized_base_b200 import qlora as Q
    return Q.bf16_from_bits(bits)


def nan(*shape):
    return torch.full(shape, float("nan"), dtype=BF, device="cuda")


class Gated:
    def __init__(self, fmt, M, N, K, r, seed=0):
        from bit_quantized_base_b200 import qlora as Q
        self.Q, self.M, self.N, self.K, self.r = Q, M, N, K, r
        self.pg, self.pu = R.problem(fmt, M, N, K, r, seed)
        w = [Q.weight_from_numpy(fmt, p["codes"], p["scales"], p["tensor_scale"], scales2=p.get("scales2"))
             for p in (self.pg, self.pu)]
        self.Wg, self.Wu = w
        self.X, self.dH = cu(self.pg["X"]), cu(self.pg["dY"])
        self.ad = [cu(p[k]) for p in (self.pg, self.pu) for k in ("A", "B")]      # Ag, Bg, Au, Bu
        self.ws = Q.alloc_workspace(Q.OP_GATED_MLP_BWD, self.Wg, M, r)

    def fwd(self, act, save=True, ws=None):
        M, N, r = self.M, self.N, self.r
        H = nan(M, N)
        G, U, T = (nan(M, N), nan(M, N), nan(2, M, r)) if save else (None, None, None)
        self.Q.qlora_gated_mlp_fwd(self.Wg, self.Wu, act, self.X, *self.ad, H, G, U, T, M, r, self.pg["s"],
                                   self.ws if ws is None else ws)
        return H, G, U, T

    def bwd(self, act, G, U, T, want_dx=True):
        M, N, K, r = self.M, self.N, self.K, self.r
        dX = nan(M, K) if want_dx else None
        out = nan(r, K), nan(N, r), nan(r, K), nan(N, r)
        self.Q.qlora_gated_mlp_bwd(self.Wg, self.Wu, act, self.X, *self.ad, T, G, U, self.dH, dX, *out, M, r,
                                   self.pg["s"], self.ws)
        return (dX, *out)

    def ok(self):
        torch.cuda.synchronize()
        assert self.Q.qlora_get_device_status(self.ws) == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_parity(fmt, i, shape):
    act = R.ACTS[(i + FMTS.index(fmt)) % 4]
    g = Gated(fmt, *shape, seed=i)
    H, G, U, T = g.fwd(act)
    H2, *_ = g.fwd(act, save=False)
    g.ok()
    X = R.f64(g.pg["X"])
    Wg, Wu = R.decoded(g.pg), R.decoded(g.pu)
    Gr, Tg = R.layer(g.pg, X, Wg)
    Ur, Tu = R.layer(g.pu, X, Wu)
    assert_close(to_f64(G), Gr, "G")
    assert_close(to_f64(U), Ur, "U")
    assert_close(to_f64(T), np.stack([Tg, Tu]), "T")
    assert_close(to_f64(H), R.act(act, Gr)[0] * Ur, "H")
    assert torch.equal(H, H2)
    # backward from the saved tensors, T given and recomputed
    outs = g.bwd(act, G, U, T)
    again = g.bwd(act, G, U, None)
    no_dx = g.bwd(act, G, U, T, want_dx=False)
    g.ok()
    a, da = R.act(act, to_f64(G))
    dH = R.f64(g.pg["dY"])
    dG, dU = dH * to_f64(U) * da, dH * a
    xg, dAg, dBg = R.layer_grad(g.pg, X, to_f64(T)[0], dG, Wg)
    xu, dAu, dBu = R.layer_grad(g.pu, X, to_f64(T)[1], dU, Wu)
    for name, got, ref in zip(("dX", "dAg", "dBg", "dAu", "dBu"), outs, (xg + xu, dAg, dBg, dAu, dBu)):
        assert_close(to_f64(got), ref, name)
    for x, y in zip(outs, again):
        assert torch.equal(x, y)                       # T recomputed bit for bit; deterministic
    for x, y in zip(outs[1:], no_dx[1:]):
        assert torch.equal(x, y)


def test_gradients_against_differences():
    # L = sum C * H in binary64: the library's gradients, from its own saved (rounded) tensors, against
    # central differences of L.  The bound is the first-order one, element by element: with e = 2^-8
    # the largest relative error of a bf16 rounding, T is off by e of its value, G and U by e of
    # theirs and by the two roundings (T, s T) of their LoRA operand (act' moves by at most max |silu''| = 1/2 per unit of G), dG and dU, the rank-r products (once
    # as stored, once scaled for dX) and the outputs are rounded once more.
    M, N, K, r, h = 3, 16, 64, 8, 1e-5
    g = Gated("mxfp4", M, N, K, r, seed=77)
    H, G, U, T = g.fwd("silu")
    dX, dAg, dBg, dAu, dBu = g.bwd("silu", G, U, T)
    g.ok()
    C = R.f64(g.pg["dY"])
    Wg, Wu = R.decoded(g.pg), R.decoded(g.pu)
    v = {"X": R.f64(g.pg["X"]), "Ag": R.f64(g.pg["A"]), "Bg": R.f64(g.pg["B"]), "Au": R.f64(g.pu["A"]),
         "Bu": R.f64(g.pu["B"])}
    s = g.pg["s"]

    def loss(q):
        Gz = q["X"] @ Wg.T + s * (q["X"] @ q["Ag"].T) @ q["Bg"].T
        Uz = q["X"] @ Wu.T + s * (q["X"] @ q["Au"].T) @ q["Bu"].T
        return float((C * R.act("silu", Gz)[0] * Uz).sum())

    e, ab = 2.0 ** -8, np.abs
    Gz = v["X"] @ Wg.T + s * (v["X"] @ v["Ag"].T) @ v["Bg"].T
    Uz = v["X"] @ Wu.T + s * (v["X"] @ v["Au"].T) @ v["Bu"].T
    act, dact = R.act("silu", Gz)
    dG, dU = C * Uz * dact, C * act
    oG, oU = (e * ab(z) + 2 * e * s * ab(v["X"] @ v["A" + n].T) @ ab(v["B" + n]).T for n, z in (("g", Gz), ("u", Uz)))
    eG = ab(C) * (oU * ab(dact) + ab(Uz) * 0.5 * oG) + e * ab(dG)
    eU = ab(C) * ab(dact) * oG + e * ab(dU)
    bound, bx = {}, e * ab(dG @ Wg + dU @ Wu + s * (dG @ v["Bg"]) @ v["Ag"] + s * (dU @ v["Bu"]) @ v["Au"])
    for n, d, ed, W in (("g", dG, eG, Wg), ("u", dU, eU, Wu)):
        A, B = v["A" + n], v["B" + n]
        u, eu = d @ B, ed @ ab(B) + e * ab(d @ B)
        bx = bx + ed @ ab(W) + s * (eu + e * ab(u)) @ ab(A)
        bound["A" + n] = s * eu.T @ ab(v["X"]) + e * s * ab(u.T @ v["X"])
        T64 = v["X"] @ A.T
        bound["B" + n] = s * (ed.T @ ab(T64) + ab(d).T @ (e * ab(T64))) + e * s * ab(d.T @ T64)
    bound["X"] = bx
    for name, got in (("X", dX), ("Ag", dAg), ("Bg", dBg), ("Au", dAu), ("Bu", dBu)):
        num = np.empty_like(v[name])
        for idx in np.ndindex(num.shape):
            q = {k: x.copy() for k, x in v.items()}
            q[name][idx] += h
            up = loss(q)
            q[name][idx] -= 2 * h
            num[idx] = (up - loss(q)) / (2 * h)
        err, most = ab(to_f64(got) - num), bound[name] * (1 + 8 * e) + 1e-6    # + second order, h^2
        assert np.all(err <= most), (name, (err / most).max())
        # the bound says something: a lost factor or term of the formula is past it
        assert np.linalg.norm(most) < 0.25 * np.linalg.norm(num), name


def test_no_rows():
    g = Gated("nf4", 4, 64, 128, 8)
    g.M = 0
    g.X, g.dH = g.X[:0], g.dH[:0]
    H, G, U, T = g.fwd("silu")
    outs = g.bwd("silu", G, U, T)
    g.ok()
    for o in outs[1:]:
        assert torch.count_nonzero(o) == 0


def test_rows_behind_the_last_stay():
    M, N, K, r = 130, 208, 192, 16
    g = Gated("nvfp4", M, N, K, r)
    buf = torch.full((M + 3, N), 7.0, dtype=BF, device="cuda")
    g.Q.qlora_gated_mlp_fwd(g.Wg, g.Wu, "silu", g.X, *g.ad, buf[1:M + 1], None, None, None, M, r, 2.0, g.ws)
    big = torch.full((M + 3, K), 7.0, dtype=BF, device="cuda")
    H, G, U, T = g.fwd("silu")
    dA, dB = nan(r, K), nan(N, r)
    g.Q.qlora_gated_mlp_bwd(g.Wg, g.Wu, "silu", g.X, *g.ad, T, G, U, g.dH, big[1:M + 1], dA, dB, nan(r, K), nan(N, r),
                            M, r, 2.0, g.ws)
    g.ok()
    assert torch.equal(buf[1:M + 1], H)
    for b in (buf, big):
        assert torch.all(b[0] == 7) and torch.all(b[M + 1:] == 7)


def test_a_larger_workspace_serves_fewer_rows():
    big, small = Gated("nf4", 300, 208, 192, 16, seed=3), Gated("nf4", 20, 208, 192, 16, seed=3)
    H, *_ = small.fwd("gelu")
    H2, *_ = small.fwd("gelu", ws=big.ws)
    torch.cuda.synchronize()
    assert_close(to_f64(H), to_f64(H2), "H")


def test_captured_with_an_eager_call_between():
    g = Gated("mxfp4", 100, 272, 320, 16)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        H, G, U, T = g.fwd("silu")
        want = g.bwd("silu", G, U, T)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        H2, G2, U2, T2 = g.fwd("silu")
        got = g.bwd("silu", G2, U2, T2)
    for _ in range(2):
        for t in (H2, *got):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(H, H2)
        for x, y in zip(want, got):
            assert torch.equal(x, y)
        g.fwd("none")                                    # another call on the same workspace between
    g.ok()
