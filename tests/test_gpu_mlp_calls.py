"""Batch sizes around every change of kernel, and the ways of calling the MLP operators: two calls at
once, captured calls that share a workspace, one workspace for several operators."""
import numpy as np
import pytest
import torch

import mlp_ref as R
from gpu_util import assert_close, to_f64
from test_gpu_gated_mlp import Gated, nan
from test_gpu_linear_act import Linear

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# one below and above: 8 and 16 rows (narrow), 64 (down-projection), 128 (a row tile), 256 (one MMA block)
ROWS = (8, 15, 16, 17, 31, 63, 64, 65, 127, 129, 255, 256, 257)
# few tiles and a deep contraction: the contraction is split, also where the last item is short
DEEP = [(17, 64, 4160, 8), (48, 272, 8192, 16), (256, 144, 2112, 64), (300, 528, 4096, 16), (520, 272, 1984, 32)]


def check_gated(fmt, shape, act, seed):
    g = Gated(fmt, *shape, seed=seed)
    H, G, U, T = g.fwd(act)
    outs = g.bwd(act, G, U, T)
    g.ok()
    X, Wg, Wu = R.f64(g.pg["X"]), R.decoded(g.pg), R.decoded(g.pu)
    Gr, Tg = R.layer(g.pg, X, Wg)
    Ur, Tu = R.layer(g.pu, X, Wu)
    for name, got, ref in (("G", G, Gr), ("U", U, Ur), ("T", T, np.stack([Tg, Tu])), ("H", H, R.act(act, Gr)[0] * Ur)):
        assert_close(to_f64(got), ref, name)
    a, da = R.act(act, to_f64(G))
    dH = R.f64(g.pg["dY"])
    dG, dU = dH * to_f64(U) * da, dH * a
    xg, dAg, dBg = R.layer_grad(g.pg, X, to_f64(T)[0], dG, Wg)
    xu, dAu, dBu = R.layer_grad(g.pu, X, to_f64(T)[1], dU, Wu)
    for name, got, ref in zip(("dX", "dAg", "dBg", "dAu", "dBu"), outs, (xg + xu, dAg, dBg, dAu, dBu)):
        assert_close(to_f64(got), ref, name)


def check_linear(fmt, shape, act, seed):
    g = Linear(fmt, *shape, seed=seed)
    Y, Z, T = g.fwd(act)
    dX, dA, dB, db = g.bwd(act, Z if act != "none" else None, T)
    g.ok()
    X, W = R.f64(g.p["X"]), R.decoded(g.p)
    Zr, Tr = R.layer(g.p, X, W)
    Zr = Zr + to_f64(g.bias)[None, :]
    assert_close(to_f64(Z), Zr, "Z")
    assert_close(to_f64(T), Tr, "T")
    assert_close(to_f64(Y), R.act(act, Zr)[0] + to_f64(g.res), "Y")
    dZ = R.f64(g.p["dY"]) * R.act(act, to_f64(Z))[1]
    for name, got, ref in zip(("dX", "dA", "dB"), (dX, dA, dB), R.layer_grad(g.p, X, to_f64(T), dZ, W)):
        assert_close(to_f64(got), ref, name)
    # dbias: binary32 sums of values that carry at most 2^-18 of |dY| from the derivative, rounded once
    slack = (2.0 ** -18 + (shape[0] + 4) * 2.0 ** -24) * 2 * np.abs(R.f64(g.p["dY"])).sum(axis=0)
    assert np.all(np.abs(to_f64(db) - dZ.sum(axis=0)) <= 2.0 ** -8 * np.abs(dZ.sum(axis=0)) + slack)


@pytest.mark.parametrize("M", ROWS)
def test_rows_around_every_kernel(M):
    fmt, act = ("nf4", "mxfp4", "nvfp4", "nf4dq")[M % 4], R.ACTS[M % 3 + 1]
    check_gated(fmt, (M, 272, 448, 16), act, seed=M)
    check_linear(fmt, (M, 272, 448, 16), act, seed=M)


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4", "nvfp4", "nf4dq"])
@pytest.mark.parametrize("i,shape", list(enumerate(DEEP)))
def test_split_contractions(fmt, i, shape):
    M, N, K, r = shape
    check_gated(fmt, shape, R.ACTS[i % 4], seed=i)
    check_linear(fmt, shape, R.ACTS[(i + 1) % 4], seed=i)
    check_linear(fmt, (M, K, -(-N // 64) * 64, r), R.ACTS[(i + 2) % 4], seed=i)     # the deep one is dX's


def test_largest_magnitudes_and_nan_rows():
    """A row of NaN or infinities leaves the other rows as they are (a split contraction, dX of 40 rows)."""
    M, N, K, r = 40, 64, 4160, 16
    g = Gated("mxfp4", M, N, K, r, seed=5)
    H, G, U, T = g.fwd("silu")
    g.X[7] = float("nan")
    g.X[21] = float("inf")
    H2, G2, U2, T2 = g.fwd("silu")
    g.ok()
    keep = [m for m in range(M) if m not in (7, 21)]
    for x, y in ((H, H2), (G, G2), (U, U2)):
        assert torch.equal(x[keep], y[keep])
    assert torch.isnan(H2[7]).all() and not torch.isfinite(G2[21].float()).any()
    assert torch.equal(T[:, keep], T2[:, keep])


@pytest.mark.parametrize("M", [3, 40, 200, 300])
def test_two_graphs_share_a_workspace(M):
    """Two captured calls on one workspace, replayed in turn and with an eager call between: each gives its
    own results every time."""
    a, b = Gated("nf4", M, 272, 4160, 16, seed=1), Gated("nf4", M, 272, 4160, 16, seed=2)
    b.ws = a.ws
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        want = []
        for g in (a, b):
            H, G, U, T = g.fwd("gelu")
            want.append((H, *g.bwd("gelu", G, U, T)))
    st.synchronize()
    graphs, got = [], []
    for g in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            H, G, U, T = g.fwd("gelu")
            got.append((H, *g.bwd("gelu", G, U, T)))
        graphs.append(graph)
    for k in (0, 1, 1, 0, 0, 1):
        for t in got[k]:
            t.zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        for x, y in zip(want[k], got[k]):
            assert torch.equal(x, y)
        if k:
            b.fwd("silu")
    a.ok()


@pytest.mark.parametrize("M", [2, 40, 300])
def test_two_calls_at_once(M):
    """Calls on two streams with a workspace each, many in flight, each as if alone."""
    gs = [Gated("mxfp4", M, 528, 2112, 16, seed=s) for s in (1, 2)]
    ls = [Linear("nvfp4", M, 528, 2112, 16, seed=s) for s in (3, 4)]
    want = []
    for g, l in zip(gs, ls):
        H, G, U, T = g.fwd("silu")
        Y, Z, T1 = l.fwd("gelu_tanh")
        want.append((H, *g.bwd("silu", G, U, T), Y, *l.bwd("gelu_tanh", Z, T1)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    for _ in range(4):
        got = []
        for st, g, l in zip(streams, gs, ls):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                H, G, U, T = g.fwd("silu")
                Y, Z, T1 = l.fwd("gelu_tanh")
                got.append((H, *g.bwd("silu", G, U, T), Y, *l.bwd("gelu_tanh", Z, T1)))
        for g, l in zip(gs, ls):
            g.ok()
            l.ok()
        for w, q in zip(want, got):
            for x, y in zip(w, q):
                assert torch.equal(x, y)


def test_one_workspace_for_all_operators():
    """A workspace of the largest call serves every operator of the layer in turn, in any order."""
    from bit_quantized_base_b200 import qlora as Q
    M, N, K, r = 200, 528, 2112, 16
    g = Gated("nf4", M, N, K, r, seed=8)
    l = {m: Linear("nf4", m, N, K, r, seed=9) for m in (1, 16, 40, 100, 200)}
    size = max([g.ws.numel()] + [x.ws.numel() for x in l.values()]
               + [Q.alloc_workspace(op, g.Wg, M, r).numel() for op in (Q.OP_FWD, Q.OP_BWD)])
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    alone = {}
    for turn in range(3):
        for m in (16, 200, 1, 100, 40) if turn else (1, 16, 40, 100, 200):
            x = l[m]
            if turn:
                x.ws = ws
            Y, Z, T = x.fwd("silu")
            out = [Y, *x.bwd("silu", Z, T)]
            plain = nan(m, N)
            Q.qlora_linear_fwd(x.W, x.X, x.A, x.B, plain, None, m, r, x.p["s"], ws)
            out.append(plain)
            H, G, U, T = g.fwd("gelu", ws=ws if turn else None)
            out.append(H)
            x.ok()
            if turn == 0:
                alone[m] = out
            for a, b in zip(alone[m], out):
                assert_close(to_f64(b), to_f64(a), "result")


@pytest.mark.parametrize("M", [1, 16, 40, 100])
def test_a_larger_workspace_serves_the_gradients_of_fewer_rows(M):
    big, g = Gated("mxfp4", 700, 272, 2112, 16, seed=4), Gated("mxfp4", M, 272, 2112, 16, seed=4)
    H, G, U, T = g.fwd("gelu")
    want = g.bwd("gelu", G, U, T)
    g.ws = big.ws
    got = g.bwd("gelu", G, U, T)
    g.ok()
    for x, y in zip(want, got):
        assert_close(to_f64(y), to_f64(x), "gradient")


def test_offsets_past_32_bits():
    """More than 2^31 elements in the widest tensors: the last rows are those of a call on them alone."""
    from bit_quantized_base_b200 import qlora as Q
    M, N, K, r, n, s = 140000, 16384, 64, 8, 300, 2.0
    small = Gated("mxfp4", n, N, K, r, seed=6)
    X = torch.randn(M, K, device="cuda").to(BF)
    dH = torch.randn(M, N, dtype=BF, device="cuda")
    H, G, U = (torch.empty(M, N, dtype=BF, device="cuda") for _ in range(3))
    T, dX = torch.empty(2, M, r, dtype=BF, device="cuda"), nan(M, K)
    outs = nan(r, K), nan(N, r), nan(r, K), nan(N, r)
    ws = Q.alloc_workspace(Q.OP_GATED_MLP_BWD, small.Wg, M, r)
    Q.qlora_gated_mlp_fwd(small.Wg, small.Wu, "silu", X, *small.ad, H, G, U, T, M, r, s, ws)
    Q.qlora_gated_mlp_bwd(small.Wg, small.Wu, "silu", X, *small.ad, T, G, U, dH, dX, *outs, M, r, s, ws)
    torch.cuda.synchronize()
    assert Q.qlora_get_device_status(ws) == 0
    x, dh, t = X[M - n:].clone(), dH[M - n:].clone(), T[:, M - n:].clone()
    g, u = G[M - n:].clone(), U[M - n:].clone()
    h2, g2, u2, t2, dx2 = nan(n, N), nan(n, N), nan(n, N), nan(2, n, r), nan(n, K)
    Q.qlora_gated_mlp_fwd(small.Wg, small.Wu, "silu", x, *small.ad, h2, g2, u2, t2, n, r, s, small.ws)
    Q.qlora_gated_mlp_bwd(small.Wg, small.Wu, "silu", x, *small.ad, t, g, u, dh, dx2, nan(r, K), nan(N, r),
                          nan(r, K), nan(N, r), n, r, s, small.ws)
    small.ok()
    for name, a, b in (("H", H[M - n:], h2), ("G", g, g2), ("U", u, u2), ("T", t, t2), ("dX", dX[M - n:], dx2)):
        assert_close(to_f64(a), to_f64(b), name)
    for o in outs:
        assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("M", [1, 2, 5, 16, 77])
def test_few_rows_lose_no_precision_in_the_adapter_gradients(M):
    """dA of few rows: U = dU B is only M r values, so a rounding of dU is not averaged out.  dU enters U in two
    bf16 terms and U enters dA in two (2^-17 each), so dA is off by its own rounding alone: a relative
    Frobenius error of at most 2^-8 / sqrt(3) (uniform within half a step of the smallest of a binade) plus
    1e-4 for those terms and the binary32 activations."""
    bound = 2.0 ** -8 / np.sqrt(3) + 1e-4
    for seed in range(6):
        fmt, act = ("nf4", "mxfp4", "nvfp4")[seed % 3], R.ACTS[seed % 3 + 1]
        g = Gated(fmt, M, 528, 192, 8, seed=40 + seed)
        H, G, U, T = g.fwd(act)
        dX, dAg, dBg, dAu, dBu = g.bwd(act, G, U, T)
        l = Linear(fmt, M, 528, 192, 8, seed=40 + seed)
        Y, Z, T1 = l.fwd(act)
        dX1, dA, dB, db = l.bwd(act, Z, T1)
        g.ok()
        l.ok()
        a, da = R.act(act, to_f64(G))
        dH, X = R.f64(g.pg["dY"]), R.f64(g.pg["X"])
        dZ = R.f64(l.p["dY"]) * R.act(act, to_f64(Z))[1]
        for name, got, p, d, x in (("dAg", dAg, g.pg, dH * to_f64(U) * da, X), ("dAu", dAu, g.pu, dH * a, X),
                                   ("dA", dA, l.p, dZ, R.f64(l.p["X"]))):
            ref = p["s"] * ((d @ R.f64(p["B"])).T @ x)
            err = np.linalg.norm(to_f64(got) - ref) / np.linalg.norm(ref)
            assert err <= bound, (name, seed, err)
