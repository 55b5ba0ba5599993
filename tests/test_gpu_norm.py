"""GPU parity of the RMS norm with the residual's addition, and of its gradients.

Reference: the formulas in binary64 (numpy / torch on the CPU).  Tolerances: an output rounded once
to bf16 is off by at most 2^-8 of its value; binary32 arithmetic in front of that rounding adds
at most a few 2^-24 of the sum of the magnitudes that enter it.  The MXFP8 output is compared
bit for bit."""
import numpy as np
import pytest
import torch

from oracle import oracle as O

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
EPS = 1e-5


def round_bf16(x):
    """The nearest bf16 value of each binary64 value, ties to even."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 256.0), e - 8)


def bits(x):
    """bf16-representable float64 -> bf16 bit patterns."""
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def bf16(rng, shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(BF)


def f64(t):
    return t.double().cpu().numpy()


def reference(X, R, gamma, eps=EPS):
    S = f64(X) if R is None else round_bf16(f64(X) + f64(R))
    rstd = 1.0 / np.sqrt((S * S).mean(axis=1) + eps)
    g = 1.0 if gamma is None else f64(gamma)[None, :]
    return S, rstd, S * rstd[:, None] * g


def close(got, ref, slack, name):
    err = np.abs(f64(got) - ref)
    bound = 2.0 ** -8 * np.abs(ref) + slack
    bad = ~(err <= bound)
    assert not bad.any(), f"{name}: {bad.sum()} outside, worst {np.max(err / np.maximum(bound, 1e-300))}"


SHAPES = [(1, 8), (1, 4096), (3, 64), (5, 1000), (2, 32768), (37, 7168), (700, 40), (1500, 1024), (601, 4096),
          (4, 28672)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_forward(M, K, res):
    from bit_quantized_base_b200 import qlora as Q
    rng = np.random.default_rng(M * 31 + K + res)
    X, R = bf16(rng, (M, K)), bf16(rng, (M, K), 2.0) if res else None
    gamma = bf16(rng, (K,)) if K % 64 else None
    if M > 2:
        X[1] = 0                                    # a row of zeros
        if res:
            R[1] = 0
    S64, rstd64, Y64 = reference(X, R, gamma)
    Y = torch.full((M, K), float("nan"), dtype=BF, device="cuda")
    S = torch.full((M, K), float("nan"), dtype=BF, device="cuda") if res else None
    rstd = torch.full((M,), float("nan"), device="cuda")
    Q.qlora_rmsnorm_fwd(X.cuda(), R.cuda() if res else None, None if gamma is None else gamma.cuda(), EPS, S, Y,
                        None, None, rstd, M, K)
    torch.cuda.synchronize()
    if res:
        assert np.array_equal(f64(S), S64)
    assert np.all(np.abs(f64(rstd) / rstd64 - 1) <= 2.0 ** -22)
    close(Y, Y64, 2.0 ** -21 * np.abs(Y64), "Y")


@pytest.mark.parametrize("M,K", [(1, 32), (1, 4096), (3, 96), (130, 2048), (37, 7168), (2, 32768), (1000, 1024)])
def test_mxfp8_output_is_bit_exact(M, K):
    from bit_quantized_base_b200 import qlora as Q
    rng = np.random.default_rng(M + K)
    X, R, gamma = bf16(rng, (M, K)), bf16(rng, (M, K), 2.0), bf16(rng, (K,))
    gamma[: min(K, 32)] = 0                          # blocks of zeros
    _, _, Y64 = reference(X, R, gamma)
    yb = bits(round_bf16(Y64))
    want_y = torch.from_numpy(yb.view(np.int16)).view(BF).reshape(M, K)
    args = (X.cuda(), R.cuda(), gamma.cuda(), EPS)
    codes = torch.full((M, K), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((M, K // 32), 0xEE, dtype=torch.uint8, device="cuda")
    Y = torch.empty((M, K), dtype=BF, device="cuda")
    Q.qlora_rmsnorm_fwd(*args, None, Y, codes, scales, None, M, K)
    torch.cuda.synchronize()
    assert torch.equal(Y.cpu().view(torch.int16) & 0x7FFF, want_y.view(torch.int16) & 0x7FFF)
    if K % 128 == 0:                                 # the library's own quantiser on the same Y
        c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
        Q.qlora_mxfp8_quantize(Y, M, K, c2, s2)
        torch.cuda.synchronize()
        assert torch.equal(codes, c2) and torch.equal(scales, s2)
        oc, os_ = O.mxfp8_quantize(round_bf16(Y64))
        assert np.array_equal(codes.cpu().numpy(), oc) and np.array_equal(scales.cpu().numpy(), os_)
    c3, s3 = torch.empty_like(codes), torch.empty_like(scales)     # without Y: the same codes
    Q.qlora_rmsnorm_fwd(*args, None, None, c3, s3, None, M, K)
    torch.cuda.synchronize()
    assert torch.equal(codes, c3) and torch.equal(scales, s3)


def grads64(S, rstd, gamma, dY, dS_in):
    g = 1.0 if gamma is None else f64(gamma)[None, :]
    v, K = g * dY, S.shape[1]
    c = (v * S).mean(axis=1, keepdims=True)
    r = rstd[:, None]
    dS = r * (v - S * r * r * c)
    mag = r * (np.abs(v) + np.abs(S) * r * r * (np.abs(v * S).mean(axis=1, keepdims=True)))
    if dS_in is not None:
        dS, mag = dS + dS_in, mag + np.abs(dS_in)
    t = dY * S * r
    return dS, mag, t.sum(axis=0), np.abs(t).sum(axis=0)


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("res,dg", [(True, True), (False, False), (True, False), (False, True)])
def test_backward(M, K, res, dg):
    from bit_quantized_base_b200 import qlora as Q
    rng = np.random.default_rng(M * 7 + K + 2 * res + dg)
    S, dY = bf16(rng, (M, K), 2.0), bf16(rng, (M, K), 0.1)
    dS_in = bf16(rng, (M, K), 0.1) if res else None
    gamma = bf16(rng, (K,)) if dg or K % 64 else None
    rstd64 = 1.0 / np.sqrt((f64(S) ** 2).mean(axis=1) + EPS)
    rstd32 = torch.from_numpy(rstd64.astype(np.float32))
    want, mag, dgam, dgmag = grads64(f64(S), f64(rstd32), gamma, f64(dY), None if dS_in is None else f64(dS_in))
    ws = torch.full((Q.qlora_rmsnorm_workspace_size(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    cu = lambda t: None if t is None else t.cuda()      # noqa: E731
    outs = []
    for give in (rstd32.cuda(), None):
        dS = torch.full((M, K), float("nan"), dtype=BF, device="cuda")
        dgamma = torch.full((K,), float("nan"), dtype=BF, device="cuda") if dg else None
        Q.qlora_rmsnorm_bwd(S.cuda(), give, cu(gamma), EPS, dY.cuda(), cu(dS_in), dS, dgamma, M, K,
                            ws if dg else None)
        torch.cuda.synchronize()
        # dot products of K terms in binary32 (at most 32 per thread, then a tree of 10 levels)
        close(dS, want, 48 * 2.0 ** -24 * mag, "dS")
        if dg:
            close(dgamma, dgam, (M + 32) * 2.0 ** -24 * dgmag, "dgamma")
        outs.append((dS, dgamma))
    again = torch.empty_like(outs[1][0])                 # deterministic
    dg2 = torch.empty_like(outs[1][1]) if dg else None
    Q.qlora_rmsnorm_bwd(S.cuda(), None, cu(gamma), EPS, dY.cuda(), cu(dS_in), again, dg2, M, K, ws if dg else None)
    torch.cuda.synchronize()
    assert torch.equal(again, outs[1][0]) and (not dg or torch.equal(dg2, outs[1][1]))


def test_gradient_against_differences():
    # L = <C, Y(S)> + <D, S> in binary64: the library's dS and dgamma against central differences
    from bit_quantized_base_b200 import qlora as Q
    M, K, h = 3, 64, 1e-5
    rng = np.random.default_rng(5)
    S, C, D, gamma = bf16(rng, (M, K)), bf16(rng, (M, K)), bf16(rng, (M, K)), bf16(rng, (K,))

    def loss(s, g):
        return float((f64(C) * (s / np.sqrt((s * s).mean(axis=1, keepdims=True) + EPS) * g)).sum() + (f64(D) * s).sum())

    s0, g0 = f64(S), f64(gamma)
    num_s, num_g = np.empty_like(s0), np.empty_like(g0)
    for i in range(M):
        for k in range(K):
            a, b = s0.copy(), s0.copy()
            a[i, k] += h
            b[i, k] -= h
            num_s[i, k] = (loss(a, g0) - loss(b, g0)) / (2 * h)
    for k in range(K):
        a, b = g0.copy(), g0.copy()
        a[k] += h
        b[k] -= h
        num_g[k] = (loss(s0, a) - loss(s0, b)) / (2 * h)
    dS, dgamma = torch.empty((M, K), dtype=BF, device="cuda"), torch.empty(K, dtype=BF, device="cuda")
    ws = torch.empty(Q.qlora_rmsnorm_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    Q.qlora_rmsnorm_bwd(S.cuda(), None, gamma.cuda(), EPS, C.cuda(), D.cuda(), dS, dgamma, M, K, ws)
    torch.cuda.synchronize()
    close(dS, num_s, 1e-6, "dS")          # differences: h^2 and 1e-16 / h errors, both below 1e-6
    close(dgamma, num_g, 1e-6, "dgamma")


def test_in_place_and_empty():
    from bit_quantized_base_b200 import qlora as Q
    M, K = 67, 1024
    rng = np.random.default_rng(9)
    X, R, dY = bf16(rng, (M, K)).cuda(), bf16(rng, (M, K)).cuda(), bf16(rng, (M, K)).cuda()
    S, Y = torch.empty_like(X), torch.empty_like(X)
    Q.qlora_rmsnorm_fwd(X, R, None, EPS, S, Y, None, None, None, M, K)
    X2, R2 = X.clone(), R.clone()
    Q.qlora_rmsnorm_fwd(X2, R2, None, EPS, R2, X2, None, None, None, M, K)   # S over R, Y over X
    torch.cuda.synchronize()
    assert torch.equal(R2, S) and torch.equal(X2, Y)
    dS = torch.empty_like(X)
    Q.qlora_rmsnorm_bwd(S, None, None, EPS, dY, R, dS, None, M, K)
    for over in range(3):
        b = [S.clone(), dY.clone(), R.clone()]
        Q.qlora_rmsnorm_bwd(b[0], None, None, EPS, b[1], b[2], b[over], None, M, K)
        torch.cuda.synchronize()
        assert torch.equal(b[over], dS), over
    # M = 0: nothing but a zero dgamma
    dgamma = torch.full((K,), float("nan"), dtype=BF, device="cuda")
    empty = torch.empty((0, K), dtype=BF, device="cuda")
    Q.qlora_rmsnorm_fwd(empty, None, None, EPS, None, empty, None, None, None, 0, K)
    ws = torch.empty(Q.qlora_rmsnorm_workspace_size(0, K), dtype=torch.uint8, device="cuda")
    Q.qlora_rmsnorm_bwd(empty, None, None, EPS, empty, None, empty, dgamma, 0, K, ws)
    torch.cuda.synchronize()
    assert torch.equal(dgamma, torch.zeros_like(dgamma))


def test_outputs_leave_their_surroundings_alone():
    from bit_quantized_base_b200 import qlora as Q
    M, K = 5, 1000
    rng = np.random.default_rng(2)
    X = bf16(rng, (M, K)).cuda()
    buf = torch.full((M + 2, K), 7.0, dtype=BF, device="cuda")
    Q.qlora_rmsnorm_fwd(X, None, None, EPS, None, buf[1:M + 1], None, None, None, M, K)
    torch.cuda.synchronize()
    assert torch.all(buf[0] == 7) and torch.all(buf[M + 1] == 7)


def test_captured_and_on_another_stream():
    from bit_quantized_base_b200 import qlora as Q
    M, K = 300, 2048
    rng = np.random.default_rng(3)
    X, R, gamma = bf16(rng, (M, K)).cuda(), bf16(rng, (M, K)).cuda(), bf16(rng, (K,)).cuda()
    want = torch.empty_like(X)
    Q.qlora_rmsnorm_fwd(X, R, gamma, EPS, None, want, None, None, None, M, K)

    S, Y, dS = (torch.empty_like(X) for _ in range(3))
    dgamma = torch.empty(K, dtype=BF, device="cuda")
    ws = torch.empty(Q.qlora_rmsnorm_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        Q.qlora_rmsnorm_fwd(X, R, gamma, EPS, S, Y, None, None, None, M, K)
        Q.qlora_rmsnorm_bwd(S, None, gamma, EPS, Y, None, dS, dgamma, M, K, ws)
    Y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)
    d1, g1 = dS.clone(), dgamma.clone()
    X.mul_(2)                                        # new inputs in the same buffers
    g.replay()
    Q.qlora_rmsnorm_fwd(X, R, gamma, EPS, None, want, None, None, None, M, K)
    torch.cuda.synchronize()
    assert torch.equal(Y, want) and not torch.equal(dS, d1) and not torch.equal(dgamma, g1)
    with torch.cuda.stream(st):                      # the current stream of the caller is used
        Y.zero_()
        Q.qlora_rmsnorm_fwd(X, R, gamma, EPS, None, Y, None, None, None, M, K)
    st.synchronize()
    assert torch.equal(Y, want)


def test_w4a8_takes_the_norm_s_codes():
    from bit_quantized_base_b200 import qlora as Q, synth
    M, N, K, r = 130, 256, 512, 16
    p = synth.small_layer("mxfp4", M, N, K, r, seed=4)
    W = Q.weight_from_numpy("mxfp4", p["codes"], p["scales"])
    X, A, B = (Q.bf16_from_bits(p[k]) for k in ("X", "A", "B"))
    Yn = torch.empty((M, K), dtype=BF, device="cuda")
    codes = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty((M, K // 32), dtype=torch.uint8, device="cuda")
    Q.qlora_rmsnorm_fwd(X, None, None, EPS, None, Yn, codes, scales, None, M, K)
    ws = Q.alloc_workspace(Q.OP_FWD_W4A8, W, M, r)
    out = [torch.empty((M, N), dtype=BF, device="cuda") for _ in range(2)]
    T = [torch.empty((M, r), dtype=BF, device="cuda") for _ in range(2)]
    Q.qlora_linear_fwd_w4a8(W, Yn, A, B, out[0], T[0], M, r, 2.0, ws)
    Q.qlora_linear_fwd_w4a8_codes(W, Yn, codes, scales, A, B, out[1], T[1], M, r, 2.0, ws)
    torch.cuda.synchronize()
    assert Q.qlora_get_device_status(ws) == 0
    assert torch.equal(out[0], out[1]) and torch.equal(T[0], T[1])


@pytest.mark.parametrize("M,K", [(1, 512), (3, 96), (600, 40), (593, 4096)])
def test_gain_gradient_without_epsilon_and_rstd(M, K):
    """eps = 0 with rstd recomputed: the row slots behind the last row add nothing to dgamma."""
    from bit_quantized_base_b200 import qlora as Q
    rng = np.random.default_rng(M + K)
    S, dY = bf16(rng, (M, K)), bf16(rng, (M, K))
    g = bf16(rng, (K,))
    dS, dg = torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(K, dtype=BF, device="cuda")
    ws = torch.zeros(Q.qlora_rmsnorm_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    Q.qlora_rmsnorm_bwd(S.cuda(), None, g.cuda(), 0.0, dY.cuda(), None, dS, dg, M, K, ws)
    torch.cuda.synchronize()
    rstd = 1.0 / np.sqrt((f64(S) ** 2).mean(axis=1))
    terms = f64(dY) * f64(S) * rstd[:, None]
    # binary32 sums of at most M terms, each with a few roundings of its own
    close(dg, terms.sum(axis=0), (M + 16) * 2.0 ** -24 * np.abs(terms).sum(axis=0), "dgamma")


@pytest.mark.parametrize("M,K", [(64, 1024), (700, 1024), (40, 4096), (640, 8192), (3, 32768)])
def test_mxfp8_products_over_a_wide_range(M, K):
    """With codes wanted, Y is the definition's value rounded once, for rows and gains of any magnitude:
    equal to the rounded binary64 value, but for values within 2^-40 of a border of two bf16 values."""
    from bit_quantized_base_b200 import qlora as Q
    rng = np.random.default_rng(M + K)
    X = rng.standard_normal((M, K)) * 2.0 ** rng.integers(-50, 51, (M, 1)) * 2.0 ** rng.integers(-6, 7, (M, K))
    X[rng.random((M, K)) < 0.01] = 0.0
    g = rng.standard_normal(K) * 2.0 ** rng.integers(-20, 21, K)
    X, g = (torch.from_numpy(t.astype(np.float32)).to(BF) for t in (X, g))
    Y, R = torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(M, dtype=torch.float32, device="cuda")
    C, E = (torch.empty(M, k, dtype=torch.uint8, device="cuda") for k in (K, K // 32))
    Q.qlora_rmsnorm_fwd(X.cuda(), None, g.cuda(), 0.0, None, Y, C, E, R, M, K)
    C2, E2 = torch.empty_like(C), torch.empty_like(E)
    Q.qlora_mxfp8_quantize(Y, M, K, C2, E2)
    torch.cuda.synchronize()
    x = f64(X)
    ref = x / np.sqrt((x * x).mean(axis=1, keepdims=True)) * f64(g)[None, :]
    m, e = np.frexp(ref)
    frac = np.abs(m * 256.0 - np.floor(m * 256.0) - 0.5)
    sure = (frac > 2.0 ** -32) & ((np.abs(ref) > 2.0 ** -100) | (ref == 0))
    assert sure.mean() > 0.999
    assert np.array_equal(f64(Y)[sure], round_bf16(ref)[sure])
    assert torch.equal(C, C2) and torch.equal(E, E2)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are those of a call on them alone."""
    from bit_quantized_base_b200 import qlora as Q
    M, K, n = 66000, 32768, 16
    X = torch.randn(M, K, dtype=BF, device="cuda")
    g = torch.randn(K, device="cuda").to(BF)
    rstd = torch.empty(M, dtype=torch.float32, device="cuda")
    Y, dS = torch.empty_like(X), torch.empty_like(X)
    Q.qlora_rmsnorm_fwd(X, None, g, EPS, None, Y, None, None, rstd, M, K)
    Q.qlora_rmsnorm_bwd(X, rstd, g, EPS, Y, X, dS, None, M, K, None)
    x = X[M - n:].clone()
    y, ds, rs = torch.empty_like(x), torch.empty_like(x), torch.empty(n, dtype=torch.float32, device="cuda")
    Q.qlora_rmsnorm_fwd(x, None, g, EPS, None, y, None, None, rs, n, K)
    Q.qlora_rmsnorm_bwd(x, rs, g, EPS, y, x, ds, None, n, K, None)
    torch.cuda.synchronize()
    for a, b in ((Y[M - n:], y), (dS[M - n:], ds), (rstd[M - n:], rs)):
        assert torch.equal(a, b)
