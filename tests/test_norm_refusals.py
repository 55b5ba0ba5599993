"""Argument checks of the RMS norm entry points and of the W4A8 forward on stored codes: refused on
the host before anything is enqueued (no GPU needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def Q():
    from bit_quantized_base_b200 import build
    build.build()
    from bit_quantized_base_b200 import qlora
    return qlora


FWD = dict(X=0x10000, R=None, gamma=None, eps=1e-5, S=None, Y=0x20000, codes=None, scales=None, rstd=None, M=4, K=64)


@pytest.mark.parametrize("change,status", [
    (dict(X=None), "INVALID_ARG"), (dict(X=0x10008), "INVALID_ARG"), (dict(Y=None), "INVALID_ARG"),
    (dict(Y=0x20002), "INVALID_ARG"), (dict(R=0x30004), "INVALID_ARG"), (dict(gamma=0x30002), "INVALID_ARG"),
    (dict(S=0x40000), "INVALID_ARG"),                       # S without R
    (dict(codes=0x50000), "INVALID_ARG"), (dict(scales=0x60000), "INVALID_ARG"),
    (dict(codes=0x50000, scales=0x60000, K=72), "INVALID_ARG"),
    (dict(K=0), "INVALID_ARG"), (dict(K=12), "INVALID_ARG"), (dict(K=32776), "UNSUPPORTED"),
    (dict(M=-1), "INVALID_ARG"), (dict(M=(1 << 31)), "INVALID_ARG"), (dict(eps=-1e-5), "INVALID_ARG"),
    (dict(eps=float("nan")), "INVALID_ARG"), (dict(eps=float("inf")), "INVALID_ARG"),
])
def test_forward(Q, change, status):
    a = dict(FWD, **change)
    rc = Q.lib.qlora_rmsnorm_fwd(a["X"], a["R"], a["gamma"], a["eps"], a["S"], a["Y"], a["codes"], a["scales"],
                                 a["rstd"], a["M"], a["K"], None)
    assert Q.STATUS[rc] == "QLORA_ERR_" + status


BWD = dict(S=0x10000, rstd=None, gamma=None, eps=1e-5, dY=0x20000, dS_in=None, dS=0x30000, dgamma=None, M=4, K=64,
           ws=None, n=0)


@pytest.mark.parametrize("change,status", [
    (dict(S=None), "INVALID_ARG"), (dict(dY=None), "INVALID_ARG"), (dict(dS=None), "INVALID_ARG"),
    (dict(dS=0x30004), "INVALID_ARG"), (dict(dS_in=0x40002), "INVALID_ARG"), (dict(rstd=0x40004), "INVALID_ARG"),
    (dict(dgamma=0x50000), "WORKSPACE"), (dict(dgamma=0x50000, ws=0x60000, n=64), "WORKSPACE"),
    (dict(dgamma=0x50000, ws=0x60008, n=1 << 30), "WORKSPACE"), (dict(K=12), "INVALID_ARG"),
    (dict(K=40000), "UNSUPPORTED"), (dict(eps=-1.0), "INVALID_ARG"), (dict(M=-3), "INVALID_ARG"),
])
def test_backward(Q, change, status):
    a = dict(BWD, **change)
    rc = Q.lib.qlora_rmsnorm_bwd(a["S"], a["rstd"], a["gamma"], a["eps"], a["dY"], a["dS_in"], a["dS"], a["dgamma"],
                                 a["M"], a["K"], a["ws"], a["n"], None)
    assert Q.STATUS[rc] == "QLORA_ERR_" + status


def test_workspace_size(Q):
    assert Q.qlora_rmsnorm_workspace_size(0, 64) > 0
    assert Q.qlora_rmsnorm_workspace_size(4096, 4096) >= 4096 * 4
    assert Q.qlora_rmsnorm_workspace_size(-1, 64) == 0
    assert Q.qlora_rmsnorm_workspace_size(4, 12) == 0
    assert Q.qlora_rmsnorm_workspace_size(4, 40000) == 0


def test_binding_refuses_tensors_that_are_not_what_the_call_reads(Q):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)            # on the host
    with pytest.raises(Q.QLoraError):
        Q.qlora_rmsnorm_fwd(x, None, None, 1e-5, None, x.clone(), None, None, None, 4, 64)
    with pytest.raises(Q.QLoraError):
        Q.qlora_rmsnorm_fwd(None, None, None, 1e-5, None, None, None, None, None, 4, 64)
    with pytest.raises(Q.QLoraError):
        Q.qlora_rmsnorm_bwd(x, None, None, 1e-5, x, None, x.clone(), None, 4, 64)


def test_w4a8_codes(Q):
    W = Q.Weight.__new__(Q.Weight)
    W.c = Q.qlora_weight_t(Q.FMT["mxfp4"], 0, 256, 512, 0x1000, 0x2000, None)

    def call(xc, xs, M=64, ws=0x50000, n=1 << 30):
        import ctypes
        return Q.STATUS[Q.lib.qlora_linear_fwd_w4a8_codes(ctypes.byref(W.c), 0x10000, xc, xs, 0x20000, 0x30000, 0x40000,
                                                          None, M, 16, 2.0, ws, n, None)]
    assert call(None, 0x70000) == "QLORA_ERR_INVALID_ARG"
    assert call(0x70000, None) == "QLORA_ERR_INVALID_ARG"
    assert call(0x70004, 0x80000) == "QLORA_ERR_INVALID_ARG"
    assert call(0x70000, 0x80000, ws=None) == "QLORA_ERR_WORKSPACE"
    assert call(None, None, M=0) == "QLORA_OK"


def test_sum_and_output_in_one_buffer(Q):
    a = dict(FWD, R=0x30000, S=0x20000)                      # S is Y's buffer
    rc = Q.lib.qlora_rmsnorm_fwd(a["X"], a["R"], a["gamma"], a["eps"], a["S"], a["Y"], a["codes"], a["scales"],
                                 a["rstd"], a["M"], a["K"], None)
    assert Q.STATUS[rc] == "QLORA_ERR_INVALID_ARG"
