"""Argument checks of the gated MLP and of the linear layer with an epilogue: refused on the host before
anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def Q():
    from bit_quantized_base_b200 import build
    build.build()
    from bit_quantized_base_b200 import qlora
    return qlora


def weight(Q, fmt="nf4", N=256, K=512, codes=0x1000, ts=None):
    return Q.qlora_weight_t(Q.FMT[fmt], 0, N, K, codes, 0x2000, ts)


BIG = 1 << 34
GATED_F = dict(act=1, X=0x10000, Ag=0x20000, Bg=0x30000, Au=0x40000, Bu=0x50000, H=0x60000, G=None, U=None, T=None,
               M=64, r=16, ws=0x70000, n=BIG)
GATED_B = dict(act=1, X=0x10000, Ag=0x20000, Bg=0x30000, Au=0x40000, Bu=0x50000, T=None, G=0x60000, U=0x61000,
               dH=0x62000, dX=None, dAg=0x63000, dBg=0x64000, dAu=0x65000, dBu=0x66000, M=64, r=16, ws=0x70000, n=BIG)
ACT_F = dict(X=0x10000, A=0x20000, B=0x30000, bias=None, act=1, res=None, Y=0x40000, Z=None, T=None, M=64, r=16,
             ws=0x70000, n=BIG)
ACT_B = dict(X=0x10000, A=0x20000, B=0x30000, T=None, Z=0x31000, act=1, dY=0x40000, dX=None, dA=0x50000, dB=0x60000,
             dbias=None, M=64, r=16, ws=0x70000, n=BIG)


def call(Q, fn, weights, a):
    w = [ctypes.byref(x) if x is not None else None for x in weights]
    vals = [v for k, v in a.items() if k not in ("M", "r", "ws", "n")]
    return Q.STATUS[getattr(Q.lib, fn)(*w, *vals, a["M"], a["r"], 2.0, a["ws"], a["n"], None)][len("QLORA_ERR_"):]


COMMON = [(dict(act=4), "INVALID_ARG"), (dict(act=-1), "INVALID_ARG"), (dict(X=None), "INVALID_ARG"),
          (dict(X=0x10008), "INVALID_ARG"), (dict(M=-1), "INVALID_ARG"), (dict(M=1 << 31), "INVALID_ARG"),
          (dict(r=12), "UNSUPPORTED"), (dict(r=0), "INVALID_ARG"), (dict(ws=None), "WORKSPACE"),
          (dict(ws=0x70008), "WORKSPACE"), (dict(n=8192), "WORKSPACE")]


@pytest.mark.parametrize("change,status", COMMON + [(dict([(k, None)]), "INVALID_ARG") for k in ("Ag", "Bg", "Au", "Bu", "H")]
                         + [(dict([(k, 0x60004)]), "INVALID_ARG") for k in ("Ag", "Bu", "H", "G", "U", "T")])
def test_gated_forward(Q, change, status):
    assert call(Q, "qlora_gated_mlp_fwd", (weight(Q), weight(Q)), dict(GATED_F, **change)) == status


@pytest.mark.parametrize("change,status", COMMON + [(dict([(k, None)]), "INVALID_ARG")
                                                    for k in ("Ag", "Bu", "G", "U", "dH", "dAg", "dBg", "dAu", "dBu")]
                         + [(dict([(k, 0x60004)]), "INVALID_ARG") for k in ("T", "G", "dH", "dX", "dBu")])
def test_gated_backward(Q, change, status):
    assert call(Q, "qlora_gated_mlp_bwd", (weight(Q), weight(Q)), dict(GATED_B, **change)) == status


@pytest.mark.parametrize("wg,wu,status", [
    (dict(), dict(N=272), "INVALID_ARG"), (dict(), dict(K=576), "INVALID_ARG"), (dict(), dict(fmt="mxfp4"), "UNSUPPORTED"),
    (dict(codes=0x1008), dict(), "INVALID_ARG"), (dict(), dict(codes=None), "INVALID_ARG"),
    (dict(fmt="nvfp4", ts=0x3000), dict(fmt="nvfp4"), "INVALID_ARG"), (dict(N=40), dict(N=40), "INVALID_ARG")])
def test_gated_weights(Q, wg, wu, status):
    for fn, a in (("qlora_gated_mlp_fwd", GATED_F), ("qlora_gated_mlp_bwd", GATED_B)):
        assert call(Q, fn, (weight(Q, **wg), weight(Q, **wu)), a) == status
        assert call(Q, fn, (weight(Q, **wg), None), a) == "INVALID_ARG"


@pytest.mark.parametrize("change,status", COMMON + [(dict([(k, None)]), "INVALID_ARG") for k in ("A", "B", "Y")]
                         + [(dict([(k, 0x60004)]), "INVALID_ARG") for k in ("A", "bias", "res", "Y", "Z", "T")])
def test_act_forward(Q, change, status):
    assert call(Q, "qlora_linear_act_fwd", (weight(Q),), dict(ACT_F, **change)) == status


@pytest.mark.parametrize("change,status", COMMON + [(dict([(k, None)]), "INVALID_ARG") for k in ("A", "B", "Z", "dY", "dA", "dB")]
                         + [(dict([(k, 0x60004)]), "INVALID_ARG") for k in ("T", "Z", "dY", "dX", "dA", "dbias")])
def test_act_backward(Q, change, status):
    assert call(Q, "qlora_linear_act_bwd", (weight(Q),), dict(ACT_B, **change)) == status


def test_workspace_sizes(Q):
    W = Q.Weight.__new__(Q.Weight)
    W.c = weight(Q)
    for op in (Q.OP_GATED_MLP_FWD, Q.OP_GATED_MLP_BWD, Q.OP_ACT_FWD, Q.OP_ACT_BWD):
        assert Q.qlora_workspace_size(op, W, 100, 16) >= 8192
        assert Q.qlora_workspace_size(op, W, 100, 12) == 0
        assert Q.qlora_workspace_size(op, W, -1, 16) == 0
    assert Q.qlora_workspace_size(Q.OP_GATED_MLP_BWD, W, 100, 16) >= Q.qlora_workspace_size(Q.OP_GATED_MLP_FWD, W, 100, 16)
    assert Q.qlora_workspace_size(Q.OP_ACT_BWD, W, 100, 16) >= Q.qlora_workspace_size(Q.OP_BWD, W, 100, 16)
    assert Q.qlora_workspace_size(9, W, 100, 16) == 0


def test_binding_refuses_host_tensors_and_unknown_names(Q):
    W = Q.Weight.__new__(Q.Weight)
    W.c, W.N, W.K = weight(Q), 256, 512
    x, ad, y = (torch.zeros(s, dtype=torch.bfloat16) for s in ((64, 512), (16, 512), (64, 256)))
    b = torch.zeros((256, 16), dtype=torch.bfloat16)
    with pytest.raises(Q.QLoraError):
        Q.qlora_linear_act_fwd(W, x, ad, b, None, "silu", None, y, None, None, 64, 16, 2.0, None)
    with pytest.raises(Q.QLoraError):
        Q.qlora_gated_mlp_fwd(W, W, "silu", x, ad, b, ad, b, y, None, None, None, 64, 16, 2.0, None)
    with pytest.raises(KeyError):
        Q._act("swish9")
