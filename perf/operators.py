"""Workloads of the MLP-block operators of the 4-bit-base LoRA library.

A decoder layer's MLP block on a frozen 4-bit base is  S = X + R,  Y = rmsnorm(S),
H = act(gate(Y)) * up(Y),  out = down(H) + S,  each projection a LoRA layer on its 4-bit weight.
The operators measured here are its parts and their gradients:

  norm_fwd   S = bf16(X + R); rstd = (mean S^2 + eps)^-1/2; Y = S rstd gamma, written as bf16 or as
             MXFP8 (E4M3 codes and one E8M0 scale per 32, of the Y rounded to bf16)
  norm_bwd   dS = dS_in + rstd (gamma dY - S rstd^2 mean(gamma dY S)),  dgamma = sum_m dY S rstd
  gated_fwd  H = act(G) * U,  G = X Wg^T + s (X Ag^T) Bg^T,  U the same with the up projection
  gated_bwd  dG = dH U act'(G), dU = dH act(G); dX and the four adapter gradients
  act_fwd    Y = act(Z) + residual,  Z = X W^T + s (X A^T) B^T + bias
  act_bwd    dZ = dY act'(Z); dX, dA, dB, dbias

With `own` false `run` computes them from elementary torch operations in 32 bits, rounded once at
the end; with `own` true it makes the library's calls.  `exact` restates them in 64 bits.
Sizes are those of the 8B and 70B decoder layers and of the mixture-of-experts projections that
the benchmark uses, cut down where a single pass would be long.
"""
import math

import torch

own = False

# ----------------------------------------------------------------------------------- cases


def listed():
    return [
        # one new token through the norm in front of the MLP block: pure latency
        dict(name="norm_fwd_token", op="norm_fwd", M=1, K=4096, residual=True, out="bf16", save=False),
        # a prefill or training batch whose norm feeds the block-scaled W4A8 projections
        dict(name="norm_fwd_mxfp8", op="norm_fwd", M=4096, K=8192, residual=True, out="mxfp8", save=True),
        # training step, long batch: the gradient through the norm joined with the residual path's
        dict(name="norm_bwd_long", op="norm_bwd", M=16384, K=4096, residual=True, dgamma=True),
        # a ragged micro-batch at the width of the expert projections, the norm's gain frozen
        dict(name="norm_bwd_ragged", op="norm_bwd", M=517, K=7168, residual=True, dgamma=False),
        # decoding: one token through gate and up of the 8B layer, nothing saved
        dict(name="gated_fwd_token", op="gated_fwd", fmt="nf4", M=1, N=14336, K=4096, r=64, act="silu", save=False),
        # a handful of sequences decoded together through an expert-sized block
        dict(name="gated_fwd_batch33", op="gated_fwd", fmt="nvfp4", M=33, N=2048, K=7168, r=16, act="silu", save=False),
        # training forward of the 8B block, pre-activations kept for the backward pass
        dict(name="gated_fwd_train", op="gated_fwd", fmt="nf4", M=4096, N=14336, K=4096, r=64, act="silu", save=True),
        # a short ragged micro-batch's gradient
        dict(name="gated_bwd_short", op="gated_bwd", fmt="mxfp4", M=77, N=2048, K=7168, r=8, act="gelu_tanh"),
        # training backward of the 8B block
        dict(name="gated_bwd_train", op="gated_bwd", fmt="nf4", M=4096, N=14336, K=4096, r=64, act="silu"),
        # decoding: one token through the 8B down projection, added to the residual stream
        dict(name="act_fwd_token", op="act_fwd", fmt="nvfp4", M=1, N=4096, K=14336, r=16, act="none", bias=False, residual=True, save=False),
        # the 70B down projection of a training batch, added to the residual stream
        dict(name="act_fwd_down", op="act_fwd", fmt="nvfp4", M=2048, N=8192, K=28672, r=16, act="none", bias=False, residual=True, save=False),
        # an odd batch's gradient through a projection with bias and an activation behind it
        dict(name="act_bwd_gelu", op="act_bwd", fmt="mxfp4", M=1021, N=8192, K=2048, r=16, act="gelu", bias=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "gated_fwd", "gated_fwd", "gated_bwd", "gated_bwd", "act_fwd", "act_bwd"])
    if op in ("norm_fwd", "norm_bwd"):
        K = _log(rng, 64, 28672, 32)
        M = _log(rng, 1, max(1, min(32768, (1 << 25) // K)))
        if op == "norm_fwd":
            out = rng.choice(["bf16", "mxfp8"])
            if out == "mxfp8":
                K = max(128, K // 128 * 128)
            return dict(op=op, M=M, K=K, residual=rng.random() < 0.7, out=out, save=rng.random() < 0.5)
        return dict(op=op, M=M, K=K, residual=rng.random() < 0.7, dgamma=rng.random() < 0.5)
    fmt = rng.choice(["nf4", "nf4dq", "mxfp4", "nvfp4"])
    N, K = _log(rng, 256, 14336, 16), _log(rng, 256, 8192, 64)
    r = rng.choice([8, 16, 32, 64])
    act = rng.choice(["none", "silu", "silu", "gelu", "gelu_tanh"])
    # up to a fifth of the largest listed case's products
    M = _log(rng, 1, max(1, min(4096, int(4.5e10) // (N * K))))
    case = dict(op=op, fmt=fmt, M=M, N=N, K=K, r=r, act=act)
    if op == "gated_fwd":
        case["save"] = rng.random() < 0.5
    if op == "act_fwd":
        case.update(bias=rng.random() < 0.5, residual=rng.random() < 0.7, save=rng.random() < 0.5)
    if op == "act_bwd":
        case["bias"] = rng.random() < 0.5
    return case


EPS = 1e-5
BLOCK = {"nf4": 64, "nf4dq": 64, "mxfp4": 32, "nvfp4": 16}
SCALE = 2.0      # alpha / r

# The 16 NF4 levels (quantiles of the standard normal, normalised to [-1, 1]).
NF4 = [-1.0, -0.6961928009986877, -0.5250729322433472, -0.39491742849349976, -0.2844413220882416,
       -0.18477340042591095, -0.09104997664690018, 0.0, 0.07958031445741653, 0.16093014180660248,
       0.24611225724220276, 0.3379151225090027, 0.4407097399234772, 0.5626168847084045,
       0.722956657409668, 1.0]
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ---------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _normal(g, shape, std):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _nearest(v, grid):
    grid = torch.tensor(grid, device="cuda")
    return torch.bucketize(v, (grid[1:] + grid[:-1]) * 0.5)


def _e2m1_code(v):
    mag = _nearest(v.abs().clamp(max=6.0), E2M1[:8])
    return mag + 8 * ((v < 0) & (mag > 0))


def _weight(g, fmt, N, K):
    """A frozen weight as it is stored: N(0, 0.02) quantised block by block."""
    v = torch.randn((N, K), generator=g, device="cuda") * 0.02
    bs = BLOCK[fmt]
    b = v.view(N, K // bs, bs)
    amax = b.abs().amax(dim=2)
    w = dict(fmt=fmt, N=N, K=K, tensor_scale=None, scales2=None)
    if fmt in ("nf4", "nf4dq"):
        scale = amax
        if fmt == "nf4dq":       # E4M3 absmax codes times one fp32 scale per 256 blocks
            flat = amax.reshape(-1)
            groups = (flat.numel() + 255) // 256
            pad = torch.zeros(groups * 256, device="cuda")
            pad[: flat.numel()] = flat
            w["scales2"] = pad.view(groups, 256).amax(dim=1) / 448.0
            per = w["scales2"].repeat_interleave(256)[: flat.numel()].view_as(amax)
            c1 = (amax / per).to(torch.float8_e4m3fn)
            scale = c1.float() * per
            w["scales"] = c1.view(torch.uint8)
        else:
            w["scales"] = scale.contiguous()
        codes = _nearest((b / scale[:, :, None].clamp(min=1e-30)).clamp(-1, 1), NF4)
    elif fmt == "mxfp4":
        e = torch.floor(torch.log2(amax.clamp(min=1e-30))) - 2
        codes = _e2m1_code(b / torch.exp2(e)[:, :, None])
        w["scales"] = (e + 127).to(torch.uint8)
    else:
        ts = v.abs().max() / 2688.0
        c = (amax / (6.0 * ts)).to(torch.float8_e4m3fn)
        codes = _e2m1_code(b / (c.float() * ts)[:, :, None].clamp(min=1e-30))
        w["scales"], w["tensor_scale"] = c.view(torch.uint8), ts.reshape(1).clone()
    codes = codes.to(torch.uint8).view(N, K // 2, 2)
    w["codes"] = (codes[:, :, 0] | (codes[:, :, 1] << 4)).contiguous()
    return w


def _adapter(g, N, K, r):
    bound = 1.0 / math.sqrt(K)
    A = ((torch.rand((r, K), generator=g, device="cuda") * 2 - 1) * bound).to(torch.bfloat16)
    return A, _normal(g, (N, r), 0.01)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    M, K, op = c["M"], c["K"], c["op"]
    s = dict(case=c)
    if op == "norm_fwd":
        s["X"] = _normal(g, (M, K), 1.0)
        s["R"] = _normal(g, (M, K), 2.0) if c["residual"] else None
        s["gamma"] = (1.0 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
    elif op == "norm_bwd":
        s["S"] = _normal(g, (M, K), 2.0)
        s["gamma"] = (1.0 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
        s["rstd"] = (s["S"].double().square().mean(dim=1) + EPS).rsqrt().float()
        s["dY"] = _normal(g, (M, K), 0.01)
        s["dS_in"] = _normal(g, (M, K), 0.01) if c["residual"] else None
    else:
        N, r, fmt = c["N"], c["r"], c["fmt"]
        names = ("g", "u") if op.startswith("gated") else ("",)
        s["X"] = _normal(g, (M, K), 1.0)
        for n in names:
            s["W" + n] = _weight(g, fmt, N, K)
            s["A" + n], s["B" + n] = _adapter(g, N, K, r)
        if op == "gated_bwd":       # what the forward kept: pre-activations of unit size, T = X A^T
            s["G"], s["U"] = _normal(g, (M, N), 1.3), _normal(g, (M, N), 1.3)
            s["T"] = torch.stack([(s["X"].float() @ s["A" + n].float().t()).to(torch.bfloat16) for n in names])
            s["dH"] = _normal(g, (M, N), 0.01)
        if op == "act_fwd":
            s["bias"] = _normal(g, (N,), 0.5) if c["bias"] else None
            s["residual"] = _normal(g, (M, N), 1.0) if c["residual"] else None
        if op == "act_bwd":
            s["Z"] = _normal(g, (M, N), 1.3) if c["act"] != "none" else None
            s["T"] = (s["X"].float() @ s["A"].float().t()).to(torch.bfloat16)
            s["dY"] = _normal(g, (M, N), 0.01)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The buffers and handles that a program keeps: outputs, workspace, weight structs."""
    from bit_quantized_base_b200 import qlora as Q
    c, o = s["case"], {}
    M, K, op = c["M"], c["K"], c["op"]

    def bf(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda")

    if op == "norm_fwd":
        o["S"] = bf(M, K) if c["residual"] else None
        o["Y"] = bf(M, K) if c["out"] == "bf16" else None
        mx = c["out"] == "mxfp8"
        o["codes"] = torch.empty((M, K), dtype=torch.uint8, device="cuda") if mx else None
        o["scales"] = torch.empty((M, K // 32), dtype=torch.uint8, device="cuda") if mx else None
        o["rstd"] = torch.empty(M, device="cuda") if c["save"] else None
    elif op == "norm_bwd":
        o["dS"] = bf(M, K)
        o["dgamma"] = bf(K) if c["dgamma"] else None
        o["ws"] = torch.zeros(Q.qlora_rmsnorm_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    else:
        N, r = c["N"], c["r"]
        for n in ("Wg", "Wu", "W"):
            if n in s:
                w = s[n]
                s["h" + n] = Q.Weight(w["fmt"], N, K, w["codes"], w["scales"], w["tensor_scale"], w["scales2"])
        code = {"gated_fwd": Q.OP_GATED_MLP_FWD, "gated_bwd": Q.OP_GATED_MLP_BWD, "act_fwd": Q.OP_ACT_FWD,
                "act_bwd": Q.OP_ACT_BWD}[op]
        o["ws"] = Q.alloc_workspace(code, s["hWg"] if "hWg" in s else s["hW"], M, r)
        if op == "gated_fwd":
            o["H"] = bf(M, N)
            o["G"], o["U"], o["T"] = (bf(M, N), bf(M, N), bf(2, M, r)) if c["save"] else (None, None, None)
        elif op == "gated_bwd":
            o.update(dX=bf(M, K), dAg=bf(r, K), dBg=bf(N, r), dAu=bf(r, K), dBu=bf(N, r))
        elif op == "act_fwd":
            o["Y"] = bf(M, N)
            o["Z"] = bf(M, N) if c["save"] and c["act"] != "none" else None
            o["T"] = bf(M, r) if c["save"] else None
        else:
            o.update(dX=bf(M, K), dA=bf(r, K), dB=bf(N, r), dbias=bf(N) if c["bias"] else None)
    s["out"] = o


# ------------------------------------------------------------------- plain form, in 32 bits
def _decode(w, dtype=torch.float32):
    """deq(W) [N, K]: each element rounded to bf16 as the format defines it (NVFP4: the tensor
    scale multiplies the rounded block product, as it multiplies the accumulated products)."""
    codes = torch.stack([w["codes"] & 15, w["codes"] >> 4], dim=2).view(w["N"], w["K"]).to(torch.int32)
    bs = BLOCK[w["fmt"]]
    if w["fmt"] in ("nf4", "nf4dq"):
        scale = w["scales"]
        if w["fmt"] == "nf4dq":
            c1 = scale.view(torch.float8_e4m3fn).float()
            scale = c1 * w["scales2"].repeat_interleave(256)[: c1.numel()].view_as(c1)
        v = torch.tensor(NF4, device="cuda")[codes].view(w["N"], -1, bs) * scale[:, :, None]
    elif w["fmt"] == "mxfp4":
        v = torch.tensor(E2M1, device="cuda")[codes].view(w["N"], -1, bs) * (w["scales"].to(torch.int32) << 23).view(torch.float32)[:, :, None]
    else:
        v = torch.tensor(E2M1, device="cuda")[codes].view(w["N"], -1, bs) * w["scales"].view(torch.float8_e4m3fn).float()[:, :, None]
    v = v.to(torch.bfloat16).to(dtype)
    if w["fmt"] == "nvfp4":
        v = v * w["tensor_scale"].to(dtype)
    return v.view(w["N"], w["K"])


def _act(name, z):
    if name == "none":
        return z
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_grad(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _mxfp8(y):
    """E4M3 codes and E8M0 scales of a bf16 tensor: the shared exponent is floor(log2 amax) - 8."""
    b = y.float().view(y.shape[0], -1, 32)
    amax = b.abs().amax(dim=2)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - 8, -127).clamp(-127, 127)
    q = (b * ((127 - e.to(torch.int32)) << 23).view(torch.float32)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    q = torch.where(q.float() == 0, 0.0, q.float()).to(torch.float8_e4m3fn)
    scales = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return q.view(y.shape), scales


def _plain(s):
    c = s["case"]
    op = c["op"]
    bf = torch.bfloat16
    if op == "norm_fwd":
        S = s["X"] if s["R"] is None else (s["X"].float() + s["R"].float()).to(bf)
        f = S.float()
        rstd = 1 / torch.sqrt((f * f).mean(dim=1, keepdim=True) + EPS)
        y = (f * rstd * s["gamma"].float()).to(bf)
        out = {"S": None if s["R"] is None else S, "rstd": rstd[:, 0] if c["save"] else None}
        if c["out"] == "bf16":
            out["Y"] = y
        else:
            out["codes"], out["scales"] = _mxfp8(y)
        return out
    if op == "norm_bwd":
        S, dY, rstd = s["S"].float(), s["dY"].float(), s["rstd"][:, None]
        gd = dY * s["gamma"].float()
        dS = rstd * (gd - S * rstd * rstd * (gd * S).mean(dim=1, keepdim=True))
        if s["dS_in"] is not None:
            dS = dS + s["dS_in"].float()
        return {"dS": dS.to(bf), "dgamma": (dY * S * rstd).sum(dim=0).to(bf) if c["dgamma"] else None}
    X = s["X"].float()
    if op == "gated_fwd":
        z, T = [], []
        for n in ("g", "u"):
            T.append(X @ s["A" + n].float().t())
            z.append(X @ _decode(s["W" + n]).t() + SCALE * (T[-1] @ s["B" + n].float().t()))
        out = {"H": (_act(c["act"], z[0]) * z[1]).to(bf)}
        if c["save"]:
            out.update(G=z[0].to(bf), U=z[1].to(bf), T=torch.stack(T).to(bf))
        return out
    if op == "gated_bwd":
        dH, G, U = s["dH"].float(), s["G"].float(), s["U"].float()
        grads = {"g": dH * U * _act_grad(c["act"], G), "u": dH * _act(c["act"], G)}
        out, dX = {}, 0
        for i, n in enumerate(("g", "u")):
            d, A, B = grads[n], s["A" + n].float(), s["B" + n].float()
            u = d @ B
            dX = dX + d @ _decode(s["W" + n]) + SCALE * (u @ A)
            out["dA" + n] = (SCALE * (u.t() @ X)).to(bf)
            out["dB" + n] = (SCALE * (d.t() @ s["T"][i].float())).to(bf)
        out["dX"] = dX.to(bf)
        return out
    if op == "act_fwd":
        T = X @ s["A"].float().t()
        z = X @ _decode(s["W"]).t() + SCALE * (T @ s["B"].float().t())
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(c["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        keep = c["save"] and c["act"] != "none"
        return {"Y": y.to(bf), "Z": z.to(bf) if keep else None, "T": T.to(bf) if c["save"] else None}
    d = s["dY"].float()
    if c["act"] != "none":
        d = d * _act_grad(c["act"], s["Z"].float())
    A, B = s["A"].float(), s["B"].float()
    u = d @ B
    return {"dX": (d @ _decode(s["W"]) + SCALE * (u @ A)).to(bf), "dA": (SCALE * (u.t() @ X)).to(bf),
            "dB": (SCALE * (d.t() @ s["T"].float())).to(bf), "dbias": d.sum(dim=0).to(bf) if c["bias"] else None}


# ----------------------------------------------------------------------- the library's calls
def _library(s):
    from bit_quantized_base_b200 import qlora as Q
    c, o = s["case"], s["out"]
    M, K, op = c["M"], c["K"], c["op"]
    if op == "norm_fwd":
        Q.qlora_rmsnorm_fwd(s["X"], s["R"], s["gamma"], EPS, o["S"], o["Y"], o["codes"], o["scales"], o["rstd"], M, K)
        out = {"S": o["S"], "rstd": o["rstd"]}
        if c["out"] == "bf16":
            out["Y"] = o["Y"]
        else:            # the stored bytes, read as the 8-bit floats they are
            out["codes"] = o["codes"].view(torch.float8_e4m3fn)
            out["scales"] = o["scales"].view(torch.float8_e8m0fnu)
        return out
    if op == "norm_bwd":
        Q.qlora_rmsnorm_bwd(s["S"], s["rstd"], s["gamma"], EPS, s["dY"], s["dS_in"], o["dS"], o["dgamma"], M, K, o["ws"])
        return {"dS": o["dS"], "dgamma": o["dgamma"]}
    r, act = c["r"], c["act"]
    if op == "gated_fwd":
        Q.qlora_gated_mlp_fwd(s["hWg"], s["hWu"], act, s["X"], s["Ag"], s["Bg"], s["Au"], s["Bu"], o["H"], o["G"],
                              o["U"], o["T"], M, r, SCALE, o["ws"])
        return {k: o[k] for k in (("H", "G", "U", "T") if c["save"] else ("H",))}
    if op == "gated_bwd":
        Q.qlora_gated_mlp_bwd(s["hWg"], s["hWu"], act, s["X"], s["Ag"], s["Bg"], s["Au"], s["Bu"], s["T"], s["G"],
                              s["U"], s["dH"], o["dX"], o["dAg"], o["dBg"], o["dAu"], o["dBu"], M, r, SCALE, o["ws"])
        return {k: o[k] for k in ("dX", "dAg", "dBg", "dAu", "dBu")}
    if op == "act_fwd":
        Q.qlora_linear_act_fwd(s["hW"], s["X"], s["A"], s["B"], s["bias"], act, s["residual"], o["Y"], o["Z"], o["T"],
                               M, r, SCALE, o["ws"])
        return {k: o[k] for k in ("Y", "Z", "T")}
    Q.qlora_linear_act_bwd(s["hW"], s["X"], s["A"], s["B"], s["T"], s["Z"], act, s["dY"], o["dX"], o["dA"], o["dB"],
                           o["dbias"], M, r, SCALE, o["ws"])
    return {k: o[k] for k in ("dX", "dA", "dB", "dbias")}


def run(state):
    return _library(state) if own else _plain(state)


# ----------------------------------------------------------------------------------- work
def _weight_bytes(fmt, N, K):
    return N * K // 2 + N * K // BLOCK[fmt] * (4 if fmt == "nf4" else 1)


def work(case):
    c = case
    M, K, op = c["M"], c["K"], c["op"]
    if op == "norm_fwd":
        b = 2 * M * K * (3 if c["residual"] else 1) + 2 * K + (4 * M if c["save"] else 0)
        b += 2 * M * K if c["out"] == "bf16" else M * K + M * K // 32
        return {"bytes": b, "flops": 5 * M * K}
    if op == "norm_bwd":
        b = 2 * M * K * (4 if c["residual"] else 3) + 2 * K + 4 * M + (2 * K if c["dgamma"] else 0)
        return {"bytes": b, "flops": 9 * M * K}
    N, r = c["N"], c["r"]
    n = 2 if op.startswith("gated") else 1
    weights = n * (_weight_bytes(c["fmt"], N, K) + 2 * r * (N + K))
    base, lora = 2 * M * N * K * n, 2 * M * r * (N + K) * n
    if op == "gated_fwd":
        return {"bytes": weights + 2 * M * K + 2 * M * N * (3 if c["save"] else 1) + (4 * M * r if c["save"] else 0),
                "flops": base + lora}
    if op == "act_fwd":
        rows = 1 + (1 if c["residual"] else 0) + (1 if c["save"] and c["act"] != "none" else 0)
        return {"bytes": weights + 2 * M * K + 2 * M * N * rows + (2 * N if c["bias"] else 0) + (2 * M * r if c["save"] else 0),
                "flops": base + lora}
    rows = 3 if n == 2 else 1 + (1 if c["act"] != "none" else 0)
    return {"bytes": weights + 2 * M * K * 2 + 2 * M * N * rows + 2 * M * r * n + n * 2 * r * (N + K) + (2 * N if c.get("bias") else 0),
            "flops": base + 2 * lora}


# --------------------------------------------------------------------- 64-bit restatement
def _pow2(e):
    """2^e in 64 bits, exactly (e an integer tensor in the normal range)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_bf16(x):
    """The nearest bf16 value of each double (8 significant bits, ties to even; normal range)."""
    m, e = torch.frexp(x)
    return torch.round(m * 256.0) * _pow2(e - 8)


def _weight64(w):
    """deq(W) from the stored bytes, element by element, in 64 bits."""
    N, K, fmt = w["N"], w["K"], w["fmt"]
    n = torch.empty((N, K), dtype=torch.uint8, device="cuda")
    n[:, 0::2] = w["codes"].bitwise_and(15)
    n[:, 1::2] = w["codes"].bitwise_right_shift(4)

    def e4m3(b):
        b = b.to(torch.int64)
        e, m = (b >> 3) & 15, (b & 7).double()
        v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _pow2(e - 7))
        return torch.where(b >= 128, -v, v)

    if fmt in ("nf4", "nf4dq"):
        if fmt == "nf4":
            a = w["scales"].double()
        else:            # the absmax is formed in binary32
            flat = torch.arange(N * (K // 64), device="cuda") // 256
            a = (e4m3(w["scales"]).reshape(-1) * w["scales2"].double()[flat]).float().double().view(N, -1)
        out = torch.empty((N, K), dtype=torch.float64, device="cuda")
        levels = torch.tensor(NF4, device="cuda").double()
        for k in range(K // 64):       # the product is a binary32 one, then bf16
            p = (levels[n[:, 64 * k: 64 * k + 64].long()] * a[:, k: k + 1]).float().double()
            out[:, 64 * k: 64 * k + 64] = _round_bf16(p)
        return out
    n = n.long()
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _pow2(e - 1))
    v = torch.where(n >= 8, -v, v)
    if fmt == "mxfp4":
        return (v.view(N, -1, 32) * _pow2(w["scales"].to(torch.int64) - 127)[:, :, None]).view(N, K)
    return (v.view(N, -1, 16) * e4m3(w["scales"])[:, :, None]).view(N, K) * w["tensor_scale"].double()


def _sigmoid64(x):
    return torch.where(x >= 0, 1 / (1 + torch.exp(-x.abs())), torch.exp(-x.abs()) / (1 + torch.exp(-x.abs())))


def _act64(name, z):
    """(act(z), act'(z)) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "silu":
        p = _sigmoid64(z)
        return z * p, p + z * p * _sigmoid64(-z)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) * 0.3989422804014326779
    inner = 2 * 0.7978845608028653559 * (z + 0.044715 * z ** 3)     # 0.5 (1 + tanh u) = sigmoid(2 u)
    p = _sigmoid64(inner)
    return z * p, p + z * p * _sigmoid64(-inner) * 2 * 0.7978845608028653559 * (1 + 0.134145 * z * z)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        S = s["X"].double()
        if s["R"] is not None:
            S = _round_bf16(S + s["R"].double())
        rstd = ((S ** 2).sum(dim=1) / c["K"] + EPS) ** -0.5
        Y = S * rstd[:, None] * s["gamma"].double()
        out = {"S": S if s["R"] is not None else None, "rstd": rstd if c["save"] else None}
        if c["out"] == "bf16":
            out["Y"] = Y
            return out
        b = _round_bf16(Y).view(c["M"], -1, 32)
        top = b.abs().amax(dim=2)
        e = torch.where(top > 0, torch.frexp(top)[1] - 9, -127).clamp(-127, 127)
        v = b / _pow2(e)[:, :, None]
        step = _pow2(torch.frexp(v.abs().clamp(min=2.0 ** -6))[1] - 4)
        out["codes"] = (torch.round(v / step) * step).clamp(-448, 448).view(c["M"], c["K"])
        out["scales"] = _pow2(e)
        return out
    if op == "norm_bwd":
        S, dY, gamma, r = s["S"].double(), s["dY"].double(), s["gamma"].double(), s["rstd"].double()
        xhat = S * r[:, None]
        v = gamma * dY
        dS = r[:, None] * (v - xhat * ((v * xhat).sum(dim=1) / c["K"])[:, None])
        if s["dS_in"] is not None:
            dS = dS + s["dS_in"].double()
        return {"dS": dS, "dgamma": torch.einsum("mk,mk->k", dY, xhat) if c["dgamma"] else None}
    X = s["X"].double()

    def layer(n):
        T = X @ s["A" + n].double().T
        return X @ _weight64(s["W" + n]).T + (SCALE * T) @ s["B" + n].double().T, T

    def layer_grad(n, d, T):
        u = d @ s["B" + n].double()
        return d @ _weight64(s["W" + n]) + (SCALE * u) @ s["A" + n].double(), SCALE * (u.T @ X), SCALE * (d.T @ T.double())

    if op == "gated_fwd":
        (G, Tg), (U, Tu) = layer("g"), layer("u")
        out = {"H": _act64(c["act"], G)[0] * U}
        if c["save"]:
            out.update(G=G, U=U, T=torch.stack([Tg, Tu]))
        return out
    if op == "gated_bwd":
        a, da = _act64(c["act"], s["G"].double())
        dH = s["dH"].double()
        xg, dAg, dBg = layer_grad("g", dH * s["U"].double() * da, s["T"][0])
        xu, dAu, dBu = layer_grad("u", dH * a, s["T"][1])
        return {"dX": xg + xu, "dAg": dAg, "dBg": dBg, "dAu": dAu, "dBu": dBu}
    if op == "act_fwd":
        Z, T = layer("")
        if s["bias"] is not None:
            Z = Z + s["bias"].double()
        Y = _act64(c["act"], Z)[0]
        if s["residual"] is not None:
            Y = Y + s["residual"].double()
        return {"Y": Y, "Z": Z if c["save"] and c["act"] != "none" else None, "T": T if c["save"] else None}
    d = s["dY"].double()
    if c["act"] != "none":
        d = d * _act64(c["act"], s["Z"].double())[1]
    dX, dA, dB = layer_grad("", d, s["T"])
    return {"dX": dX, "dA": dA, "dB": dB, "dbias": d.sum(dim=0) if c["bias"] else None}
