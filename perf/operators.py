"""Measured cases of the 8-bit activation checkpoints and of the norm step.

Four operators of the library (all tensors on the GPU, tokens flattened to N):

  checkpoint           checkpoint_save then checkpoint_load: bf16 rows to MXFP8 codes and block
                       scales and back, the values a backward pass gets to see.
  step_backward        fused_step_backward_ckpt: the gradients of the fused multi-stream step from
                       checkpoints of its X and F.
  norm_step            a block's output normalised, gated and scaled, added to the residual streams,
                       and the norm of the next block's input.
  norm_step_backward   its gradients, from bf16 X and F or from their checkpoints.

`run` computes them from elementary torch operations in float32; with `own` set, by the library's
calls. `exact` restates the definitions in float64.
"""
import math

import torch

own = False

BLOCK = 32              # features per checkpoint block
MIX = 24                # mix numbers of a 4-stream token
EPS = 1e-6


# ----------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # the saved streams of one odd-sized microbatch: rows whose last block is short
        dict(name="ckpt_ragged", op="checkpoint", rows=4 * 1031, d=1000),
        # the streams of the B=4, T=8192 workload, saved once a sublayer
        dict(name="ckpt_prefill32k", op="checkpoint", rows=4 * 32768, d=5120),
        # the B=1, T=8 workload: launches and weight traffic, hardly any tokens
        dict(name="step_bwd_tiny", op="step_backward", N=8, d=5120, iters=20, row_dest=False),
        # a ragged microbatch of a narrower model, the other reading of comb
        dict(name="step_bwd_ragged", op="step_backward", N=1333, d=2560, iters=20, row_dest=True),
        # the training step of the B=4, T=8192 workload
        dict(name="step_bwd_prefill32k", op="step_backward", N=32768, d=5120, iters=20, row_dest=False),
        # one token of one request
        dict(name="norm_decode1", op="norm_step", N=1, n=4, d=5120, gate="none", post_norm=True,
             shared=False, row_dest=False, scale=1.0),
        # the decode batch of 256
        dict(name="norm_decode256", op="norm_step", N=256, n=4, d=5120, gate="sigmoid", post_norm=True,
             shared=False, row_dest=False, scale=0.5),
        # a plain residual model of an odd width, ragged tokens
        dict(name="norm_plain_ragged", op="norm_step", N=4099, n=1, d=1992, gate="sigmoid", post_norm=True,
             shared=False, row_dest=False, scale=0.22),
        # the B=4, T=8192 prefill
        dict(name="norm_prefill32k", op="norm_step", N=32768, n=4, d=5120, gate="linear", post_norm=True,
             shared=False, row_dest=False, scale=1.0),
        # a microbatch of 8 tokens from checkpoints
        dict(name="norm_bwd_tiny_ckpt", op="norm_step_backward", N=8, n=4, d=5120, gate="sigmoid",
             post_norm=True, shared=False, row_dest=False, scale=1.0, ckpt=True),
        # the plain residual model's backward
        dict(name="norm_bwd_plain_ragged", op="norm_step_backward", N=4099, n=1, d=1992, gate="sigmoid",
             post_norm=True, shared=False, row_dest=False, scale=0.22, ckpt=False),
        # a long training microbatch of four streams with weights shared by all tokens
        dict(name="norm_bwd_train16k", op="norm_step_backward", N=16384, n=4, d=5120, gate="linear",
             post_norm=True, shared=True, row_dest=False, scale=1.0, ckpt=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["checkpoint", "step_backward", "norm_step", "norm_step_backward"])
    if op == "checkpoint":
        d = 8 * _log(rng, 1, 1024)
        return dict(op=op, rows=min(_log(rng, 1, 131072), 131072 * 5120 // d), d=d)
    if op == "step_backward":
        # widths the step takes: 128 to 640 columns for each of 1 to 32 CTAs
        d = 64 * rng.randint(2, 10) * 2 ** rng.randint(0, 3)
        return dict(op=op, N=min(_log(rng, 1, 32768), 32768 * 5120 // (2 * d)), d=d,
                    iters=rng.choice([1, 3, 20]), row_dest=rng.random() < 0.5)
    n = rng.choice([1, 4])
    d = 8 * _log(rng, 8, 1024)
    case = dict(op=op, N=min(_log(rng, 1, 16384), 16384 * 5120 // d), n=n, d=d,
                gate=rng.choice(["none", "linear", "sigmoid"]), post_norm=rng.random() < 0.75,
                shared=rng.random() < 0.3, row_dest=rng.random() < 0.3,
                scale=rng.choice([1.0, 0.5, 0.22]))
    if op == "norm_step_backward":
        case["ckpt"] = rng.random() < 0.5
    return case


# ----------------------------------------------------------------------------------------------
# inputs


def _encode(x):
    """MXFP8 codes and scale codes of bf16 rows [..., d] (uint8), as a training program holds them."""
    d = x.shape[-1]
    pad = -d % BLOCK
    v = torch.nn.functional.pad(x.float(), (0, pad)).view(*x.shape[:-1], -1, BLOCK)
    amax = v.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 1 - 8 + 127).clamp_min(0)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    q = torch.ldexp(v, (127 - e)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    codes = q.view(torch.uint8).view(*x.shape[:-1], d + pad)[..., :d].contiguous()
    return codes, e.to(torch.uint8).contiguous()


def _decode(codes, scale):
    """float32 values of codes [..., d] with scale codes [..., ceil(d / 32)]."""
    d = codes.shape[-1]
    s = torch.exp2(scale.float() - 127.0).repeat_interleave(BLOCK, -1)[..., :d]
    return codes.view(torch.float8_e4m3fn).float() * s


def _weights(shape, gen, n):
    """Stream weights as a trained block has them: reading and writing weights, and a combination
    near the identity whose columns sum to about one."""
    dev = torch.device("cuda")
    pre = torch.rand(*shape, n, generator=gen, device=dev)
    post = 2 * torch.rand(*shape, n, generator=gen, device=dev)
    comb = torch.rand(*shape, n, n, generator=gen, device=dev) + 2 * torch.eye(n, device=dev)
    return pre, post, comb / comb.sum(-2, keepdim=True)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def streams(N, n, d):
        # streams of different sizes, a few features far larger than the rest, one quiet token
        x = normal(N, n, d).mul_(0.5 + torch.rand(n, 1, generator=gen, device="cuda"))
        x[..., torch.randint(0, d, (max(1, d // 512),), generator=gen, device="cuda")] *= 30.0
        x[N // 2] *= 1e-3
        return x.bfloat16()

    st = dict(case)
    if case["op"] == "checkpoint":
        st["x"] = streams(case["rows"], 1, case["d"])[:, 0].contiguous()
        return st
    N, d = case["N"], case["d"]
    n = case.get("n", 4)
    X = streams(N, n, d)
    F = normal(N, d).bfloat16()
    st["gXp"], st["gy"] = normal(N, n, d).bfloat16(), normal(N, d).bfloat16()
    if case["op"] == "step_backward":
        pre, post, comb = _weights((N,), gen, 4)
        st.update(pre=pre, post=post, comb=comb, W=0.02 * normal(MIX, 4 * d), base=normal(MIX),
                  sc=0.5 + 1.5 * torch.rand(3, generator=gen, device="cuda"),
                  gain=1.0 + 0.1 * normal(d), gpre=normal(N, 4), gpost=normal(N, 4),
                  gcomb=normal(N, 4, 4))
        Xp = _post(X.float(), F.float(), post, comb, case["row_dest"]).bfloat16().float().view(N, -1)
        st["mixes"] = ((Xp @ st["W"].T) * torch.rsqrt(Xp.square().mean(1, keepdim=True) + EPS)).contiguous()
        del Xp
    else:
        given = n == 4 or case["shared"]
        pre, post, comb = _weights(() if case["shared"] else (N,), gen, n) if given else (None,) * 3
        st.update(pre=pre, post=post, comb=comb, case_gate=case["gate"],
                  gate=None if case["gate"] == "none" else normal(N, d).bfloat16(),
                  gain_post=1.0 + 0.1 * normal(d) if case["post_norm"] else None,
                  gain_pre=1.0 + 0.1 * normal(d))
    if case["op"] == "step_backward" or case.get("ckpt"):
        st["X_codes"], st["X_scale"] = _encode(X)
        st["F_codes"], st["F_scale"] = _encode(F)
    else:
        st["X"], st["F"] = X, F
    return st


# ----------------------------------------------------------------------------------------------
# the plain forms


def _post(X, F, post, comb, row_dest):
    """X'_k = u_k F + sum_j C_jk X_j, each product and sum rounded to float32, in stream order."""
    C = comb.transpose(1, 2) if row_dest else comb
    s = X[:, 0, None] * C[:, 0, :, None]
    s = s + X[:, 1, None] * C[:, 1, :, None]
    s = s + X[:, 2, None] * C[:, 2, :, None]
    s = s + X[:, 3, None] * C[:, 3, :, None]
    return post[:, :, None] * F[:, None] + s


def _plain_step_backward(st):
    N, d, iters = st["N"], st["d"], st["iters"]
    K = 4 * d
    X, F = _decode(st["X_codes"], st["X_scale"]), _decode(st["F_codes"], st["F_scale"])
    p, m, s, b = st["pre"], st["mixes"], st["sc"], st["base"]
    # the streams and the block input are bf16 tensors
    Xp = _post(X, F, st["post"], st["comb"], st["row_dest"]).bfloat16().float()
    yh = p[:, 0, None] * Xp[:, 0]
    yh = yh + p[:, 1, None] * Xp[:, 1]
    yh = yh + p[:, 2, None] * Xp[:, 2]
    yh = (yh + p[:, 3, None] * Xp[:, 3]).bfloat16().float()
    # split, softmax and the normalisation rounds, walked back
    zp, zu = torch.sigmoid(s[0] * m[:, :4] + b[:4]), torch.sigmoid(s[1] * m[:, 4:8] + b[4:8])
    gzp = st["gpre"] * zp * (1 - zp)
    gzu = 2 * st["gpost"] * zu * (1 - zu)
    L = (s[2] * m[:, 8:] + b[8:]).view(N, 4, 4)
    e = torch.exp(L - L.amax(2, keepdim=True))
    sm = e / e.sum(2, keepdim=True)
    c, tape = sm + EPS, []
    for i in range(2 * iters - 1):
        t = c.sum(1 + i % 2, keepdim=True) + EPS
        tape.append((c, t))
        c = c / t
    g = st["gcomb"]
    for i in reversed(range(2 * iters - 1)):
        c, t = tape[i]
        g = g / t - (g * c).sum(1 + i % 2, keepdim=True) / (t * t)
    gL = (sm * (g - (g * sm).sum(2, keepdim=True))).view(N, 16)
    gz = torch.cat([gzp, gzu, gL], 1)
    gs = torch.stack([(gzp * m[:, :4]).sum(), (gzu * m[:, 4:8]).sum(), (gL * m[:, 8:]).sum()])
    gm = torch.cat([s[0] * gzp, s[1] * gzu, s[2] * gL], 1)
    # projection and its scale, norm, streams
    x = Xp.view(N, K)
    r = torch.rsqrt(x.square().mean(1) + EPS)
    ga = gm * r[:, None]
    gW = ga.T @ x
    G = (ga @ st["W"]).view(N, 4, d)
    G -= Xp * (r * r / K * (gm * m).sum(1))[:, None, None]
    ry = torch.rsqrt(yh.square().mean(1) + EPS)
    gy = st["gy"].float()
    ggain = (gy * yh * ry[:, None]).sum(0)
    T = (st["gain"] * gy * yh).sum(1)
    gyh = (ry[:, None] * st["gain"]) * gy - yh * (ry ** 3 * T / d)[:, None]
    gp = (gyh[:, None] * Xp).sum(2)
    del Xp, x
    G += st["gXp"]
    G += p[:, :, None] * gyh[:, None]
    C = st["comb"].transpose(1, 2) if st["row_dest"] else st["comb"]
    gF = (st["post"][:, :, None] * G).sum(1)
    gu = (G * F[:, None]).sum(2)
    gC = torch.bmm(X, G.transpose(1, 2))
    gX = torch.bmm(C, G)
    if st["row_dest"]:
        gC = gC.transpose(1, 2).contiguous()
    return dict(gX=gX.bfloat16(), gF=gF.bfloat16(), gpre_prev=gp, gpost_prev=gu, gcomb_prev=gC, gW=gW,
                gbase=gz.sum(0), gscale=gs, ggain=ggain)


def _gate(st):
    """(the gate's values, its derivative) or (1, None)."""
    if st["gate"] is None:
        return 1.0, None
    g = st["gate"].float()
    if st["case_gate"] == "linear":
        return g, 1.0
    a = torch.sigmoid(g)
    return a, a * (1 - a)


def _norm_forward(st, X, F):
    n = st["n"]
    r = torch.rsqrt(F.square().mean(1, keepdim=True) + EPS) if st["post_norm"] else 1.0
    gain = st["gain_post"] if st["post_norm"] else 1.0
    a, da = _gate(st)
    h = st["scale"] * a * gain
    Z = h * F * r
    if st["pre"] is None:
        return r, gain, a, da, h, Z, X + Z[:, None], None
    C = st["comb"].expand(X.shape[0], n, n)
    C = C if st["row_dest"] else C.transpose(1, 2)
    Xp = torch.bmm(C, X) + st["post"][..., None] * Z[:, None]
    return r, gain, a, da, h, Z, Xp, C


def _plain_norm_step(st):
    Xp = _norm_forward(st, st["X"].float(), st["F"].float())[6]
    yh = Xp[:, 0] if st["pre"] is None else (st["pre"][..., None] * Xp).sum(1)
    y = st["gain_pre"] * yh * torch.rsqrt(yh.square().mean(1, keepdim=True) + EPS)
    return dict(Xp=Xp.bfloat16(), y=y.bfloat16())


def _plain_norm_step_backward(st):
    if st["ckpt"]:
        X, F = _decode(st["X_codes"], st["X_scale"]), _decode(st["F_codes"], st["F_scale"])
    else:
        X, F = st["X"].float(), st["F"].float()
    d = st["d"]
    r, gain, a, da, h, Z, Xp, C = _norm_forward(st, X, F)
    yh = Xp[:, 0] if C is None else (st["pre"][..., None] * Xp).sum(1)
    ry = torch.rsqrt(yh.square().mean(1, keepdim=True) + EPS)
    gy = st["gy"].float()
    out = dict(ggain_pre=(gy * yh * ry).sum(0))
    q = st["gain_pre"] * gy
    gyh = ry * q - yh * (ry ** 3 / d * (q * yh).sum(1, keepdim=True))
    G = st["gXp"].float()
    if C is None:
        G = G + gyh[:, None]
        gX, gZ = G, G[:, 0]
    else:
        gp = (gyh[:, None] * Xp).sum(2)
        del Xp
        G += st["pre"][..., None] * gyh[:, None]
        gX = torch.bmm(C.transpose(1, 2), G)
        gC = torch.bmm(G, X.transpose(1, 2))
        gu = (G * Z[:, None]).sum(2)
        gZ = (st["post"][..., None] * G).sum(1)
        gC = gC if st["row_dest"] else gC.transpose(1, 2).contiguous()
        out.update(gpre=gp.sum(0) if st["shared"] else gp, gpost=gu.sum(0) if st["shared"] else gu,
                   gcomb=gC.sum(0) if st["shared"] else gC)
    hz = h * gZ
    if st["post_norm"]:
        gF = r * hz - F * (r ** 3 / d * (hz * F).sum(1, keepdim=True))
        out["ggain_post"] = (st["scale"] * a * F * r * gZ).sum(0)
    else:
        gF = hz
    if da is not None:
        out["ggate"] = (st["scale"] * gain * F * r * gZ * da).bfloat16()
    return dict(out, gX=gX.bfloat16(), gF=gF.bfloat16())


# ----------------------------------------------------------------------------------------------
# one pass


def _own(st):
    from stream_residual_fusion_gb300 import mhc

    if st["op"] == "checkpoint":
        codes, scale = mhc.checkpoint_save(st["x"])
        return mhc.checkpoint_load(codes, scale)
    flags = mhc.COMB_ROW_DEST if st["row_dest"] else 0
    if st["op"] == "step_backward":
        return mhc.fused_step_backward_ckpt(
            st["X_codes"], st["X_scale"], st["F_codes"], st["F_scale"], st["mixes"], st["pre"],
            st["post"], st["comb"], st["W"], st["sc"], st["base"], st["gain"], st["gXp"], st["gy"],
            st["gpre"], st["gpost"], st["gcomb"], iters=st["iters"], hc_eps=EPS, norm_eps=EPS,
            flags=flags)
    if st["case_gate"] == "sigmoid":
        flags |= mhc.GATE_SIGMOID
    if st["shared"]:
        flags |= mhc.WEIGHTS_SHARED
    kw = dict(gate=st["gate"], pre=st["pre"], post=st["post"], comb=st["comb"], res_scale=st["scale"],
              norm_eps=EPS, flags=flags)
    if st["op"] == "norm_step":
        return mhc.norm_step(st["X"], st["F"], st["gain_post"], st["gain_pre"], **kw)
    if st["ckpt"]:
        return mhc.norm_step_backward_ckpt(st["X_codes"], st["X_scale"], st["F_codes"], st["F_scale"],
                                           st["gXp"], st["gy"], st["gain_post"], st["gain_pre"], **kw)
    return mhc.norm_step_backward(st["X"], st["F"], st["gXp"], st["gy"], st["gain_post"], st["gain_pre"],
                                  **kw)


def run(st):
    if own:
        return _own(st)
    if st["op"] == "checkpoint":
        return _decode(*_encode(st["x"])).bfloat16()
    if st["op"] == "step_backward":
        return _plain_step_backward(st)
    return _plain_norm_step(st) if st["op"] == "norm_step" else _plain_norm_step_backward(st)


# ----------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    d = case["d"]
    if case["op"] == "checkpoint":
        # the rows read, codes and scales written, read again, and the rows written
        return {"bytes": case["rows"] * (4 * d + 2 * (d + -(-d // BLOCK))), "flops": 6 * case["rows"] * d}
    N = case["N"]
    if case["op"] == "step_backward":
        token = 5 * (d + d // BLOCK) + 20 * d + 4 * (MIX + 24 + 24 + 24)
        return {"bytes": N * token + 2 * 4 * MIX * 4 * d + 8 * d, "flops": N * (2 * 2 * MIX * 4 * d + 160 * d)}
    n, gate = case["n"], case["gate"] != "none"
    given = 4 * (2 * n + n * n) if n == 4 or case["shared"] else 0
    once, each = (given, 0) if case["shared"] else (0, given)
    if case["op"] == "norm_step":
        return {"bytes": N * ((4 * n + 4 + 2 * gate) * d + each) + once + 8 * d,
                "flops": N * d * (2 * n * n + 6 * n + 12)}
    saved = (n + 1) * (d + -(-d // BLOCK)) if case["ckpt"] else (2 * n + 2) * d
    return {"bytes": N * (saved + (4 * n + 4 + 4 * gate) * d + 2 * each) + 2 * once + 16 * d,
            "flops": N * d * (8 * n * n + 16 * n + 40)}


# ----------------------------------------------------------------------------------------------
# the definitions in float64


def _values(codes, scale):
    """float64 values of codes from their bit fields."""
    c = codes.to(torch.int64)
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, f * 2.0 ** -9, torch.ldexp(8 + f, e - 10))
    v = torch.where(c >= 128, -mag, mag)
    return torch.ldexp(v, scale.to(torch.int64).repeat_interleave(BLOCK, -1)[..., :v.shape[-1]] - 127)


def _binade(x):
    """The power of two at or below each positive value."""
    return torch.exp2(torch.frexp(x)[1].double() - 1)


def _nearest(x):
    """Rows of bf16 values rounded to the grid of their block's scale."""
    rows, d = x.shape
    v = torch.zeros(rows, -(-d // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    v[:, :d] = x
    v = v.view(rows, -1, BLOCK)
    unit = _binade(v.abs().amax(2, keepdim=True).clamp_min(2.0 ** -119)) / 256
    v = v / unit
    grid = _binade(v.abs().clamp_min(2.0 ** -6)) / 8
    v = (torch.round(v / grid) * grid).clamp(-448, 448) * unit
    return v.view(rows, -1)[:, :d]


def _exact_step_backward(st, sl):
    X, F = _values(st["X_codes"][sl], st["X_scale"][sl]), _values(st["F_codes"][sl], st["F_scale"][sl])
    N, d, iters = X.shape[0], st["d"], st["iters"]
    C32 = st["comb"][sl].transpose(1, 2) if st["row_dest"] else st["comb"][sl]
    p32, C, u, p = st["pre"][sl], C32.double(), st["post"][sl].double(), st["pre"][sl].double()
    # X' and the block input are bf16 tensors whose float32 evaluation is part of the definition
    acc = None
    for j in range(4):
        t = C32[:, j, :, None] * X[:, j, None].float()
        acc = t if acc is None else acc + t
    Xp = (st["post"][sl][:, :, None] * F[:, None].float() + acc).bfloat16()
    acc = None
    for j in range(4):
        t = p32[:, j, None] * Xp[:, j].float()
        acc = t if acc is None else acc + t
    yh, Xp = acc.bfloat16().double(), Xp.double()
    s, b, m = st["sc"].double(), st["base"].double(), st["mixes"][sl].double()
    z = torch.cat([s[0] * m[:, :4], s[1] * m[:, 4:8], s[2] * m[:, 8:]], 1) + b
    sg = torch.sigmoid(z[:, :8])
    gsp = torch.cat([st["gpre"][sl].double(), 2 * st["gpost"][sl].double()], 1) * sg * (1 - sg)
    soft = torch.softmax(z[:, 8:].view(N, 4, 4), 2)
    seen, c = [], soft + EPS
    for i in range(2 * iters - 1):
        seen.append(c)
        c = c / (c.sum(2 if i % 2 else 1, keepdim=True) + EPS)
    g = st["gcomb"][sl].double()
    for i in range(2 * iters - 2, -1, -1):
        c, ax = seen[i], 2 if i % 2 else 1
        den = c.sum(ax, keepdim=True) + EPS
        g = (g - (g * c / den).sum(ax, keepdim=True)) / den
    gl = soft * (g - (soft * g).sum(2, keepdim=True))
    gz = torch.cat([gsp, gl.view(N, 16)], 1)
    gsc = torch.stack([(gz * m)[:, q].sum() for q in (slice(0, 4), slice(4, 8), slice(8, 24))])
    gm = gz * torch.cat([s[0].expand(4), s[1].expand(4), s[2].expand(16)])
    x = Xp.reshape(N, 4 * d)
    r = (x.square().mean(1, keepdim=True) + EPS).rsqrt()
    gW = (gm * r).T @ x
    gx = (gm * r) @ st["W"].double() - x * (r * r * (gm * m).sum(1, keepdim=True) / (4 * d))
    ry = (yh.square().mean(1, keepdim=True) + EPS).rsqrt()
    gy, gain = st["gy"][sl].double(), st["gain"].double()
    nrm = yh * ry
    gyh = ry * (gain * gy - nrm * (gain * gy * nrm).mean(1, keepdim=True))
    G = st["gXp"][sl].double() + gx.view(N, 4, d) + p[:, :, None] * gyh[:, None]
    gC = torch.einsum("njd,nkd->njk", X, G)
    each = dict(gX=torch.einsum("njk,nkd->njd", C, G), gF=torch.einsum("nk,nkd->nd", u, G),
                gpre_prev=torch.einsum("nd,njd->nj", gyh, Xp), gpost_prev=torch.einsum("nkd,nd->nk", G, F),
                gcomb_prev=gC.transpose(1, 2) if st["row_dest"] else gC)
    return each, dict(gW=gW, gbase=gz.sum(0), gscale=gsc, ggain=(gy * nrm).sum(0))


def _exact_norm(st, sl, back):
    if "X_codes" in st:
        X, F = _values(st["X_codes"][sl], st["X_scale"][sl]), _values(st["F_codes"][sl], st["F_scale"][sl])
    else:
        X, F = st["X"][sl].double(), st["F"][sl].double()
    N, n = X.shape[:2]
    one = torch.ones(N, n, dtype=torch.float64, device=X.device)
    if st["pre"] is None:
        p, u, C = one, one, one[:, :, None]
    else:
        p, u, C = (w.double().expand(N, *w.shape) if st["shared"] else w[sl].double()
                   for w in (st["pre"], st["post"], st["comb"]))
    C = C.transpose(1, 2) if st["row_dest"] else C
    if st["post_norm"]:
        r = (F.square().mean(1, keepdim=True) + EPS).rsqrt()
        V, k = F * r, st["gain_post"].double()
    else:
        r, V, k = one[:, :1], F, 1.0
    a = 1.0 if st["gate"] is None else st["gate"][sl].double()
    if st["case_gate"] == "sigmoid":
        a = torch.sigmoid(a)
    Z = st["scale"] * a * k * V
    Xp = torch.einsum("njk,njd->nkd", C, X) + u[:, :, None] * Z[:, None]
    yh = torch.einsum("nk,nkd->nd", p, Xp)
    ry = (yh.square().mean(1, keepdim=True) + EPS).rsqrt()
    nrm, gain = yh * ry, st["gain_pre"].double()
    if not back:
        return dict(Xp=Xp, y=gain * nrm), {}
    gy = st["gy"][sl].double()
    gyh = ry * (gain * gy - nrm * (gain * gy * nrm).mean(1, keepdim=True))
    G = st["gXp"][sl].double() + p[:, :, None] * gyh[:, None]
    gZ = torch.einsum("nk,nkd->nd", u, G)
    each, total = dict(gX=torch.einsum("njk,nkd->njd", C, G)), dict(ggain_pre=(gy * nrm).sum(0))
    gV = st["scale"] * a * k * gZ
    each["gF"] = r * (gV - V * (gV * V).mean(1, keepdim=True)) if st["post_norm"] else gV
    if st["post_norm"]:
        total["ggain_post"] = (st["scale"] * a * V * gZ).sum(0)
    if st["gate"] is not None:
        ga = st["scale"] * k * V * gZ
        each["ggate"] = ga * a * (1 - a) if st["case_gate"] == "sigmoid" else ga
    if st["pre"] is not None:
        gC = torch.einsum("njd,nkd->njk", X, G)
        w = dict(gpre=torch.einsum("nd,nkd->nk", gyh, Xp), gpost=torch.einsum("nkd,nd->nk", G, Z),
                 gcomb=gC.transpose(1, 2) if st["row_dest"] else gC)
        if st["shared"]:
            total.update({key: v.sum(0) for key, v in w.items()})
        else:
            each.update(w)
    return each, total


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "checkpoint":
        return torch.cat([_nearest(x.double()) for x in st["x"].split(1 << 14)])
    parts, total = [], {}
    for t in range(0, case["N"], 2048):
        sl = slice(t, t + 2048)
        if case["op"] == "step_backward":
            each, some = _exact_step_backward(st, sl)
        else:
            each, some = _exact_norm(st, sl, case["op"] == "norm_step_backward")
        parts.append(each)
        total = {k: total[k] + v if total else v for k, v in some.items()}
    return dict(total, **{k: torch.cat([q[k] for q in parts]) for k in parts[0]})
