"""The activation checkpoints, the step's gradients from them and the norm step with its gradients on the
GPU, against their float64 oracles.

Tolerances:
  * checkpoints: codes, scales and loaded values equal the oracle's, bit for bit.
  * the step's gradients from checkpoints: those of the step's gradients (tests/test_gpu_backward.py).
  * norm step: every float32 evaluation in it is a chain of at most three sums over the width (64
    additions each at the widths here: at most 16 in a thread, 5 across its warp, and the rest across
    warps) and about 60 other operations, under 512 roundings in all, so it is within 2^-15 of the result's
    magnitude (the formula with every term's absolute value; oracle/norm_step.py). A bf16 output adds half
    a step, 2^-8 of the value; a sum over N tokens N more roundings.
"""
import numpy as np
import pytest
import torch

from oracle import checkpoint as OC
from oracle import norm_step as ON
from tests.parity import to64
from tests.test_gpu_backward import _check as check_step_gradients

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def M():
    from stream_residual_fusion_gb300 import build
    build.build()
    import stream_residual_fusion_gb300.mhc as m
    return m


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _equal_with_nan(a, b):
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


# ----------------------------------------------------------------------------------------------
# checkpoints


def _rows(rows, d, seed):
    g = _gen(seed)
    x = _normal(g, rows, d) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g, device=DEV).float())
    if d > 16:
        x[:, 3] *= 100.0                       # an outlier feature: the rest of its block in few bits
    x[rows // 2, : d // 2] = 0.0
    return x.bfloat16()


@pytest.mark.parametrize("rows,d", [(1, 8), (3, 40), (5, 32), (7, 72), (129, 1000), (4 * 33, 5120), (2, 32768)])
def test_checkpoint_parity(M, rows, d):
    x = _rows(rows, d, 10 * rows + d)
    codes, scales = M.checkpoint_save(x)
    want_c, want_s = OC.checkpoint_save(to64(x))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    back = M.checkpoint_load(codes, scales)
    assert np.array_equal(to64(back), OC.checkpoint_load(want_c, want_s))


def test_checkpoint_of_special_values(M):
    """Infinities, NaNs, signed zeros, the largest and the subnormal values, each alone in its block's
    place and all in one block; every code with every scale loads as the oracle says."""
    special = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 3.3895e38, -3.3895e38, 1e-40,
                            -9.2e-41, 1.1754944e-38, 2.0, 447.0, 464.0, 480.0, -1.0, 1e-30])
    x = torch.cat([special, special.flip(0)]).repeat(33, 1)
    for i in range(32):
        x[i] = torch.where(torch.arange(32) <= i, x[i], torch.full((32,), 0.3 * (i + 1)))
    x = x.to(DEV).bfloat16()
    codes, scales = M.checkpoint_save(x)
    want_c, want_s = OC.checkpoint_save(to64(x))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    gc = codes.cpu().numpy()
    nan = ~np.isfinite(to64(x))
    assert np.array_equal(gc[~nan], want_c[~nan])
    assert ((gc[nan] & 0x7F) == 0x7F).all()
    every = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(256, 1)
    es = torch.arange(256, dtype=torch.uint8, device=DEV)[:, None].repeat(1, 8).contiguous()
    got = M.checkpoint_load(every, es)
    want = torch.tensor(OC.checkpoint_load(every.cpu().numpy(), es.cpu().numpy()))
    assert _equal_with_nan(got.double().cpu(), want)


def test_checkpoint_saved_again_is_the_same(M):
    """What a checkpoint loads as has that same checkpoint (wherever its values are bf16's)."""
    x = _rows(64, 512, 5)
    codes, scales = M.checkpoint_save(x)
    back = M.checkpoint_load(codes, scales)
    c2, s2 = M.checkpoint_save(back)
    assert torch.equal(M.checkpoint_load(c2, s2), back)


def test_checkpoint_shapes_bounds_and_streams(M):
    """Leading dimensions, no rows, outputs within their bounds, another stream, a captured graph."""
    x = _rows(3 * 4, 104, 6)
    c, s = M.checkpoint_save(x.view(3, 4, 104))
    assert c.shape == (3, 4, 104) and s.shape == (3, 4, 4)
    c0, s0 = M.checkpoint_save(x[:0])
    assert c0.shape == (0, 104) and M.checkpoint_load(c0, s0).shape == (0, 104)
    big_c = torch.full((12 * 104 + 64,), 99, dtype=torch.uint8, device=DEV)
    big_s = torch.full((12 * 4 + 64,), 99, dtype=torch.uint8, device=DEV)
    out = (big_c[:12 * 104].view(12, 104), big_s[:48].view(12, 4))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.checkpoint_save(x, out=out, stream=side)
    y = M.checkpoint_load(*out, stream=side)
    side.synchronize()
    assert torch.equal(out[0], c.view(12, 104)) and torch.equal(out[1], s.view(12, 4))
    assert bool((big_c[12 * 104:] == 99).all()) and bool((big_s[48:] == 99).all())
    g = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(g):
        gc, gs = M.checkpoint_save(xs)
        gy = M.checkpoint_load(gc, gs)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gy, y)
    xs.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gy, y.flip(0))


# ----------------------------------------------------------------------------------------------
# the step's gradients from checkpoints


def _step_inputs(M, N, d, seed):
    from stream_residual_fusion_gb300 import synth
    inp = synth.make_inputs(N, 4, d, seed=seed, device=DEV, scale_uniform=True, x_stream_std=True)
    up = synth.make_upstream(N, 4, d, seed=seed + 1, device=DEV)
    return inp, up, M.checkpoint_save(inp["X"]), M.checkpoint_save(inp["F"])


def _step_backward(M, inp, up, cX, cF, mixes, **kw):
    return M.fused_step_backward_ckpt(*cX, *cF, mixes, inp["pre"], inp["post"], inp["comb"], inp["W"],
                                      inp["scale"], inp["base"], inp["gain"], up["gXp"], up["gy"], up["gpre"],
                                      up["gpost"], up["gcomb"], **kw)


@pytest.mark.parametrize("N,d,iters,row_dest", [
    (300, 5120, 20, False), (300, 5120, 20, True), (1000, 512, 20, False), (200, 256, 1, False),
    (129, 128, 3, True), (1, 5120, 20, False), (113, 192, 2, False), (17, 1088, 20, True), (65, 64, 20, False),
    (2, 10240, 20, False)])
def test_step_backward_ckpt_parity(M, N, d, iters, row_dest):
    """A training step's chain: the fused step, the checkpoints of its inputs, its gradients from them."""
    inp, up, cX, cF = _step_inputs(M, N, d, 8000 + N + d)
    flags = M.COMB_ROW_DEST if row_dest else 0
    Xp = M.hc_post(inp["X"], inp["F"], inp["post"], inp["comb"], flags=flags)
    x = Xp.double().view(N, -1)
    mixes = ((x @ inp["W"].double().T) * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt()).float()
    got = _step_backward(M, inp, up, cX, cF, mixes, iters=iters, flags=flags)
    torch.cuda.synchronize()
    assert M.get_status() == M.MHC_OK
    X, F = (OC.checkpoint_values(c.cpu().numpy(), s.cpu().numpy()) for c, s in (cX, cF))
    u = {k: to64(v) for k, v in up.items()}
    ref = OC.fused_step_backward_ckpt(X, F, to64(mixes), *(to64(inp[k]) for k in (
        "pre", "post", "comb", "W", "scale", "base", "gain")), u["gXp"], u["gy"], u["gpre"], u["gpost"], u["gcomb"],
        iters=iters, comb_row_dest=row_dest)
    check_step_gradients(got, ref)


@pytest.mark.parametrize("N,d", [(1, 256), (129, 512), (300, 5120)])
def test_step_backward_ckpt_agrees_with_the_step_backward(M, N, d):
    """On streams that checkpoints hold exactly, the gradients from checkpoints and from X, F and X' are
    the same to the last rounding of sums; outputs stay within their bounds and inputs as they were."""
    inp, up, cX, cF = _step_inputs(M, N, d, 8100 + N)
    inp["X"], inp["F"] = M.checkpoint_load(*cX), M.checkpoint_load(*cF)
    fw = M.fused_step(inp["X"], inp["F"], inp["pre"], inp["post"], inp["comb"], inp["W"], inp["scale"],
                      inp["base"], inp["gain"], with_mixes=True)
    want = M.fused_step_backward(inp["X"], inp["F"], fw["Xp"], fw["mixes"], inp["pre"], inp["post"],
                                 inp["comb"], inp["W"], inp["scale"], inp["base"], inp["gain"], up["gXp"],
                                 up["gy"], up["gpre"], up["gpost"], up["gcomb"])
    big, out = {}, {}
    for k, v in want.items():
        big[k] = torch.full((v.numel() + 4096,), -7.0, dtype=v.dtype, device=DEV)
        out[k] = big[k][:v.numel()].view(v.shape)
    before = [t.clone() for t in (*cX, *cF)]
    _step_backward(M, inp, up, cX, cF, fw["mixes"], out=out)
    torch.cuda.synchronize()
    assert M.get_status() == M.MHC_OK
    for k, v in want.items():
        assert bool((big[k][v.numel():] == -7.0).all()), k
        a, b = out[k].double(), v.double()
        # one rounding each of bf16 outputs from sums in another order; 2^-17 of the largest for the sums
        lim = 2.0 ** -7 * b.abs() + 2.0 ** -14 * b.abs().max()
        assert bool(((a - b).abs() <= lim).all()), k
    for a, b in zip((*cX, *cF), before):
        assert torch.equal(a, b)


def test_step_backward_ckpt_of_no_tokens(M):
    inp, up, cX, cF = _step_inputs(M, 4, 256, 8200)
    e = {k: (v[:0] if k in ("pre", "post", "comb") else v) for k, v in inp.items()}
    out = {"gW": torch.full_like(inp["W"], 7.0), "gbase": torch.full((24,), 7.0, device=DEV),
           "gscale": torch.full((3,), 7.0, device=DEV), "ggain": torch.full((256,), 7.0, device=DEV)}
    got = _step_backward(M, e, {k: v[:0] for k, v in up.items()}, tuple(t[:0] for t in cX),
                         tuple(t[:0] for t in cF), torch.empty(0, 24, device=DEV), out=out)
    torch.cuda.synchronize()
    for k in out:
        assert torch.count_nonzero(got[k]).item() == 0, k


def test_step_backward_ckpt_twice_and_in_a_graph(M):
    """The same bits from the same call, also when captured, with a shared workspace reused between."""
    inp, up, cX, cF = _step_inputs(M, 260, 512, 8300)
    mixes = _normal(_gen(1), 260, 24)
    ws = torch.empty(M.backward_ckpt_workspace_bytes(260, 512), dtype=torch.uint8, device=DEV)
    a = _step_backward(M, inp, up, cX, cF, mixes, workspace=ws)
    a = {k: v.clone() for k, v in a.items()}
    ws.fill_(0x7F)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = _step_backward(M, inp, up, cX, cF, mixes, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]), k


# ----------------------------------------------------------------------------------------------
# the norm step


def _norm_inputs(N, n, d, gate, post_norm, weights, shared, seed, masked=False):
    g = _gen(seed)
    X, F = _normal(g, N, n, d).bfloat16(), _normal(g, N, d).bfloat16()
    a = dict(X=X, F=F, gXp=_normal(g, N, n, d).bfloat16(), gy=_normal(g, N, d).bfloat16(),
             gain_post=1 + 0.2 * _normal(g, d) if post_norm else None, gain_pre=1 + 0.2 * _normal(g, d))
    a["gate"] = (2 * _normal(g, N, d)).bfloat16() if gate != "none" else None
    rows = () if shared else (N,)
    a["w"] = (torch.rand(*rows, n, generator=g, device=DEV), 2 * torch.rand(*rows, n, generator=g, device=DEV),
              _normal(g, *rows, n, n)) if weights else (None,) * 3
    return a


def _norm_kw(M, a, gate, shared, row_dest, scale, eps):
    flags = (M.GATE_SIGMOID if gate == "sigmoid" else 0) | (M.WEIGHTS_SHARED if shared else 0)
    flags |= M.COMB_ROW_DEST if row_dest else 0
    kw = dict(gate=a["gate"], pre=a["w"][0], post=a["w"][1], comb=a["w"][2], res_scale=scale, norm_eps=eps,
              flags=flags)
    okw = dict(gate=None if a["gate"] is None else to64(a["gate"]),
               weights=None if a["w"][0] is None else [to64(w) for w in a["w"]], scale=scale, eps=eps,
               sigmoid=gate == "sigmoid", row_dest=row_dest)
    return kw, okw


def _opt64(t):
    return None if t is None else to64(t)


def _check_norm(got, ref, mag, N):
    assert set(got) == set(ref)
    for k, r in ref.items():
        g = to64(got[k])
        assert g.shape == r.shape, k
        lim = (2.0 ** -15 + N * 2.0 ** -24) * mag[k]
        if got[k].dtype == torch.bfloat16:
            lim = lim + 2.0 ** -8 * np.abs(r) + 2.0 ** -134
        bad = ~(np.abs(g - r) <= lim)
        assert not bad.any(), (k, int(bad.sum()), np.argwhere(bad)[:3].tolist(), g[bad][:3], r[bad][:3])


# N, n, d, gate, post_norm, weights, shared, row_dest
NORM_CASES = [
    (1, 4, 5120, "none", True, True, False, False),
    (300, 4, 512, "sigmoid", True, True, False, False),
    (200, 4, 5120, "linear", True, True, False, True),
    (153, 4, 2056, "sigmoid", False, True, True, False),
    (33, 4, 8, "linear", True, True, False, False),
    (7, 4, 10248, "sigmoid", True, True, True, True),
    (3, 4, 32768, "linear", True, True, False, False),
    (311, 1, 1992, "sigmoid", True, False, False, False),
    (5, 1, 4096, "none", True, False, False, False),
    (64, 1, 640, "none", False, False, False, False),
    (9, 1, 8, "linear", True, True, False, False),
    (40, 1, 5120, "linear", True, True, True, False),
    (2, 1, 32768, "sigmoid", True, False, False, False),
    (1, 1, 16, "none", False, True, False, True),
    (77, 4, 64, "sigmoid", True, True, True, False),
    (260, 4, 248, "none", True, True, False, True),
    (19, 4, 1032, "sigmoid", True, True, False, False),
    (130, 1, 200, "linear", True, True, True, False),
    (600, 1, 1024, "sigmoid", False, False, False, False),
    (6, 4, 7168, "none", False, True, True, False),
    (1, 1, 520, "linear", True, False, False, False),      # codes of 8 bytes beyond whole 16: one row, and more
    (306, 1, 1000, "sigmoid", True, True, False, False),
    (457, 4, 520, "linear", True, True, False, False),
    (458, 4, 1000, "none", True, True, False, True),
    (153, 1, 5128, "none", True, False, False, False),
    (170, 1, 2688, "sigmoid", True, False, False, False),
    (331, 1, 1160, "linear", False, True, False, False),
    (155, 1, 7168, "sigmoid", True, True, True, False),
    (160, 1, 3344, "none", True, False, False, False),
]


@pytest.mark.parametrize("N,n,d,gate,post_norm,weights,shared,row_dest", NORM_CASES)
def test_norm_step_parity(M, N, n, d, gate, post_norm, weights, shared, row_dest):
    a = _norm_inputs(N, n, d, gate, post_norm, weights, shared, 100 * N + d)
    kw, okw = _norm_kw(M, a, gate, shared, row_dest, 0.7, 1e-6)
    got = M.norm_step(a["X"], a["F"], a["gain_post"], a["gain_pre"], **kw)
    ref, mag = ON.norm_step(to64(a["X"]), to64(a["F"]), _opt64(a["gain_post"]), to64(a["gain_pre"]), **okw)
    _check_norm(got, ref, mag, 0)
    # in place, on another stream
    X = a["X"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = M.norm_step(X, a["F"], a["gain_post"], a["gain_pre"], out={"Xp": X}, stream=side, **kw)
    side.synchronize()
    assert torch.equal(X, got["Xp"]) and torch.equal(again["y"], got["y"])


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("N,n,d,gate,post_norm,weights,shared,row_dest", NORM_CASES)
def test_norm_step_backward_parity(M, N, n, d, gate, post_norm, weights, shared, row_dest, ckpt):
    a = _norm_inputs(N, n, d, gate, post_norm, weights, shared, 100 * N + d + 1)
    kw, okw = _norm_kw(M, a, gate, shared, row_dest, 0.7, 1e-6)
    args = (a["gXp"], a["gy"], a["gain_post"], a["gain_pre"])
    X, F = to64(a["X"]), to64(a["F"])
    if ckpt:
        cX, cF = M.checkpoint_save(a["X"]), M.checkpoint_save(a["F"])
        got = M.norm_step_backward_ckpt(*cX, *cF, *args, **kw)
        X, F = (OC.checkpoint_values(c.cpu().numpy(), s.cpu().numpy()) for c, s in (cX, cF))
    else:
        got = M.norm_step_backward(a["X"], a["F"], *args, **kw)
    ref, mag = ON.norm_step_backward(X, F, to64(a["gXp"]), to64(a["gy"]), _opt64(a["gain_post"]),
                                     to64(a["gain_pre"]), shared=shared, **okw)
    _check_norm(got, ref, mag, N)


@pytest.mark.parametrize("n", [1, 4])
def test_norm_step_of_zeros_and_values_that_are_not_finite(M, n):
    """A row of zeros (also with a zero residual scale), a quiet row where eps decides, and a NaN and
    an infinity in one token, which stay in that token's outputs."""
    N, d = 6, 512
    a = _norm_inputs(N, n, d, "sigmoid", True, n == 4, False, 77)
    a["F"][1] = 0
    a["X"][2], a["F"][2] = 0, 0
    a["X"][3], a["F"][3] = a["X"][3] * 1e-4, a["F"][3] * 1e-4
    clean, _ = _norm_kw(M, a, "sigmoid", False, False, 0.7, 1e-6)
    a["gate"][5, :4] = torch.tensor([-200.0, 200.0, float("inf"), -float("inf")])
    kw, okw = _norm_kw(M, a, "sigmoid", False, False, 0.7, 1e-6)
    with np.errstate(over="ignore"):
        ref, mag = ON.norm_step(to64(a["X"]), to64(a["F"]), to64(a["gain_post"]), to64(a["gain_pre"]), **okw)
        refb, magb = ON.norm_step_backward(to64(a["X"]), to64(a["F"]), to64(a["gXp"]), to64(a["gy"]),
                                           to64(a["gain_post"]), to64(a["gain_pre"]), **okw)
    _check_norm(M.norm_step(a["X"], a["F"], a["gain_post"], a["gain_pre"], **kw), ref, mag, 0)
    good = M.norm_step_backward(a["X"], a["F"], a["gXp"], a["gy"], a["gain_post"], a["gain_pre"], **kw)
    _check_norm(good, refb, magb, N)
    a["X"][4, 0, 7], a["F"][0, 9] = float("nan"), float("inf")
    out = M.norm_step(a["X"], a["F"], a["gain_post"], a["gain_pre"], **kw)
    back = M.norm_step_backward(a["X"], a["F"], a["gXp"], a["gy"], a["gain_post"], a["gain_pre"], **kw)
    rest = [1, 2, 3, 5]
    for k in ("Xp", "y"):
        assert np.isfinite(to64(out[k])[rest]).all()
        assert not np.isfinite(to64(out[k])[0]).all() and not np.isfinite(to64(out[k])[4]).all()
    for k in ("gX", "gF", "ggate"):
        assert torch.equal(back[k][rest], good[k][rest]), k
        assert not np.isfinite(to64(back[k])[4]).all() or k != "gX"


def test_norm_step_bounds_empty_and_refusals(M):
    a = _norm_inputs(131, 4, 520, "linear", True, True, False, 5)
    kw, _ = _norm_kw(M, a, "linear", False, False, 1.0, 1e-6)
    pos = (a["gain_post"], a["gain_pre"])
    want = M.norm_step(a["X"], a["F"], *pos, **kw)
    wantb = M.norm_step_backward(a["X"], a["F"], a["gXp"], a["gy"], *pos, **kw)
    before = {k: a[k].clone() for k in ("X", "F", "gXp", "gy", "gate")}

    def padded(like):
        big = {k: torch.full((v.numel() + 256,), -7.0, dtype=v.dtype, device=DEV) for k, v in like.items()}
        return big, {k: big[k][:v.numel()].view(v.shape) for k, v in like.items()}
    for like, call in ((want, lambda o: M.norm_step(a["X"], a["F"], *pos, out=o, **kw)),
                       (wantb, lambda o: M.norm_step_backward(a["X"], a["F"], a["gXp"], a["gy"], *pos, out=o, **kw))):
        big, out = padded(like)
        call(out)
        torch.cuda.synchronize()
        for k, v in like.items():
            assert torch.equal(out[k], v), k
            assert bool((big[k][v.numel():] == -7.0).all()), k
    for k, v in before.items():
        assert torch.equal(a[k], v), k
    # no tokens
    e = {k: (v[:0] if v is not None else None) for k, v in a.items() if k in ("X", "F", "gXp", "gy", "gate")}
    ekw = dict(kw, gate=e["gate"], pre=kw["pre"][:0], post=kw["post"][:0], comb=kw["comb"][:0])
    assert M.norm_step(e["X"], e["F"], *pos, **ekw)["y"].shape == (0, 520)
    out = {"ggain_pre": torch.full((520,), 7.0, device=DEV), "ggain_post": torch.full((520,), 7.0, device=DEV)}
    M.norm_step_backward(e["X"], e["F"], e["gXp"], e["gy"], *pos, out=out, **ekw)
    shared = dict(kw, gate=e["gate"], pre=kw["pre"][0], post=kw["post"][0], comb=kw["comb"][0],
                  flags=M.WEIGHTS_SHARED)
    g = M.norm_step_backward(e["X"], e["F"], e["gXp"], e["gy"], *pos, **shared)
    torch.cuda.synchronize()
    for t in (*out.values(), g["gpre"], g["gpost"], g["gcomb"]):
        assert torch.count_nonzero(t).item() == 0
    # wrong shapes, types, devices
    for bad in (dict(gate=a["gate"][:, :8]), dict(gate=a["gate"].float()), dict(pre=kw["pre"][:5]),
                dict(comb=kw["comb"].transpose(1, 2)), dict(comb=kw["comb"].cpu())):
        with pytest.raises((TypeError, ValueError)):
            M.norm_step(a["X"], a["F"], *pos, **dict(kw, **bad))
    with pytest.raises(ValueError):
        M.norm_step_backward_ckpt(*M.checkpoint_save(a["X"]), a["F"].view(torch.uint8)[:, :520].contiguous(),
                                  torch.empty(131, 16, dtype=torch.uint8, device=DEV), a["gXp"], a["gy"], *pos, **kw)
    with pytest.raises(M.MhcError) as err:
        M.norm_step_backward(a["X"], a["F"], a["gXp"], a["gy"], *pos, **kw,
                             workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert err.value.code == M.MHC_ERR_WORKSPACE
    for some in (dict(post=None), dict(pre=None), dict(pre=None, comb=None)):   # weights: all or none
        with pytest.raises(M.MhcError):
            M.norm_step(a["X"], a["F"], *pos, **dict(kw, **some))
        with pytest.raises(M.MhcError):
            M.norm_step_backward(a["X"], a["F"], a["gXp"], a["gy"], *pos, **dict(kw, **some))


@pytest.mark.parametrize("N,n,d", [(70, 1, 72), (700, 4, 64), (331, 1, 1992), (309, 4, 1032), (3, 4, 32768)])
def test_norm_step_in_place(M, N, n, d):
    a = _norm_inputs(N, n, d, "sigmoid", True, True, False, 8)
    kw, _ = _norm_kw(M, a, "sigmoid", False, False, 0.5, 1e-6)
    want = M.norm_step(a["X"], a["F"], a["gain_post"], a["gain_pre"], **kw)
    X = a["X"].clone()
    got = M.norm_step(X, a["F"], a["gain_post"], a["gain_pre"], **kw, out={"Xp": X})
    assert got["Xp"] is X and torch.equal(X, want["Xp"]) and torch.equal(got["y"], want["y"])


@pytest.mark.parametrize("n,shared", [(1, False), (4, True)])
def test_norm_step_same_bits_and_graph(M, n, shared):
    """The same bits from the same call, eager or captured with new inputs copied in."""
    a = _norm_inputs(700, n, 1024, "sigmoid", True, n == 4, shared, 9)
    kw, _ = _norm_kw(M, a, "sigmoid", shared, False, 0.5, 1e-6)
    pos = (a["gain_post"], a["gain_pre"])
    first = {**M.norm_step(a["X"], a["F"], *pos, **kw),
             **M.norm_step_backward(a["X"], a["F"], a["gXp"], a["gy"], *pos, **kw)}
    X = torch.zeros_like(a["X"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = {**M.norm_step(X, a["F"], *pos, **kw), **M.norm_step_backward(X, a["F"], a["gXp"], a["gy"], *pos, **kw)}
    X.copy_(a["X"])
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(first[k], out[k]), k


def test_two_residual_steps_trained_from_checkpoints(M):
    """A chain as a training step runs it: two norm steps around two blocks, their inputs kept as
    checkpoints, and the gradients walked back through both; against the oracle at the decoded values."""
    N, n, d = 70, 4, 768
    first = _norm_inputs(N, n, d, "sigmoid", True, True, False, 31)
    second = _norm_inputs(N, n, d, "linear", True, True, True, 32)
    kw1, ok1 = _norm_kw(M, first, "sigmoid", False, False, 0.7, 1e-6)
    kw2, ok2 = _norm_kw(M, second, "linear", True, False, 1.0, 1e-6)
    o1 = M.norm_step(first["X"], first["F"], first["gain_post"], first["gain_pre"], **kw1)
    c1 = (*M.checkpoint_save(first["X"]), *M.checkpoint_save(first["F"]))
    F2 = (o1["y"].float() * 0.5).bfloat16()                    # the second block: half its input
    c2 = (*M.checkpoint_save(o1["Xp"]), *M.checkpoint_save(F2))
    o2 = M.norm_step(o1["Xp"], F2, second["gain_post"], second["gain_pre"], **kw2)
    assert torch.isfinite(o2["y"].float()).all()
    b2 = M.norm_step_backward_ckpt(*c2, second["gXp"], second["gy"], second["gain_post"], second["gain_pre"], **kw2)
    gy1 = (b2["gF"].float() * 0.5).bfloat16()
    b1 = M.norm_step_backward_ckpt(*c1, b2["gX"], gy1, first["gain_post"], first["gain_pre"], **kw1)

    def values(c):
        c = [t.cpu().numpy() for t in c]
        return OC.checkpoint_values(c[0], c[1]), OC.checkpoint_values(c[2], c[3])
    r2, m2 = ON.norm_step_backward(*values(c2), to64(second["gXp"]), to64(second["gy"]), to64(second["gain_post"]),
                                   to64(second["gain_pre"]), shared=True, **ok2)
    r1, m1 = ON.norm_step_backward(*values(c1), to64(b2["gX"]), to64(gy1), to64(first["gain_post"]),
                                   to64(first["gain_pre"]), **ok1)
    _check_norm(b2, r2, m2, N)
    _check_norm(b1, r1, m1, N)
