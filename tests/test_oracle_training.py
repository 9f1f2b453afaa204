"""The oracles of the activation checkpoints and of the norm step (CPU): the encoding against an
exhaustive search, the gradients against central differences and against torch's autograd of the same
forward, and the checkpointed step gradients against those of the plain oracle."""
import numpy as np
import pytest
import torch

from oracle import backward as OB
from oracle import checkpoint as OC
from oracle import mhc as O
from oracle import mx
from oracle import norm_step as ON


def _bf16(rng, *shape):
    return O.bf16_round(rng.standard_normal(shape))


def test_checkpoint_codes_are_the_nearest_values():
    rng = np.random.default_rng(1)
    x = _bf16(rng, 6, 72) * np.exp2(rng.integers(-20, 20, (6, 1)))
    codes, scales = OC.checkpoint_save(x)
    assert codes.shape == (6, 72) and scales.shape == (6, 3)
    grid = mx.e4m3_decode(np.arange(256))
    grid = np.unique(grid[np.isfinite(grid)])
    for r in range(6):
        for b in range(3):
            blk = x[r, 32 * b:32 * b + 32]
            s = 2.0 ** (np.floor(np.log2(np.abs(blk).max())) - 8)
            assert scales[r, b] == int(np.log2(s)) + 127
            got = OC.checkpoint_values(codes, scales)[r, 32 * b:32 * b + 32]
            best = np.abs(blk[:, None] - s * grid[None]).min(axis=1)
            assert np.array_equal(np.abs(blk - got), best)


def test_checkpoint_of_values_that_are_not_finite():
    x = np.zeros((1, 40))
    x[0, :6] = [np.inf, -np.inf, np.nan, 3.0, -0.0, 2.0 ** -133]
    codes, scales = OC.checkpoint_save(x)
    assert codes[0, 0] == 0x7F and codes[0, 1] == 0xFF and codes[0, 2] & 0x7F == 0x7F and codes[0, 4] == 0x80
    assert scales.tolist() == [[1 - 8 + 127, 0]]            # the largest finite value is 3
    v = OC.checkpoint_load(codes, scales)
    assert np.isnan(v[0, :3]).all() and v[0, 3] == 3.0 and (v[0, 4:] == 0).all()
    assert np.isnan(OC.checkpoint_values(codes, np.full((1, 2), 255, np.uint8))).all()


CASES = [(n, gate, sigmoid, post_norm, row_dest, shared)
         for n in (1, 4)
         for gate, sigmoid in ((False, False), (True, False), (True, True))
         for post_norm in (True, False)
         for row_dest, shared in ((False, False), (True, True))]


def _inputs(n, gate, post_norm, shared, N=3, d=16, seed=3):
    rng = np.random.default_rng(seed)
    r = rng.standard_normal
    rows = () if shared else (N,)
    return dict(X=r((N, n, d)), F=r((N, d)), gain_post=1 + 0.3 * r(d) if post_norm else None,
                gain_pre=1 + 0.3 * r(d), gate=r((N, d)) if gate else None,
                weights=(r((*rows, n)), r((*rows, n)), r((*rows, n, n)))), r((N, n, d)), r((N, d))


@pytest.mark.parametrize("n,gate,sigmoid,post_norm,row_dest,shared", CASES)
def test_norm_step_gradients_against_differences(n, gate, sigmoid, post_norm, row_dest, shared):
    a, gXp, gy = _inputs(n, gate, post_norm, shared)
    kw = dict(scale=0.7, eps=1e-3, sigmoid=sigmoid, row_dest=row_dest)
    got, mag = ON.norm_step_backward(a["X"], a["F"], gXp, gy, a["gain_post"], a["gain_pre"], gate=a["gate"],
                                     weights=a["weights"], shared=shared, **kw)

    def loss(X, F, gain_post, gain_pre, gate, pre, post, comb):
        o, _ = ON.norm_step(X, F, gain_post, gain_pre, gate=gate, weights=(pre, post, comb), **kw)
        return (o["Xp"] * gXp).sum() + (o["y"] * gy).sum()

    args = [a["X"], a["F"], a["gain_post"], a["gain_pre"], a["gate"], *a["weights"]]
    names = ["gX", "gF", "ggain_post", "ggain_pre", "ggate", "gpre", "gpost", "gcomb"]
    rng = np.random.default_rng(4)
    for i, (v, name) in enumerate(zip(args, names)):
        if v is None:
            assert name not in got
            continue
        assert got[name].shape == v.shape == mag[name].shape
        assert (np.abs(got[name]) <= mag[name] * (1 + 1e-12)).all()
        e, h = rng.standard_normal(v.shape), 1e-5
        up, down = list(args), list(args)
        up[i], down[i] = v + h * e, v - h * e
        want = (loss(*up) - loss(*down)) / (2 * h)
        assert abs((got[name] * e).sum() - want) <= 1e-6 * (np.abs(got[name] * e).sum() + 1e-3), name


def test_norm_step_of_one_stream_is_the_plain_residual():
    a, gXp, gy = _inputs(1, True, True, False)
    o, _ = ON.norm_step(a["X"], a["F"], a["gain_post"], a["gain_pre"], gate=a["gate"], scale=0.5)
    Z = 0.5 * a["gate"] * a["gain_post"] * a["F"] / np.sqrt((a["F"] ** 2).mean(1, keepdims=True) + 1e-6)
    x = a["X"][:, 0] + Z
    assert np.allclose(o["Xp"][:, 0], x, atol=1e-14)
    assert np.allclose(o["y"], a["gain_pre"] * x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6), atol=1e-13)
    g, _ = ON.norm_step_backward(a["X"], a["F"], gXp, gy, a["gain_post"], a["gain_pre"], gate=a["gate"], scale=0.5)
    assert "gcomb" not in g and g["gX"].shape == (3, 1, 16)


@pytest.mark.parametrize("row_dest", [False, True])
def test_norm_step_gradients_against_autograd(row_dest):
    a, gXp, gy = _inputs(4, True, True, False, seed=9)
    t = {k: torch.tensor(v, requires_grad=True) for k, v in a.items() if k != "weights"}
    p, u, C = (torch.tensor(w, requires_grad=True) for w in a["weights"])
    Z = 0.5 * torch.sigmoid(t["gate"]) * t["gain_post"] * t["F"] * (t["F"].square().mean(1, keepdim=True) + 1e-6).rsqrt()
    Xp = torch.einsum("nkj,njd->nkd" if row_dest else "njk,njd->nkd", C, t["X"]) + u[:, :, None] * Z[:, None]
    yh = (p[:, :, None] * Xp).sum(1)
    y = t["gain_pre"] * yh * (yh.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    ((Xp * torch.tensor(gXp)).sum() + (y * torch.tensor(gy)).sum()).backward()
    got, _ = ON.norm_step_backward(a["X"], a["F"], gXp, gy, a["gain_post"], a["gain_pre"], gate=a["gate"],
                                   weights=a["weights"], scale=0.5, sigmoid=True, row_dest=row_dest)
    want = dict(gX=t["X"], gF=t["F"], ggain_post=t["gain_post"], ggain_pre=t["gain_pre"], ggate=t["gate"],
                gpre=p, gpost=u, gcomb=C)
    for k, v in want.items():
        assert np.allclose(got[k], v.grad.numpy(), rtol=1e-9, atol=1e-11), k


def test_checkpointed_step_gradients_are_the_steps_at_the_decoded_values():
    """With the mix numbers of the decoded values themselves, the gradients are those of the step."""
    rng = np.random.default_rng(11)
    N, n, d = 3, 4, 64
    X, F = _bf16(rng, N * n, d), _bf16(rng, N, d)
    X = OC.checkpoint_load(*OC.checkpoint_save(X)).reshape(N, n, d)
    F = OC.checkpoint_load(*OC.checkpoint_save(F))
    r = rng.standard_normal
    pre, post, comb = rng.random((N, n)), 2 * rng.random((N, n)), rng.random((N, n, n))
    W, scale, base, gain = 0.1 * r((24, n * d)), np.ones(3), r(24), 1 + 0.1 * r(d)
    ups = [r((N, n, d)), r((N, d)), r((N, n)), r((N, n)), r((N, n, n))]
    for row_dest in (False, True):
        want = OB.fused_step_backward(X, F, pre, post, comb, W, scale, base, gain, *ups, iters=4,
                                      comb_row_dest=row_dest)
        x = O.hc_post(X, F, post, comb, row_dest).reshape(N, n * d)
        m = (x @ W.T) / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6)
        got = OC.fused_step_backward_ckpt(X, F, m, pre, post, comb, W, scale, base, gain, *ups, iters=4,
                                          comb_row_dest=row_dest)
        for k, v in got.items():
            assert np.allclose(v, want[k], rtol=1e-10, atol=1e-12), k
