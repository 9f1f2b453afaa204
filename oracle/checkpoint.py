"""8-bit activation checkpoints and the step's gradients from them (oracle; test infrastructure only).

A checkpoint holds rows of d bf16 features as MXFP8 blocks of 32 consecutive features (oracle.mx has
the format), the last block of a row possibly shorter. Two rules beyond the format: the largest
magnitude of a block is taken over its finite values, and an infinity or NaN is stored as a NaN code
(sign kept), so that a checkpoint never turns it into a finite value.
"""
from __future__ import annotations

import numpy as np

from .backward import rmsnorm_backward, sinkhorn_backward, sinkhorn_taped, split_backward
from .mhc import bf16_round, hc_post, hc_pre
from .mx import MX_BLOCK, e4m3_decode, e4m3_encode, e4m3_round, mx_scale_code

__all__ = ["checkpoint_save", "checkpoint_values", "checkpoint_load", "fused_step_backward_ckpt"]


def checkpoint_save(x):
    """x [rows, d] float64 (bf16 values) -> (codes uint8 [rows, d], scales uint8 [rows, ceil(d/32)])."""
    x = np.asarray(x, dtype=np.float64)
    rows, d = x.shape
    nb = -(-d // MX_BLOCK)
    finite = np.isfinite(x)
    v = np.zeros((rows, nb * MX_BLOCK))
    v[:, :d] = np.where(finite, x, 0.0)
    blocks = v.reshape(rows, nb, MX_BLOCK)
    scale = mx_scale_code(np.abs(blocks).max(axis=2))
    q = blocks / np.exp2(scale.astype(np.float64) - 127.0)[:, :, None]
    codes = e4m3_encode(e4m3_round(q)).reshape(rows, nb * MX_BLOCK)[:, :d]
    # the sign of a zero is its input's; what is not finite is the NaN code
    codes = np.where((codes & 0x7F) == 0, np.where(np.signbit(x), 0x80, 0), codes)
    codes = np.where(finite, codes, np.where(np.signbit(x), 0xFF, 0x7F))
    return codes.astype(np.uint8), scale


def checkpoint_values(codes, scales) -> np.ndarray:
    """The float64 values code * 2^(scale - 127) of a checkpoint's rows; NaN for scale code 255."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    d = codes.shape[-1]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return e4m3_decode(codes) * np.repeat(s, MX_BLOCK, axis=-1)[..., :d]


def checkpoint_load(codes, scales) -> np.ndarray:
    """Those values rounded to bf16 (float64)."""
    v = checkpoint_values(codes, scales)
    out = np.full_like(v, np.nan)
    ok = np.isfinite(v)
    out[ok] = bf16_round(v[ok])
    return out


def fused_step_backward_ckpt(X, F, mixes, pre_prev, post_prev, comb_prev, W, scale, base, gain, gXp, gy,
                             gpre, gpost, gcomb, *, iters: int = 20, hc_eps: float = 1e-6,
                             norm_eps: float = 1e-6, comb_row_dest: bool = False) -> dict:
    """Gradients of the step at the values X, F of their checkpoints: X' = hc_post(X, F) and
    y_hat = hc_pre(X') as the forward evaluates and rounds them, the forward's mix numbers `mixes`
    given (oracle.backward has the formulas)."""
    X, F, m, W, gXp = (np.asarray(a, dtype=np.float64) for a in (X, F, mixes, W, gXp))
    N, n, d = X.shape
    Xp = hc_post(X, F, post_prev, comb_prev, comb_row_dest)
    y_hat = hc_pre(Xp, pre_prev)
    s, b = np.asarray(scale, dtype=np.float64), np.asarray(base, dtype=np.float64)
    _, tape = sinkhorn_taped((s[2] * m[:, 2 * n:] + b[2 * n:]).reshape(N, n, n), iters, hc_eps)
    gm, gbase, gscale = split_backward(m, scale, base, gpre, gpost, sinkhorn_backward(gcomb, tape), n)
    x = Xp.reshape(N, n * d)
    r = 1.0 / np.sqrt((x * x).sum(axis=1) / (n * d) + norm_eps)
    ga = gm * r[:, None]
    gx = (ga @ W - (r * r / (n * d) * (gm * m).sum(axis=1))[:, None] * x).reshape(N, n, d)
    gyh, ggain, _, _ = rmsnorm_backward(y_hat, gain, gy, norm_eps)
    p, u, C = (np.asarray(a, dtype=np.float64) for a in (pre_prev, post_prev, comb_prev))
    G = gXp + gx + p[:, :, None] * gyh[:, None, :]
    C = np.swapaxes(C, 1, 2) if comb_row_dest else C
    gC = np.einsum("nkd,njd->njk", G, X)
    return {"gX": np.einsum("njk,nkd->njd", C, G), "gF": np.einsum("nk,nkd->nd", u, G),
            "gpre_prev": np.einsum("nd,njd->nj", gyh, Xp), "gpost_prev": np.einsum("nkd,nd->nk", G, F),
            "gcomb_prev": np.swapaxes(gC, 1, 2) if comb_row_dest else gC, "gW": ga.T @ x,
            "gbase": gbase, "gscale": gscale, "ggain": ggain, "gXp_total": G}
