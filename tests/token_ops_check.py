"""Helpers of the token operators' GPU parity tests: inputs and tolerances.

Derived from the kernels' fp32 arithmetic.  Every exponential is 2^y with
y = x log2(e) / T less a row constant, formed by at most two roundings, so its
relative error (and lse's, which sums them) is below

    eps = 4e-7 max(1, max |x| / T)     (finite logits of the row; ex2.approx 2^-22)

* logprob, top_logprob:  2 eps + 2^-22 |log p|       (the exponent and lse)
* lse:                   eps + 2^-22 |lse|
* entropy:               eps (2 + 2 H)               (sum p |log p + H| <= 2 H)
* logits gradient of (g_l, g_H): one rounding of the output (eps/2 of its type
  relative to the value; 2^-22 for fp32, whose sums round more than once) and,
  through p and log p, (1/T) p (|g_l| + |g_H| (|log p| + H + 1)) (eps +
  2^-22 max(1, |lse|)), the given lse being rounded to fp32; at the given token
  also 2^-22 |g_l| / T.
* distillation: row loss T^2 (2 eps Q + 2^-19 sum q (|log q| + |log p| + 1) +
  2^-22 Q max |v| / T); gradient one rounding of the output and
  scale T (Q p (eps + 2^-20) + q (2^-20 + 2^-22 max |v| / T)).
"""
import numpy as np
import torch

import oracle

OUT_EPS = {torch.float32: 2.0 ** -22, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}
TINY = 2.0 ** -120  # results flushed to zero


def logits(B, V, dtype, seed, pad=0, sigma=3.0):
    """[B, V] CUDA logits with rows V + pad apart, and the same in float64."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (sigma * torch.randn(B, V + pad, generator=g, device="cuda")).to(dtype)[:, :V]
    return x


def f64(t):
    return t.detach().double().cpu().numpy()


def row_eps(x64, T):
    a = np.where(np.isfinite(x64), np.abs(x64), 0.0)
    return 4e-7 * np.maximum(1.0, a.max(axis=1) / T)


def close(got, want, tol, what):
    """Equal where `want` is not finite, within `tol` elsewhere."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    tol = np.broadcast_to(tol, want.shape)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), f"{what}: infinities differ"
    err = np.abs(got[fin] - want[fin])
    bad = err > tol[fin]
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {err[bad].max():.3g} (bound {tol[fin][bad].min():.3g})"


def check_logprobs(x, index, k, T, out, ignore_index=-100, what=""):
    x64, t = f64(x), index.cpu().numpy()
    lp, ent, lse, top, ids = oracle.token_logprobs(x64, t, k, T, ignore_index)
    eps = row_eps(x64, T)
    close(f64(out[0]), lp, 2 * eps + 2.0 ** -22 * np.abs(lp), what + " logprob")
    close(f64(out[1]), ent, eps * (2 + 2 * ent), what + " entropy")
    with np.errstate(over="ignore"):
        lse = lse.astype(np.float32).astype(np.float64)  # beyond fp32's range the rounded value is infinite
    lse_tol = eps + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    close(f64(out[2]), lse, lse_tol, what + " lse")
    if k:
        assert np.array_equal(out[4].cpu().numpy(), ids), what + " top_index"
        tol = 2 * eps[:, None] + 2.0 ** -22 * np.abs(np.where(np.isfinite(top), top, 0.0))
        close(f64(out[3]), top, tol, what + " top_logprob")
    else:
        assert out[3] is None and out[4] is None


def check_vjp(x, index, gl, gH, T, grad, ignore_index=-100, what=""):
    x64, t = f64(x), index.cpu().numpy()
    gl64, gH64 = f64(gl), np.zeros(len(t)) if gH is None else f64(gH)
    want = oracle.token_logprobs_vjp(x64, t, gl64, gH64, T, ignore_index)
    valid = t != ignore_index
    _, ent, lse, _, _ = oracle.token_logprobs(x64, t, 0, T, ignore_index)
    logp = np.where(valid[:, None], x64 / T - lse[:, None], 0.0)
    p = np.exp(logp)
    alog = np.where(p > 0, np.abs(np.maximum(logp, -1e5)), 0.0)
    # beyond 1024 the kernel does not use the given lse
    eps = row_eps(x64, T) + 2.0 ** -22 * np.clip(np.abs(lse), 1.0, 1024.0)
    tol = OUT_EPS[x.dtype] * np.abs(want) + TINY
    tol = tol + p * (np.abs(gl64)[:, None] + np.abs(gH64)[:, None] * (alog + ent[:, None] + 1)) * (eps / T)[:, None]
    rows = np.nonzero(valid)[0]
    tol[rows, t[rows]] += 2.0 ** -22 * np.abs(gl64[rows]) / T
    close(f64(grad), want, tol, what)
    assert not f64(grad)[~valid].any(), what + ": ignored rows must be zero"


def check_distill(x, ids, values, T, renorm, reduction, loss, grad, row_loss=None, what=""):
    x64, i64, v64 = f64(x), ids.cpu().numpy(), f64(values)
    r = oracle.topk_distill(x64, i64, v64, T, renorm, reduction)
    B = x64.shape[0]
    scale = 1.0 / max(r["n_valid"], 1) if reduction == "mean" else 1.0
    eps = row_eps(x64, T)
    row_tol, tol = np.zeros(B), np.zeros_like(x64)
    for b in range(B):
        ok = (i64[b] != -1) & (v64[b] != -np.inf)
        if not ok.any():
            continue
        v, at = v64[b][ok], i64[b][ok]
        log_q = v / T - (np.max(v / T) + np.log(np.exp(v / T - np.max(v / T)).sum())) if renorm else v
        q = np.exp(log_q)
        z = x64[b] / T
        logp = z - (z.max() + np.log(np.exp(z - z.max()).sum()))
        vmax = np.abs(v).max() / T
        big = np.where(q > 0, q * (np.abs(log_q) + np.abs(logp[at]) + 1), 0.0).sum()
        row_tol[b] = T * T * (2 * eps[b] * q.sum() + 2.0 ** -19 * big + 2.0 ** -22 * q.sum() * vmax)
        tol[b] = scale * T * q.sum() * np.exp(logp) * (eps[b] + 2.0 ** -20)
        np.add.at(tol[b], at, scale * T * q * (2.0 ** -20 + 2.0 ** -22 * vmax))
    if row_loss is not None:
        close(f64(row_loss), r["row_loss"], row_tol, what + " row loss")
    assert abs(loss.item() - r["loss"]) <= scale * row_tol.sum() + 2.0 ** -22 * abs(r["loss"]), what + " loss"
    if grad is not None:
        close(f64(grad), r["grad"], tol + OUT_EPS[x.dtype] * np.abs(r["grad"]) + TINY, what + " grad")


def straddling_rows(B, V, T, seed):
    """fp32 rows whose logits times log2(e) / T lie on both sides of -2^20, where
    sums relative to 0 end: the lower ones just below it, the higher ones just
    above, in places that fall to other batches, warps and CTAs of a row.  Equal
    steps of 1 nat (T = 1) or 3 (T = 1e-4), at most 6 of them in a row."""
    low, high = (-726818.0, -726817.0) if T == 1.0 else (-72.6820, -72.6817)
    x = torch.full((B, V), low, device="cuda")
    x[0, V - 10:] = high           # the lower ones first
    x[1, :10] = high               # the higher ones first
    x[2, V // 2] = high
    x[3, 3 * V // 4:] = high
    x[4, ::777] = high
    x[5] = high                    # none below
    x[6, V // 3:] = high - 3 * (high - low)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x[7:] = low + (high - low) * torch.randint(-3, 4, (B - 7, V), generator=g, device="cuda").float()
    return x


# The bound for these rows: a logit times c is one fused multiply-add from its
# row's reference, or a product of its exact distance to the row's maximum, so
# that neither's size matters: y is off by |y| 2^-23 for c's rounding and its own,
# |y| <= 27 (18 nats and the reference's rounding), which 2^y has as 27 ln 2 2^-23
# < 2^-18.7 relative; with 2^-22 of ex2, 2^-20 of the sums and a few roundings of
# 2^-24 that is below 2^-17 for p, log p and the entropy's p (log p + H).
STRADDLE = 2.0 ** -17
