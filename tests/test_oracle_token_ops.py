"""Pins of the oracle's token operators: closed forms, torch in float64 and
central differences (CPU)."""
import math

import numpy as np
import pytest
import torch

import oracle


def problem(B=5, V=23, seed=0, banned=0.0):
    rng = np.random.default_rng(seed)
    x = 3.0 * rng.normal(size=(B, V))
    t = rng.integers(0, V, size=B)
    if banned:
        mask = rng.random((B, V)) < banned
        mask[np.arange(B), t] = False
        x[mask] = -np.inf
    return x, t, rng


def test_uniform_row_closed_form():
    lp, ent, lse, top, ids = oracle.token_logprobs(np.zeros((1, 8)), [3], 3, 0.5)
    assert abs(lp[0] + math.log(8)) < 1e-14 and abs(ent[0] - math.log(8)) < 1e-14 and abs(lse[0] - math.log(8)) < 1e-14
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(top, -math.log(8))


@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
@pytest.mark.parametrize("banned", [0.0, 0.4])
def test_logprobs_against_torch(T, banned):
    x, t, _ = problem(seed=1, banned=banned)
    lp, ent, lse, top, ids = oracle.token_logprobs(x, t, 5, T)
    z = torch.from_numpy(x) / T
    logp = torch.log_softmax(z, dim=1)
    assert np.allclose(lp, logp[torch.arange(5), torch.from_numpy(t)])
    assert np.allclose(ent, torch.distributions.Categorical(logits=z.clamp_min(-1e9)).entropy())
    assert np.allclose(lse, torch.logsumexp(z, dim=1))
    want = torch.sort(torch.from_numpy(x), dim=1, descending=True, stable=True).indices[:, :5]
    assert np.array_equal(ids, want.numpy()) and np.allclose(top, logp.gather(1, want))


def test_logprobs_rows_without_a_distribution_and_ignored_rows():
    x = np.zeros((4, 3))
    x[0], x[1, 1], x[2, 0] = -np.inf, np.inf, np.nan
    lp, ent, lse, top, ids = oracle.token_logprobs(x, [0, 0, 1, -100], 2)
    for r in range(3):
        assert np.isnan([lp[r], ent[r], lse[r], *top[r]]).all() and (ids[r] == -1).all()
    assert lp[3] == ent[3] == lse[3] == 0 and np.isneginf(top[3]).all() and (ids[3] == -1).all()


@pytest.mark.parametrize("T", [0.7, 1.0])
def test_vjp_against_autograd_and_differences(T):
    x, t, rng = problem(seed=2)
    gl, gh = rng.normal(size=5), rng.normal(size=5)
    t[2] = -100
    got = oracle.token_logprobs_vjp(x, t, gl, gh, T)
    z = torch.from_numpy(x).requires_grad_(True)
    logp = torch.log_softmax(z / T, dim=1)
    keep = torch.from_numpy(t != -100)
    lp = logp[torch.arange(5), torch.from_numpy(np.maximum(t, 0))]
    ent = -(logp.exp() * logp).sum(dim=1)
    ((torch.from_numpy(gl) * lp + torch.from_numpy(gh) * ent) * keep).sum().backward()
    assert np.allclose(got, z.grad.numpy(), atol=1e-14)
    h = 1e-6
    for r, j in [(0, 0), (1, 7), (3, int(t[3]))]:
        vals = []
        for s in (h, -h):
            y = x.copy()
            y[r, j] += s
            a = oracle.token_logprobs(y, t, 0, T)
            vals.append((gl * a[0] + gh * a[1]).sum())
        assert abs((vals[0] - vals[1]) / (2 * h) - got[r, j]) < 1e-7


def test_vjp_at_masked_logits_is_zero():
    x, t, rng = problem(seed=3, banned=0.5)
    got = oracle.token_logprobs_vjp(x, t, rng.normal(size=5), rng.normal(size=5))
    assert np.isfinite(got).all() and not got[np.isneginf(x)].any()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_distill_against_autograd(renorm, reduction):
    x, _, rng = problem(B=6, seed=4)
    T = 2.0
    ids = np.stack([rng.choice(23, size=4, replace=False) for _ in range(6)])
    ids[1, 2:], ids[4], ids[5, 3] = -1, -1, ids[5, 0]  # short row, empty row, an id twice
    v = rng.normal(size=(6, 4)) if renorm else np.log(rng.dirichlet(np.ones(5), size=6)[:, :4])
    v[0, 1] = -np.inf
    r = oracle.topk_distill(x, ids, v, T, renorm, reduction)
    z = torch.from_numpy(x).requires_grad_(True)
    logp = torch.log_softmax(z / T, dim=1)
    total = 0.0
    for row in (0, 1, 2, 3, 5):
        ok = [k for k in range(4) if ids[row, k] >= 0 and v[row, k] > -np.inf]
        w = torch.tensor(v[row, ok])
        q = torch.softmax(w / T, dim=0) if renorm else w.exp()
        total = total + T * T * (q * (q.log() - logp[row, ids[row, ok]])).sum()
    total = total / 5 if reduction == "mean" else total
    total.backward()
    assert r["n_valid"] == 5 and abs(r["loss"] - total.item()) < 1e-12
    assert np.allclose(r["grad"], z.grad.numpy(), atol=1e-14) and not r["grad"][4].any()


def test_distill_from_the_students_own_top_entries_has_no_gradient_when_all_are_kept():
    x, t, _ = problem(V=9, seed=5)
    _, _, _, top, ids = oracle.token_logprobs(x, t, 9, 1.5)
    r = oracle.topk_distill(x, ids, top, 1.5, False, "sum")
    assert abs(r["loss"]) < 1e-13 and np.abs(r["grad"]).max() < 1e-15
