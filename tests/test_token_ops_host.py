"""Refusals of the token operators' entry points, before anything reaches the
GPU (no GPU needed)."""
import pytest
import torch

import lm_head_cross_gh_b200 as gh

FAKE = 0x7F0000000000  # a well-aligned non-null address; never dereferenced


def at(k):
    return FAKE + (k << 32)


@pytest.fixture(scope="module")
def L():
    from lm_head_cross_gh_b200 import _build
    _build.build()
    return gh.lib()


BAD, UNSUPPORTED = gh.GH_ERR_INVALID_ARG, gh.GH_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), BAD), (dict(V=0), BAD), (dict(V=1 << 31, ld=1 << 31), BAD), (dict(ld=99), BAD), (dict(dtype=2), BAD),
    (dict(T=0.0), BAD), (dict(T=-1.0), BAD), (dict(T=float("nan")), BAD), (dict(T=float("inf")), BAD),
    (dict(T=1e-5), BAD), (dict(T=1e5), BAD),
    (dict(k=-1), BAD), (dict(k=101), BAD), (dict(k=129, V=1000, ld=1000), UNSUPPORTED),
    (dict(logits=None), BAD), (dict(index=None), BAD), (dict(logprob=None), BAD), (dict(entropy=None), BAD),
    (dict(lse=None), BAD), (dict(top=None), BAD), (dict(ids=None), BAD),
    (dict(logits=at(0) + 1), BAD), (dict(index=at(1) + 4), BAD), (dict(lse=at(4) + 2), BAD), (dict(ids=at(6) + 4), BAD),
    (dict(B=0, logits=None), gh.GH_OK),
    (dict(B=1 << 31), UNSUPPORTED), (dict(B=1, V=1 << 26, ld=1 << 26), UNSUPPORTED),  # grid; a row of 128 MiB
])
def test_token_logprobs_refusals(L, kw, expect):
    a = dict(logits=at(0), ld=100, index=at(1), B=16, V=100, dtype=gh.GH_BF16, T=1.0, k=5, logprob=at(2),
             entropy=at(3), lse=at(4), top=at(5), ids=at(6))
    a.update(kw)
    assert L.gh_token_logprobs(a["logits"], a["ld"], a["index"], a["B"], a["V"], a["dtype"], -100, a["T"], a["k"],
                               a["logprob"], a["entropy"], a["lse"], a["top"], a["ids"], None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), BAD), (dict(V=0), BAD), (dict(ld=99), BAD), (dict(ldg=99), BAD), (dict(dtype=-1), BAD),
    (dict(T=0.0), BAD), (dict(T=float("nan")), BAD),
    (dict(logits=None), BAD), (dict(index=None), BAD), (dict(lse=None), BAD), (dict(entropy=None), BAD),
    (dict(gl=None), BAD), (dict(grad=None), BAD), (dict(grad=at(6) + 1), BAD), (dict(gH=at(5) + 2), BAD),
    (dict(grad=at(0) + 64), BAD),            # partial overlap
    (dict(grad=at(0), ldg=128), BAD),        # in place with another row stride
    (dict(B=0, grad=None), gh.GH_OK),
    (dict(B=1 << 31, V=1, ld=1, ldg=1), UNSUPPORTED),
])
def test_token_logprobs_vjp_refusals(L, kw, expect):
    a = dict(logits=at(0), ld=100, index=at(1), B=16, V=100, dtype=gh.GH_F32, T=1.0, lse=at(2), entropy=at(3),
             gl=at(4), gH=at(5), grad=at(6), ldg=100)
    a.update(kw)
    assert L.gh_token_logprobs_vjp(a["logits"], a["ld"], a["index"], a["B"], a["V"], a["dtype"], -100, a["T"],
                                   a["lse"], a["entropy"], a["gl"], a["gH"], a["grad"], a["ldg"], None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), BAD), (dict(V=0), BAD), (dict(K=0), BAD), (dict(K=129), UNSUPPORTED), (dict(ld=99), BAD),
    (dict(ldg=99), BAD), (dict(dtype=5), BAD), (dict(T=0.0), BAD), (dict(T=float("inf")), BAD), (dict(renorm=2), BAD),
    (dict(red=3), BAD), (dict(logits=None), BAD), (dict(ids=None), BAD), (dict(vals=None), BAD), (dict(loss=None), BAD),
    (dict(loss=at(4) + 2), BAD), (dict(total=at(7) + 4), BAD), (dict(row=at(5) + 1), BAD), (dict(vals=at(2) + 2), BAD),
    (dict(grad=at(0) + 64), BAD), (dict(grad=at(0), ldg=128), BAD),
    (dict(B=1 << 31, grad=None), UNSUPPORTED),
])
def test_topk_distill_refusals(L, kw, expect):
    a = dict(logits=at(0), ld=100, ids=at(1), vals=at(2), B=16, V=100, K=8, dtype=gh.GH_BF16, T=1.0, renorm=1, red=0,
             total=None, loss=at(4), row=None, grad=at(6), ldg=100)
    a.update(kw)
    assert L.gh_topk_distill(a["logits"], a["ld"], a["ids"], a["vals"], a["B"], a["V"], a["K"], a["dtype"], a["T"],
                             a["renorm"], a["red"], a["total"], a["loss"], a["row"], a["grad"], a["ldg"],
                             None) == expect


def test_distill_count_refusals(L):
    assert L.gh_distill_count(at(0), at(1), -1, 8, 100, at(2), None) == BAD
    assert L.gh_distill_count(at(0), at(1), 4, 0, 100, at(2), None) == BAD
    assert L.gh_distill_count(at(0), at(1), 4, 129, 100, at(2), None) == UNSUPPORTED
    assert L.gh_distill_count(at(0), at(1), 4, 8, 100, None, None) == BAD
    assert L.gh_distill_count(None, at(1), 4, 8, 100, at(2), None) == BAD
    assert L.gh_distill_count(at(0), at(1), 4, 8, 100, at(2) + 4, None) == BAD


def test_python_binding_refuses_cpu_tensors():
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    f, ids = torch.zeros(4), torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(ValueError):
        gh.gh_token_logprobs(x, t)
    with pytest.raises(ValueError):
        gh.gh_token_logprobs_vjp(x, t, f, f, f)
    with pytest.raises(ValueError):
        gh.gh_topk_distill(x, ids, torch.zeros(4, 2))
    with pytest.raises(ValueError):
        gh.gh_distill_count(ids, torch.zeros(4, 2), 8)


def test_threshold_search_ends_for_every_key(tmp_path):
    """The alternatives' search over order keys (tests/threshold_search_check.cpp):
    a NaN's key beside lanes without a key spans the whole 32-bit range."""
    import os
    import shutil
    import subprocess
    gxx = shutil.which("g++") or shutil.which("c++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "threshold_search_check")
    build = subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
                            os.path.join(here, "threshold_search_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr[:2000]
    assert " 0 failed checks" in run.stdout


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), BAD), (dict(V=0), BAD), (dict(ld=98), BAD), (dict(ldo=98), BAD), (dict(dtype=2), BAD),
    (dict(grad=None), BAD), (dict(g=None), BAD), (dict(out=None), BAD), (dict(grad=at(0) + 1), BAD),
    (dict(out=at(2) + 1), BAD), (dict(g=at(1) + 2), BAD),
    (dict(out=at(0) + 64), BAD),           # partial overlap
    (dict(out=at(0), ldo=128), BAD),       # in place with another row stride
    (dict(B=0, grad=None, g=None, out=None), gh.GH_OK),
    (dict(B=1 << 31), UNSUPPORTED), (dict(B=1 << 40, ld=1 << 40), UNSUPPORTED),
])
def test_scale_grad_refusals(L, kw, expect):
    a = dict(grad=at(0), ld=100, B=16, V=99, dtype=gh.GH_BF16, g=at(1), out=at(100), ldo=100)
    a.update(kw)
    assert L.gh_scale_grad(a["grad"], a["ld"], a["B"], a["V"], a["dtype"], a["g"], a["out"], a["ldo"], None) == expect


def test_a_bf16_gradient_is_scaled_by_the_unrounded_upstream_gradient():
    from lm_head_cross_gh_b200 import functional as GF
    torch.manual_seed(0)
    x = torch.randn(64, 100).to(torch.bfloat16)
    for g in (0.3, 1.0 / 3.0, -1.37):
        got = GF._scaled(x, torch.tensor(g))
        assert torch.equal(got, (x.float() * g).to(torch.bfloat16))
        # over many elements the roundings' mean is far below g's own in bf16 (0.1 to 0.3%):
        # 6400 of at most 2^-8 each, 2^-8 / 80 as a random walk, bounded at 5 of those
        ratio = float((got.double() * x.double()).sum() / (x.double() ** 2).sum()) / float(torch.tensor(g))
        assert abs(ratio - 1.0) <= 5 * 2.0 ** -8 / 80


def test_functional_forms_refuse_companions_of_another_shape():
    """Rows of an index, ids or values of another shape than the logits' would be
    paired wrongly, whatever their number."""
    from lm_head_cross_gh_b200 import functional as GF
    x, i, v = torch.zeros(2, 6, 9), torch.zeros(2, 6, 3, dtype=torch.int64), torch.zeros(2, 6, 3)
    for index in (i[..., 0].t(), i[0, :, 0], i.reshape(4, 9), i[..., :2], i[:1, :, 0], i[0, 0, 0]):
        with pytest.raises(ValueError, match="index"):
            GF.token_logprobs(x, index)
    for ids, values, name in ((i.transpose(0, 1), v, "teacher_index"), (i[:1], v, "teacher_index"),
                              (i.reshape(4, 9), v, "teacher_index"), (i, v.transpose(0, 1), "teacher_logits"),
                              (i, v.reshape(2, 9, 2), "teacher_logits"), (i, v[..., :2], "teacher_logits"),
                              (i, v.reshape(4, 9), "teacher_logits")):
        with pytest.raises(ValueError, match=name):
            GF.topk_distillation(x, ids, values)
    X, W = torch.zeros(12, 8), torch.zeros(9, 8)
    for ids, values, name in ((i[0], v[0], "teacher_index"), (i.reshape(12, 3), v[0], "teacher_logits"),
                              (i, v, "teacher_index"), (i.reshape(12, 3), v.reshape(3, 12).t()[:, :2], "teacher_logits")):
        with pytest.raises(ValueError, match=name):
            GF.chunked_linear_topk_distillation(X, W, ids, values)


def test_dense_rows_of_a_vocabulary_of_one():
    """Rows that share their one logit (a broadcast) are copied like any others that overlap."""
    from lm_head_cross_gh_b200 import functional as GF
    for V in (1, 3):
        x = GF._dense_rows(torch.ones(1, V).expand(4, V))
        assert x.shape == (4, V) and x.stride(0) >= V and (V == 1 or x.stride(1) == 1)
    x = torch.ones(4, 6)[:, :1]
    assert GF._dense_rows(x) is x


@pytest.mark.parametrize("dtype,step", [(torch.float32, 4), (torch.bfloat16, 8)])
def test_the_gradient_of_rows_far_apart_is_not_as_wide(dtype, step):
    """The gradient's own rows (one position's logits out of [B, S, V]): close
    together, each at its logits' offset from 16 bytes; a padded head's keep their stride."""
    for S, V in ((64, 101), (3, 64), (1000, 7), (5, 1)):
        x = torch.zeros(6, S, V, dtype=dtype)[:, -1]
        grad, ld = gh._grad_like(None, x, 6, V, S * V, torch)
        assert grad.shape == (6, V) and grad.stride(0) == ld and V <= ld < V + step and (ld - S * V) % step == 0
        assert grad.untyped_storage().nbytes() <= 6 * (V + step) * grad.element_size()
    x = torch.zeros(6, 104, dtype=dtype)[:, :101]
    assert gh._grad_like(None, x, 6, 101, 104, torch)[1] == 104
