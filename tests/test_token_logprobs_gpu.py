"""GPU parity of gh_token_logprobs and gh_token_logprobs_vjp against the float64
oracle (tolerances: token_ops_check)."""
import math

import numpy as np
import pytest
import torch

import lm_head_cross_gh_b200 as gh
from lm_head_cross_gh_b200 import functional as GF
from token_ops_check import STRADDLE, check_logprobs, check_vjp, logits, straddling_rows

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]


def given(B, V, seed, ignored=0.2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.randint(0, V, (B,), generator=g, device="cuda")
    t[torch.rand(B, generator=g, device="cuda") < ignored] = -100
    return t


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 63, 64, 65, 129, 1023, 1025, 4099, 8191, 8193, 50257])
def test_sizes(cuda_device, dtype, V):
    B = 11 if V < 9000 else 5
    for k, T, pad in ((0, 1.0, 0), (min(V, 1), 0.7, 3), (min(V, 20), 2.0, 0), (min(V, 128), 1.0, 5)):
        x, t = logits(B, V, dtype, V + k, pad), given(B, V, V + k)
        out = gh.gh_token_logprobs(x, t, k, T)
        check_logprobs(x, t, k, T, out, what=f"{dtype} V={V} k={k} T={T} pad={pad}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V,k", [(1, 50257, 20), (2, 262144, 128), (150, 5003, 64), (300, 1000, 5),
                                   (1300, 2003, 33), (2500, 131, 128), (1200, 8200, 20)])
def test_batches(cuda_device, dtype, B, V, k):
    x, t = logits(B, V, dtype, B), given(B, V, B)
    out = gh.gh_token_logprobs(x, t, k, 1.3)
    check_logprobs(x, t, k, 1.3, out, what=f"{dtype} {B}x{V}")
    again = gh.gh_token_logprobs(x, t, k, 1.3)
    for a, b in zip(out, again):
        assert torch.equal(a, b), "two calls differ"


def test_long_rows_of_a_few_tokens(cuda_device):
    # rows far longer than any vocabulary: still one answer per row
    x, t = logits(3, 3_000_001, torch.bfloat16, 1, sigma=2.0), given(3, 3_000_001, 1, 0.0)
    check_logprobs(x, t, 40, 1.0, gh.gh_token_logprobs(x, t, 40))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [6, 1250])
def test_ties_go_to_the_lowest_index(cuda_device, dtype, B):
    V = 3001
    x = logits(B, V, dtype, 3).round()  # a few dozen distinct values
    x[0] = 0.25                          # all alike
    x[1] = torch.arange(V, device="cuda").to(dtype)          # rising (bf16: runs of equal values)
    x[2] = -torch.arange(V, device="cuda").to(dtype)
    x[3] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0).to(dtype)  # both zeros are one value
    x[4] = -5.0
    x[4, -60:] = 7.0
    t = given(B, V, 4, 0.0)
    for k in (1, 20, 128):
        check_logprobs(x, t, k, 1.0, gh.gh_token_logprobs(x, t, k), what=f"k={k}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [7, 1250])
def test_masked_and_non_finite_logits(cuda_device, dtype, B):
    V, k = 2053, 20
    low = torch.finfo(dtype).min
    x = logits(B, V, dtype, 5)
    t = given(B, V, 6, 0.0)
    x[0, 3:] = -math.inf                 # fewer tokens than alternatives
    x[1] = -math.inf                     # nothing left: no distribution
    x[2] = low                           # a mask of the lowest value that leaves nothing: uniform
    x[3, ::2] = low
    x[4, 100] = math.nan
    x[5, 2000] = math.inf
    x[6, : V - 1] = -math.inf            # one token left
    if B > 10:
        x[7] = low
        x[7, 5:900] = -math.inf          # lowest values and -inf: uniform over the former
        x[8] = -1000.0
        x[9] = x[9] * 50.0
    check_logprobs(x, t, k, 1.0, gh.gh_token_logprobs(x, t, k), what="T=1")
    check_logprobs(x, t, k, 0.5, gh.gh_token_logprobs(x, t, k, 0.5), what="T=0.5")
    # the gradient: zero at masked logits, NaN rows where there is no distribution
    for T in (1.0, 0.5):
        lp, ent, lse, _, _ = gh.gh_token_logprobs(x, t, 0, T)
        gl, gH = torch.randn(B, device="cuda"), torch.randn(B, device="cuda")
        grad = gh.gh_token_logprobs_vjp(x, t, lse, ent, gl, gH, T)
        assert torch.isnan(grad[[1, 4, 5]]).all()
        keep = [r for r in range(B) if r not in (1, 4, 5)]
        gone = torch.isneginf(x[keep]) & (torch.arange(V, device="cuda")[None] != t[keep][:, None])
        assert not grad[keep][gone].any()
        check_vjp(x[keep], t[keep], gl[keep], gH[keep], T, grad[keep], what=f"vjp T={T}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [3, 1250])
@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
def test_rows_far_from_zero_keep_their_distribution(cuda_device, dtype, B, T):
    """All logits at one value far below 0 (a mask that leaves nothing): the
    uniform distribution, in closed form.  2^-20 relative covers log2 and the
    few roundings; the row constant is exact because every difference is 0."""
    V = 1537
    x = logits(B, V, dtype, 51)
    t = given(B, V, 52, 0.0)
    for r, low in enumerate((torch.finfo(dtype).min, -1e9, -3e4)):
        x[r] = low
    lp, ent, lse, top, ids = gh.gh_token_logprobs(x, t, 3, T)
    want = torch.full((3,), math.log(V), device="cuda")
    assert torch.allclose(lp[:3], -want, rtol=2.0 ** -20, atol=0)
    assert torch.allclose(ent[:3], want, rtol=2.0 ** -20, atol=0)
    assert torch.allclose(top[:3], -want[:, None].expand(3, 3), rtol=2.0 ** -20, atol=0)
    assert (ids[:3] == torch.arange(3, device="cuda")).all()
    gl, gH = torch.full((B,), 2.0, device="cuda"), torch.full((B,), 3.0, device="cuda")
    grad = gh.gh_token_logprobs_vjp(x, t, lse, ent, gl, gH, T)[:3].float()
    expect = torch.full((3, V), -2.0 / V / T, device="cuda")
    expect[torch.arange(3), t[:3]] += 2.0 / T
    # the entropy's part is 3 p (log p + H) / T = 0 up to the rounding of log p + H (2^-19 log V)
    tol = expect.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -18) + 3.0 * math.log(V) * 2.0 ** -19 / V / T
    assert ((grad - expect).abs() <= tol).all()


def test_extreme_temperatures(cuda_device):
    x, t = logits(9, 777, torch.float32, 7), given(9, 777, 7)
    for T in (1e-4, 1e4):
        check_logprobs(x, t, 9, T, gh.gh_token_logprobs(x, t, 9, T), what=f"T={T}")


def test_index_out_of_range_and_ignore_index_inside_the_vocabulary(cuda_device):
    gh.gh_get_device_status()
    x = logits(4, 300, torch.bfloat16, 8)
    t = torch.tensor([5, 300, 7, -3], device="cuda")
    out = gh.gh_token_logprobs(x, t, 4)
    torch.cuda.synchronize()
    assert gh.gh_get_device_status() == gh.GH_ERR_TARGET_RANGE
    for v in out[:4]:
        assert torch.isnan(v[[1, 3]]).all()
    assert (out[4][[1, 3]] == -1).all()
    check_logprobs(x[[0, 2]], t[[0, 2]], 4, 1.0, [v[[0, 2]] for v in out])
    g = gh.gh_token_logprobs_vjp(x, t, out[2], out[1], torch.ones(4, device="cuda"))
    assert gh.gh_get_device_status() == gh.GH_ERR_TARGET_RANGE
    assert not g[[1, 3]].any()
    t = torch.tensor([5, 5, 7, 5], device="cuda")
    check_logprobs(x, t, 3, 1.0, gh.gh_token_logprobs(x, t, 3, 1.0, 5), ignore_index=5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 100, 1023, 1025, 8191, 50257])
def test_vjp_sizes(cuda_device, dtype, V):
    B = 37 if V < 20000 else 9
    for T, pad, with_h in ((1.0, 0, True), (0.6, 3, True), (2.0, 0, False)):
        x, t = logits(B, V, dtype, V, pad), given(B, V, V)
        _, ent, lse, _, _ = gh.gh_token_logprobs(x, t, 0, T)
        gl = torch.randn(B, device="cuda")
        gH = torch.randn(B, device="cuda") if with_h else None
        gl[::5] = 0.0
        grad = gh.gh_token_logprobs_vjp(x, t, lse, ent, gl, gH, T)
        check_vjp(x, t, gl, gH, T, grad, what=f"{dtype} V={V} T={T}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_vjp_in_place_other_phase_and_untouched_padding(cuda_device, dtype):
    B, V = 40, 3001
    x, t = logits(B, V, dtype, 11, pad=7), given(B, V, 11)
    _, ent, lse, _, _ = gh.gh_token_logprobs(x, t)
    gl, gH = torch.randn(B, device="cuda"), torch.randn(B, device="cuda")
    want = gh.gh_token_logprobs_vjp(x, t, lse, ent, gl, gH)
    check_vjp(x, t, gl, gH, 1.0, want)
    buf = torch.full((B * 3050 + 16,), 9.0, dtype=dtype, device="cuda")
    shifted = buf[3:3 + B * 3050].view(B, 3050)[:, :V]   # another 16-byte phase and row stride
    gh.gh_token_logprobs_vjp(x, t, lse, ent, gl, gH, grad=shifted)
    assert torch.equal(shifted, want)
    rest = buf.clone()
    rest[3:3 + B * 3050].view(B, 3050)[:, :V] = 9.0
    assert (rest == 9.0).all(), "wrote outside the gradient"
    whole = torch.full((B, V + 7), 9.0, dtype=dtype, device="cuda")
    whole[:, :V] = x
    y = whole[:, :V]
    gh.gh_token_logprobs_vjp(y, t, lse, ent, gl, gH, grad=y)
    assert torch.equal(y, want) and (whole[:, V:] == 9.0).all()


def test_vjp_many_rows(cuda_device):
    x, t = logits(1500, 5003, torch.bfloat16, 12), given(1500, 5003, 12)
    _, ent, lse, _, _ = gh.gh_token_logprobs(x, t)
    gl, gH = torch.randn(1500, device="cuda"), torch.randn(1500, device="cuda")
    check_vjp(x, t, gl, gH, 1.0, gh.gh_token_logprobs_vjp(x, t, lse, ent, gl, gH))


def test_offsets_beyond_32_bits(cuda_device):
    B, V = 17000, 131072  # 2.2e9 logits
    x = torch.zeros(B, V, dtype=torch.bfloat16, device="cuda")
    tail = logits(8, V, torch.bfloat16, 13)
    x[-8:] = tail
    t = torch.full((B,), -100, dtype=torch.int64, device="cuda")
    t[-8:] = given(8, V, 13, 0.0)
    out = gh.gh_token_logprobs(x, t, 16)
    check_logprobs(tail, t[-8:], 16, 1.0, [v[-8:] for v in out])
    gl = torch.ones(B, device="cuda")
    g = gh.gh_token_logprobs_vjp(x, t, out[2], out[1], gl, gl, grad=x)
    check_vjp(tail, t[-8:], gl[-8:], gl[-8:], 1.0, g[-8:])
    assert not g[:-8].any()


def test_empty_batch(cuda_device):
    x, t = torch.empty(0, 5, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    lp, ent, lse, top, ids = gh.gh_token_logprobs(x, t, 2)
    assert lp.shape == ent.shape == lse.shape == (0,) and top.shape == ids.shape == (0, 2)
    z = torch.empty(0, device="cuda")
    assert gh.gh_token_logprobs_vjp(x, t, z, z, z).shape == (0, 5)


@pytest.mark.parametrize("B,V", [(3, 50257), (1300, 2003)])
def test_captured_graphs_and_streams(cuda_device, B, V):
    # two graphs of the same call on other inputs, replayed in turn and on two streams
    k = 20
    xs = [logits(B, V, torch.bfloat16, s) for s in (21, 22)]
    ts = [given(B, V, s) for s in (21, 22)]
    want = [gh.gh_token_logprobs(x, t, k) for x, t in zip(xs, ts)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for x, t in zip(xs, ts):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gh.gh_token_logprobs(x, t, k))
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            for v in o:
                v.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for a, b in zip(o, w):
                assert torch.equal(a, b)
    # two calls at once on two streams
    with torch.cuda.stream(side):
        a = gh.gh_token_logprobs(xs[0], ts[0], k)
    b = gh.gh_token_logprobs(xs[1], ts[1], k)
    torch.cuda.synchronize()
    for o, w in zip((a, b), want):
        assert all(torch.equal(p, q) for p, q in zip(o, w))


def test_given_outputs_are_written_and_nothing_behind_them(cuda_device):
    B, V, k = 13, 1001, 7
    x, t = logits(B, V, torch.float32, 31), given(B, V, 31)
    f = torch.full((4, B + 3), 5.0, device="cuda")
    top, ids = torch.full((B + 2, k), 5.0, device="cuda"), torch.full((B + 2, k), 5, device="cuda")
    out = gh.gh_token_logprobs(x, t, k, logprob=f[0, :B], entropy=f[1, :B], lse=f[2, :B], top_logprob=top[:B],
                               top_index=ids[:B])
    check_logprobs(x, t, k, 1.0, out)
    assert (f[:3, B:] == 5.0).all() and (top[B:] == 5.0).all() and (ids[B:] == 5).all()


def test_functional_gradients(cuda_device):
    """Autograd against the formula (float64 autograd) and against differences."""
    torch.manual_seed(1)
    x = torch.randn(2, 3, 50, device="cuda", requires_grad=True)
    t = torch.randint(0, 50, (2, 3), device="cuda")
    t[0, 1] = -100
    gl, gH = torch.randn(2, 3, device="cuda"), torch.randn(2, 3, device="cuda")
    lp, ent, top, ids = GF.token_logprobs(x, t, 4, 0.8)
    assert lp.shape == ent.shape == (2, 3) and top.shape == ids.shape == (2, 3, 4)
    assert not top.requires_grad and not ids.requires_grad
    (gl * lp + gH * ent).sum().backward()
    y = x.detach().double().requires_grad_(True)

    def value(z):
        logp = torch.log_softmax(z / 0.8, dim=-1)
        l = logp.gather(-1, t.clamp_min(0)[..., None])[..., 0]
        h = -(logp.exp() * logp).sum(-1)
        return ((gl * l + gH * h) * (t != -100)).sum()

    value(y).backward()
    assert torch.allclose(x.grad.double(), y.grad, rtol=1e-5, atol=1e-6)
    d = torch.randn(2, 3, 50, device="cuda", dtype=torch.float64)
    diff = (value(y.detach() + 1e-5 * d) - value(y.detach() - 1e-5 * d)) / 2e-5
    assert abs((x.grad.double() * d).sum() - diff) < 1e-4
    with torch.no_grad():
        lp2, ent2 = GF.token_logprobs(x, t, temperature=0.8)
    assert torch.equal(lp2, lp) and torch.equal(ent2, ent)
    # a sequence dimension that is not dense, and a broadcast upstream gradient
    xt = x.detach().transpose(0, 1)
    assert torch.equal(GF.token_logprobs(xt, t.t(), temperature=0.8)[0], lp.t())
    xb = x.detach().clone().requires_grad_(True)
    GF.token_logprobs(xb, t, temperature=0.8)[0].sum().backward()
    assert torch.allclose(xb.grad.sum(-1), torch.zeros(2, 3, device="cuda"), atol=1e-5)


def test_selected_value_agrees_with_selective_log_softmax(cuda_device):
    x, t = logits(200, 50257, torch.bfloat16, 41), given(200, 50257, 41, 0.0)
    lp = gh.gh_token_logprobs(x, t)[0]
    sel = gh.gh_selective_log_softmax(x, t)
    eps = 4e-7 * max(1.0, float(x.abs().max()))
    assert (lp - sel).abs().max().item() <= 4 * eps + 2.0 ** -21 * float(sel.abs().max())


def test_keyword_arguments(cuda_device):
    x, t = logits(5, 333, torch.float32, 61), given(5, 333, 61)
    out = gh.gh_token_logprobs(logits=x, index=t, top_k=3, temperature=0.9)
    check_logprobs(x, t, 3, 0.9, out)
    g = torch.ones(5, device="cuda")
    a = gh.gh_token_logprobs_vjp(logits=x, index=t, lse=out[2], entropy=out[1], g_logprob=g, temperature=0.9)
    check_vjp(x, t, g, None, 0.9, a)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V,k", [(2, 60001, 20), (20, 33000, 128), (3, 400_003, 7)])
def test_rows_split_over_a_cluster_with_odd_contents(cuda_device, dtype, B, V, k):
    """Small batches: a row's CTAs each see a part of it."""
    x = logits(B, V, dtype, 71, pad=5).round()               # ties across the parts
    t = given(B, V, 71, 0.0)
    check_logprobs(x, t, k, 1.0, gh.gh_token_logprobs(x, t, k), what="ties")
    x[0] = -math.inf
    x[0, V // 2: V // 2 + 3] = 1.0                            # one part has all the mass
    check_logprobs(x, t, k, 0.7, gh.gh_token_logprobs(x, t, k, 0.7), what="one part")
    x[0, 5] = math.nan                                        # and a NaN in another
    check_logprobs(x, t, k, 0.7, gh.gh_token_logprobs(x, t, k, 0.7), what="NaN")
    x[0] = math.nan
    x[1] = torch.finfo(dtype).min
    check_logprobs(x, t, k, 1.0, gh.gh_token_logprobs(x, t, k), what="all NaN, all lowest")
    x[0] = torch.arange(V, device="cuda").to(dtype) / 1000    # the last part has every alternative
    check_logprobs(x, t, k, 1.0, gh.gh_token_logprobs(x, t, k), what="rising")


@pytest.mark.parametrize("k", [1, 128])
def test_more_candidates_than_are_kept(cuda_device, k):
    """One segment of large equal logits, and a plateau over half the row: more
    logits reach the threshold than the candidates' buffer holds."""
    B, V = 1100, 9001
    x = logits(B, V, torch.bfloat16, 81)
    x[0, 4000:] = 30.0
    x[1, 1000:1700] = 30.0
    x[2, ::3] = 30.0
    x[3, 3000:3000 + 4 * k] = torch.arange(4 * k, device="cuda").to(torch.bfloat16)
    t = given(B, V, 81, 0.0)
    rows = slice(0, 40)
    out = gh.gh_token_logprobs(x, t, k)
    check_logprobs(x[rows], t[rows], k, 1.0, [v[rows] for v in out])
    few = gh.gh_token_logprobs(x[:4], t[:4], k)  # four rows: other kernels
    check_logprobs(x[:4], t[:4], k, 1.0, few)


def test_nearly_certain_rows(cuda_device):
    """log p near 0 is held to about 1e-7 absolute: the rest's sum, not 1 + rest."""
    x = logits(64, 50257, torch.float32, 91)
    t = given(64, 50257, 91, 0.0)
    x[torch.arange(64), t] = torch.linspace(14.0, 30.0, 64, device="cuda")
    lp, ent, _, _, _ = gh.gh_token_logprobs(x, t)
    z = x.double()
    z[torch.arange(64), t] = -math.inf
    rest = torch.exp(torch.logsumexp(z, 1) - x.double()[torch.arange(64), t])
    # 50257 terms in 512 running sums of fp32: the sum that holds the 1 loses at
    # most 98 half steps of 2^-24, half a step's random walk 10; 2^-20 covers both
    assert ((lp.double() + torch.log1p(rest)).abs() <= 2.0 ** -20).all()
    assert (ent >= -2.0 ** -20).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_vjp_in_place_of_long_and_far_rows(cuda_device, dtype):
    """Rows of several parts, in place: rows far from 0 have their sums taken again
    by one of the parts, before any of the row is overwritten."""
    B, V = 6, 70001
    x, t = logits(B, V, dtype, 95), given(B, V, 95, 0.0)
    x[1] -= 30000.0
    x[2] = torch.finfo(dtype).min
    for T in (1.0, 0.5):
        _, ent, lse, _, _ = gh.gh_token_logprobs(x, t, 0, T)
        gl, gH = torch.randn(B, device="cuda"), torch.randn(B, device="cuda")
        want = gh.gh_token_logprobs_vjp(x, t, lse, ent, gl, gH, T)
        check_vjp(x, t, gl, gH, T, want)
        for _ in range(5):
            y = x.clone()
            gh.gh_token_logprobs_vjp(y, t, lse, ent, gl, gH, T, grad=y)
            assert torch.equal(y, want)


def test_backward_captured_beside_an_eager_graph(cuda_device):
    """The functional forward and backward in a CUDA graph, replayed on new inputs,
    while eager calls of other leaves go on."""
    x = logits(300, 2003, torch.bfloat16, 97)
    t = given(300, 2003, 97)
    leaf = x.clone().requires_grad_(True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            lp, ent = GF.token_logprobs(leaf, t)
            torch.autograd.grad((lp + 0.1 * ent).sum(), leaf)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lp, ent = GF.token_logprobs(leaf, t)
        (grad,) = torch.autograd.grad((lp + 0.1 * ent).sum(), leaf)
    for seed in (98, 99):
        y = logits(300, 2003, torch.bfloat16, seed)
        with torch.no_grad():
            leaf.copy_(y)
        g.replay()
        other = y.clone().requires_grad_(True)
        lp2, ent2 = GF.token_logprobs(other, t)
        (lp2 + 0.1 * ent2).sum().backward()
        torch.cuda.synchronize()
        assert torch.equal(grad, other.grad) and torch.equal(lp, lp2)


@pytest.mark.parametrize("shape", [(0,), (2, 0), ()])
def test_functional_shapes_without_rows_and_of_one_row(cuda_device, shape):
    torch.manual_seed(2)
    x = torch.randn(*shape, 9, device="cuda", requires_grad=True)
    t = torch.ones(shape, dtype=torch.int64, device="cuda")
    lp, ent, top, ids = GF.token_logprobs(x, t, 3)
    assert lp.shape == ent.shape == shape and top.shape == ids.shape == (*shape, 3)
    (lp.sum() + ent.sum()).backward()
    assert x.grad.shape == x.shape
    if shape == ():
        assert torch.allclose(lp, torch.log_softmax(x.detach(), -1)[1], atol=1e-6)


def test_a_second_derivative_is_refused(cuda_device):
    x = torch.randn(4, 9, device="cuda", requires_grad=True)
    w = torch.ones(4, device="cuda", requires_grad=True)
    lp, _ = GF.token_logprobs(x, torch.zeros(4, dtype=torch.int64, device="cuda"))
    (g,) = torch.autograd.grad((w * lp).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V", [(4, 333), (1300, 1537), (4, 70001)])
@pytest.mark.parametrize("T", [1e-4, 1.0, 1e4])
def test_largest_finite_logits(cuda_device, dtype, B, V, T):
    """Rows whose n largest logits are equal and out of the others' reach, at the
    ends of the type's range: the uniform distribution over those n, in closed
    form (2^-20 relative for log2 and the few roundings, the gradient as for
    rows far from zero)."""
    big = torch.finfo(dtype).max
    x = torch.zeros(B, V, device="cuda", dtype=dtype)
    at = torch.tensor([V - 1, V // 2, 3], device="cuda")
    for r, (low, high) in enumerate(((-big, big), (0.0, big), (-big, 0.0), (big, big))):
        x[r::4] = low
        x[r::4, at] = high
    n = torch.full((B,), 3.0, device="cuda")
    n[3::4] = V
    t = torch.full((B,), V // 2, dtype=torch.int64, device="cuda")
    lp, ent, lse, top, ids = gh.gh_token_logprobs(x, t, 3, T)
    want = n.log()
    assert torch.allclose(lp, -want, rtol=2.0 ** -20, atol=0)
    assert torch.allclose(ent, want, rtol=2.0 ** -20, atol=0)
    assert torch.allclose(top, -want[:, None].expand(B, 3), rtol=2.0 ** -20, atol=0)
    order = torch.tensor([3, V // 2, V - 1], device="cuda").expand(B, 3).clone()
    order[3::4] = torch.arange(3, device="cuda")
    assert torch.equal(ids, order)
    gl, gH = torch.full((B,), 2.0, device="cuda"), torch.full((B,), 3.0, device="cuda")
    grad = gh.gh_token_logprobs_vjp(x, t, lse, ent, gl, gH, T).double()
    p = torch.zeros(B, V, device="cuda", dtype=torch.float64)
    p[:, at] = 1.0 / 3.0
    p[3::4] = 1.0 / V
    expect = -2.0 * p / T
    expect[:, V // 2] += 2.0 / T
    tol = expect.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -18) + 3.0 * math.log(V) * 2.0 ** -19 * p / T
    assert ((grad - expect).abs() <= tol).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V", [(6, 70001), (6, 700), (1300, 1537), (1300, 20001)])
def test_rows_of_nan_write_every_alternative(cuda_device, dtype, B, V):
    """Rows of NaN throughout, but for three logits, or for one half: every place
    of the given outputs is written."""
    x = logits(B, V, dtype, 17)
    x[0] = math.nan
    x[1] = math.nan
    x[1, 5:8] = 1.0
    x[2, : V // 2] = math.nan
    x[3, V // 2:] = math.nan
    k = 40
    top = torch.full((B, k), 5.0, device="cuda")
    ids = torch.full((B, k), 5, dtype=torch.int64, device="cuda")
    t = given(B, V, 18, 0.0)
    lp, ent, lse, _, _ = gh.gh_token_logprobs(x, t, k, top_logprob=top, top_index=ids)
    assert torch.isnan(torch.stack((lp[:4], ent[:4], lse[:4]))).all()
    assert torch.isnan(top[:4]).all() and (ids[:4] == -1).all()
    check_logprobs(x[4:], t[4:], k, 1.0, [v[4:] for v in (lp, ent, lse, top, ids)])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [4, 1300])
@pytest.mark.parametrize("mask", [None, -math.inf, "lowest"])
def test_alternatives_nearly_as_many_as_logits(cuda_device, dtype, B, mask):
    """Short rows whose alternatives are most of their logits, the ragged ends
    among them, at every alignment and with most logits masked."""
    for V in (9, 12, 18, 25, 73, 139, 150):
        for k in {1, 2, V // 2, min(V - 1, 128), min(V - 5, 128), min(V, 128)}:
            pad = (V + k) % 8
            x = logits(B, V, dtype, V + k, pad)
            if mask is not None:
                x[1::2, V // 5:] = torch.finfo(dtype).min if mask == "lowest" else mask
            t = torch.zeros(B, dtype=torch.int64, device="cuda")
            out = gh.gh_token_logprobs(x, t, k, 0.8)
            order = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :k]
            assert torch.equal(out[4], order), f"V={V} k={k}"
            if B < 10 and mask != "lowest":
                check_logprobs(x, t, k, 0.8, out, what=f"V={V} k={k}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [9, 1250])
@pytest.mark.parametrize("V,k", [(3900, 1), (3900, 8), (2053, 5), (700, 1), (300, 1), (450, 8), (250, 4), (80, 2),
                                 (110, 12), (52, 6), (29, 4), (31, 20)])
def test_nan_in_rows_of_few_segments(cuda_device, dtype, B, V, k):
    """Rows with a NaN that have fewer segments than a warp has lanes, of each
    segment kind (fp32: a warp's load, four lanes', one lane's, one logit)."""
    x = logits(B, V, dtype, V + k)
    bad = {0: [0], 1: [V - 1], 2: [V // 2], 3: [1, V // 3, V // 2 + 1, V - 2], 4: list(range(0, V, 2)), 5: list(range(V))}
    for r, at in bad.items():
        x[r, at] = math.nan
    x[6, V // 2] = math.inf
    t = given(B, V, V, 0.0)
    top = torch.full((B, k), 5.0, device="cuda")
    ids = torch.full((B, k), 5, dtype=torch.int64, device="cuda")
    out = gh.gh_token_logprobs(x, t, k, top_logprob=top, top_index=ids)
    for v in out[:4]:
        assert torch.isnan(v[:7]).all()
    assert (out[4][:7] == -1).all()
    rows = slice(0, 64)
    check_logprobs(x[rows], t[rows], k, 1.0, [v[rows] for v in out], what=f"V={V} k={k}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k", [20, 33, 128])
def test_a_cluster_of_nan_parts_and_one_plateau(cuda_device, dtype, k):
    """One CTA's part of a row holds a plateau (more candidates than are kept) and
    a NaN, the others nothing but NaN: places without a key beside a NaN's key."""
    V = 70001
    x = logits(4, V, dtype, 5)
    for r, (a, b) in enumerate(((9000, 17000), (0, 8000), (62000, V))):
        x[r] = math.nan
        x[r, a:b] = 5.0
        x[r, (a + b) // 2] = math.nan
    t = given(4, V, 5, 0.0)
    out = gh.gh_token_logprobs(x, t, k)
    for v in out[:4]:
        assert torch.isnan(v[:3]).all()
    assert (out[4][:3] == -1).all()
    check_logprobs(x[3:], t[3:], k, 1.0, [v[3:] for v in out])


@pytest.mark.parametrize("B,V", [(3, 70001), (1100, 20011), (3, 1_000_003)])
@pytest.mark.parametrize("at", [-2000.0, -2e6])
def test_long_rows_far_from_zero(cuda_device, at, B, V):
    """Rows far from 0 whose logits have three values one nat apart: their sums
    hold for any length, in the gradient (at -2000) and in the log-probabilities
    too (at -2e6).  Exponentials are off by |y| 2^-23 <= 3 2^-23 and 2^-22 of ex2, a
    chain of 32 terms by 31 2^-25 < 2^-20 and the rest of the sums by a few 2^-24:
    together below 2^-19 for the sum and p; the entropy has that twice, and log p and
    the entropy 2^-22 of themselves."""
    x = at + torch.arange(V, device="cuda").remainder(3).float().expand(B, V).contiguous()
    t = torch.arange(B, device="cuda") * 7
    lp, ent, lse, top, ids = gh.gh_token_logprobs(x, t, 3)
    logp = torch.log_softmax(x[0].double() - at, 0)
    p, H = logp.exp(), -(logp.exp() * logp).sum()
    assert ((lp.double() - logp[t]).abs() <= 2.0 ** -19 + 2.0 ** -22 * logp[t].abs()).all()
    assert ((ent.double() - H).abs() <= 2.0 ** -18 + 2.0 ** -22 * H).all()
    assert (ids == torch.tensor([2, 5, 8], device="cuda")).all()
    assert ((top.double() - logp[2]).abs() <= 2.0 ** -19 + 2.0 ** -22 * logp[2].abs()).all()
    g = gh.gh_token_logprobs_vjp(x, t, lse, ent, torch.ones(B, device="cuda"))
    for r in range(min(B, 3)):
        want = -p
        want[t[r]] += 1.0
        assert ((g[r].double() - want).abs() <= 2.0 ** -19 * p + 2.0 ** -22 * want.abs()).all()
    q, loss = torch.zeros(B, 1, device="cuda"), torch.empty(B, device="cuda")
    _, g = gh.gh_topk_distill(x, t[:, None].contiguous(), q, 1.0, True, "sum", row_loss=loss)
    assert ((loss.double() + logp[t]).abs() <= 2.0 ** -19 + 2.0 ** -21 * logp[t].abs()).all()
    for r in range(min(B, 3)):
        want = p.clone()
        want[t[r]] -= 1.0
        assert ((g[r].double() - want).abs() <= 2.0 ** -19 * p + 2.0 ** -22 * want.abs()).all()


@pytest.mark.parametrize("B,V,k", [(9, 30, 3), (9, 2050, 5), (1250, 2050, 5), (1250, 5003, 20), (9, 16001, 0), (9, 70001, 20)])
@pytest.mark.parametrize("T", [1.0, 1e-4])
def test_rows_on_both_sides_of_the_far_limit(cuda_device, T, B, V, k):
    x = straddling_rows(B, V, T, V)
    t = given(B, V, V, 0.0)
    t[::2] = V // 2
    T = float(torch.tensor(T))
    lp, ent, lse, top, ids = gh.gh_token_logprobs(x, t, k, T)
    z = x.double() / T
    z = z - z.amax(1, keepdim=True)
    logp = torch.log_softmax(z, 1)
    want = logp.gather(1, t[:, None])[:, 0]
    H = -(logp.exp() * logp).sum(1)
    assert ((lp.double() - want).abs() <= STRADDLE + 2.0 ** -22 * want.abs()).all()
    assert ((ent.double() - H).abs() <= STRADDLE * (2 + 2 * H)).all()
    w = torch.logsumexp(x.double() / T, 1)
    assert ((lse.double() - w).abs() <= 2.0 ** -22 * w.abs()).all()
    if k:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(ids, order)
        want = logp.gather(1, order)
        assert ((top.double() - want).abs() <= STRADDLE + 2.0 ** -22 * want.abs()).all()


def test_functional_companions_may_be_flat(cuda_device):
    x = logits(12, 77, torch.float32, 3).view(3, 4, 77)
    t = given(12, 77, 3)
    a, b = GF.token_logprobs(x, t, 5), GF.token_logprobs(x, t.view(3, 4), 5)
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and a[0].shape == (3, 4)
    assert torch.equal(GF.token_logprobs(x, t.view(3, 4, 1), 5)[0], a[0])
    ids, top = a[3], a[2]
    l1 = GF.topk_distillation(x, ids, top, 2.0)
    l2 = GF.topk_distillation(x, ids.reshape(12, 5), top.reshape(12, 5), 2.0)
    assert torch.equal(l1, l2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_far_apart(cuda_device, dtype):
    """One position's logits out of [B, S, V]: values, gradients, and memory of their own size."""
    B, S, V, k = 40, 33, 2003, 6
    whole = logits(B * S, V, dtype, 7).view(B, S, V)
    t = given(B, V, 7)
    x = whole[:, -1]
    out = gh.gh_token_logprobs(x, t, k)
    check_logprobs(x, t, k, 1.0, out)
    gl, gH = torch.randn(B, device="cuda"), torch.randn(B, device="cuda")
    grad = gh.gh_token_logprobs_vjp(x, t, out[2], out[1], gl, gH)
    assert grad.stride(0) < V + 8
    check_vjp(x, t, gl, gH, 1.0, grad)
    leaf = whole.clone().requires_grad_(True)
    lp, ent = GF.token_logprobs(leaf[:, -1], t)
    (gl * lp + gH * ent).sum().backward()
    assert torch.equal(leaf.grad[:, -1], grad) and not leaf.grad[:, :-1].any()
