"""GPU parity of gh_topk_distill against the float64 oracle (tolerances:
token_ops_check), and of a teacher's top logits carried through to a linear
student's gradients."""
import math

import numpy as np
import pytest
import torch

import lm_head_cross_gh_b200 as gh
import oracle
from lm_head_cross_gh_b200 import functional as GF
from token_ops_check import STRADDLE, check_distill, f64, logits, straddling_rows

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]


def entries(x, K, T, renorm, seed, ragged=True):
    """A teacher near the student: its top K entries, some rows short, some empty."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, V = x.shape
    z = torch.nan_to_num(x.float(), neginf=-50.0) + torch.randn(B, V, generator=g, device="cuda")
    if not renorm:
        z = torch.log_softmax(z / T, dim=1)
    v, i = torch.topk(z, K, dim=1)
    if ragged:
        n = torch.randint(0, K + 1, (B,), generator=g, device="cuda")
        n[::3] = K
        none = torch.arange(K, device="cuda")[None] >= n[:, None]
        i = i.masked_fill(none, -1)
        v[:, K // 2] = torch.where(torch.rand(B, generator=g, device="cuda") < 0.2, -math.inf, v[:, K // 2])
    return i.contiguous(), v.contiguous()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 64, 65, 1023, 1025, 8191, 50257])
def test_sizes(cuda_device, dtype, V):
    B = 13 if V < 9000 else 6
    for K, T, renorm, red, pad in ((1, 1.0, True, "mean", 0), (min(V, 8), 2.0, True, "sum", 3),
                                   (min(V, 128), 1.5, False, "mean", 0)):
        x = logits(B, V, dtype, V + K, pad)
        i, v = entries(x, K, T, renorm, V)
        row = torch.full((B,), 7.0, device="cuda")
        loss, grad = gh.gh_topk_distill(x, i, v, T, renorm, red, row_loss=row)
        check_distill(x, i, v, T, renorm, red, loss, grad, row, f"{dtype} V={V} K={K}")
        only, none = gh.gh_topk_distill(x, i, v, T, renorm, red, with_grad=False)
        assert none is None
        check_distill(x, i, v, T, renorm, red, only, None, None, f"loss only {dtype} V={V} K={K}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V,K", [(1, 50257, 32), (2, 262144, 128), (160, 5003, 17), (1300, 2003, 32),
                                   (1250, 8200, 128), (2500, 131, 5), (1200, 66001, 8)])
def test_batches(cuda_device, dtype, B, V, K):
    x = logits(B, V, dtype, B)
    i, v = entries(x, K, 2.0, True, B)
    loss, grad = gh.gh_topk_distill(x, i, v, 2.0)
    if B * V < 30_000_000:
        check_distill(x, i, v, 2.0, True, "mean", loss, grad)
    else:  # a sample of the rows, each as a batch of its own
        n = int(gh.gh_distill_count(i, v, V).item())
        for r in (0, 3, B - 1):
            l1, g1 = gh.gh_topk_distill(x[r:r + 1], i[r:r + 1], v[r:r + 1], 2.0, True, "sum")
            check_distill(x[r:r + 1], i[r:r + 1], v[r:r + 1], 2.0, True, "sum", l1, g1)
            d = (grad[r].double() * n - g1[0].double()).abs()
            assert (d <= 2 * torch.finfo(dtype).eps * g1[0].double().abs() + 1e-5 * g1.abs().max().item()).all()
    l2, g2 = gh.gh_topk_distill(x, i, v, 2.0)
    assert torch.equal(l2, loss) and torch.equal(g2, grad), "two calls differ"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [5, 1250])
def test_duplicate_ids_add_up(cuda_device, dtype, B):
    x = logits(B, 515, dtype, 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    i = torch.randint(0, 4, (B, 12), generator=g, device="cuda") * 128 + 1
    i[:, 11] = 514
    v = torch.randn(B, 12, generator=g, device="cuda")
    loss, grad = gh.gh_topk_distill(x, i, v, 1.0)
    check_distill(x, i, v, 1.0, True, "mean", loss, grad)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [8, 1250])
def test_masks_and_non_finite_values(cuda_device, dtype, B):
    V, K = 2053, 6
    low = torch.finfo(dtype).min
    x = logits(B, V, dtype, 3)
    i, v = entries(x, K, 1.0, True, 4, ragged=False)
    x[0, 1000:] = low
    x[1] = low                                  # uniform
    i[0], i[1] = torch.arange(6, device="cuda") * 7, torch.arange(6, device="cuda") * 300
    i[2] = -1                                   # no entry: not read
    x[2] = math.nan
    v[3] = -math.inf                            # no entry either
    v[4, 1:] = -2e4                             # teacher probabilities that underflow to zero
    x[4, i[4, 2]] = -math.inf                   # the student has none there: 0 log 0
    x[4, i[4, 0]] = 1.0
    row = torch.empty(B, device="cuda")
    loss, grad = gh.gh_topk_distill(x, i, v, 1.0, True, "sum", row_loss=row)
    xc = x.clone()
    xc[2] = 0.0
    check_distill(xc, i, v, 1.0, True, "sum", loss, grad, row)
    # a student without mass at an entry: an infinite loss, a finite gradient
    y = x[5:8].clone()
    y[0, i[5, 0]] = -math.inf
    loss, grad = gh.gh_topk_distill(y, i[5:8], v[5:8], 1.0, True, "sum")
    assert loss.item() == math.inf and torch.isfinite(grad).all()
    # no distribution, or a NaN among the values: NaN in that row alone
    y = x[5:8].clone()
    y[0, 5], y[1] = math.nan, -math.inf
    w = v[5:8].clone()
    w[2, 0] = math.nan
    row = torch.empty(3, device="cuda")
    loss, grad = gh.gh_topk_distill(torch.cat([y, x[6:7]]), torch.cat([i[5:8], i[6:7]]), torch.cat([w, v[6:7]]), 1.0,
                                    True, "sum", row_loss=torch.empty(4, device="cuda"))
    assert math.isnan(loss.item()) and torch.isnan(grad[:3]).all() and torch.isfinite(grad[3]).all()


def test_no_row_has_an_entry(cuda_device):
    x = logits(5, 100, torch.bfloat16, 5)
    i = torch.full((5, 3), -1, dtype=torch.int64, device="cuda")
    loss, grad = gh.gh_topk_distill(x, i, torch.zeros(5, 3, device="cuda"))
    assert loss.item() == 0.0 and not grad.any()
    e = torch.empty(0, 100, device="cuda")
    loss, grad = gh.gh_topk_distill(e, i[:0], torch.zeros(0, 3, device="cuda"))
    assert loss.item() == 0.0 and grad.shape == (0, 100)


def test_id_out_of_range_is_no_entry(cuda_device):
    for total in (None, torch.tensor(3, device="cuda")):
        gh.gh_get_device_status()
        x = logits(3, 100, torch.float32, 6)
        i = torch.tensor([[1, 2], [100, 5], [-7, 6]], device="cuda")
        v = torch.randn(3, 2, device="cuda")
        loss, grad = gh.gh_topk_distill(x, i, v, n_valid_total=total)
        assert gh.gh_get_device_status() == gh.GH_ERR_TARGET_RANGE
        j = i.clone()
        j[1, 0] = j[2, 0] = -1
        check_distill(x, j, v, 1.0, True, "mean", loss, grad)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [9, 1250])
def test_in_place_padding_and_other_phase(cuda_device, dtype, B):
    V = 3001
    whole = torch.full((B, V + 7), 9.0, dtype=dtype, device="cuda")
    whole[:, :V] = logits(B, V, dtype, 7)
    x = whole[:, :V]
    i, v = entries(x, 16, 1.0, True, 8)
    loss, want = gh.gh_topk_distill(x, i, v)
    check_distill(x, i, v, 1.0, True, "mean", loss, want)
    buf = torch.full((B * 3050 + 16,), 9.0, dtype=dtype, device="cuda")
    other = buf[3:3 + B * 3050].view(B, 3050)[:, :V]
    l2, _ = gh.gh_topk_distill(x, i, v, grad=other)
    assert torch.equal(l2, loss) and torch.equal(other, want)
    other.fill_(9.0)
    assert (buf == 9.0).all()
    l3, _ = gh.gh_topk_distill(x, i, v, grad=x)
    assert torch.equal(l3, loss) and torch.equal(x, want) and (whole[:, V:] == 9.0).all()


def test_a_batch_in_chunks_has_one_mean(cuda_device):
    x = logits(700, 999, torch.float32, 9)
    i, v = entries(x, 10, 1.0, True, 10)
    loss, grad = gh.gh_topk_distill(x, i, v)
    n = gh.gh_distill_count(i, v, 999)
    parts = [gh.gh_topk_distill(x[a:b], i[a:b], v[a:b], n_valid_total=n) for a, b in ((0, 300), (300, 700))]
    assert abs(sum(p[0].item() for p in parts) - loss.item()) <= 2.0 ** -22 * abs(loss.item())
    assert torch.allclose(torch.cat([p[1] for p in parts]), grad, rtol=1e-6, atol=1e-12)


def test_offsets_beyond_32_bits(cuda_device):
    B, V = 17000, 131072
    x = torch.zeros(B, V, dtype=torch.bfloat16, device="cuda")
    tail = logits(6, V, torch.bfloat16, 13)
    x[-6:] = tail
    i = torch.full((B, 4), -1, dtype=torch.int64, device="cuda")
    v = torch.zeros(B, 4, device="cuda")
    i[-6:], v[-6:] = entries(tail, 4, 1.0, True, 14, ragged=False)
    loss, grad = gh.gh_topk_distill(x, i, v, 1.0, True, "sum", grad=x)
    check_distill(tail, i[-6:], v[-6:], 1.0, True, "sum", loss, grad[-6:])
    assert not grad[:-6].any()


@pytest.mark.parametrize("B,V", [(3, 50257), (1300, 2003)])
def test_captured_graphs(cuda_device, B, V):
    xs = [logits(B, V, torch.bfloat16, s) for s in (21, 22)]
    es = [entries(x, 9, 1.0, True, s) for s, x in enumerate(xs)]
    want = [gh.gh_topk_distill(x, *e) for x, e in zip(xs, es)]
    graphs, outs = [], []
    for x, e in zip(xs, es):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gh.gh_topk_distill(x, *e))
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_functional_gradient_against_formula_and_differences(cuda_device):
    torch.manual_seed(3)
    x = torch.randn(2, 4, 60, device="cuda", requires_grad=True)
    i, v = entries(torch.randn(8, 60, device="cuda"), 5, 2.0, True, 1, ragged=False)
    i, v = i.view(2, 4, 5), v.view(2, 4, 5)
    loss = GF.topk_distillation(x, i, v, 2.0)
    (3.0 * loss).backward()

    def value(z):
        q = torch.softmax(v.double() / 2.0, dim=-1)
        logp = torch.log_softmax(z / 2.0, dim=-1).gather(-1, i)
        return 3.0 * 4.0 * (q * (q.log() - logp)).sum(-1).mean()

    y = x.detach().double().requires_grad_(True)
    value(y).backward()
    assert abs(3.0 * loss.item() - value(y).item()) < 1e-5
    assert torch.allclose(x.grad.double(), y.grad, rtol=1e-5, atol=1e-7)
    d = torch.randn_like(y)
    diff = (value(y.detach() + 1e-5 * d) - value(y.detach() - 1e-5 * d)) / 2e-5
    assert abs((x.grad.double() * d).sum() - diff) < 1e-5


@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_teacher_to_linear_student(cuda_device, reduction):
    """The operators as they are used together: a teacher's logits are scored
    and its top entries written out, then a linear student is distilled from
    them in chunks, against the materialised float64 computation on the bf16
    logits that the chunk loop forms (gradients: 1e-2 relative Frobenius, the
    linear cross-entropy's bar)."""
    torch.manual_seed(4)
    N, D, V, K, T = 700, 128, 3001, 20, 2.0
    X = torch.randn(N, D, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, D, device="cuda") * 0.2).to(torch.bfloat16)
    teacher = (X.float() @ W.float().t() + torch.randn(N, V, device="cuda")).to(torch.bfloat16)
    token = torch.randint(0, V, (N,), device="cuda")
    token[:30] = -100
    logprob, entropy, lse, top, ids = gh.gh_token_logprobs(teacher, token, K)
    assert (ids[:30] == -1).all()
    Xg, Wg = X.clone().requires_grad_(True), W.clone().requires_grad_(True)
    loss = GF.chunked_linear_topk_distillation(Xg, Wg, ids, top, T, True, reduction, chunk_size=256)
    loss.backward()
    z = f64((X.float() @ W.float().t()).to(torch.bfloat16))
    r = oracle.topk_distill(z, ids.cpu().numpy(), f64(top), T, True, reduction)
    assert r["n_valid"] == N - 30
    assert abs(loss.item() - r["loss"]) <= 1e-3 * abs(r["loss"])
    dX, dW = r["grad"] @ f64(W), r["grad"].T @ f64(X)
    for got, want in ((f64(Xg.grad), dX), (f64(Wg.grad), dW)):
        assert np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want)
    assert not Xg.grad[:30].any()
    assert gh.gh_get_device_status() == gh.GH_OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V", [(3, 70001), (200, 90001), (9, 300_001)])
def test_in_place_over_a_cluster(cuda_device, dtype, B, V):
    """Rows split over several CTAs, in place: entries and rows far from 0 are read
    before any CTA of the row stores."""
    x = logits(B, V, dtype, 31)
    x[1] -= 30000.0
    x[2] = torch.finfo(dtype).min
    i, v = entries(x, 64, 1.0, True, 32, ragged=False)
    loss, want = gh.gh_topk_distill(x, i, v, 1.0, True, "sum")
    rows = slice(0, 3)
    l3, g3 = gh.gh_topk_distill(x[rows], i[rows], v[rows], 1.0, True, "sum")
    check_distill(x[rows], i[rows], v[rows], 1.0, True, "sum", l3, g3)
    tol = 4e-7 * 8 + 2.0 ** -18 + 2 * torch.finfo(dtype).eps
    assert ((want[rows].float() - g3.float()).abs() <= tol * g3.float().abs() + 1e-6).all()
    for _ in range(5):
        y = x.clone()
        l2, _ = gh.gh_topk_distill(y, i, v, 1.0, True, "sum", grad=y)
        assert torch.equal(y, want) and torch.equal(l2, loss)


@pytest.mark.parametrize("B,K", [(1, 1), (16, 128), (17, 128), (63, 32), (64, 32), (65, 32), (64, 33)])
def test_counts_of_small_batches(cuda_device, B, K):
    """Both ways of counting the rows with an entry, at their border."""
    x = logits(B, 1000, torch.float32, B)
    i, v = entries(x, K, 1.0, True, K)
    if B > 1:
        i[0] = -1
        i[B - 1, : K - 1] = -1   # only the last entry
    n = int(((i >= 0) & (v > -math.inf)).any(1).sum())
    assert int(gh.gh_distill_count(i, v, 1000)) == n
    loss, grad = gh.gh_topk_distill(x, i, v)
    check_distill(x, i, v, 1.0, True, "mean", loss, grad)


def test_two_calls_at_once(cuda_device):
    xs = [logits(1300, 5003, torch.bfloat16, s) for s in (41, 42)]
    es = [entries(x, 16, 1.0, True, s) for s, x in enumerate(xs)]
    want = [gh.gh_topk_distill(x, *e) for x, e in zip(xs, es)]
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a = gh.gh_topk_distill(xs[0], *es[0])
        b = gh.gh_topk_distill(xs[1], *es[1])
        torch.cuda.synchronize()
        for o, w in zip((a, b), want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


@pytest.mark.parametrize("shape", [(0,), (2, 0), ()])
def test_functional_shapes_without_rows_and_of_one_row(cuda_device, shape):
    torch.manual_seed(2)
    x = torch.randn(*shape, 9, device="cuda", requires_grad=True)
    i = torch.arange(4, device="cuda").expand(*shape, 4)
    loss = GF.topk_distillation(x, i, torch.zeros(*shape, 4, device="cuda"))
    loss.backward()
    assert loss.shape == () and x.grad.shape == x.shape
    assert (loss.item() > 0.0) == (shape == ()) and torch.isfinite(loss)


def test_linear_student_without_rows(cuda_device):
    X = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    W = torch.randn(100, 64, device="cuda").to(torch.bfloat16).requires_grad_(True)
    loss = GF.chunked_linear_topk_distillation(X, W, torch.empty(0, 3, dtype=torch.int64, device="cuda"),
                                               torch.empty(0, 3, device="cuda"))
    loss.backward()
    assert loss.item() == 0.0 and X.grad.shape == (0, 64) and not W.grad.any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V", [(4, 333), (1300, 1537), (4, 70001)])
@pytest.mark.parametrize("T", [1e-4, 1.0, 1e4])
def test_largest_finite_logits(cuda_device, dtype, B, V, T):
    """Rows whose n largest logits are equal and out of the others' reach, at the
    ends of the type's range, and one entry of all the teacher's probability: in
    closed form, row loss T^2 log n and gradient T (1 / n - [j = id]) (2^-20
    relative for log2 and the few roundings, one rounding of the output)."""
    big = torch.finfo(dtype).max
    x = torch.zeros(B, V, device="cuda", dtype=dtype)
    at = torch.tensor([V - 1, V // 2, 3], device="cuda")
    for r, (low, high) in enumerate(((-big, big), (0.0, big), (-big, 0.0), (big, big))):
        x[r::4] = low
        x[r::4, at] = high
    n = torch.full((B,), 3.0, device="cuda", dtype=torch.float64)
    n[3::4] = V
    i = torch.tensor([V // 2, -1], device="cuda").expand(B, 2).contiguous()
    row = torch.empty(B, device="cuda")
    _, grad = gh.gh_topk_distill(x, i, torch.zeros(B, 2, device="cuda"), T, True, "sum", row_loss=row)
    assert torch.allclose(row.double(), T * T * n.log(), rtol=2.0 ** -19, atol=0)
    p = torch.zeros(B, V, device="cuda", dtype=torch.float64)
    p[:, at] = 1.0 / 3.0
    p[3::4] = 1.0 / V
    want = T * p
    want[:, V // 2] -= T
    assert ((grad.double() - want).abs() <= want.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -19)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [4, 1300])
@pytest.mark.parametrize("T", [0.5, 2.0])
def test_entry_at_a_logit_of_the_lowest_value(cuda_device, dtype, B, T):
    """The student's mask has its type's lowest value where the teacher has an
    entry: log p is beyond fp32, the loss T q |x| is not (2^-19 relative: q's and
    the sums' few roundings)."""
    V = 1537
    x = logits(B, V, dtype, 91)
    x[:, 7] = torch.finfo(dtype).min
    i = torch.tensor([11, 7, 30], device="cuda").expand(B, 3).contiguous()
    v = torch.tensor([1.0, 0.2, 0.4], device="cuda").expand(B, 3).contiguous()
    row = torch.empty(B, device="cuda")
    loss, grad = gh.gh_topk_distill(x, i, v, T, row_loss=row)
    r = oracle.topk_distill(f64(x), i.cpu().numpy(), f64(v), T)
    assert np.isfinite(f64(row)).all() and (np.abs(f64(row) - r["row_loss"]) <= 2.0 ** -19 * r["row_loss"]).all()
    assert torch.isfinite(grad).all()


def test_entry_of_vanishing_probability_at_a_masked_logit(cuda_device):
    """An entry whose probability is fp32's smallest, or 0, at a logit of -inf:
    an infinite loss or none, never NaN (0 log 0 = 0)."""
    x = logits(64, 300, torch.float32, 5)
    x[:, 7] = -math.inf
    i = torch.tensor([11, 7], device="cuda").expand(64, 2).contiguous()
    v = torch.zeros(64, 2, device="cuda")
    v[:, 1] = -torch.linspace(80, 120, 64, device="cuda")
    for T in (0.05, 1.0, 8.0):
        row = torch.empty(64, device="cuda")
        _, grad = gh.gh_topk_distill(x, i, v * T, T, True, "sum", row_loss=row)
        assert not torch.isnan(row).any() and torch.isfinite(grad).all()
        assert torch.isposinf(row[0]) and torch.isfinite(row[-1])


@pytest.mark.parametrize("B,V", [(9, 30), (9, 2050), (1250, 2050), (1250, 5003), (9, 70001), (500, 40001)])
@pytest.mark.parametrize("T", [1.0, 1e-4])
def test_rows_on_both_sides_of_the_far_limit(cuda_device, T, B, V):
    x = straddling_rows(B, V, T, V)
    T = float(torch.tensor(T))
    i = torch.tensor([0, V // 2, V - 1], device="cuda").expand(B, 3).contiguous()
    v = T * torch.tensor([1.0, 0.5, -0.25], device="cuda").expand(B, 3).contiguous()
    row = torch.empty(B, device="cuda")
    _, grad = gh.gh_topk_distill(x, i, v, T, True, "sum", row_loss=row)
    z = x.double() / T
    logp = torch.log_softmax(z - z.amax(1, keepdim=True), 1)
    log_q = torch.log_softmax(v.double() / T, 1)
    q, log_p = log_q.exp(), logp.gather(1, i)
    want = T * T * (q * (log_q - log_p)).sum(1)
    # the log-probabilities' bound for log p and p; q's few roundings as 2^-19
    tol = T * T * (STRADDLE + 2.0 ** -19 * (q * (log_q.abs() + log_p.abs() + 1)).sum(1))
    assert ((row.double() - want).abs() <= tol).all()
    want = T * logp.exp()
    tol = STRADDLE * want
    want.scatter_add_(1, i, -T * q)
    tol.scatter_add_(1, i, T * q * 2.0 ** -19)
    assert ((grad.double() - want).abs() <= tol + 2.0 ** -22 * want.abs()).all()
