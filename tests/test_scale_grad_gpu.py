"""gh_scale_grad and the autograd forms' upstream gradients (GPU): the product
of a stored gradient and an fp32 scalar in fp32, rounded to the gradient's type, so
bit for bit what torch's fp32 product rounds to."""
import pytest
import torch

import lm_head_cross_gh_b200 as gh
from lm_head_cross_gh_b200 import functional as GF

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]


def data(shape, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def product(x, g):
    return (x.float() * g).to(x.dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 63, 1000, 4099, 16384, 16385, 100_003, 5_000_011])
def test_dense(cuda_device, dtype, n):
    g = torch.tensor(0.3, device="cuda")
    buf = torch.full((n + 40,), 5.0, dtype=dtype, device="cuda")
    for phase, ophase in ((0, 0), (3, 3), (1, 6)):
        x = data((n + 8,), dtype, n)[phase:phase + n]
        buf.fill_(5.0)
        out = buf[16 + ophase:16 + ophase + n]
        assert gh.gh_scale_grad(x, g, out=out) is out
        assert torch.equal(out, product(x, g))
        assert (buf[:16 + ophase] == 5.0).all() and (buf[16 + ophase + n:] == 5.0).all()
    y = data((n,), dtype, n)
    want = product(y, g)
    assert torch.equal(gh.gh_scale_grad(y, g), want)
    gh.gh_scale_grad(y, g, out=y)
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V", [(1, 50257), (13, 1001), (2500, 129), (40, 70001)])
def test_rows_apart(cuda_device, dtype, B, V):
    g = torch.tensor(-1.7, device="cuda")
    whole = data((B, V + 5), dtype, V)
    x = whole[:, :V]
    want = product(x, g)
    out = gh.gh_scale_grad(x, g)
    assert torch.equal(out, want) and out.stride(1) == 1
    other = torch.full((B, V + 9), 5.0, dtype=dtype, device="cuda")
    gh.gh_scale_grad(x, g, out=other[:, 2:V + 2])
    assert torch.equal(other[:, 2:V + 2], want) and (other[:, :2] == 5.0).all() and (other[:, V + 2:] == 5.0).all()
    keep = whole[:, V:].clone()
    gh.gh_scale_grad(x, g, out=x)
    assert torch.equal(x, want) and torch.equal(whole[:, V:], keep)


def test_shapes_values_and_refusals(cuda_device):
    g = torch.tensor(0.3, device="cuda")
    for shape in ((0,), (0, 5), (3, 0), (2, 3, 4), ()):
        x = torch.randn(shape, device="cuda")
        assert torch.equal(gh.gh_scale_grad(x, g), x * g)
    x = torch.tensor([0.0, -0.0, float("inf"), float("-inf"), float("nan"), 3e38, 1e-40], device="cuda")
    for s in (0.3, 0.0, 4.0, -1.0, float("nan"), float("inf")):
        s = torch.tensor(s, device="cuda")
        assert torch.equal(torch.nan_to_num(gh.gh_scale_grad(x, s), nan=7.0), torch.nan_to_num(x * s, nan=7.0))
    with pytest.raises(ValueError):
        gh.gh_scale_grad(x, g.double())
    with pytest.raises(ValueError):
        gh.gh_scale_grad(x, g.cpu())
    with pytest.raises(ValueError):
        gh.gh_scale_grad(x.half(), g)
    with pytest.raises(ValueError):
        gh.gh_scale_grad(x, g, out=x[:3])


def test_offsets_beyond_32_bits(cuda_device):
    x = torch.zeros(2_300_000_017, dtype=torch.bfloat16, device="cuda")
    x[:5], x[-5:] = 1.0, 3.0
    g = torch.tensor(0.3, device="cuda")
    gh.gh_scale_grad(x, g, out=x)
    ends = torch.cat([x[:6], x[-6:]])
    assert torch.equal(ends, product(torch.tensor([1.0] * 5 + [0.0, 0.0] + [3.0] * 5, device="cuda").to(torch.bfloat16), g))
    assert int((x != 0).sum()) == 10


@pytest.mark.parametrize("g", [0.3, 1.0 / 3.0, -2.0])
def test_autograd_forms_round_the_product_once(cuda_device, g):
    """Each form's gradient for an upstream g is the direct call's times g,
    rounded once."""
    up = torch.tensor(g, device="cuda")
    x = data((200, 1003), torch.bfloat16, 1)
    t = torch.randint(0, 1003, (200,), device="cuda")
    _, _, _, top, ids = gh.gh_token_logprobs(data((200, 1003), torch.bfloat16, 2), t, 16)
    leaf = x.clone().requires_grad_(True)
    (g * GF.topk_distillation(leaf, ids, top, 2.0)).backward()
    assert torch.equal(leaf.grad, product(gh.gh_topk_distill(x, ids, top, 2.0)[1], up))
    # rows apart, as a slice of a padded head's logits
    wide = torch.zeros(200, 1010, device="cuda", dtype=torch.bfloat16)
    wide[:, :1003] = x
    wide.requires_grad_(True)
    (g * GF.topk_distillation(wide[:, :1003], ids, top, 2.0)).backward()
    direct = gh.gh_topk_distill(wide.detach()[:, :1003], ids, top, 2.0)[1]  # (another phase: sums in another order)
    assert torch.equal(wide.grad[:, :1003], product(direct, up)) and not wide.grad[:, 1003:].any()
    leaf = x.clone().requires_grad_(True)
    (g * GF.cross_entropy(leaf, t)).backward()
    assert torch.equal(leaf.grad, product(gh.gh_ce_fwd_bwd(x, t)[1], up))
    X, W = data((200, 64), torch.bfloat16, 3), data((1003, 64), torch.bfloat16, 4)
    Xg, Wg = X.clone().requires_grad_(True), W.clone().requires_grad_(True)
    (g * GF.chunked_linear_cross_entropy(Xg, Wg, t)).backward()
    _, dX, dW = gh.gh_linear_ce(X, W, t)
    assert torch.equal(Xg.grad, product(dX, up)) and torch.equal(Wg.grad, product(dW, up))


def test_upstream_gradient_keeps_its_graph(cuda_device):
    """With create_graph the product stays differentiable by the upstream gradient."""
    x = data((20, 103), torch.float32, 5).requires_grad_(True)
    t = torch.randint(0, 103, (20,), device="cuda")
    w = torch.tensor(0.7, device="cuda", requires_grad=True)
    (grad,) = torch.autograd.grad(w * GF.cross_entropy(x, t), x, create_graph=True)
    (gw,) = torch.autograd.grad(grad.sum(0)[3], w)
    assert torch.allclose(gw, grad.detach().sum(0)[3] / 0.7, rtol=1e-5, atol=1e-7)


def test_captured_and_replayed(cuda_device):
    x = data((300, 2003), torch.bfloat16, 6)
    g = torch.tensor(0.3, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gh.gh_scale_grad(x, g)
    for s in (0.3, -1.1):
        g.fill_(s)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, product(x, g))
