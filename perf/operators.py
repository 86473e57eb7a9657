"""Measured cases of the token log-probability and top-logits distillation operators.

Each case names one operator, its sizes and its types.  ``run`` makes one pass:
the operator's plain form in elementary torch operations (``own`` false), or the
library call a user makes (``own`` true).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
IGNORE = -100
MOST_BYTES = 8192 * 50257 * 2  # logits of the largest listed cases


def listed():
    return [
        # serving: the log probabilities of one sequence's step, with 20 alternatives
        dict(name="logprobs_decode_one", op="logprobs", B=1, V=50257, ld=50257, dtype="bf16", k=20, T=0.8,
             ignored=0.0, banned=0.0),
        # serving: a batch's step under a grammar that bans most of the vocabulary
        dict(name="logprobs_decode_masked", op="logprobs", B=64, V=128256, ld=128256, dtype="bf16", k=5, T=1.0,
             ignored=0.0, banned=0.9),
        # fine-tuning: scoring a batch of sequences, padding ignored
        dict(name="logprobs_score", op="logprobs", B=8192, V=50257, ld=50257, dtype="bf16", k=0, T=1.0,
             ignored=0.02, banned=0.0),
        # writing out a teacher's top logits, head padded to a round vocabulary
        dict(name="logprobs_teacher", op="logprobs", B=4096, V=50257, ld=50304, dtype="bf16", k=32, T=1.0,
             ignored=0.02, banned=0.0),
        # the same with a large vocabulary and many entries
        dict(name="logprobs_teacher_wide", op="logprobs", B=1024, V=262144, ld=262144, dtype="bf16", k=128, T=2.0,
             ignored=0.0, banned=0.0),
        # evaluation in full precision, odd sizes
        dict(name="logprobs_f32_odd", op="logprobs", B=2047, V=8191, ld=8191, dtype="f32", k=8, T=1.0,
             ignored=0.1, banned=0.0),
        # a toy model's policy gradient
        dict(name="vjp_small", op="vjp", B=64, V=1024, ld=1024, dtype="f32", T=1.0, ignored=0.1, banned=0.0),
        # policy gradient with an entropy bonus over a batch of sequences
        dict(name="vjp_policy", op="vjp", B=8192, V=50257, ld=50257, dtype="bf16", T=1.0, ignored=0.02, banned=0.0),
        # the same in full precision on a wide head
        dict(name="vjp_f32_wide", op="vjp", B=1024, V=128256, ld=128256, dtype="f32", T=0.7, ignored=0.0,
             banned=0.1),
        # distilling a toy model
        dict(name="distill_small", op="distill", B=64, V=1024, ld=1024, dtype="f32", K=8, T=2.0, renorm=True,
             reduction="mean", ignored=0.1),
        # distilling a batch of sequences from 32 stored entries a token
        dict(name="distill_batch", op="distill", B=8192, V=50257, ld=50257, dtype="bf16", K=32, T=2.0, renorm=True,
             reduction="mean", ignored=0.02),
        # many entries of a large vocabulary, stored as log probabilities
        dict(name="distill_wide", op="distill", B=1024, V=262144, ld=262144, dtype="bf16", K=128, T=1.0,
             renorm=False, reduction="sum", ignored=0.0),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["logprobs", "logprobs", "vjp", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    V = spread(1000, 262144)
    ld = V + rng.choice([0, 0, 47, 64])
    es = 4 if dtype == "f32" else 2
    B = spread(1, max(1, min(8192, MOST_BYTES // (ld * es))))
    c = dict(op=op, B=B, V=V, ld=ld, dtype=dtype, T=rng.choice([1.0, 1.0, 0.6, 2.0]), ignored=rng.choice([0.0, 0.05]))
    if op == "distill":
        c.update(K=spread(1, 128), renorm=rng.random() < 0.6, reduction=rng.choice(["mean", "sum"]))
    else:
        c.update(banned=rng.choice([0.0, 0.0, 0.5]))
        if op == "logprobs":
            c.update(k=rng.choice([0, spread(1, 128)]))
    return c


def _ignored_rows(case):
    return int(case["ignored"] * case["B"])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, V, ld, dt = case["B"], case["V"], case["ld"], DTYPES[case["dtype"]]
    buf = torch.randn(B, ld, generator=g, device=dev, dtype=dt).mul_(2.0)
    x = buf[:, :V]
    rows = torch.arange(B, device=dev)
    # each row has a likely token, as a trained head's rows do
    likely = torch.randint(0, V, (B,), generator=g, device=dev)
    x[rows, likely] += (torch.rand(B, generator=g, device=dev) * 12.0 + 2.0).to(dt)
    drop = torch.randperm(B, generator=g, device=dev)[:_ignored_rows(case)]
    s = dict(case=dict(case), logits=x)
    if case["op"] == "distill":
        K = case["K"]
        teacher = x.float() + torch.randn(B, V, generator=g, device=dev) * 0.5
        if not case["renorm"]:
            teacher = torch.log_softmax(teacher / case["T"], dim=1)
        val, idx = torch.topk(teacher, K, dim=1)
        del teacher
        # ragged rows: some tokens were stored with fewer entries, some with none
        count = torch.where(torch.rand(B, generator=g, device=dev) < 0.1,
                            torch.randint(1, K + 1, (B,), generator=g, device=dev), K)
        count[drop] = 0
        none = torch.arange(K, device=dev)[None, :] >= count[:, None]
        s["teacher_index"] = idx.masked_fill(none, -1).contiguous()
        s["teacher_logits"] = val.float().masked_fill(none, 0.0).contiguous()
        return s
    other = torch.randint(0, V, (B,), generator=g, device=dev)
    index = torch.where(torch.rand(B, generator=g, device=dev) < 0.7, likely, other)
    if case["banned"] > 0.0:
        keep = torch.rand(B, V, generator=g, device=dev) >= case["banned"]
        keep[rows, likely] = True
        keep[rows, index] = True
        x.masked_fill_(~keep, -math.inf)
        del keep
    index[drop] = IGNORE
    s["index"] = index
    if case["op"] == "vjp":
        d = x.double() / case["T"]
        lse = torch.logsumexp(d, dim=1)
        p = torch.exp(d - lse[:, None])
        ent = lse - torch.where(p > 0, p * d, 0.0).sum(dim=1)
        del d, p
        gone = index == IGNORE
        s["lse"] = lse.masked_fill(gone, 0.0).float()
        s["entropy"] = ent.masked_fill(gone, 0.0).float()
        s["g_logprob"] = torch.randn(B, generator=g, device=dev)
        s["g_entropy"] = torch.randn(B, generator=g, device=dev) * 0.1
    return s


# ---- plain forms ------------------------------------------------------------------------------------------------


def _strided(values, like):
    """`values` in a buffer with `like`'s strides."""
    return torch.empty_strided(like.shape, like.stride(), dtype=like.dtype, device=like.device).copy_(values)


def _plain_logprobs(x, index, k, T):
    z = x.float() / T
    d = z - z.amax(dim=1, keepdim=True)
    e = torch.exp(d)
    s = e.sum(dim=1)
    log_s = torch.log(s)
    entropy = log_s - torch.where(e > 0, e * d, 0.0).sum(dim=1) / s
    lse = z.amax(dim=1) + log_s
    gone = index == IGNORE
    at = index.masked_fill(gone, 0)[:, None]
    logprob = d.gather(1, at)[:, 0] - log_s
    out = [logprob.masked_fill(gone, 0.0), entropy.masked_fill(gone, 0.0), lse.masked_fill(gone, 0.0)]
    if not k:
        return out + [None, None]
    # the k largest by (value descending, index ascending): one integer key for both
    bits = (x.float() + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64)
    key = (key << 32) - torch.arange(x.shape[1], device=x.device)
    top = torch.topk(key, k, dim=1).indices
    top_logprob = d.gather(1, top) - log_s[:, None]
    return out + [top_logprob.masked_fill(gone[:, None], -math.inf), top.masked_fill(gone[:, None], -1)]


def _plain_vjp(x, index, lse, entropy, g_logprob, g_entropy, T):
    logp = x.float() / T - lse[:, None]
    p = torch.exp(logp)
    inner = torch.where(p > 0, g_entropy[:, None] * (logp + entropy[:, None]), 0.0)
    grad = -p * (g_logprob[:, None] + inner)
    gone = index == IGNORE
    grad.scatter_add_(1, index.masked_fill(gone, 0)[:, None], g_logprob[:, None])
    grad = (grad / T).masked_fill(gone[:, None], 0.0)
    return _strided(grad, x)


def _plain_distill(x, ids, vals, T, renorm, reduction):
    z = x.float() / T
    d = z - z.amax(dim=1, keepdim=True)
    log_s = torch.log(torch.exp(d).sum(dim=1, keepdim=True))
    logp = d - log_s
    ok = (ids >= 0) & (vals > -math.inf)
    v = vals.masked_fill(~ok, -math.inf)
    if renorm:
        v = v / T
        v = v - v.amax(dim=1, keepdim=True).clamp_min(-1e30)
        log_q = v - torch.log(torch.exp(v).sum(dim=1, keepdim=True).clamp_min(1e-30))
    else:
        log_q = v
    q = torch.exp(log_q)
    at = ids.clamp_min(0)
    row = T * T * torch.where(q > 0, q * (log_q - logp.gather(1, at)), 0.0).sum(dim=1)
    valid = ok.any(dim=1)
    scale = 1.0 / valid.sum().clamp_min(1).float() if reduction == "mean" else 1.0
    loss = row.masked_fill(~valid, 0.0).double().sum().float() * scale
    grad = q.sum(dim=1, keepdim=True) * torch.exp(logp)
    grad.scatter_add_(1, at, -q)
    grad = (grad * (T * scale)).masked_fill(~valid[:, None], 0.0)
    return [loss, _strided(grad, x)]


def run(s):
    c = s["case"]
    if own:
        import lm_head_cross_gh_b200 as gh
        if c["op"] == "logprobs":
            return gh.gh_token_logprobs(s["logits"], s["index"], c["k"], c["T"], IGNORE)
        if c["op"] == "vjp":
            return gh.gh_token_logprobs_vjp(s["logits"], s["index"], s["lse"], s["entropy"], s["g_logprob"],
                                            s["g_entropy"], c["T"], IGNORE)
        return gh.gh_topk_distill(s["logits"], s["teacher_index"], s["teacher_logits"], c["T"], c["renorm"],
                                  c["reduction"])
    if c["op"] == "logprobs":
        return _plain_logprobs(s["logits"], s["index"], c["k"], c["T"])
    if c["op"] == "vjp":
        return _plain_vjp(s["logits"], s["index"], s["lse"], s["entropy"], s["g_logprob"], s["g_entropy"], c["T"])
    return _plain_distill(s["logits"], s["teacher_index"], s["teacher_logits"], c["T"], c["renorm"], c["reduction"])


# ---- what a pass cannot do without ---------------------------------------------------------------------------------


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    B, V = case["B"], case["V"]
    valid = B - _ignored_rows(case)
    if case["op"] == "logprobs":
        return {"bytes": valid * V * es + B * 8 + B * 12 + B * 12 * case["k"], "flops": 7.0 * valid * V}
    if case["op"] == "vjp":
        return {"bytes": (valid + B) * V * es + B * 24, "flops": 7.0 * valid * V}
    return {"bytes": (valid + B) * V * es + B * case["K"] * 12 + 4, "flops": 6.0 * valid * V}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

ROWS = 256  # rows at a time


def exact(case, seed):
    s = prepare(case, seed)
    x, T = s["logits"], float(case["T"])
    B, V = x.shape
    blocks = [slice(r, min(B, r + ROWS)) for r in range(0, B, ROWS)]
    if case["op"] == "logprobs":
        parts = [_exact_logprobs_rows(x[b].double(), s["index"][b], case["k"], T) for b in blocks]
        out = [torch.cat([p[i] for p in parts]) for i in range(3)]
        return out + ([torch.cat([p[i] for p in parts]) for i in (3, 4)] if case["k"] else [None, None])
    out = torch.empty(B, V, dtype=torch.float64, device=x.device)
    if case["op"] == "vjp":
        for b in blocks:
            y = torch.nan_to_num(x[b].double() / T, neginf=-1e300)
            logp = y - s["lse"][b, None].double()
            t = s["index"][b, None]
            hit = (torch.arange(V, device=x.device) == t).double()
            gl, gh_, h = (s[n][b, None].double() for n in ("g_logprob", "g_entropy", "entropy"))
            p = torch.where(logp < -800, 0.0, torch.exp(logp))
            rows = (gl * (hit - p) - gh_ * p * (logp.clamp_min(-1e4) + h)) / T
            out[b] = rows * (t != IGNORE)
        return out
    total, n = 0.0, 0
    for b in blocks:
        loss, rows, count = _exact_distill_rows(x[b].double(), s["teacher_index"][b], s["teacher_logits"][b].double(), T,
                                                case["renorm"])
        out[b] = rows
        total, n = total + loss, n + count
    if case["reduction"] == "mean":
        total, out = total / max(n, 1), out.div_(max(n, 1))
    return [torch.tensor(total, dtype=torch.float64), out]


def _exact_logprobs_rows(x, t, k, T):
    z = x / T
    lse = torch.logsumexp(z, dim=1)
    logp = z - lse[:, None]
    p = torch.exp(logp)
    entropy = -torch.xlogy(p, p).sum(dim=1)
    gone = t == IGNORE
    lp = logp[torch.arange(x.shape[0], device=x.device), torch.where(gone, 0, t)]
    out = [torch.where(gone, 0.0, v) for v in (lp, entropy, lse)]
    if k:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
        vals = logp.gather(1, order)
        vals[gone], order[gone] = -math.inf, -1
        out += [vals, order]
    return out


def _exact_distill_rows(x, ids, vals, T, renorm):
    p = torch.softmax(x / T, dim=1)
    q = torch.zeros_like(p)
    ok = ids >= 0
    w = torch.where(ok, vals / T if renorm else vals, -math.inf)
    some = ok.any(dim=1)
    qk = torch.zeros_like(w)
    qk[some] = torch.softmax(w[some], dim=1) if renorm else torch.exp(w[some])
    q.scatter_add_(1, torch.where(ok, ids, 0), qk)
    logp = torch.log_softmax(x / T, dim=1).gather(1, torch.where(ok, ids, 0))
    row = (torch.xlogy(qk, qk) - torch.where(ok, qk * logp, 0.0)).sum(dim=1)
    grad = T * (q.sum(dim=1, keepdim=True) * p - q) * some[:, None]
    return T * T * float(row[some].sum()), grad, int(some.sum())
