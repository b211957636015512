"""Cases for measuring the logits operators around a policy's LM head: the sampler's rules on
logits (penalties, biases, grammar masks), a teacher's top log-probs, and the distillation
loss on them.

``own`` chooses between the plain torch form of each operator and this package's entry points;
``prepare`` makes what a program has in hand before the call, ``run`` is one pass.
"""

import math

import torch

own = False

NEG_INF = -math.inf
REST_MIN = 2.0 ** -20   # least teacher mass outside its list
CELLS = 4 * 2048 * 151936   # rows x vocabulary of the largest listed case


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request being decoded: 600 tokens so far, penalties and a few biases
        dict(name="rules_decode_b1_v32000", op="rules", B=1, L=1, V=32000, dtype="bf16", hist=600, bias=8, mask=False,
             train=False, strided=False),
        # a decode batch under grammars, long histories
        dict(name="rules_decode_b64_v151936", op="rules", B=64, L=1, V=151936, dtype="bf16", hist=4096, bias=32,
             mask=True, train=False, strided=False),
        # a short odd-sized scoring batch, fp32, one row cut off each sequence's logits
        dict(name="rules_score_b3_l170_v32003", op="rules", B=3, L=170, V=32003, dtype="fp32", hist=77, bias=5,
             mask=True, train=True, strided=True),
        # policy logits under the sampler's penalties, forward and backward, prompts of 512
        dict(name="rules_train_b4_l1024_v151936", op="rules", B=4, L=1024, V=151936, dtype="bf16", hist=512, bias=16,
             mask=False, train=True, strided=False),
        # the top log-probs a serving endpoint returns with one token
        dict(name="topk_decode_b1_v151936_k20", op="topk", B=1, L=1, V=151936, dtype="bf16", K=20, T=1.0,
             strided=False),
        # the same for a batch, fp32 logits, odd vocabulary
        dict(name="topk_decode_b48_v50001_k5", op="topk", B=48, L=1, V=50001, dtype="fp32", K=5, T=0.7, strided=False),
        # a teacher scoring a batch of completions
        dict(name="topk_b4_l512_v32000_k128", op="topk", B=4, L=512, V=32000, dtype="bf16", K=128, T=1.0,
             strided=True),
        dict(name="topk_b4_l2048_v151936_k64", op="topk", B=4, L=2048, V=151936, dtype="bf16", K=64, T=1.0,
             strided=False),
        # the smallest training step: a unit test's batch
        dict(name="distill_b2_l16_v512_k8", op="distill", B=2, L=16, V=512, dtype="fp32", K=8, T=1.0, beta=0.0,
             tail=False, fused=False, strided=False),
        # forward KL on a teacher's renormalised list, loss weights known in advance
        dict(name="distill_b4_l512_v32000_k64", op="distill", B=4, L=512, V=32000, dtype="bf16", K=64, T=0.9, beta=0.0,
             tail=False, fused=True, strided=False),
        # reverse KL with the rest of the vocabulary as one bucket, odd vocabulary, fp32
        dict(name="distill_b3_l333_v50001_k32", op="distill", B=3, L=333, V=50001, dtype="fp32", K=32, T=1.0, beta=1.0,
             tail=True, fused=False, strided=True),
        # the largest: mixture divergence, forward then backward as autograd calls them
        dict(name="distill_b4_l2048_v151936_k64", op="distill", B=4, L=2048, V=151936, dtype="bf16", K=64, T=1.0,
             beta=0.5, tail=True, fused=False, strided=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rules", "topk", "distill"])
    V = _log_int(rng, 600, 151936)
    if rng.random() < 0.5:
        V = max(600, V // 8 * 8)
    B = _log_int(rng, 1, 64)
    L = 1 if op != "distill" and rng.random() < 0.4 else _log_int(rng, 1, 2048)
    B = max(1, min(B, CELLS // 4 // V)) if B * V > CELLS // 4 else B
    L = max(1, min(L, CELLS // 4 // (B * V)))
    c = dict(op=op, B=B, L=L, V=V, dtype=rng.choice(["bf16", "bf16", "fp32"]), strided=L > 1 and rng.random() < 0.3)
    if op == "rules":
        c.update(hist=_log_int(rng, 1, 8192 if L == 1 else 1024), bias=rng.randint(0, 64), mask=rng.random() < 0.5,
                 train=L > 1)
    else:
        c.update(K=_log_int(rng, 1, 256), T=rng.choice([0.6, 0.8, 1.0, 1.3]))
    if op == "distill":
        beta = rng.choice([0.0, 0.0, 0.3, 0.5, 1.0])
        c.update(beta=beta, tail=beta == 1.0 or rng.random() < 0.5, fused=rng.random() < 0.4)
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _logits(c, g):
    """Logits of spread 2, one row in twenty with a token far above the others."""
    B, L, V = c["B"], c["L"], c["V"]
    Lb = L + 1 if c["strided"] else L
    x = torch.randn(B, Lb, V, generator=g, device="cuda").mul_(2.0)
    peaked = torch.rand(B, Lb, generator=g, device="cuda") < 0.05
    at = torch.randint(0, V, (B, Lb, 1), generator=g, device="cuda")
    x.scatter_add_(2, at, peaked[..., None] * 20.0)
    return x.to(_dtype(c))


def _view(c, x):
    return x[:, :-1, :] if c["strided"] else x


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, L, V = c["B"], c["L"], c["V"]
    R = B * L
    s = dict(case=c, logits=_view(c, _logits(c, g)))
    rnd = lambda *n: torch.rand(*n, generator=g, device="cuda")  # noqa: E731
    if c["op"] == "rules":
        P = c["hist"]
        # a few tokens come often, most seldom
        s["tokens"] = (rnd(B, P + L) ** 3 * V).long().clamp_(max=V - 1)
        prompt = torch.randint(0, P + 1, (B,), generator=g, device="cuda")
        if L == 1:   # decoding: prompt and generated tokens make up the history
            hist = P - torch.randint(0, P // 4 + 1, (B, 1), generator=g, device="cuda")
            prompt = torch.minimum(prompt, hist[:, 0])
        else:        # scoring: each position's history is its sequence up to there
            prompt = P - prompt // 2
            hist = prompt[:, None] + torch.arange(L, device="cuda")[None, :]
        s["hist_len"] = hist.reshape(R).to(torch.int32)
        s["prompt_len"] = prompt.to(torch.int32)
        s["repetition"] = 1.0 + 0.5 * rnd(B)
        s["frequency"] = 0.8 * rnd(B) - 0.2
        s["presence"] = 0.8 * rnd(B) - 0.2
        s["bias_ids"] = s["bias"] = s["allowed"] = None
        if c["bias"]:
            s["bias_ids"] = rnd(B, V).topk(c["bias"], dim=1).indices
            s["bias"] = 10.0 * rnd(B, c["bias"]) - 5.0
        if c["mask"]:   # grammars: a few tokens left, about half, or nearly all
            share = torch.tensor([0.002, 0.5, 0.98], device="cuda")[
                torch.randint(0, 3, (B, L), generator=g, device="cuda")]
            W = (V + 31) // 32
            bits = rnd(B, L, W, 32) < share[:, :, None, None]
            weight = (torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda"))
            words = (bits * weight).sum(-1)
            s["allowed"] = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
        if c["train"]:
            s["dout"] = torch.randn(B, L, V, generator=g, device="cuda").mul_(1e-3).to(_dtype(c))
        return s
    if c["op"] == "topk":
        return s
    # distill: the teacher's list is the top of logits near the student's own
    x = s["logits"]
    t = x.float() + 0.5 * torch.randn(B, L, V, generator=g, device="cuda")
    top = t.reshape(R, V).topk(c["K"], dim=1)
    s["ids"] = top.indices
    s["teacher_logp"] = (top.values - torch.logsumexp(t.reshape(R, V), 1, keepdim=True)).contiguous()
    length = torch.randint(max(1, L // 2), L + 1, (B, 1), generator=g, device="cuda")
    mask = torch.arange(L, device="cuda")[None, :] < length
    s["mask"] = mask.reshape(R).to(torch.uint8)
    s["dloss"] = (mask / mask.sum().float()).reshape(R).contiguous()
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_history(s):
    c, tokens = s["case"], s["tokens"]
    B, L, V = c["B"], c["L"], c["V"]
    pos = torch.arange(tokens.shape[1], device="cuda")
    hist = pos < s["hist_len"].view(B, L, 1)
    made = hist & (pos >= s["prompt_len"].view(B, 1, 1))
    at = tokens[:, None, :].expand(B, L, -1)
    zero = torch.zeros(B, L, V, device="cuda")
    return zero.scatter_add(2, at, hist.float()) > 0, zero.scatter_add(2, at, made.float())


def _plain_allowed(s):
    c = s["case"]
    bits = (s["allowed"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    return bits.reshape(c["B"], c["L"], -1)[..., :c["V"]] != 0


def _plain_rules(s):
    c, x = s["case"], s["logits"].float()
    row = lambda v: v.view(-1, 1, 1)  # noqa: E731
    seen, count = _plain_history(s)
    rep = row(s["repetition"])
    y = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    y = y - row(s["frequency"]) * count - row(s["presence"]) * (count > 0)
    if s["bias"] is not None:
        y = y + torch.zeros(c["B"], c["V"], device="cuda").scatter(1, s["bias_ids"], s["bias"])[:, None, :]
    if s["allowed"] is not None:
        y = torch.where(_plain_allowed(s), y, NEG_INF)
    out = dict(out=y.to(_dtype(c)))
    if c["train"]:
        d = s["dout"].float()
        d = torch.where(seen, torch.where(x > 0, d / rep, d * rep), d)
        if s["allowed"] is not None:
            d = torch.where(_plain_allowed(s), d, 0.0)
        out["dlogits"] = d.to(_dtype(c))
    return out


def _plain_topk(s):
    c = s["case"]
    x = s["logits"].float().reshape(-1, c["V"])
    z = x / c["T"]
    m = z.amax(1, keepdim=True)
    lse = m[:, 0] + (z - m).exp().sum(1).log()
    # order by value, then by the lowest index: one integer key for both
    b = (x + 0.0).contiguous().view(torch.int32).long()
    b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    key = (b << 32) | (c["V"] - 1 - torch.arange(c["V"], device="cuda"))
    ids = c["V"] - 1 - (key.topk(c["K"], dim=1).values & 0xFFFFFFFF)
    return dict(ids=ids, logp=z.gather(1, ids) - lse[:, None], lse=lse)


def _plain_distill(s):
    c, ids, lq = s["case"], s["ids"], s["teacher_logp"].double()
    T, beta = c["T"], c["beta"]
    z = s["logits"].float().reshape(-1, c["V"]) / T
    m = z.amax(1, keepdim=True)
    # the buckets in 64 bits: a divergence is a small difference of log-probs around 10
    e = (z - m).exp()
    zk = s["logits"].reshape(-1, c["V"]).gather(1, ids).double() / T - m.double()
    rest = e.scatter(1, ids, 0.0).sum(1, keepdim=True).double()
    total = rest + zk.exp().sum(1, keepdim=True)
    lse = m.double() + total.log()
    p, rest, lp = e / total.float(), rest / total, zk - total.log()
    if c["tail"]:
        q_rest = (1.0 - lq.exp().sum(1, keepdim=True)).clamp(min=REST_MIN)
    else:
        lq = lq - lq.exp().sum(1, keepdim=True).log()
        q_rest = torch.zeros_like(rest)
    # buckets: the list's tokens, then the rest of the vocabulary
    p_b, lp_b = torch.cat([lp.exp(), rest], 1), torch.cat([lp, rest.log()], 1)
    q_b, lq_b = torch.cat([lq.exp(), q_rest], 1), torch.cat([lq, q_rest.log()], 1)
    none = torch.zeros_like(p_b)
    if beta == 0.0:
        term, grad = torch.where(q_b > 0, q_b * (lq_b - lp_b), none), -q_b
    elif beta == 1.0:
        term = torch.where(p_b > 0, p_b * (lp_b - lq_b), none)
        grad = term + p_b
    else:
        lm = (beta * q_b + (1.0 - beta) * p_b).log()
        mine = torch.where(p_b > 0, p_b * (lp_b - lm), none)
        term = beta * torch.where(q_b > 0, q_b * (lq_b - lm), none) + (1.0 - beta) * mine
        grad = (1.0 - beta) * mine
    total = grad.sum(1, keepdim=True)
    d = p * (torch.where(rest > 0, grad[:, -1:] / rest, 0.0) - total).float()
    d = d.scatter(1, ids, (grad[:, :-1] - p_b[:, :-1] * total).float())
    live = s["mask"] != 0
    d = torch.where(live[:, None], d * (s["dloss"] / T)[:, None], 0.0)
    keep = lambda v: torch.where(live, v, 0.0).float()  # noqa: E731
    return dict(loss=keep(term.sum(1)), lse=keep(lse[:, 0]), p_rest=keep(rest[:, 0]),
                dlogits=d.to(_dtype(c)).view(c["B"], c["L"], c["V"]))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own_rules(s):
    import rl_fine_tuning_pass_gb300 as rp
    rules = dict(tokens=s["tokens"], hist_len=s["hist_len"], prompt_len=s["prompt_len"], repetition=s["repetition"],
                 frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"], bias=s["bias"],
                 allowed=s["allowed"])
    out = dict(out=rp.process_logits_fwd(s["logits"], **rules))
    if s["case"]["train"]:
        out["dlogits"] = rp.process_logits_bwd(s["logits"], s["dout"], **rules)
    return out


def _own_topk(s):
    import rl_fine_tuning_pass_gb300 as rp
    ids, logp, lse = rp.topk_log_softmax(s["logits"], s["case"]["K"], T=s["case"]["T"])
    return dict(ids=ids, logp=logp, lse=lse)


def _own_distill(s):
    import rl_fine_tuning_pass_gb300 as rp
    c = s["case"]
    how = dict(T=c["T"], beta=c["beta"], tail=c["tail"], mask=s["mask"])
    if c["fused"]:
        return rp.distill_topk_fused(s["logits"], s["ids"], s["teacher_logp"], s["dloss"], **how)
    out = rp.distill_topk_fwd(s["logits"], s["ids"], s["teacher_logp"], **how)
    out["dlogits"] = rp.distill_topk_bwd(s["logits"], s["ids"], s["teacher_logp"], s["dloss"], out["lse"],
                                         out["p_rest"], **how)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rules": _own_rules, "topk": _own_topk, "distill": _own_distill}[op](state)
    return {"rules": _plain_rules, "topk": _plain_topk, "distill": _plain_distill}[op](state)


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    R = c["B"] * c["L"]
    cells = R * c["V"]
    if c["op"] == "rules":
        passes = 2 if c["train"] else 1
        aux = 8 * c["B"] * (c["hist"] + c["L"] + 2 * c["bias"]) + 4 * R + (cells // 8 if c["mask"] else 0)
        return dict(bytes=passes * (2 * cells * es + aux), flops=2 * passes * cells)
    if c["op"] == "topk":
        return dict(bytes=cells * es + R * (12 * c["K"] + 4), flops=4 * cells)
    return dict(bytes=2 * cells * es + R * (12 * c["K"] + 20), flops=8 * cells)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, a block of rows at a time
# ---------------------------------------------------------------------------
def _exact_rules(s):
    c = s["case"]
    B, L, V = c["B"], c["L"], c["V"]
    out = torch.empty(B, L, V, dtype=torch.float64, device="cuda")
    grad = torch.empty_like(out) if c["train"] else None
    ones = torch.ones(s["tokens"].shape[1], dtype=torch.float64, device="cuda")
    for b in range(B):
        for l0 in range(0, L, 256):
            l1 = min(L, l0 + 256)
            # prefix counts: those of the block's first row, then one row's new tokens at a time
            n = s["hist_len"].view(B, L)[b, l0:l1].tolist()
            p = int(s["prompt_len"][b])
            seen = torch.zeros(l1 - l0, V, dtype=torch.float64, device="cuda")
            made = torch.zeros_like(seen)
            for r in range(l1 - l0):
                a = n[r - 1] if r else 0
                if r:
                    seen[r], made[r] = seen[r - 1], made[r - 1]
                seen[r].index_add_(0, s["tokens"][b, a:n[r]], ones[a:n[r]])
                a = max(a, p)
                if n[r] > a:
                    made[r].index_add_(0, s["tokens"][b, a:n[r]], ones[a:n[r]])
            x = s["logits"][b, l0:l1].double()
            rep, freq, pres = (float(s[k][b]) for k in ("repetition", "frequency", "presence"))
            slope = torch.where(seen > 0, torch.where(x > 0, 1.0 / rep, rep), 1.0)
            y = x * slope - freq * made - pres * made.clamp(max=1.0)
            if s["bias"] is not None:
                y[:, s["bias_ids"][b]] += s["bias"][b].double()
            if s["allowed"] is not None:
                j = torch.arange(V, device="cuda")
                no = ((s["allowed"][b, l0:l1].long()[:, j // 32] >> (j % 32)) & 1) == 0
                y[no] = NEG_INF
                slope = slope.masked_fill(no, 0.0)
            out[b, l0:l1] = y
            if grad is not None:
                grad[b, l0:l1] = s["dout"][b, l0:l1].double() * slope
    return dict(out=out, dlogits=grad) if c["train"] else dict(out=out)


def _exact_topk(s):
    c = s["case"]
    x = s["logits"]
    logp, lse = [], []
    for b in range(c["B"]):
        for l0 in range(0, c["L"], 512):
            z = x[b, l0:l0 + 512].double() / c["T"]
            lse.append(torch.logsumexp(z, 1))
            logp.append(z.topk(c["K"], dim=1).values - lse[-1][:, None])
    return dict(ids=None, logp=torch.cat(logp), lse=torch.cat(lse))


def _divergence(p, q, beta):
    """(terms, d terms / d p) of beta KL(q|m) + (1 - beta) KL(p|m), m = beta q + (1 - beta) p, with the limits
    KL(q|p) at beta = 0 and KL(p|q) at beta = 1."""
    if beta == 0.0:
        return torch.xlogy(q, q) - torch.xlogy(q, p), -q / p
    if beta == 1.0:
        return torch.xlogy(p, p) - torch.xlogy(p, q), (p / q).log() + 1.0
    m = beta * q + (1.0 - beta) * p
    return (beta * (torch.xlogy(q, q) - torch.xlogy(q, m)) + (1.0 - beta) * (torch.xlogy(p, p) - torch.xlogy(p, m)),
            (1.0 - beta) * (p / m).log())


def _exact_distill(s):
    c = s["case"]
    T, R, V = c["T"], c["B"] * c["L"], c["V"]
    loss = torch.zeros(R, dtype=torch.float64, device="cuda")
    lse, p_rest = torch.zeros_like(loss), torch.zeros_like(loss)
    grad = torch.zeros(R, V, dtype=torch.float64, device="cuda")
    for r0 in range(0, R, 512):
        r = torch.arange(r0, min(R, r0 + 512), device="cuda")
        r = r[s["mask"][r] != 0]
        if not len(r):
            continue
        z = s["logits"][r // c["L"], r % c["L"]].double() / T
        lse[r] = torch.logsumexp(z, 1)
        p = torch.softmax(z, 1)
        ids, q = s["ids"][r], s["teacher_logp"][r].double().exp()
        inside = torch.zeros_like(p, dtype=torch.bool).scatter_(1, ids, True)
        p_rest[r] = p.masked_fill(inside, 0.0).sum(1)
        if c["tail"]:
            q_rest = (1.0 - q.sum(1)).clamp(min=REST_MIN)
        else:
            q, q_rest = q / q.sum(1, keepdim=True), torch.zeros_like(p_rest[r])
        terms, slope = _divergence(p.gather(1, ids), q, c["beta"])
        rest_term, rest_slope = _divergence(p_rest[r], q_rest, c["beta"])
        loss[r] = terms.sum(1) + rest_term
        f = rest_slope[:, None].expand_as(p).scatter(1, ids, slope)
        grad[r] = p * (f - (p * f).sum(1, keepdim=True)) * (s["dloss"][r].double() / T)[:, None]
    return dict(loss=loss, lse=lse, p_rest=p_rest, dlogits=grad.view(c["B"], c["L"], V))


def exact(case, seed):
    s = prepare(case, seed)
    return {"rules": _exact_rules, "topk": _exact_topk, "distill": _exact_distill}[case["op"]](s)
