"""fp64 CPU oracle of the operators next to the row pass: the sampler's rules on logits, the
top log-probs of a row, and the distillation loss on a teacher's top log-probs.

Test infrastructure only, with no code shared with the CUDA library: plain loops over the
rows, from the definitions.  Pinned by ``tests/test_logits_ops_oracle.py`` (closed forms,
finite differences, invariants).
"""

from __future__ import annotations

import numpy as np

__all__ = ["process_logits", "process_logits_bwd", "topk_log_softmax", "distill_topk", "REST_MIN"]

REST_MIN = 2.0 ** -20


def _row_rules(V, row, tokens, hist, prompt, bias_ids, bias, allowed):
    """(seen, generated count, bias, allowed) of each column of one row."""
    seen = np.zeros(V, bool)
    count = np.zeros(V)
    if tokens is not None:
        for i in range(max(0, min(int(hist), len(tokens)))):
            t = int(tokens[i])
            if 0 <= t < V:
                seen[t] = True
                if i >= prompt:
                    count[t] += 1
    add = np.zeros(V)
    if bias_ids is not None:
        for t, v in zip(bias_ids, bias):
            if 0 <= int(t) < V:
                add[int(t)] = float(v)   # the last entry of a column counts
    ok = np.ones(V, bool) if allowed is None else np.asarray(
        [(int(allowed[j // 32]) >> (j % 32)) & 1 == 1 for j in range(V)]) if V < 2000 else _bits(allowed, V)
    return seen, count, add, ok


def _bits(words, V):
    w = np.ascontiguousarray(np.asarray(words, dtype=np.int32)).view(np.uint8)
    return np.unpackbits(w, bitorder="little")[:V].astype(bool)


def _rows(B, L, tokens, hist_len, prompt_len, bias_ids, bias, allowed):
    for b in range(B):
        for l in range(L):
            r = b * L + l
            n = 0 if tokens is None else (tokens.shape[1] if hist_len is None else hist_len[r])
            yield r, b, (None if tokens is None else tokens[b], n, 0 if prompt_len is None else int(prompt_len[b]),
                         None if bias_ids is None else bias_ids[b], None if bias is None else bias[b],
                         None if allowed is None else allowed[r])


def process_logits(x, L, *, tokens=None, hist_len=None, prompt_len=None, repetition=None, frequency=None,
                   presence=None, bias_ids=None, bias=None, allowed=None):
    """x [B*L, V] fp64, allowed [B*L, W] int32 -> (y, size): the processed logits and the sum of
    the magnitudes of the terms each was formed from (for rounding bounds)."""
    R, V = x.shape
    y, size = np.empty_like(x), np.empty_like(x)
    for r, b, args in _rows(R // L, L, tokens, hist_len, prompt_len, bias_ids, bias, allowed):
        seen, count, add, ok = _row_rules(V, r, *args)
        v = x[r].copy()
        if repetition is not None:
            rho = float(repetition[b])
            v = np.where(seen, np.where(v > 0, v / rho, v * rho), v)
        f = 0.0 if frequency is None else float(frequency[b])
        a = 0.0 if presence is None else float(presence[b])
        s = np.abs(v) + abs(f) * count + abs(a) * (count > 0) + np.abs(add)
        v = np.where(count > 0, v - f * count - a, v)
        v = v + add
        y[r] = np.where(ok, v, -np.inf)
        size[r] = s
    return y, size


def process_logits_bwd(x, dy, L, *, tokens=None, hist_len=None, prompt_len=None, repetition=None, frequency=None,
                       presence=None, bias_ids=None, bias=None, allowed=None):
    R, V = x.shape
    d = np.empty_like(x)
    for r, b, args in _rows(R // L, L, tokens, hist_len, prompt_len, bias_ids, bias, allowed):
        seen, _, _, ok = _row_rules(V, r, *args)
        g = dy[r].copy()
        if repetition is not None:
            rho = float(repetition[b])
            g = np.where(seen, np.where(x[r] > 0, g / rho, g * rho), g)
        d[r] = np.where(ok, g, 0.0)
    return d


def topk_log_softmax(x, K, T):
    """x [R, V] fp64 -> (ids, logp, lse); rows without a finite lse get ids 0..K-1 and NaN."""
    R, V = x.shape
    ids, logp, lse = np.empty((R, K), np.int64), np.empty((R, K)), np.empty(R)
    for r in range(R):
        z = x[r] / T
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            m = z.max()
            ln_s = np.log(np.exp(z - m).sum()) if m != -np.inf else 0.0
            lse[r] = m + ln_s
        if not np.isfinite(lse[r]):
            ids[r], logp[r] = np.arange(K), np.nan
            continue
        order = np.lexsort((np.arange(V), -x[r]))[:K]
        ids[r], logp[r] = order, (z[order] - m) - ln_s   # m + ln_s may absorb ln_s
    return ids, logp, lse


def _kl(a, log_a, log_b):
    """a log(a / b) per bucket, 0 where a is 0."""
    with np.errstate(invalid="ignore"):
        return np.where(a == 0, 0.0, a * (log_a - log_b))


def _log_sum(z):
    """log sum exp(z), -inf of nothing."""
    m = z.max() if len(z) else -np.inf
    return m if np.isneginf(m) else m + np.log(np.exp(z - m).sum())


def distill_topk(x, ids, tlogp, T, beta, tail, mask=None, dloss=None):
    """x [R, V] fp64, ids / tlogp [R, K] -> dict of loss, lse, p_rest, and with dloss dlogits;
    also "G" [R] = sum |G_b| + |S|, "terms" [R] = sum of the terms' magnitudes, "F" [R] =
    |G_rest / p_rest| (for error bounds)."""
    R, V = x.shape
    out = {k: np.zeros(R) for k in ("loss", "lse", "p_rest", "G", "terms", "F")}
    if dloss is not None:
        out["dlogits"] = np.zeros((R, V))
    for r in range(R):
        if mask is not None and mask[r] == 0:
            continue
        use = np.asarray([i >= 0 for i in ids[r]], bool)
        at, lq = np.asarray(ids[r])[use].astype(np.int64), np.asarray(tlogp[r], dtype=np.float64)[use]
        if np.any(at >= V) or len(set(at.tolist())) < len(at):
            for k in ("loss", "lse", "p_rest"):
                out[k][r] = np.nan
            if dloss is not None and dloss[r] != 0:
                out["dlogits"][r] = np.nan
            continue
        z = x[r] / T
        m = z.max()
        lse = m + np.log(np.exp(z - m).sum())
        p = np.exp(z - lse)
        inside = np.zeros(V, bool)
        inside[at] = True
        q = np.exp(lq)
        # without a column that has any mass outside the list there is no rest, as without the tail
        if tail and not np.all(np.isneginf(x[r][~inside])):
            q_rest = max(1.0 - q.sum(), REST_MIN)
        else:
            q, q_rest = (q / q.sum() if len(q) else q), 0.0
        P, Q = np.append(p[at], p[~inside].sum()), np.append(q, q_rest)
        # log-probs of the buckets from the logits: a mass may be less than 64 bits hold
        rest = _log_sum(z[~inside])
        with np.errstate(divide="ignore", invalid="ignore"):
            LP, LQ = np.append(z[at], rest) - lse, np.log(Q)
            if beta == 0.0:
                terms, slope = _kl(Q, LQ, LP), None
            elif beta == 1.0:
                terms, slope = _kl(P, LP, LQ), LP - LQ + 1.0
            else:
                LM = np.logaddexp(np.log(beta) + LQ, np.log1p(-beta) + LP)
                terms = beta * _kl(Q, LQ, LM) + (1.0 - beta) * _kl(P, LP, LM)
                slope = (1.0 - beta) * (LP - LM)
        # G = p dL/dp: at p = 0 the limit, -q for the forward divergence and 0 for the others
        G = -Q if beta == 0.0 else np.where(P == 0, 0.0, P * np.where(P == 0, 0.0, slope))
        S = G.sum()
        F = G[-1] / P[-1] if P[-1] > 0 else 0.0
        out["loss"][r], out["lse"][r], out["p_rest"][r] = terms.sum(), lse, P[-1]
        out["G"][r], out["terms"][r], out["F"][r] = np.abs(G).sum() + abs(S), np.abs(terms).sum(), abs(F)
        if dloss is not None:
            # p_j G_rest / p_rest with p_j / p_rest from the logits
            with np.errstate(invalid="ignore", over="ignore"):   # of listed columns, set below
                d = (np.exp(z - rest) * G[-1] if rest > -np.inf else 0.0) - p * S
            d[at] = G[:-1] - p[at] * S
            out["dlogits"][r] = d * (float(dloss[r]) / T)
    return out
