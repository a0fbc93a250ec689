"""64-bit plain implementations of the rotary append, scored attention, eviction and
draft verification, written from their definitions for the tests (numpy, loops)."""
import math

import numpy as np
import torch


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to("cpu").to(torch.float64).numpy()


def e4m3_values(codes: torch.Tensor) -> np.ndarray:
    return f64(codes.view(torch.float8_e4m3fn))


def rope(x, positions, inv_freq, pair_axis, interleaved):
    """x [tokens, heads, dim] float64 -> rotated; positions [axes][tokens]."""
    half = len(inv_freq)
    theta = positions[pair_axis].T.astype(np.float64) * np.asarray(inv_freq)  # [tokens, half]
    c, s = np.cos(theta)[:, None], np.sin(theta)[:, None]
    y = x.copy()
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + (1 if interleaved else half)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def rope_slack(x, half, interleaved):
    """Bound on the fp32 error of a rotated element, before its rounding.  The half
    turn's rounding to fp32 (relative 2^-24 of at most 1, times pi) is 1.9e-7, sincospi
    within 2 ulp 2.4e-7, two products and a sum 2 * 2^-24 = 1.2e-7: 5.5e-7 of |a| + |b|."""
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + (1 if interleaved else half)
    d = np.zeros_like(x)
    m = 5.5e-7 * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    d[..., ia] = m
    d[..., ib] = m
    return d


def rows_of(cache, table, length):
    """Logical rows [heads, length, dim] of one sequence (cache float64)."""
    nb, h, bs, d = cache.shape
    n = -(-length // bs)
    x = cache[table[:n]].transpose(1, 0, 2, 3).reshape(h, n * bs, d)
    return x[:, :length]


def scored(q, k_cache, v_cache, tables, lens, scale, scores):
    """q [n, u, hq, d]; returns out [n, u, hq, d], scores, share (all float64), and the
    largest sum of |q_d k_d| * scale (for error bounds)."""
    n, u, hq, d = q.shape
    h = k_cache.shape[1]
    g = hq // h
    out = np.zeros_like(q)
    new = scores.copy()
    share = np.zeros_like(scores)
    biggest = 0.0
    for i in range(n):
        L = int(lens[i])
        if L == 0:
            continue
        k, v = rows_of(k_cache, tables[i], L), rows_of(v_cache, tables[i], L)
        new[i, :, max(0, L - u):L] = 0.0
        for j in range(u):
            T = L - u + j + 1
            if T <= 0:
                continue
            for head in range(hq):
                kh, qv = k[head // g, :T], q[i, j, head]
                s = scale * (kh @ qv)
                biggest = max(biggest, float((np.abs(kh) @ np.abs(qv)).max()) * abs(scale))
                w = np.exp(s - s.max())
                w /= w.sum()
                out[i, j, head] = w @ v[head // g, :T]
                share[i, head // g, :T] += w
    return out, new + share, share, biggest


def evict(k_cache, v_cache, scores, row_pos, tables, lens, seq_lens, budget, sinks, recent):
    """In place on copies; returns (k, v, scores, row_pos, new_lens)."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    s_out, p_out = scores.copy(), row_pos.copy()
    bs = k_cache.shape[2]
    new_lens = np.minimum(lens, budget)
    for i in range(len(lens)):
        L = int(lens[i])
        if L <= budget:
            continue
        for h in range(scores.shape[1]):
            def rank(r):
                pos = int(row_pos[i, h, r])
                if pos < sinks or pos >= int(seq_lens[i]) - recent:
                    return (0, 0.0, r)
                x = float(scores[i, h, r])
                return (2, 0.0, r) if math.isnan(x) else (1, -x, r)
            kept = sorted(sorted(range(L), key=rank)[:budget])
            inside = set(kept)
            holes = [r for r in range(budget) if r not in inside]
            late = [r for r in kept if r >= budget]
            assert len(holes) == len(late)
            for to, frm in zip(holes, late):
                s_out[i, h, to], p_out[i, h, to] = scores[i, h, frm], row_pos[i, h, frm]
                bt, bf = tables[i, to // bs], tables[i, frm // bs]
                k_cache[bt, h, to % bs] = k_cache[bf, h, frm % bs]
                v_cache[bt, h, to % bs] = v_cache[bf, h, frm % bs]
    return k_cache, v_cache, s_out, p_out, new_lens


def verify(p, q, tokens, given, accept_u, sample_u):
    """p [n, k+1, V], q [n, k, V] or None; all float64 / ints.  (tokens, accepted)."""
    n, k = tokens.shape
    vocab = p.shape[2]
    out = np.full((n, k + 1), -1, dtype=np.int64)
    count = np.zeros(n, dtype=np.int64)

    def clean(w):
        return np.where(np.isfinite(w) & (w > 0), w, 0.0)

    for i in range(n):
        a = 0
        while a < given[i]:
            x = int(tokens[i, a])
            if not 0 <= x < vocab:
                break
            qx = 1.0 if q is None else q[i, a, x]
            if not accept_u[i, a] * qx < p[i, a, x]:
                break
            out[i, a] = x
            a += 1
        count[i] = a
        w = p[i, a]
        if a < given[i]:
            if q is None:
                w = w.copy()
                if 0 <= tokens[i, a] < vocab:
                    w[tokens[i, a]] = 0.0
            else:
                w = w - q[i, a]
        w = clean(w)
        if w.sum() == 0:
            w = clean(p[i, a])
        if w.sum() == 0:
            continue
        c = np.array([math.fsum(w[:v + 1]) for v in range(vocab)]) if vocab <= 64 else np.cumsum(w)
        over = np.nonzero(c > sample_u[i] * c[-1])[0]
        out[i, a] = over[0] if len(over) else np.nonzero(w)[0][-1]
    return out, count
