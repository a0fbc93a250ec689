"""64-bit plain implementations of the block-scaled cache, the block pool's bookkeeping and
the logits' adjustment, written from their definitions for the tests (numpy, loops)."""
import numpy as np
import torch

E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
_POS = E4M3[:127]          # codes 0 .. 126 in ascending order of value, 448 last
LEAST, MOST = 2.0 ** -40, 2.0 ** 40


def e4m3(x):
    """Codes of float64 values: nearest, ties to even, saturating; NaN to 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=1e300)), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    mid = (_POS[lo] + _POS[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    code = np.where(np.signbit(x), code + 128, code)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def clamp(s):
    s = np.asarray(s, np.float64)
    return np.where(np.isnan(s), LEAST, np.clip(s, LEAST, MOST))


def need(top):
    """The least power of two s with top <= 448 s, in the range of scales."""
    if top <= 0:
        return LEAST
    e = -200
    while 448.0 * 2.0 ** e < top and e < 200:
        e += 1
    return float(np.clip(2.0 ** e, LEAST, MOST))


def append(kc, vc, scales, k_new, v_new, tables, lens, q_len):
    """In place: codes uint8 [nb, h, bs, d], scales float32 [nb, h, 2]; rows float64."""
    nb, h, bs, d = kc.shape
    for i, L in enumerate(int(x) for x in lens):
        first = L - q_len
        for lb in range(max(0, first) // bs, -(-L // bs) if L > 0 else 0):
            if lb >= tables.shape[1] or not 0 <= tables[i, lb] < nb:
                continue
            b = tables[i, lb]
            r0, r1 = max(0, first - lb * bs), min(bs, L - lb * bs)
            for which, (cache, rows) in enumerate(((kc, k_new), (vc, v_new))):
                for head in range(h):
                    t0 = i * q_len + lb * bs + r0 - first
                    x = rows[t0:t0 + r1 - r0, head]
                    fin = np.abs(x[np.isfinite(x)])
                    s = need(fin.max() if fin.size else 0.0)
                    if r0 > 0:
                        old = float(clamp(scales[b, head, which]))
                        s = max(s, old)
                        if s > old:
                            f = np.float32(np.float32(old) / np.float32(s))
                            v = E4M3[cache[b, head, :r0]].astype(np.float32)
                            cache[b, head, :r0] = e4m3((v * f).astype(np.float64))
                    with np.errstate(over="ignore", invalid="ignore"):
                        y = (x.astype(np.float32) / np.float32(s)).astype(np.float64)
                    cache[b, head, r0:r1] = e4m3(y)
                    scales[b, head, which] = s


def attend(q, kc, vc, scales, tables, lens, scale):
    """q [n, u, hq, d] float64; codes and scales as above.  Returns out, and a bound on a
    kernel's error before its output's rounding (derived in the tests) from: sum of w |v|,
    largest base-2 score magnitude, sum |q k| scale, largest V scale of the row's blocks."""
    n, u, hq, d = q.shape
    nb, h, bs, _ = kc.shape
    g = hq // h
    out, wv, mags = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:3] + (4,))
    sc = clamp(scales)
    for i, L in enumerate(int(x) for x in lens):
        if L <= 0:
            continue
        ids = [int(b) for b in tables[i, :-(-L // bs)]]

        def rows(cache, which):
            page = [E4M3[cache[b]] * sc[b, :, which][:, None, None] if 0 <= b < nb else np.zeros((h, bs, d))
                    for b in ids]
            return np.concatenate(page, axis=1)[:, :L]

        k, v = rows(kc, 0), rows(vc, 1)
        sv = np.repeat(np.array([sc[b, :, 1] if 0 <= b < nb else np.ones(h) for b in ids]), bs, axis=0)[:L]
        for j in range(u):
            T = L - u + j + 1
            if T <= 0:
                continue
            for head in range(hq):
                kh, vh, x = k[head // g, :T], v[head // g, :T], q[i, j, head]
                s = scale * (kh @ x)
                w = np.exp(s - s.max())
                w /= w.sum()
                out[i, j, head] = w @ vh
                wv[i, j, head] = w @ np.abs(vh)
                mags[i, j, head] = (np.abs(s).max() * 1.4427, (np.abs(kh) @ np.abs(x)).max() * abs(scale) * 1.4427,
                                    sv[:T, head // g].max(), np.abs(kh).sum(1).max() * np.abs(x).max() *
                                    abs(scale) * 1.4427)
    return out, wv, mags


# ------------------------------------------------------------------------- pool
def free(tables, refs, keep, bs):
    for i in range(tables.shape[0]):
        for j in range(tables.shape[1]):
            if tables[i, j] >= 0 and j >= -(-max(0, int(keep[i])) // bs):
                refs[tables[i, j]] -= 1
                tables[i, j] = -1


def reserve(tables, refs, lens, bs):
    pool = [b for b in range(len(refs)) if refs[b] == 0]
    missing = 0
    for i in range(tables.shape[0]):
        for j in range(min(tables.shape[1], -(-max(0, int(lens[i])) // bs))):
            if tables[i, j] < 0:
                if pool:
                    tables[i, j] = pool.pop(0)
                    refs[tables[i, j]] = 1
                else:
                    missing += 1
    return missing


def fork(tables, lens, refs, src, dst, bs):
    """Returns (pairs, missing)."""
    pool = [b for b in range(len(refs)) if refs[b] == 0]
    pairs, missing = [], 0
    was, length = tables.copy(), lens.copy()
    for s, d in zip(src, dst):
        L = int(length[s])
        full = L // bs
        row = np.full(tables.shape[1], -1, tables.dtype)
        row[:full] = was[s, :full]
        for b in row[:full]:
            refs[b] += 1
        lens[d] = L
        if L % bs:
            if pool:
                row[full] = pool.pop(0)
                refs[row[full]] = 1
                pairs.append((was[s, full], row[full]))
            else:
                missing += 1
                lens[d] = full * bs
        tables[d] = row
    return pairs, missing


def compact(tables, refs):
    """Returns (tables, refs, pairs, live), new arrays."""
    live = int((refs != 0).sum())
    frm = [b for b in range(live, len(refs)) if refs[b] != 0]
    to = [b for b in range(live) if refs[b] == 0]
    name = np.arange(len(refs))
    new = refs.copy()
    for f, t in zip(frm, to):
        name[f] = t
        new[t], new[f] = refs[f], 0
    return np.where(tables >= 0, name[np.maximum(tables, 0)], tables).astype(tables.dtype), new, list(zip(frm, to)), live


# ----------------------------------------------------------------------- logits
def adjusted(x, history, prompt, drafts, rep, pres, freq, bias, allowed):
    """One row in float32 steps as defined: x float32 [v]; history / drafts lists of ids,
    prompt how many of the history; bias [(id, value)]; allowed bool [v] or None."""
    f = np.float32
    v = len(x)
    y = x.astype(f).copy()
    ok = [int(t) for t in history[:prompt] if 0 <= t < v]
    said = [int(t) for t in list(history[prompt:]) + list(drafts) if 0 <= t < v]
    count = np.bincount(said, minlength=v) if said else np.zeros(v, int)
    seen = count > 0
    seen[ok] = True
    with np.errstate(over="ignore", invalid="ignore"):
        y = np.where(seen, np.where(y > 0, y / f(rep), y * f(rep)), y).astype(f)
        y = np.where(count > 0, (y - (count.astype(f) * f(freq)).astype(f)).astype(f) - f(pres), y).astype(f)
        for t, b in bias:
            if 0 <= t < v:
                y[t] = f(y[t] + f(b))
    if allowed is not None:
        y[~allowed] = -np.inf
    return y


def probabilities(y, t):
    y = np.where(np.isnan(y), -np.inf, y.astype(np.float64))
    if y.max() == -np.inf:
        return np.zeros_like(y)
    if not t > 0:
        p = np.zeros_like(y)
        p[int(np.argmax(y))] = 1
        return p
    if y.max() == np.inf:
        return (y == np.inf) / (y == np.inf).sum()
    with np.errstate(over="ignore"):
        p = np.exp((y - y.max()) / float(t))
    return p / p.sum()
