"""Plain 64-bit implementations of the drafted-token calls (numpy, unit by
unit, from the definitions in include/kvc.h) and the error bounds the tests
hold the kernels to."""
import numpy as np

D = 128
SCALE = 1.0 / np.sqrt(D)
E32 = 2.0 ** -24            # half a step of fp32, relative
EBF = 2.0 ** -8             # half a step of bf16, relative


def bits(word, T):
    word = int(word) & (1 << 64) - 1
    return np.array([word >> j & 1 for j in range(T)], dtype=bool)


def logit_error(q, keys):
    """Bound on a computed logit's error: 128 fp32 additions of exact products
    (counted twice, for adders that truncate), the scale, the bias."""
    return (2 * D + 4) * E32 * (np.abs(q) @ np.abs(keys).T) * SCALE


def attend(q, K, V, votes, n, kt, vt, mask, live, mom, first, correct):
    """One unit: q [T][G][D], caches [cap][D], tree rows [T][D] as float64.
    Returns o, lse and elementwise error bounds, each [live][G](...)."""
    G = q.shape[1]
    o = np.zeros((live, G, D))
    lse = np.full((live, G), -np.inf)
    bo, bl = np.zeros((live, G, D)), np.zeros((live, G))
    for t in range(live):
        see = [j for j in range(live) if int(mask[t]) >> j & 1]
        keys = np.concatenate([K[:n], kt[see]])
        vals = np.concatenate([V[:n], vt[see]])
        for h in range(G):
            f, A, ex, worst = np.zeros(D), np.zeros(D), 0.0, 0.0
            if len(keys):
                x = keys @ q[t, h] * SCALE
                if votes is not None:
                    x[:n] += np.log(votes[:n])
                top = x.max()
                e = np.exp(x - top)
                lse[t, h] = top + np.log(e.sum())
                p = e / e.sum()
                f, A = p @ vals, p @ np.abs(vals)
                err = logit_error(q[t, h], keys) + 4 * E32 * (np.abs(x) + abs(top))
                # the weights' error, the sums' (at most 128 terms a run, one
                # run per 128 slots), exp and log
                ex = float(p @ err) + (256 + len(keys) / 128) * E32 + 8 * E32
                bl[t, h] = ex + 4 * E32 * abs(lse[t, h])
                worst = float(err.max()) + ex
            b = A * (EBF + worst)
            if correct and mom[0] > 0:
                ne, mu_k, mu_v, C = mom
                ze = np.log(ne) + mu_k @ q[t, h] * SCALE
                ez = (2 * D + 4) * E32 * (np.abs(mu_k) @ np.abs(q[t, h])) * SCALE + \
                    8 * E32 * (1 + abs(ze))
                w = 1.0 / (1.0 + np.exp(min(700.0, ze - lse[t, h])))
                g, bg = mu_v.copy(), 4 * E32 * np.abs(mu_v)
                if first:
                    g = g + C @ q[t, h] * SCALE
                    # the co-moment as two bf16 terms: 2^-16 of every product
                    bg = bg + (2.0 ** -16 + (4 * D + 8) * E32) * (np.abs(C) @ np.abs(q[t, h])) * SCALE
                dw = w * (1 - w) * (ez + bl[t, h] * (np.isfinite(lse[t, h]))) + 4 * E32
                b = w * b + (1 - w) * bg + dw * (np.abs(f) + np.abs(g))
                f = w * f + (1 - w) * g
            o[t, h], bo[t, h] = f, b + EBF * (np.abs(f) + b) + 1e-30
    return o, lse, bo, bl


def weights(q, K, votes, n, kt, mask, path, w, lse):
    """One unit's S [n + a] and its bound."""
    G, a = q.shape[1], len(path)
    S, b = np.zeros(n + a), np.zeros(n + a)
    for j, c in enumerate(path):
        see = [int(mask[c]) >> r & 1 for r in path]
        keys = np.concatenate([K[:n], kt[path]]) if a else K[:n]
        for h in range(G):
            if lse[c, h] == -np.inf:
                continue
            x = keys @ q[c, h] * SCALE
            e = np.exp(x - lse[c, h])
            if votes is not None:
                e[:n] *= votes[:n]
            e[n:] = np.where(see, e[n:], 0.0)
            e = e * w[j] / G
            S += e
            b += np.where(e > 0, e, 0) * (logit_error(q[c, h], keys) + 8 * E32 * (
                np.abs(x) + abs(lse[c, h]) + 2 + abs(np.log(max(w[j], 1e-30) / G))))
    return S, b + (a * G + 16) * E32 * S + (a * G) * 2.0 ** -126 * 8


def commit(K, V, votes, pos, util, n, budget, rule, alpha, S, kt, vt, path, pos0, mom):
    """One unit, on copies.  K, V [cap][D]; returns a dict of the new state,
    the victims' slots and positions, and bounds of the moments."""
    K, V, pos, util = K.copy(), V.copy(), pos.copy(), util.copy()
    votes = None if votes is None else votes.copy()
    a = len(path)
    rk, rv = np.concatenate([K[:n], kt[path]]), np.concatenate([V[:n], vt[path]])
    rp = np.concatenate([pos[:n], pos0 + np.arange(a)])
    rw = np.concatenate([votes[:n] if votes is not None else np.ones(n, int), np.ones(a, int)])
    ru = np.concatenate([util[:n], np.full(a, np.inf)])
    if S is not None:
        fresh = np.isinf(ru)
        with np.errstate(invalid="ignore"):
            upd = {"single": S, "cumulative": ru + S, "ema": alpha * ru + (1.0 - alpha) * S}[rule]
        ru = np.where(fresh, S, upd)
    k = max(0, n + a - budget)
    order = sorted((i for i in range(n + a) if not np.isinf(ru[i])), key=lambda i: (ru[i], rp[i], i))
    vic = sorted(order[:k])
    assert len(vic) == k
    out = dict(n_evict=k, evict_idx=vic, evict_pos=[int(rp[i]) for i in vic])
    if mom is not None and k:
        n0, mu_k, mu_v, C = mom
        p = rw[vic].astype(float)
        nb, x, y = p.sum(), rk[vic], rv[vic]
        n1 = n0 + nb
        sk, sv = n0 * mu_k + p @ x, n0 * mu_v + p @ y
        raw = n0 * (C + np.outer(mu_v, mu_k)) + (y * p[:, None]).T @ x
        out.update(n=n1, mu_k=sk / n1, mu_v=sv / n1, C=raw / n1 - np.outer(sv, sk) / n1 ** 2)
        ax, ay = (p @ np.abs(x)) / nb + np.abs(mu_k), (p @ np.abs(y)) / nb + np.abs(mu_v)
        out["bound_mu"] = (k + 8) * 2 * E32
        out["bound_C"] = (2 * k + 16) * 2 * E32 * (
            n0 * np.abs(C) / n1 + (np.abs(y) * p[:, None]).T @ np.abs(x) / n1 + 4 * np.outer(ay, ax))
        out["scale_k"], out["scale_v"] = ax, ay
    end = n + a - k
    gone = set(vic)
    holes = [i for i in vic if i < end]
    fill = [i for i in range(end, n + a) if i not in gone]
    util[:n] = ru[:n]
    stay = [i for i in range(n, end) if i not in gone]
    for d, s in list(zip(holes, fill)) + [(i, i) for i in stay]:
        K[d], V[d], pos[d], util[d] = rk[s], rv[s], rp[s], ru[s]
        if votes is not None:
            votes[d] = rw[s]
    out.update(K=K, V=V, pos=pos, util=util, votes=votes, len=end)
    return out
