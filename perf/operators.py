"""Cases of the draft-tree operators over a budgeted KV cache.

A serving loop that verifies drafted tokens over the budgeted cache makes three
calls per verification: the attention of a tree of drafted tokens over the
cache (``attend``), the attention weight that the accepted tokens gave to every
slot (``weights``), and the commit of the accepted tokens with the eviction of
the slots that gathered the least (``commit``).  ``run`` makes one of them, in
elementary torch operations or, where ``own`` is set, through the library's
entry points.

A unit is one (sequence, layer, KV head); its G query heads share the KV head.
All units of a sequence share the sequence's tree and its accepted path.
"""
import math

import torch

own = False

D = 128                      # head dimension
SCALE = 1.0 / math.sqrt(D)
INF = float("inf")


# ---------------------------------------------------------------------- cases

def _attend(name, seqs, per, G, T, n, ragged=0.0, tree="tree", votes=False, moments=False):
    return dict(name=name, op="attend", seqs=seqs, per=per, G=G, T=T, n=n, ragged=ragged,
                tree=tree, votes=votes, moments=moments)


def _weights(name, seqs, per, G, T, A, n, ragged=0.0, votes=False):
    return dict(name=name, op="weights", seqs=seqs, per=per, G=G, T=T, A=A, n=n, ragged=ragged,
                tree="tree", votes=votes)


def _commit(name, seqs, per, T, A, n, rule, ragged=0.0, votes=False, moments=True):
    return dict(name=name, op="commit", seqs=seqs, per=per, T=T, A=A, n=n, ragged=ragged,
                tree="tree", rule=rule, votes=votes, moments=moments)


def listed():
    return [
        # one sequence, one layer, a single token over a 64-slot budget: the latency of a call
        _attend("attend-token", 1, 8, 4, 1, 64),
        # one layer of a batch of 16 sequences at a 10 % budget of 32768 tokens, 24-node trees,
        # a budget of its own per KV head
        _attend("attend-batch", 16, 8, 4, 24, 3277, ragged=0.4),
        # every layer of 4 sequences in one call, 16 drafted tokens, votes and the moment correction
        _attend("attend-layers", 4, 256, 4, 16, 1024, votes=True, moments=True),
        # one layer of one sequence over its whole long prompt, a 63-node tree (252 query rows)
        _attend("attend-long", 1, 8, 4, 63, 131071),
        # the accepted tokens' weights: one sequence, one layer, a 128-slot budget
        _weights("weights-token", 1, 8, 4, 8, 3, 128),
        # one layer of a batch, up to 6 accepted of 24, ragged budgets
        _weights("weights-batch", 16, 8, 4, 24, 6, 3277, ragged=0.4),
        # every layer of 4 sequences, votes
        _weights("weights-layers", 4, 256, 4, 16, 5, 1024, votes=True),
        # one layer over a whole long prompt, 17 accepted of 63
        _weights("weights-long", 1, 8, 4, 63, 17, 131071),
        # commit and eviction: one sequence, one layer, a 64-slot budget, no eviction moments
        _commit("commit-token", 1, 8, 4, 2, 64, "ema", moments=False),
        # one layer of a batch, ragged budgets
        _commit("commit-batch", 16, 8, 24, 6, 3277, "ema", ragged=0.4),
        # every layer of 4 sequences, votes and moments
        _commit("commit-layers", 4, 256, 16, 5, 1024, "cumulative", votes=True),
        # one layer over a whole long prompt
        _commit("commit-long", 1, 8, 63, 17, 131071, "cumulative"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attend", "weights", "commit"])
    per = rng.choice([1, 2, 4, 8, 8, 64, 256])
    seqs = _log(rng, 1, max(1, 1024 // per))
    n = min(_log(rng, 17, 131071), (1 << 20) // (seqs * per))
    G, T = rng.choice([1, 2, 4, 8]), _log(rng, 1, 64)
    G = max(1, min(G, 256 // T))
    G = 1 << (G.bit_length() - 1)
    A = _log(rng, 1, min(T, 24))
    ragged, votes = rng.choice([0.0, 0.3, 0.7]), rng.random() < 0.5
    if op == "attend":
        case = _attend("", seqs, per, G, T, n, ragged, rng.choice(["tree", "chain"]), votes,
                       rng.random() < 0.4)
    elif op == "weights":
        case = _weights("", seqs, per, G, T, A, n, ragged, votes)
    else:
        case = _commit("", seqs, per, T, A, n, rng.choice(["single", "cumulative", "ema"]), ragged,
                       votes, rng.random() < 0.6)
    del case["name"]
    return case


# --------------------------------------------------------------------- inputs

def _lengths(case):
    """Slots in use per unit: spread over [(1 - ragged) n, n]."""
    U = case["seqs"] * case["per"]
    return [case["n"] - int(case["ragged"] * case["n"] * ((u * 0.6180339887) % 1.0))
            for u in range(U)]


def _accepted(case):
    """Accepted tokens per sequence: spread over 0 .. A, all A for a single sequence."""
    B = case["seqs"]
    return [case["A"] - (b * (case["A"] + 1)) // B for b in range(B)]


def _live(case):
    """Drafted tokens per sequence: from T down to about three quarters of it."""
    B = case["seqs"]
    least = case.get("A", 1)
    return [max(least, case["T"] - (b * (case["T"] // 4 + 1)) // B) for b in range(B)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _trees(case, g):
    """Parents drawn among the four tokens before (a chain: the token before); a token's mask has
    its own bit and its ancestors'.  Returns int64 bit masks [seqs][T] and the parents."""
    T, B = case["T"], case["seqs"]
    back = torch.randint(1, 5, (B, T), generator=g, device="cuda").tolist()
    masks, parents = [], []
    for b in range(B):
        m, par = [], []
        for i in range(T):
            p = i - (1 if case["tree"] == "chain" else min(i, back[b][i]))
            par.append(p if i else -1)
            m.append((m[p] if i else 0) | (1 << i))
        masks.append([x - (1 << 64) if x >> 63 else x for x in m])
        parents.append(par)
    return torch.tensor(masks, dtype=torch.int64, device="cuda"), parents


def _paths(case, parents, live):
    """Root-to-node paths of the accepted counts, each the first tokens of the path to a token as
    deep as the tree has; where no path is long enough, the rest of the count is dropped."""
    A, paths, counts = case["A"], [], []
    for b, a in enumerate(_accepted(case)):
        best = []
        for leaf in range(live[b]):
            p, i = [], leaf
            while i >= 0:
                p.append(i)
                i = parents[b][i]
            if len(p) > len(best):
                best = p
            if len(best) >= a:
                break
        best = best[::-1][:a]
        counts.append(len(best))
        paths.append(best + [0] * (A - len(best)))
    return paths, counts


def prepare(case, seed):
    g = _gen(seed)
    B, per, T, n = case["seqs"], case["per"], case["T"], case["n"]
    U, G, A = B * per, case.get("G", 1), case.get("A", 1)
    cap = n + A + 16
    bf, dev = torch.bfloat16, "cuda"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case=case, U=U, G=G, cap=cap)
    order = torch.randperm(U, generator=g, device=dev)
    s["len"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)[order].contiguous()
    s["K"] = torch.empty(U, cap, D, dtype=bf, device=dev)
    s["V"] = torch.empty(U, cap, D, dtype=bf, device=dev)
    # keys share a direction of their unit, as keys do; what lies behind len is an older step's
    bias_k, bias_v = normal(U, 1, D), 0.5 * normal(U, 1, D)
    step = max(1, (1 << 20) // cap)
    for u in range(0, U, step):
        m = min(step, U - u)
        s["K"][u:u + m] = (bias_k[u:u + m] + normal(m, cap, D)).to(bf)
        s["V"][u:u + m] = (bias_v[u:u + m] + normal(m, cap, D)).to(bf)
    s["k_tree"] = (bias_k + normal(U, T, D)).to(bf)
    s["v_tree"] = (bias_v + normal(U, T, D)).to(bf)
    s["votes"] = (torch.randint(1, 9, (U, cap), generator=g, device=dev, dtype=torch.int32)
                  if case["votes"] else None)
    s["pos"] = torch.argsort(torch.rand(U, cap, generator=g, device=dev), dim=1).to(torch.int32)
    live = _live(case)
    s["n_tree"] = torch.tensor(live, dtype=torch.int32, device=dev)
    s["mask"], parents = _trees(case, g)
    if case["op"] != "commit":
        s["q"] = (1.5 * normal(U, T, G, D)).to(bf)
        s["util"] = torch.zeros(U, cap, dtype=torch.float64, device=dev)
    s["mom"] = None
    if case.get("moments"):
        s["mom"] = [torch.randint(1, 4000, (U,), generator=g, device=dev).float(),
                    (bias_k[:, 0] + 0.1 * normal(U, D)).contiguous(),
                    (bias_v[:, 0] + 0.1 * normal(U, D)).contiguous(), 0.1 * normal(U, D, D)]
    if case["op"] == "attend":
        s["o"] = torch.zeros(U, T, G, D, dtype=bf, device=dev)
        s["lse"] = torch.zeros(U, T, G, device=dev)
    else:
        paths, counts = _paths(case, parents, live)
        s["path"] = torch.tensor(paths, dtype=torch.int32, device=dev)
        s["n_path"] = torch.tensor(counts, dtype=torch.int32, device=dev)
        s["pos0"] = cap + torch.randint(0, 1000, (B,), generator=g, device=dev, dtype=torch.int32)
    if case["op"] == "weights":
        s["row_weight"] = 0.5 + 0.5 * torch.rand(B, A, generator=g, device=dev)
        s["lse"] = _attend_plain(s)[1]       # what the attention of the same tree returned
        s["S"] = torch.zeros(U, cap, device=dev)
    if case["op"] == "commit":
        # attention weights are heavy-tailed: most slots gather little
        s["util"] = 1e-3 * torch.exp(2.0 * normal(U, cap)).double()
        s["S"] = 1e-3 * torch.exp(2.0 * normal(U, cap))
        s["budget"] = s["len"].clone()
        s["evict_idx"] = torch.full((U, A), -1, dtype=torch.int32, device=dev)
        s["evict_pos"] = torch.full((U, A), -1, dtype=torch.int32, device=dev)
        s["n_evict"] = torch.zeros(U, dtype=torch.int32, device=dev)
    if own:
        # what a serving program keeps beside its cache: parameters, descriptors, workspace
        from kv_cache_eviction_kvc_gb300 import kvc
        rule = {"single": kvc.RULE_SINGLE, "cumulative": kvc.RULE_CUMULATIVE,
                "ema": kvc.RULE_EMA}[case.get("rule", "ema")]
        s["p"] = kvc.make_params(U, G, cap, n, rule=rule, alpha=0.9, budget=s.get("budget"))
        s["cache"] = kvc.make_cache(s["K"], s["V"], s["votes"], s["pos"], s["util"], s["len"])
        s["moments"] = kvc.make_moments(*s["mom"]) if s["mom"] else None
        s["tree"] = kvc.make_tree(T, per, s["mask"], s["n_tree"])
        if case["op"] != "attend":
            s["accept"] = kvc.make_path(A, s["path"], s["n_path"], s["pos0"])
        if case["op"] == "commit":
            s["ws"] = torch.empty(kvc.kvc_decode_workspace_size(s["p"]), dtype=torch.uint8,
                                  device=dev)
            kvc.kvc_decode_workspace_init(s["p"], s["ws"])
        else:
            s["ws"] = torch.zeros(kvc.kvc_tree_workspace_size(s["p"], T), dtype=torch.uint8,
                                  device=dev)
    return s


# ---------------------------------------------------------------- plain forms

def _visible(s):
    """[U][T][T] truth values: drafted token i attends drafted token j, both live."""
    T, per = s["case"]["T"], s["case"]["per"]
    j = torch.arange(T, device="cuda")
    m = ((s["mask"].unsqueeze(-1) >> j) & 1).bool()
    alive = j < s["n_tree"].unsqueeze(-1)
    m = m & alive.unsqueeze(1) & alive.unsqueeze(2)
    return m.repeat_interleave(per, 0), alive.repeat_interleave(per, 0)


def _attend_plain(s):
    """softmax(q K^T / sqrt(d) + ln votes) V over the cache and the visible drafted tokens; with
    moments, the mixture with the evicted set's estimate."""
    U, G, T = s["U"], s["G"], s["case"]["T"]
    nmax = s["case"]["n"]
    q = s["q"].float().reshape(U, T * G, D)
    see, alive = _visible(s)
    x = torch.matmul(q, s["K"][:, :nmax].float().transpose(1, 2)) * SCALE
    if s["votes"] is not None:
        x = x + s["votes"][:, :nmax].float().log().unsqueeze(1)
    x = x.masked_fill((torch.arange(nmax, device="cuda") >= s["len"].unsqueeze(-1)).unsqueeze(1),
                      -INF)
    y = torch.matmul(q, s["k_tree"].float().transpose(1, 2)) * SCALE
    y = y.masked_fill(~see.repeat_interleave(G, 1), -INF)
    top = torch.maximum(x.amax(-1), y.amax(-1))
    top = torch.where(top > -INF, top, torch.zeros_like(top)).unsqueeze(-1)
    x, y = (x - top).exp_(), (y - top).exp_()
    z = (x.sum(-1) + y.sum(-1)).unsqueeze(-1)
    f = torch.matmul(x, s["V"][:, :nmax].float()) + torch.matmul(y, s["v_tree"].float())
    f = f / z.clamp_min(1e-37)
    lse = (z.log() + top).squeeze(-1)
    if s["mom"] is not None:
        cnt, mu_k, mu_v, C = s["mom"]
        logz = cnt.log().unsqueeze(-1) + torch.matmul(q, mu_k.unsqueeze(-1)).squeeze(-1) * SCALE
        fe = mu_v.unsqueeze(1) + torch.matmul(q, C.transpose(1, 2)) * SCALE
        w = (1.0 / (1.0 + torch.exp(logz - lse))).unsqueeze(-1)
        f = w * f + (1.0 - w) * fe
    alive = alive.unsqueeze(-1)
    lse = lse.reshape(U, T, G)
    if "o" not in s:
        return None, torch.where(alive, lse, torch.zeros_like(lse))
    o = torch.where(alive.unsqueeze(-1), f.reshape(U, T, G, D).to(torch.bfloat16), s["o"])
    return o, torch.where(alive, lse, s["lse"])


def _weights_plain(s):
    """Column sums of the accepted tokens' attention, mean over the G heads, weighted per token:
    the cache slots, then the accepted tokens behind them."""
    case, U, G, cap = s["case"], s["U"], s["G"], s["cap"]
    A, per, nmax = case["A"], case["per"], case["n"]
    path = s["path"].long().repeat_interleave(per, 0)                       # [U][A]
    take = torch.arange(A, device="cuda") < s["n_path"].repeat_interleave(per, 0).unsqueeze(-1)
    w = torch.where(take, s["row_weight"].repeat_interleave(per, 0), 0.0) / G
    w = w.unsqueeze(-1).expand(U, A, G).reshape(U, 1, A * G)
    u = torch.arange(U, device="cuda").unsqueeze(-1)
    q = s["q"][u, path].float().reshape(U, A * G, D)
    lse = s["lse"][u, path].reshape(U, A * G, 1)
    x = torch.matmul(q, s["K"][:, :nmax].float().transpose(1, 2)) * SCALE
    if s["votes"] is not None:
        x = x + s["votes"][:, :nmax].float().log().unsqueeze(1)
    old = torch.matmul(w, torch.exp(x - lse)).squeeze(1)                    # [U][nmax]
    see, _ = _visible(s)
    see = see[u.unsqueeze(-1), path.unsqueeze(2), path.unsqueeze(1)]        # [U][A rows][A columns]
    y = torch.matmul(q, s["k_tree"][u, path].float().transpose(1, 2)) * SCALE - lse
    y = torch.where(see.repeat_interleave(G, 1), torch.exp(y), 0.0)
    new = torch.matmul(w, y).squeeze(1)                                     # [U][A]
    n = s["len"].long().unsqueeze(-1)
    i = torch.arange(cap, device="cuda").unsqueeze(0)
    j = i - n
    a = take.sum(1, keepdim=True)
    old = torch.nn.functional.pad(old, (0, cap - nmax))
    new = torch.gather(new, 1, j.clamp(0, A - 1))
    return torch.where(j < 0, old, torch.where(j < a, new, s["S"]))


def _commit_plain(s):
    """Append the accepted tokens, update the utilities with the gathered weight, evict the
    lowest (utility, position) down to the budget into the moments, close the gaps.  In place."""
    case, U, cap = s["case"], s["U"], s["cap"]
    A, per = case["A"], case["per"]
    ar = torch.arange(A, device="cuda")
    slot = torch.arange(cap, device="cuda")
    row = torch.arange(U, device="cuda").unsqueeze(-1)
    path = s["path"].long().repeat_interleave(per, 0)
    a = s["n_path"].long().repeat_interleave(per, 0).unsqueeze(-1)
    n = s["len"].long().unsqueeze(-1)
    total, fresh = n + a, slot - n
    is_new = (fresh >= 0) & (slot < total)
    # the rows as they stand after the append, by index: [0, cap) the cache, cap + j a new token
    source = torch.where(is_new, cap + fresh, slot)
    pos = torch.where(is_new, s["pos0"].repeat_interleave(per, 0).unsqueeze(-1) + fresh.int(),
                      s["pos"])
    S, m = s["S"].double(), s["util"]
    if case["rule"] == "single":
        upd = S
    elif case["rule"] == "cumulative":
        upd = m + S
    else:
        alpha = torch.tensor(0.9, dtype=torch.float32).item()
        upd = alpha * m + (1.0 - alpha) * S
    util = torch.where(is_new | torch.isinf(m), S, upd)
    util = torch.where(slot < total, util, m)
    # the k lowest (utility, position): a stable sort by position, then by utility
    k = (total - s["budget"].long().unsqueeze(-1)).clamp_min(0)
    key = torch.where(slot < total, util, INF)
    by_pos = torch.argsort(pos, dim=1, stable=True)
    by_util = torch.argsort(torch.gather(key, 1, by_pos), dim=1, stable=True)
    low = torch.gather(by_pos, 1, by_util)[:, :A]
    victim = torch.zeros(U, cap + 1, dtype=torch.bool, device="cuda")
    victim.scatter_(1, torch.where(ar < k, low, cap), True)
    victim = victim[:, :cap]

    def ranked(which):
        """The slots where `which` holds, ascending, in A columns; cap behind the last."""
        rank = torch.where(which, which.long().cumsum(1) - 1, A)
        out = torch.full((U, A + 1), cap, dtype=torch.int64, device="cuda")
        return out.scatter_(1, rank.clamp_max(A), slot.expand(U, cap))[:, :A], which.sum(1, True)

    gone, _ = ranked(victim)
    live = ar < k
    s["evict_idx"].copy_(torch.where(live, gone.int(), s["evict_idx"]))
    s["evict_pos"].copy_(torch.where(live, torch.gather(pos, 1, gone.clamp_max(cap - 1)),
                                     s["evict_pos"]))
    s["n_evict"].copy_(k.squeeze(1))
    take = torch.gather(source, 1, gone.clamp_max(cap - 1))

    def rows(cache, drafted, at):
        """Rows by the index after the append."""
        old = cache[row, at.clamp_max(cap - 1)]
        new = drafted[row, torch.gather(path, 1, (at - cap).clamp(0, A - 1))]
        return torch.where((at >= cap).unsqueeze(-1), new, old)

    votes = s["votes"]
    if s["mom"] is not None:
        cnt, mu_k, mu_v, C = s["mom"]
        p = (torch.ones(U, A, device="cuda") if votes is None else
             torch.where(take < cap, votes[row, take.clamp_max(cap - 1)], 1).float())
        p = torch.where(live, p, 0.0)
        vk, vv = rows(s["K"], s["k_tree"], take).float(), rows(s["V"], s["v_tree"], take).float()
        nb = p.sum(1, keepdim=True)
        safe = nb.clamp_min(1.0)
        bk = (p.unsqueeze(-1) * vk).sum(1) / safe
        bv = (p.unsqueeze(-1) * vv).sum(1) / safe
        cb = torch.matmul(((vv - bv.unsqueeze(1)) * p.unsqueeze(-1)).transpose(1, 2),
                          vk - bk.unsqueeze(1))
        n0 = cnt.unsqueeze(-1)
        n1 = n0 + nb
        dk, dv = bk - mu_k, bv - mu_v
        C.copy_((n0.unsqueeze(-1) * C + cb) / n1.unsqueeze(-1)
                + (n0 * nb / (n1 * n1)).unsqueeze(-1) * dv.unsqueeze(2) * dk.unsqueeze(1))
        mu_k.add_(dk * (nb / n1))
        mu_v.add_(dv * (nb / n1))
        cnt.copy_(n1.squeeze(1))
    # close the gaps: the r-th hole below the new length takes the r-th live slot at or above it;
    # accepted tokens that stay below the new length go where they are
    end = total - k
    holes, nh = ranked(victim & (slot < end))
    fill, _ = ranked(~victim & (slot >= end) & (slot < total))
    kept, nk = ranked(is_new & ~victim & (slot < end))
    dst = torch.cat([torch.where(ar < nh, holes, cap - 1), torch.where(ar < nk, kept, cap - 1)], 1)
    src = torch.cat([torch.where(ar < nh, fill, cap - 1), torch.where(ar < nk, kept, cap - 1)], 1)
    src = src.clamp_max(cap - 1)
    path = torch.cat([path, path], 1)
    A = 2 * A
    at = torch.gather(source, 1, src)
    new_k, new_v = rows(s["K"], s["k_tree"], at), rows(s["V"], s["v_tree"], at)
    s["K"][row, dst] = new_k
    s["V"][row, dst] = new_v
    s["pos"][row, dst] = torch.gather(pos, 1, src)
    if votes is not None:
        votes[row, dst] = torch.where(at >= cap, 1, votes[row, at.clamp_max(cap - 1)])
    moved = torch.gather(util, 1, src)
    s["util"].copy_(torch.where(slot < n, util, s["util"]))
    s["util"][row, dst] = torch.where(dst == cap - 1, s["util"][row, dst], moved)
    s["len"].copy_(end.squeeze(1))
    return _state(s)


def _state(s):
    out = {k: s[k] for k in ("K", "V", "pos", "util", "len", "evict_idx", "evict_pos", "n_evict")}
    if s["votes"] is not None:
        out["votes"] = s["votes"]
    if s["mom"] is not None:
        out |= dict(zip(("n", "mu_k", "mu_v", "C"), s["mom"]))
    return out


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from kv_cache_eviction_kvc_gb300 import kvc
        n = s["case"]["n"]
        if op == "attend":
            kvc.kvc_tree_attend(s["p"], n, s["tree"], s["q"], s["k_tree"], s["v_tree"], s["cache"],
                                s["moments"], s["o"], s["lse"], s["ws"])
            return {"o": s["o"], "lse": s["lse"]}
        if op == "weights":
            kvc.kvc_tree_weights(s["p"], n, s["tree"], s["accept"], s["row_weight"], s["q"],
                                 s["k_tree"], s["lse"], s["cache"], s["S"], s["ws"])
            return {"S": s["S"]}
        kvc.kvc_tree_commit(s["p"], n, s["tree"], s["accept"], s["k_tree"], s["v_tree"], s["S"],
                            s["cache"], s["moments"], s["case"]["A"], s["evict_idx"],
                            s["evict_pos"], s["n_evict"], s["ws"])
        return _state(s)
    if op == "attend":
        o, lse = _attend_plain(s)
        return {"o": o, "lse": lse}
    if op == "weights":
        return {"S": _weights_plain(s)}
    return _commit_plain(s)


# ----------------------------------------------------------------------- work

def work(case):
    lens = _lengths(case)
    U, T, slots = len(lens), case["T"], sum(lens)
    live = sum(_live(case)) * case["per"]                 # drafted tokens over all units
    vote = 4 * slots if case["votes"] else 0
    if case["op"] == "attend":
        rows = live * case["G"]
        pairs = sum(x * t for x, t in zip(lens, (t for t in _live(case) for _ in range(case["per"]))))
        b = slots * 4 * D + vote + live * 4 * D + rows * (4 * D + 4)
        f = pairs * case["G"] * 4 * D
        if case["moments"]:
            b, f = b + U * 4 * (D * D + 2 * D + 1), f + rows * 2 * D * D
        return {"bytes": b, "flops": f}
    acc = sum(_accepted(case)) * case["per"]
    if case["op"] == "weights":
        pairs = sum(x * t for x, t in zip(lens, (t for t in _accepted(case) for _ in range(case["per"]))))
        return {"bytes": slots * (2 * D + 4) + vote + acc * (case["G"] * (2 * D + 4) + 2 * D + 4),
                "flops": pairs * case["G"] * 2 * D}
    # utilities read and written, weights read; per accepted token a row read and written, and with
    # moments the row that goes read
    b = (slots + acc) * (8 + 8 + 4) + acc * (4 * D * 2 + 4 * 4)
    f = slots + acc
    if case["moments"]:
        b, f = b + U * 8 * (D * D + 2 * D + 1) + acc * 4 * D, f + U * 3 * D * D + acc * 2 * D * D
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in 64 bits, unit by unit."""
    s = prepare(case, seed)
    return {"attend": _exact_attend, "weights": _exact_weights, "commit": _exact_commit}[case["op"]](s)


def _bits(word, T):
    word &= (1 << 64) - 1
    return [bool(word >> j & 1) for j in range(T)]


def _exact_attend(s):
    case, G, T, per = s["case"], s["G"], s["case"]["T"], s["case"]["per"]
    o, lse = s["o"].double(), s["lse"].double()
    masks, live, lens = s["mask"].tolist(), s["n_tree"].tolist(), s["len"].tolist()
    for u in range(s["U"]):
        t, n = live[u // per], lens[u]
        keys = torch.cat([s["K"][u, :n], s["k_tree"][u, :t]]).double()
        vals = torch.cat([s["V"][u, :n], s["v_tree"][u, :t]]).double()
        q = s["q"][u, :t].double().reshape(t * G, D)
        x = q @ keys.T / math.sqrt(D)
        if s["votes"] is not None:
            x[:, :n] += s["votes"][u, :n].double().log()
        hide = ~torch.tensor([_bits(w, t) for w in masks[u // per][:t]], device="cuda")
        x[:, n:].masked_fill_(hide.repeat_interleave(G, 0), -INF)
        z = torch.logsumexp(x, 1)
        f = torch.softmax(x, 1) @ vals
        if s["mom"] is not None:
            cnt, mu_k, mu_v, C = (v[u].double() for v in s["mom"])
            ze = cnt.log() + q @ mu_k / math.sqrt(D)
            both = torch.logaddexp(z, ze)
            fe = mu_v + q @ C.T / math.sqrt(D)
            f = torch.exp(z - both)[:, None] * f + torch.exp(ze - both)[:, None] * fe
        o[u, :t], lse[u, :t] = f.reshape(t, G, D), z.reshape(t, G)
    return {"o": o, "lse": lse}


def _exact_weights(s):
    G, per = s["G"], s["case"]["per"]
    out = s["S"].double()
    masks, lens = s["mask"].tolist(), s["len"].tolist()
    paths, counts, T = s["path"].tolist(), s["n_path"].tolist(), s["case"]["T"]
    for u in range(s["U"]):
        b, n = u // per, lens[u]
        path = paths[b][:counts[b]]
        if not path:
            continue
        keys = torch.cat([s["K"][u, :n], s["k_tree"][u, path]]).double()
        q = s["q"][u, path].double()
        x = torch.einsum("ahd,nd->ahn", q, keys) / math.sqrt(D) - s["lse"][u, path].double()[..., None]
        x = x.exp()
        if s["votes"] is not None:
            x[..., :n] *= s["votes"][u, :n].double()
        see = torch.tensor([[_bits(masks[b][i], T)[j] for j in path] for i in path], device="cuda")
        x[..., n:] *= see.double().unsqueeze(1)
        out[u, :n + len(path)] = torch.einsum("a,an->n", s["row_weight"][b, :len(path)].double(), x.mean(1))
    return {"S": out}


def _exact_commit(s):
    case, per = s["case"], s["case"]["per"]
    paths, counts = s["path"].tolist(), s["n_path"].tolist()
    lens, first = s["len"].tolist(), s["pos0"].tolist()
    out = {k: v.clone() for k, v in _state(s).items()}
    budgets = s["budget"].tolist()
    alpha = float(torch.tensor(0.9, dtype=torch.float32))
    for u in range(s["U"]):
        b, n = u // per, lens[u]
        path = paths[b][:counts[b]]
        a = len(path)
        new_pos = torch.arange(first[b], first[b] + a, dtype=torch.int32, device="cuda")
        pos = torch.cat([s["pos"][u, :n], new_pos])
        keys, vals = (torch.cat([s[c][u, :n], s[t][u, path]]) for c, t in (("K", "k_tree"), ("V", "v_tree")))
        votes = (torch.ones(n + a, dtype=torch.int32, device="cuda") if s["votes"] is None else
                 torch.cat([s["votes"][u, :n], torch.ones(a, dtype=torch.int32, device="cuda")]))
        S = s["S"][u, :n + a].double()
        util, m = S.clone(), s["util"][u, :n]
        if case["rule"] == "cumulative":
            util[:n] = m + S[:n]
        elif case["rule"] == "ema":
            util[:n] = alpha * m + (1.0 - alpha) * S[:n]
        k = max(0, n + a - budgets[u])
        # among the k + 64 lowest utilities, the k lowest pairs
        low = torch.topk(util, min(n + a, k + 64), largest=False).indices.tolist()
        vs, ps = util[low].tolist(), pos[low].tolist()
        gone = sorted(i for _, _, i in sorted(zip(vs, ps, low))[:k])
        out["n_evict"][u] = k
        out["evict_idx"][u, :k] = torch.tensor(gone, dtype=torch.int32)
        out["evict_pos"][u, :k] = pos[gone]
        if s["mom"] is not None and k:
            cnt, mu_k, mu_v, C = (v[u].double() for v in s["mom"])
            p, vk, vv = votes[gone].double(), keys[gone].double(), vals[gone].double()
            # the raw sums of the set before and of the batch, added
            sk, sv = cnt * mu_k + p @ vk, cnt * mu_v + p @ vv
            raw = cnt * (C + torch.outer(mu_v, mu_k)) + (vv * p[:, None]).T @ vk
            cnt = cnt + p.sum()
            for name, v in (("n", cnt), ("mu_k", sk / cnt), ("mu_v", sv / cnt),
                            ("C", raw / cnt - torch.outer(sv / cnt, sk / cnt))):
                out[name][u] = v
        end, dead = n + a - k, set(gone)
        holes = [i for i in gone if i < end]
        fill = [i for i in range(end, n + a) if i not in dead]
        at = list(range(n, min(end, n + a)))
        at = [i for i in at if i not in dead]
        dst, src = holes + at, fill + at
        out["util"][u, :n] = util[:n]
        if dst:
            for name, v in (("K", keys), ("V", vals), ("pos", pos), ("util", util)):
                out[name][u, dst] = v[src]
            if s["votes"] is not None:
                out["votes"][u, dst] = votes[src]
        out["len"][u] = end
    return out
