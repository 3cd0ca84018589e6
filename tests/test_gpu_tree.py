"""GPU tests of the drafted-token calls (kvc_tree_attend, kvc_tree_weights,
kvc_tree_commit) against their definitions in 64 bits (tree_ref.py): head
layouts, lengths from zero on, ragged trees and budgets, masks that leave rows
empty, NaN where nothing looks, ties, every rule; then runs of the three
together against the one-token calls, streams and graphs."""
import ctypes
import sys
import threading
from fractions import Fraction

import numpy as np
import pytest
import torch

import tree_ref as R
from kv_cache_eviction_kvc_gb300 import kvc as K
from kv_cache_eviction_kvc_gb300.state import DecodeState

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

DEV = "cuda"
NAN = float("nan")


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def tree_masks(rng, B, T, kind):
    out = np.zeros((B, T), dtype=np.uint64)
    for b in range(B):
        for i in range(T):
            own = np.uint64(1) << np.uint64(i)
            if kind == "chain":
                out[b, i] = (out[b, i - 1] if i else np.uint64(0)) | own
            elif kind == "tree":
                out[b, i] = (out[b, rng.integers(max(0, i - 4), i)] if i else np.uint64(0)) | own
            elif kind == "none":
                out[b, i] = 0
            else:                                      # any bits, rows without one among them
                out[b, i] = np.uint64(rng.integers(0, 1 << 63)) if rng.random() < 0.8 else 0
    return out


class Case:
    """Inputs of one verification on both sides; rows nobody may look at are NaN."""

    def __init__(self, seed, per, G, T, lens, kind="tree", live=None, votes=False, moments=False,
                 correction=K.CORR_FIRST_ORDER, cap=None, rule="ema", L=None, budget=None,
                 q_scale=1.5, unscored=False):
        rng = self.rng = np.random.default_rng(seed)
        U = self.U = len(lens)
        B = self.B = U // per
        self.per, self.G, self.T, self.lens = per, G, T, list(lens)
        cap = self.cap = cap or max(lens) + T + 3
        self.live = list(live) if live is not None else [T] * B
        self.mask = tree_masks(rng, B, T, kind)
        D = R.D
        off = rng.standard_normal((U, 1, D))
        self.K = off + rng.standard_normal((U, cap, D))
        self.V = 0.5 + rng.standard_normal((U, cap, D))
        self.kt = off + rng.standard_normal((U, T, D))
        self.vt = 0.5 + rng.standard_normal((U, T, D))
        self.q = q_scale * rng.standard_normal((U, T, G, D))
        for u in range(U):
            self.K[u, lens[u]:], self.V[u, lens[u]:] = NAN, NAN
            t = self.live[u // per]
            self.kt[u, t:], self.vt[u, t:], self.q[u, t:] = NAN, NAN, NAN
        self.votes = rng.integers(1, 9, (U, cap)).astype(np.int32) if votes else None
        self.pos = np.stack([rng.permutation(cap) for _ in range(U)]).astype(np.int32)
        self.util = np.exp(rng.standard_normal((U, cap)) * 2)
        if unscored:
            self.util[rng.random((U, cap)) < 0.3] = np.inf
        self.mom = None
        if moments:
            n = rng.integers(0, 50, U).astype(np.float32)
            self.mom = [n, (off[:, 0] + 0.1 * rng.standard_normal((U, D))).astype(np.float32),
                        rng.standard_normal((U, D)).astype(np.float32),
                        (0.3 * rng.standard_normal((U, D, D))).astype(np.float32)]
        t = {}
        for name in ("K", "V", "kt", "vt", "q"):
            t[name] = bf(getattr(self, name)).to(DEV)
            setattr(self, name, f64(t[name]))
        t["votes"] = None if self.votes is None else torch.from_numpy(self.votes).to(DEV)
        t["pos"], t["util"] = torch.from_numpy(self.pos).to(DEV), torch.from_numpy(self.util).to(DEV)
        t["len"] = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        t["mom"] = None if self.mom is None else [torch.from_numpy(x).to(DEV) for x in self.mom]
        t["mask"] = torch.from_numpy(self.mask.view(np.int64)).to(DEV)
        t["live"] = torch.tensor(self.live, dtype=torch.int32, device=DEV)
        t["budget"] = None if budget is None else torch.tensor(budget, dtype=torch.int32, device=DEV)
        self.t = t
        self.budget = budget if budget is not None else [L or cap - 1] * U
        self.rule, self.correction = rule, correction
        code = {"single": K.RULE_SINGLE, "cumulative": K.RULE_CUMULATIVE, "ema": K.RULE_EMA}[rule]
        self.p = K.make_params(U, G, cap, L or cap - 1, rule=code, alpha=0.75, correction=correction,
                               budget=t["budget"])
        self.cache = K.make_cache(t["K"], t["V"], t["votes"], t["pos"], t["util"], t["len"])
        self.moments = None if self.mom is None else K.make_moments(*t["mom"])
        self.tree = K.make_tree(T, per, t["mask"], t["live"])
        self.ws = torch.zeros(K.kvc_tree_workspace_size(self.p, T), dtype=torch.uint8, device=DEV)
        self.dws = torch.empty(K.kvc_decode_workspace_size(self.p), dtype=torch.uint8, device=DEV)
        K.kvc_decode_workspace_init(self.p, self.dws)
        self.max_len = max(1, max(lens))

    def path(self, counts, A):
        """Paths along the visible ancestors of a live token where there are enough, else any
        live tokens."""
        tok = np.zeros((self.B, A), np.int32)
        for b, a in enumerate(counts):
            rows = sorted(range(self.live[b]), key=lambda i: -bin(int(self.mask[b, i])).count("1"))
            anc = [j for j in range(self.live[b]) if rows and int(self.mask[b, rows[0]]) >> j & 1]
            rest = [j for j in range(self.live[b]) if j not in anc]
            tok[b, :a] = (anc + rest)[:a]
        self.tok, self.counts = tok, list(counts)
        self.pos0 = (self.cap + 10 * np.arange(self.B)).astype(np.int32)
        self.t["tok"] = torch.from_numpy(tok).to(DEV)
        self.t["np"] = torch.tensor(self.counts, dtype=torch.int32, device=DEV)
        self.t["pos0"] = torch.from_numpy(self.pos0).to(DEV)
        self.accept = K.make_path(A, self.t["tok"], self.t["np"], self.t["pos0"])

    # ---------------------------------------------------------------- attend
    def run_attend(self, max_len=None):
        o = torch.full((self.U, self.T, self.G, R.D), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((self.U, self.T, self.G), 7.0, device=DEV)
        K.kvc_tree_attend(self.p, max_len or self.max_len, self.tree, self.t["q"], self.t["kt"],
                          self.t["vt"], self.cache, self.moments, o, lse, self.ws)
        self.o, self.lse = o, lse
        return o, lse

    def ref_attend(self, u):
        b = u // self.per
        mom = None if self.mom is None else [np.float64(x[u]) for x in self.mom]
        return R.attend(self.q[u], self.K[u], self.V[u],
                        None if self.votes is None else self.votes[u], self.lens[u], self.kt[u],
                        self.vt[u], self.mask[b], self.live[b], mom,
                        self.correction == K.CORR_FIRST_ORDER,
                        mom is not None and self.correction != K.CORR_OFF)

    def check_attend(self):
        o, lse = f64(self.o), f64(self.lse)
        for u in range(self.U):
            t = self.live[u // self.per]
            ro, rl, bo, bl = self.ref_attend(u)
            assert (o[u, t:] == 7).all() and (lse[u, t:] == 7).all(), "dead rows written"
            fin = np.isfinite(rl)
            assert (np.isneginf(lse[u, :t]) == ~fin).all()
            assert (np.abs(lse[u, :t][fin] - rl[fin]) <= bl[fin]).all(), (
                u, np.abs(lse[u, :t][fin] - rl[fin]).max(), bl[fin].min())
            err = np.abs(o[u, :t] - ro)
            assert np.isfinite(o[u, :t]).all()
            assert (err <= bo).all(), (u, err.max(), (err / bo).max())


ATTEND = [
    # per, G, T, lens, keywords
    (1, 1, 1, [0, 1, 2, 7], {}),
    (2, 4, 1, [64, 63, 65, 1], {}),
    (2, 4, 7, [127, 128, 129, 0], dict(live=[7, 3])),
    (2, 8, 5, [255, 256, 257, 300], dict(votes=True)),
    (1, 2, 64, [130, 1, 400], dict(kind="chain")),
    (1, 1, 64, [96, 33], dict(kind="any")),
    (2, 4, 33, [200, 511, 513, 90], dict(live=[33, 0], kind="any")),
    (1, 8, 64, [150, 700], dict(kind="any", live=[64, 50])),
    (1, 4, 63, [385, 640], dict(votes=True, moments=True)),
    (3, 4, 16, [0, 1, 300, 77, 128, 5], dict(moments=True, live=[16, 9])),
    (3, 2, 9, [0, 40, 130], dict(moments=True, correction=K.CORR_ZERO_ORDER)),
    (3, 2, 9, [0, 40, 130], dict(moments=True, correction=K.CORR_OFF)),
    (1, 4, 6, [0, 0, 5], dict(kind="none")),
    (1, 4, 6, [0, 0, 5], dict(kind="none", moments=True)),
    (1, 8, 17, [900, 1000, 3], dict(q_scale=30.0)),          # sharp attention
    (4, 1, 24, [100, 200, 300, 400] * 45, dict()),           # more units than SMs
    # parts of the line of all tiles, which begin and end inside of units
    (4, 2, 12, [(37 * i * i) % 2100 for i in range(160)], dict(votes=True, moments=True)),
    (4, 1, 5, [(53 * i * i) % 2100 for i in range(160)], dict(kind="any", live=[i % 6 for i in range(40)])),
    (2, 8, 40, [(41 * i * i) % 2900 for i in range(80)], dict(kind="any")),
    # parts of single units, some of fewer tiles than parts
    (1, 2, 12, [4000, 130, 5, 0, 2050], dict(votes=True, moments=True)),
    (1, 8, 40, [2900, 1, 260], dict(moments=True)),
    (1, 8, 3, [20000], dict(votes=True, moments=True)),      # one unit on every SM
    (1, 1, 1, [1], dict(moments=True)),
]


@pytest.mark.parametrize("i", range(len(ATTEND)))
def test_attend(i):
    per, G, T, lens, kw = ATTEND[i]
    c = Case(100 + i, per, G, T, lens, **kw)
    c.run_attend()
    assert K.kvc_get_device_status(c.ws) == 0
    c.check_attend()


def test_attend_bounds_looser_than_the_lengths():
    c = Case(3, 1, 4, 5, [17, 140], cap=1000)
    c.run_attend(max_len=1000)
    c.check_attend()


@pytest.mark.parametrize("i", [6, 8, 9, 15])
def test_attend_gives_the_same_bits_again(i):
    """Run after run, with the caches cold and warm: nothing depends on what lands first."""
    per, G, T, lens, kw = ATTEND[i]
    c = Case(100 + i, per, G, T, lens, **kw)
    first = [x.clone() for x in c.run_attend()]
    c.check_attend()
    flush = torch.empty(64 << 20, dtype=torch.int32, device=DEV)
    for r in range(40):
        if r & 1:
            flush.fill_(r)
        for x, y in zip(first, c.run_attend()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("where", ["k", "v", "both"])
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_attend_masked_branch_does_not_leak(where, value):
    """Token 1's branch is not finite: the rows that do not see it are as
    they are without it; the rows that see it are not finite."""
    ok = Case(5, 1, 4, 6, [50], kind="tree")
    mask = np.array([[1, 3, 5, 7, 17, 63]], dtype=np.uint64)
    outs = []
    for bad in (False, True):
        c = ok
        c.t["mask"].copy_(torch.from_numpy(mask.view(np.int64)))
        if bad and where in ("k", "both"):
            c.t["kt"][0, 1] = value
        if bad and where in ("v", "both"):
            c.t["vt"][0, 1] = value
        outs.append([x.clone() for x in c.run_attend()])
    clean = [t for t in range(6) if not int(mask[0, t]) >> 1 & 1]
    seen = [t for t in range(6) if int(mask[0, t]) >> 1 & 1]
    for a, b in zip(*outs):
        assert torch.equal(a[0, clean], b[0, clean])
    if where != "k" or value != value:
        assert not torch.isfinite(outs[1][0][0, seen].float()).all(-1).any()


def test_attend_refused_on_the_device():
    c = Case(6, 1, 4, 4, [50, 60, 40], live=[4, 4, 4])
    c.t["live"].copy_(torch.tensor([4, 5, 4]))
    o, lse = c.run_attend()
    assert K.kvc_get_device_status(c.ws) == 1 and K.kvc_get_device_status(c.ws) == 0
    assert (o[1] == 7).all() and (lse[1] == 7).all() and (lse[0] != 7).all()
    c.t["live"].fill_(4)
    o, lse = c.run_attend(max_len=50)
    assert K.kvc_get_device_status(c.ws) == 2
    assert (o[1] == 7).all() and (lse[1] == 7).all() and (lse[[0, 2]] != 7).all()


# --------------------------------------------------------------------- weights

WEIGHTS = [
    (1, 1, 1, [0, 1, 2], [1, 1, 0], 1, {}),
    (2, 4, 7, [127, 128, 129, 0], [3, 2], 3, {}),
    (2, 8, 5, [255, 256, 257, 300], [5, 1], 5, dict(votes=True)),
    (1, 2, 64, [130, 1, 400], [64, 64, 7], 64, dict(kind="chain")),
    (1, 8, 64, [200, 129], [64, 30], 64, dict(kind="chain")),
    (1, 1, 20, [96, 33], [20, 3], 20, dict(kind="any")),
    (1, 4, 33, [700, 511], [17, 4], 17, dict(live=[33, 20], votes=True)),
    (1, 4, 6, [0, 0, 5], [2, 3, 1], 3, dict(kind="none")),
    (4, 1, 24, [100, 200, 300, 400] * 45, [i % 7 for i in range(45)], 6, {}),
    (1, 4, 9, [300], [5], 5, dict(q_scale=30.0)),
]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("i", range(len(WEIGHTS)))
def test_weights(i, given):
    per, G, T, lens, counts, A, kw = WEIGHTS[i]
    c = Case(200 + i, per, G, T, lens, **kw)
    c.path(counts, A)
    _, lse = c.run_attend()
    w = c.rng.random((c.B, A)).astype(np.float32) if given else np.ones((c.B, A), np.float32)
    if given:
        w[0, 0] = 0.0
    S = torch.full((c.U, c.cap), -3.0, device=DEV)
    K.kvc_tree_weights(c.p, c.max_len, c.tree, c.accept,
                       torch.from_numpy(w).to(DEV) if given else None, c.t["q"], c.t["kt"], lse,
                       c.cache, S, c.ws)
    assert K.kvc_get_device_status(c.ws) == 0
    S, lse = f64(S), f64(lse)
    for u in range(c.U):
        b = u // per
        a = counts[b]
        ref, bound = R.weights(c.q[u], c.K[u], None if c.votes is None else c.votes[u], lens[u],
                               c.kt[u], c.mask[b], [int(x) for x in c.tok[b, :a]],
                               w[b].astype(np.float64), lse[u])
        got = S[u, :lens[u] + a]
        assert (np.abs(got - ref) <= bound).all(), (u, (np.abs(got - ref) / bound).max())
        assert (S[u, lens[u] + a:] == -3).all(), "entries behind the last written"


def test_weights_of_512_rows_over_many_tiles():
    """64 accepted tokens of 8 heads fill the accumulator: several tiles per CTA through one."""
    U, n, T, G = 2, 20100, 64, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(1)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV).bfloat16()

    Kc, q, kt = rnd(U, n + 70, 128), rnd(U, T, G, 128), rnd(U, T, 128)
    ln = torch.full((U,), n, dtype=torch.int32, device=DEV)
    pos = torch.zeros(U, n + 70, dtype=torch.int32, device=DEV)
    util = torch.zeros(U, n + 70, dtype=torch.float64, device=DEV)
    p = K.make_params(U, G, n + 70, n)
    cache = K.make_cache(Kc, Kc, None, pos, util, ln)
    mask = torch.from_numpy(tree_masks(np.random.default_rng(0), 1, T, "chain").view(np.int64)).to(DEV)
    tree = K.make_tree(T, U, mask)
    path = K.make_path(T, torch.arange(T, dtype=torch.int32, device=DEV)[None],
                       torch.tensor([T], dtype=torch.int32, device=DEV),
                       torch.zeros(1, dtype=torch.int32, device=DEV))
    # any normalization will do: the log of the sum over the cache
    x = torch.einsum("uthd,und->uthn", q.double(), Kc[:, :n].double()) * R.SCALE
    lse = torch.logsumexp(x, -1).float()
    S = torch.zeros(U, n + 70, device=DEV)
    ws = torch.zeros(K.kvc_tree_workspace_size(p, T), dtype=torch.uint8, device=DEV)
    K.kvc_tree_weights(p, n, tree, path, None, q, kt, lse, cache, S, ws)
    assert K.kvc_get_device_status(ws) == 0
    ref = torch.exp(x - lse.double().unsqueeze(-1)).mean(2).sum(1)
    # every term is off by the logit's error (128 additions of products, |q||k| sums to
    # about 100 here, and 16 half steps of a logarithm near 14), the sum by 512 additions
    rel = (2 * 128 + 4) * R.E32 * float((q.double().abs().amax(-1).max() * 128 * R.SCALE
                                         * Kc[:, :n].double().abs().amax())) + (16 * 14 + 512) * R.E32
    assert float(((S[:, :n].double() - ref).abs() / ref).max()) <= rel


def test_weights_sum_to_the_accepted_tokens():
    """Each accepted row's probabilities add up to 1 over the cache and its ancestors."""
    c = Case(7, 1, 4, 12, [333, 20], kind="chain", votes=True)
    c.path([9, 12], 12)
    _, lse = c.run_attend()
    S = torch.zeros(c.U, c.cap, device=DEV)
    K.kvc_tree_weights(c.p, c.max_len, c.tree, c.accept, None, c.t["q"], c.t["kt"], lse, c.cache, S,
                       c.ws)
    # each of a sums has the logits' error (64 bits of slack for the longest one here)
    assert torch.allclose(S.double().sum(1).cpu(), torch.tensor([9.0, 12.0]).double(), rtol=1e-4)


def test_weights_refused_on_the_device():
    c = Case(8, 1, 4, 6, [50, 60, 40, 30], live=[6, 6, 4, 6], cap=62)
    c.path([2, 3, 2, 3], 3)
    c.t["tok"][2, 1] = 4                               # not live
    c.t["np"][3] = 4                                   # more than A
    c.run_attend()
    S = torch.full((4, c.cap), -3.0, device=DEV)
    K.kvc_tree_weights(c.p, 60, c.tree, c.accept, None, c.t["q"], c.t["kt"], c.lse, c.cache, S, c.ws)
    assert K.kvc_get_device_status(c.ws) in (1, 2)
    assert (S[1:] == -3).all() and (S[0, :52] >= 0).all()   # unit 1: 60 + 3 > cap


# ---------------------------------------------------------------------- commit

def run_commit(c, S, kmax, mom=True):
    ei = torch.full((c.U, kmax), -9, dtype=torch.int32, device=DEV)
    ep = torch.full((c.U, kmax), -9, dtype=torch.int32, device=DEV)
    ne = torch.full((c.U,), -9, dtype=torch.int32, device=DEV)
    K.kvc_tree_commit(c.p, c.max_len, c.tree, c.accept, c.t["kt"], c.t["vt"],
                      None if S is None else torch.from_numpy(S).to(DEV), c.cache,
                      c.moments if mom else None, kmax, ei, ep, ne, c.dws)
    return ei.cpu().numpy(), ep.cpu().numpy(), ne.cpu().numpy()


def check_commit(c, S, kmax):
    ei, ep, ne = run_commit(c, S, kmax)
    assert K.kvc_get_device_status(c.dws) == 0
    got = {n: f64(c.t[n]) for n in ("K", "V")}
    pos, util, ln = c.t["pos"].cpu().numpy(), c.t["util"].cpu().numpy(), c.t["len"].tolist()
    votes = None if c.votes is None else c.t["votes"].cpu().numpy()
    for u in range(c.U):
        b = u // c.per
        a = c.counts[b]
        mom = None if c.mom is None else [np.float64(x[u]) for x in c.mom]
        ref = R.commit(c.K[u], c.V[u], None if c.votes is None else c.votes[u], c.pos[u], c.util[u],
                       c.lens[u], c.budget[u], c.rule, 0.75,
                       None if S is None else S[u, :c.lens[u] + a].astype(np.float64), c.kt[u],
                       c.vt[u], [int(x) for x in c.tok[b, :a]], int(c.pos0[b]), mom)
        k = ref["n_evict"]
        assert ne[u] == k and ei[u, :k].tolist() == ref["evict_idx"]
        assert ep[u, :k].tolist() == ref["evict_pos"]
        assert (ei[u, k:] == -9).all() and (ep[u, k:] == -9).all()
        assert ln[u] == ref["len"]
        assert np.array_equal(got["K"][u], ref["K"], equal_nan=True)
        assert np.array_equal(got["V"][u], ref["V"], equal_nan=True)
        assert np.array_equal(pos[u], ref["pos"])
        # one multiplication and one addition in 64 bits, fused or not
        np.testing.assert_allclose(util[u], ref["util"], rtol=4 * 2.0 ** -53)
        if votes is not None:
            assert np.array_equal(votes[u], ref["votes"])
        if mom is not None and k:
            n1, mk, mv, C = (f64(x[u]) for x in c.t["mom"])
            assert n1 == ref["n"]
            assert (np.abs(mk - ref["mu_k"]) <= ref["bound_mu"] * ref["scale_k"]).all()
            assert (np.abs(mv - ref["mu_v"]) <= ref["bound_mu"] * ref["scale_v"]).all()
            assert (np.abs(C - ref["C"]) <= ref["bound_C"]).all(), (
                np.abs(C - ref["C"]) / ref["bound_C"]).max()


COMMIT = [
    # per, T, lens, counts, A, keywords, scored weights given
    (1, 4, [0, 1, 2, 9], [1, 2, 0, 4], 4, dict(budget=[1, 1, 9, 9], L=9), True),
    (2, 7, [64, 63, 60, 64], [3, 5], 5, dict(L=64, votes=True, moments=True), True),
    (1, 8, [100, 100], [8, 0], 8, dict(L=100, rule="cumulative", moments=True), True),
    (1, 64, [200, 130], [64, 33], 64, dict(L=200, kind="chain", rule="single", moments=True), True),
    (1, 8, [120, 128], [3, 8], 8, dict(budget=[77, 100], L=128, votes=True, moments=True), True),
    (1, 8, [500, 90], [5, 2], 8, dict(budget=[500, 88], L=500, unscored=True, moments=True), True),
    (1, 8, [500, 90], [5, 2], 8, dict(budget=[500, 88], L=500, unscored=True, moments=True), False),
    (4, 6, [3000, 1025, 4096, 8200], [6], 6, dict(budget=[3000, 1024, 4096, 8200], L=8200), True),
    (1, 3, [5, 5], [3, 3], 3, dict(L=9), True),                        # room left: nothing goes
    (4, 24, [100, 200, 300, 400] * 45, [i % 7 for i in range(45)], 6,
     dict(budget=[100, 200, 300, 400] * 45, L=400), True),
    (1, 30, [9000, 8193, 40], [20, 3, 30], 30,                         # long units, more than 16 victims
     dict(budget=[9000, 8180, 50], L=9000, votes=True, moments=True, unscored=True), True),
    (20, 4, [5000 + 37 * i for i in range(80)], [3, 0, 4, 2], 4,       # many units, no kernel of their own
     dict(budget=[5000 + 37 * i for i in range(80)], L=7925, rule="cumulative"), True),
    # more units than fit at once
    (10, 6, [(29 * i) % 400 for i in range(650)], [i % 7 for i in range(65)], 6,
     dict(L=400, budget=[max(1, (29 * i) % 400) for i in range(650)], votes=True, moments=True), True),
]


@pytest.mark.parametrize("i", range(len(COMMIT)))
def test_commit(i):
    per, T, lens, counts, A, kw, scored = COMMIT[i]
    c = Case(300 + i, per, 1, T, lens, cap=max(lens) + A + 2, **kw)
    c.path(counts, A)
    S = np.exp(c.rng.standard_normal((c.U, c.cap)) * 2).astype(np.float32) if scored else None
    kmax = max(1, max(max(0, c.lens[u] + counts[u // per] - c.budget[u]) for u in range(c.U)))
    check_commit(c, S, kmax)


@pytest.mark.parametrize("n", [70, 1500, 6000])
@pytest.mark.parametrize("ties", ["zero", "few", "stride"])
def test_commit_ties(n, ties):
    """Weights that underflowed, few distinct ones, and the lowest all in
    slots of one residue: the lowest positions go."""
    c = Case(400 + n, 1, 1, 40, [n, n], cap=n + 44, L=n, rule="single", moments=True, kind="chain")
    c.path([40, 17], 40)
    S = np.zeros((2, c.cap), np.float32)
    if ties == "few":
        S = c.rng.integers(0, 3, S.shape).astype(np.float32)
    elif ties == "stride":
        S = (1 + c.rng.random(S.shape)).astype(np.float32)
        S[:, ::512] = 0.25
        S[:, 1:3000:3] = 0.5
    check_commit(c, S, 40)


@pytest.mark.parametrize("n", [300, 9000])
@pytest.mark.parametrize("rule", ["cumulative", "ema"])
def test_commit_utilities_to_the_bit(rule, n):
    """The new utilities are what IEEE arithmetic gives (a multiply-add of the
    rounded product under EMA), for operands all over the range."""
    c = Case(13, 1, 1, 2, [n], cap=n + 4, rule=rule)
    c.path([1], 1)
    rng = c.rng
    m = np.exp2(rng.uniform(-60, 20, n)) * (1 + rng.integers(0, 4, n) * 2.0 ** -52)
    s = np.exp2(rng.uniform(-60, 20, n)).astype(np.float32)
    m[:200:2] = np.exp2(rng.integers(-30, 3, 100).astype(np.float64))          # ties of the rounding
    s[:200:2] = (np.exp2(rng.integers(-40, 3, 100)) * rng.integers(1, 4, 100)).astype(np.float32)
    odd = [(0.0, 0.0), (0.0, 1.5), (0.25, 0.0), (5e-324, 1e-45), (1e-310, 0.0), (1e300, 1.0),
           (1e-300, 1e-38), (2.0 ** -699, 0.0), (-1.5, 1.5), (-1.5, 0.25), (1.0, 1e-45),
           (1.0, 3e38), (0.0, 1e-42), (1.0, 2.0 ** -53), (1 + 2.0 ** -52, 2.0 ** -53),
           (2 - 2.0 ** -52, 2.0 ** -53), (2.0 ** -53, 2.0 ** 60)]
    for i, (x, y) in enumerate(odd):
        m[201 + i], s[201 + i] = x, np.float32(y)
    c.t["util"][0, :n] = torch.from_numpy(m).to(DEV)
    S = np.ones((1, c.cap), np.float32)
    S[0, :n] = s
    run_commit(c, S, 1)
    got = f64(c.t["util"])[0, :n]
    if rule == "cumulative":
        want = m + s.astype(np.float64)
    else:
        want = np.array([float(Fraction(0.75) * Fraction(x) + Fraction(0.25 * float(y)))
                         for x, y in zip(m, s)])
    assert np.array_equal(got, want), np.flatnonzero(got != want)[:10]


def test_commit_of_a_token_named_twice():
    """A path is a list of live tokens; one that is named twice is appended
    twice, and its weights count twice."""
    c = Case(14, 1, 2, 4, [70, 40], cap=80, L=70, kind="chain", moments=True)
    c.path([3, 4], 4)
    c.tok[:] = [[2, 0, 2, 0], [1, 1, 1, 3]]
    c.t["tok"].copy_(torch.from_numpy(c.tok))
    o, lse = c.run_attend()
    S = torch.full((c.U, c.cap), -3.0, device=DEV)
    K.kvc_tree_weights(c.p, c.max_len, c.tree, c.accept, None, c.t["q"], c.t["kt"], lse, c.cache, S, c.ws)
    assert K.kvc_get_device_status(c.ws) == 0
    for u in range(c.U):
        n, a = c.lens[u], c.counts[u]
        rs, bs = R.weights(c.q[u], c.K[u], None, n, c.kt[u], c.mask[u], [int(x) for x in c.tok[u, :a]],
                           np.ones(4), f64(lse[u]))
        assert (np.abs(f64(S[u, :n + a]) - rs) <= bs).all()
    check_commit(c, S.cpu().numpy(), 3)


def test_commit_of_many_long_units_is_as_of_few():
    """160 units in one call and 80 at a time: the same bits (the number of
    units chooses how the work is laid out)."""
    U, n, cap, T, A = 160, 8250, 8300, 3, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(3)

    def rnd(*s, dtype=torch.bfloat16):
        return torch.randn(*s, generator=g, device=DEV).to(dtype)

    start = dict(K=rnd(U, cap, 128), V=rnd(U, cap, 128), util=rnd(U, cap, dtype=torch.float64).exp(),
                 pos=torch.randperm(cap, device=DEV, dtype=torch.int32).repeat(U, 1),
                 len=torch.full((U,), n, dtype=torch.int32, device=DEV),
                 n=torch.full((U,), 5.0, device=DEV), mu_k=rnd(U, 128, dtype=torch.float32),
                 mu_v=rnd(U, 128, dtype=torch.float32), C=rnd(U, 128, 128, dtype=torch.float32))
    kt, vt, S = rnd(U, T, 128), rnd(U, T, 128), rnd(U, cap, dtype=torch.float32).exp()
    mask = torch.tensor([[1, 3, 7]] * 4, dtype=torch.int64, device=DEV)
    tok = torch.tensor([[0, 1], [0, 2], [1, 2], [0, 1]], dtype=torch.int32, device=DEV)
    counts = torch.tensor([2, 1, 2, 0], dtype=torch.int32, device=DEV)
    first = torch.full((4,), 9000, dtype=torch.int32, device=DEV)

    def run(units):
        c = {k: v.clone() for k, v in start.items()}
        ne = torch.zeros(U, dtype=torch.int32, device=DEV)
        ev = torch.full((2, U, A), -9, dtype=torch.int32, device=DEV)
        for a in range(0, U, units):
            z, b = slice(a, a + units), slice(a // 40, (a + units) // 40)
            p = K.make_params(units, 1, cap, n, rule=K.RULE_CUMULATIVE)
            dws = torch.empty(K.kvc_decode_workspace_size(p), dtype=torch.uint8, device=DEV)
            K.kvc_decode_workspace_init(p, dws)
            K.kvc_tree_commit(p, n, K.make_tree(T, 40, mask[b]), K.make_path(A, tok[b], counts[b], first[b]),
                              kt[z], vt[z], S[z], K.make_cache(c["K"][z], c["V"][z], None, c["pos"][z],
                                                               c["util"][z], c["len"][z]),
                              K.make_moments(c["n"][z], c["mu_k"][z], c["mu_v"][z], c["C"][z]), A,
                              ev[0, z], ev[1, z], ne[z], dws)
            assert K.kvc_get_device_status(dws) == 0
        return [*c.values(), ne, ev]

    many, few = run(160), run(80)
    assert many[-2].tolist() == [2] * 40 + [1] * 40 + [2] * 40 + [0] * 40
    for x, y in zip(many, few):
        assert torch.equal(x, y)


def test_commit_in_a_graph():
    """Weights and commit captured once and replayed from two states: what
    the calls give."""
    def make(seed):
        c = Case(seed, 2, 4, 9, [700, 90, 33, 400], votes=True, moments=True,
                 budget=[700, 88, 33, 398], L=700)
        c.path([4, 2], 4)
        c.run_attend()
        return c

    def call(c):
        K.kvc_tree_weights(c.p, c.max_len, c.tree, c.accept, None, c.t["q"], c.t["kt"], c.lse, c.cache,
                           c.S, c.ws)
        K.kvc_tree_commit(c.p, c.max_len, c.tree, c.accept, c.t["kt"], c.t["vt"], c.S, c.cache,
                          c.moments, 6, None, None, c.ne, c.dws)

    def state(c):
        return [c.t[n] for n in ("K", "V", "votes", "pos", "util", "len")] + c.t["mom"] + [c.ne]

    c = make(31)
    c.S = torch.zeros(c.U, c.cap, device=DEV)
    c.ne = torch.zeros(c.U, dtype=torch.int32, device=DEV)
    first = [x.clone() for x in state(c)]
    call(c)
    want = [x.clone() for x in state(c)]
    for x, y in zip(state(c), first):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c)
    for _ in range(3):
        for x, y in zip(state(c), first):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(state(c), want):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
    assert K.kvc_get_device_status(c.dws) == 0 and K.kvc_get_device_status(c.ws) == 0


def test_commit_same_position_and_weight_goes_by_slot():
    c = Case(9, 1, 1, 4, [50], cap=60, L=50, rule="single")
    c.t["pos"].fill_(3)
    c.pos[:] = 3
    c.path([4], 4)
    c.pos0[:] = 0
    c.t["pos0"].zero_()
    check_commit(c, np.ones((1, 60), np.float32), 4)


def test_commit_refused_on_the_device():
    """Every refused unit is as it was; the others go on."""
    c = Case(10, 1, 1, 6, [50, 60, 40, 30, 20, 45], cap=64, live=[6, 6, 4, 6, 6, 6], moments=True,
             budget=[50, 60, 40, 30, 20, 0], L=60)
    c.path([2, 5, 2, 3, 3, 1], 5)
    c.t["tok"][2, 1] = 4                               # not live
    c.t["np"][3] = 6                                   # more than A
    c.t["len"][4] = 61                                 # beyond max_len
    before = {n: c.t[n].clone() for n in ("K", "V", "pos", "util", "len")}
    mom = [x.clone() for x in c.t["mom"]]
    ei, ep, ne = run_commit(c, np.ones((6, 64), np.float32), 5)
    assert K.kvc_get_device_status(c.dws) in (1, 2)
    assert ne.tolist() == [2, 0, 0, 0, 0, 0]           # unit 1: 60 + 5 > cap; unit 5: budget 0
    for n, x in before.items():
        assert torch.equal(c.t[n][1:].view(torch.uint8), x[1:].view(torch.uint8)), n
    for x, y in zip(c.t["mom"], mom):
        assert torch.equal(x[1:], y[1:])
    assert c.t["len"][0] == 50


def test_commit_more_victims_than_room_and_too_few_scored():
    c = Case(11, 1, 1, 6, [50, 50], cap=64, budget=[45, 50], L=50)
    c.path([2, 2], 2)
    ei, ep, ne = run_commit(c, np.ones((2, 64), np.float32), 2)       # unit 0 needs 7
    assert K.kvc_get_device_status(c.dws) == 2 and ne.tolist() == [0, 2]
    c = Case(12, 1, 1, 6, [50, 50], cap=64, L=50)
    c.t["util"][0, 1:] = float("inf")
    c.path([2, 2], 2)
    util = c.t["util"].clone()
    ei, ep, ne = run_commit(c, None, 2)                               # one scored, two to go
    assert K.kvc_get_device_status(c.dws) == 1 and ne.tolist() == [0, 2]
    assert torch.equal(c.t["util"][0], util[0]) and c.t["len"].tolist() == [50, 50]


# --------------------------------------------------------------------- together

def _stream(seed, U, G, n, cap, L, steps, **kw):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV)

    st = DecodeState(U, G, cap, L, rule=K.RULE_CUMULATIVE, **kw)
    st.load_prefill(rnd(U, n, 128).bfloat16(), rnd(U, n, 128).bfloat16(),
                    None, torch.arange(n, dtype=torch.int32, device=DEV).repeat(U, 1),
                    torch.full((U,), n, dtype=torch.int32, device=DEV))
    return st, rnd


def test_one_token_trees_are_decode_steps():
    """A drafted token accepted alone, with its weight as the utility's
    observation, does what the one-token calls do: the same outputs, victims
    and moments, step by step."""
    U, G, n, L = 6, 4, 90, 64
    a, rnd = _stream(1, U, G, n, n + 4, L, 8)
    b, _ = _stream(1, U, G, n, n + 4, L, 8)
    one = torch.ones(1, 1, dtype=torch.int64, device=DEV)
    zero = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    for t in range(1, 9):
        q, k, v = rnd(U, G, 128).bfloat16(), rnd(U, 128).bfloat16(), rnd(U, 128).bfloat16()
        max_len = n + 1 if t == 1 else L + 1
        b.step_calls(t, n + t - 1, q, k, v, max_len)
        if t == 1:       # the prompt goes down to the budget in the one-token calls
            a.step_calls(t, n + t - 1, q, k, v, max_len)
            continue
        tree = K.make_tree(1, U, one)
        path = K.make_path(1, zero, torch.ones(1, dtype=torch.int32, device=DEV),
                           torch.full((1,), n + t - 1, dtype=torch.int32, device=DEV))
        o, lse = a.verify(tree, q, k, v, L)
        a.accept(tree, path, q, k, v, L)
        assert a.tree_status() == 0 and a.device_status() == 0
        # the attention over every slot of the step, before the eviction
        assert torch.allclose(lse[:, 0], b.lse, atol=2e-5)
        assert torch.equal(a.n_evict, b.n_evict)
        assert torch.equal(a.tree_evict[1][:, 0], b.evict_pos[:, 0])
        assert torch.equal(a.pos[:, :L].sort(1)[0], b.pos[:, :L].sort(1)[0])
        assert torch.equal(a.n, b.n)
        assert torch.allclose(a.C, b.C, atol=1e-5)


def test_verification_run_matches_the_reference():
    """Verifications of trees with ragged acceptance on a budgeted cache, each
    against the 64-bit definitions from the state before it."""
    U, per, G, T, A, L = 8, 4, 4, 10, 5, 96
    st, rnd = _stream(2, U, G, L, L + T + 2, L, 6)
    rng = np.random.default_rng(0)
    for step in range(6):
        mask = tree_masks(rng, 2, T, "chain")
        counts = [int(x) for x in rng.integers(0, A + 1, 2)]
        tok = np.tile(np.arange(A, dtype=np.int32), (2, 1))
        tree = K.make_tree(T, per, torch.from_numpy(mask.view(np.int64)).to(DEV))
        path = K.make_path(A, torch.from_numpy(tok).to(DEV),
                           torch.tensor(counts, dtype=torch.int32, device=DEV),
                           torch.tensor([1000 + 10 * step] * 2, dtype=torch.int32, device=DEV))
        q, k, v = (rnd(U, T, G, 128).bfloat16(), rnd(U, T, 128).bfloat16(), rnd(U, T, 128).bfloat16())
        old = {x: f64(getattr(st, x)) for x in ("K", "V", "util", "n", "mu_k", "mu_v", "C")}
        pos, lens = st.pos.cpu().numpy(), st.len.tolist()
        o, lse = (x.clone() for x in st.verify(tree, q, k, v, L))
        st.accept(tree, path, q, k, v, L)
        assert st.tree_status() == 0 and st.device_status() == 0
        S = f64(st.tree_S)
        for u in range(U):
            a = counts[u // per]
            mom = [old[x][u] for x in ("n", "mu_k", "mu_v", "C")]
            ro, rl, bo, bl = R.attend(f64(q[u]), old["K"][u], old["V"][u], None, lens[u], f64(k[u]),
                                      f64(v[u]), mask[u // per], T, mom, True, True)
            assert (np.abs(f64(o[u]) - ro) <= bo).all() and (np.abs(f64(lse[u]) - rl) <= bl).all()
            p = list(range(a))
            rs, bs = R.weights(f64(q[u]), old["K"][u], None, lens[u], f64(k[u]), mask[u // per], p,
                               np.ones(A), f64(lse[u]))
            assert (np.abs(S[u, :lens[u] + a] - rs) <= bs).all()
            ref = R.commit(old["K"][u], old["V"][u], None, pos[u], old["util"][u], lens[u], L,
                           "cumulative", 0.0, S[u, :lens[u] + a], f64(k[u]), f64(v[u]), p,
                           1000 + 10 * step, mom)
            assert np.array_equal(f64(st.K[u]), ref["K"]) and np.array_equal(f64(st.V[u]), ref["V"])
            assert st.len[u] == ref["len"] and st.n_evict[u] == ref["n_evict"]
            if ref["n_evict"]:
                assert (np.abs(f64(st.C[u]) - ref["C"]) <= ref["bound_C"]).all()
    # the stream goes on with a one-token step on the same cache
    assert st.len.tolist() == [L] * U
    st.step(2, 5000, rnd(U, G, 128).bfloat16(), rnd(U, 128).bfloat16(), rnd(U, 128).bfloat16(), L + 1)
    assert st.device_status() == 0 and st.len.tolist() == [L] * U


def _graph_case(seed):
    c = Case(seed, 2, 4, 9, [700, 90, 33, 400], votes=True, moments=True)
    c.path([4, 2], 4)
    c.o = torch.zeros(c.U, c.T, c.G, R.D, dtype=torch.bfloat16, device=DEV)
    c.lse = torch.zeros(c.U, c.T, c.G, device=DEV)
    c.S = torch.zeros(c.U, c.cap, device=DEV)

    def call(stream=None):
        K.kvc_tree_attend(c.p, c.max_len, c.tree, c.t["q"], c.t["kt"], c.t["vt"], c.cache, c.moments,
                          c.o, c.lse, c.ws, stream)
        K.kvc_tree_weights(c.p, c.max_len, c.tree, c.accept, None, c.t["q"], c.t["kt"], c.lse, c.cache,
                           c.S, c.ws, stream)
    c.call = call
    return c


def test_graphs_that_share_a_workspace_and_another_stream():
    a, b = _graph_case(21), _graph_case(22)
    b.ws = a.ws
    want = []
    for c in (a, b):
        c.call()
        want.append([x.clone() for x in (c.o, c.lse, c.S)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.call(side)                                       # the caller's stream, not the current one
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for c, g, w in zip((a, b), graphs, want):
            for x in (c.o, c.lse, c.S):
                x.zero_()
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip((c.o, c.lse, c.S), w):
                assert torch.equal(x, y)               # the same bits, run after run


def test_graph_with_copies_and_branches():
    """Captured behind copies and fills, and on two branches that meet again."""
    cases = [_graph_case(51), _graph_case(52)]
    for c in cases:
        c.call()
    want = [[x.clone() for x in (c.o, c.lse, c.S)] for c in cases]
    src = [c.t["q"].clone() for c in cases]
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            cases[1].t["q"].copy_(src[1])
            cases[1].o.zero_()
            cases[1].call()
        cases[0].o.zero_()
        cases[0].t["q"].copy_(src[0])
        cases[0].call()
        main.wait_stream(side)
        cases[0].call()                                # behind both branches
    for _ in range(3):
        for c in cases:
            c.t["q"].zero_()
            c.S.zero_()
        g.replay()
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            for x, y in zip((c.o, c.lse, c.S), w):
                assert torch.equal(x, y)


def test_calls_at_once_on_two_streams():
    """Two verifications in flight together, a workspace each: the bits that
    each gives alone."""
    cases = [_graph_case(41), _graph_case(42)]
    for c in cases:
        c.call()
    want = [[x.clone() for x in (c.o, c.lse, c.S)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for c, s in zip(cases, streams):
            c.call(s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        for x, y in zip((c.o, c.lse, c.S), w):
            assert torch.equal(x, y)
        assert K.kvc_get_device_status(c.ws) == 0


def test_state_keeps_buffers_of_every_tree_size():
    """A graph of a verification stays valid when the same state verifies
    trees of another size in between."""
    U, G, L = 4, 4, 80
    st, rnd = _stream(5, U, G, L, L + 20, L, 1)
    trees, args = {}, {}
    for T in (3, 7):
        mask = tree_masks(np.random.default_rng(T), 1, T, "chain")
        trees[T] = K.make_tree(T, U, torch.from_numpy(mask.view(np.int64)).to(DEV))
        args[T] = (rnd(U, T, G, 128).bfloat16(), rnd(U, T, 128).bfloat16(), rnd(U, T, 128).bfloat16())
    path = K.make_path(2, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV),
                       torch.tensor([2], dtype=torch.int32, device=DEV),
                       torch.tensor([500], dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        st.accept(trees[3], path, *args[3], L)          # nothing verified yet
    o, lse = st.verify(trees[3], *args[3], L)
    want = o.clone(), lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.verify(trees[3], *args[3], L)
    o7 = [x.clone() for x in st.verify(trees[7], *args[7], L)]
    o.zero_(), lse.zero_()
    g.replay()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    again = st.verify(trees[7], *args[7], L)
    assert torch.equal(again[0], o7[0]) and torch.equal(again[1], o7[1])
    assert st.verify(trees[3], *args[3], L)[0].data_ptr() == o.data_ptr()
    st.accept(trees[3], path, *args[3], L)
    assert st.tree_status() == 0 and st.device_status() == 0
    assert st.len.tolist() == [L] * U and st.n_evict.tolist() == [2] * U


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes (and 2^31 elements) of keys: the last
    unit is where it should be."""
    U, cap, n, T, G = 34, 1 << 19, 300, 3, 2
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    Kc = torch.zeros(U, cap, 128, dtype=torch.bfloat16, device=DEV)
    Vc = torch.zeros(U, cap, 128, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV).bfloat16()

    Kc[-1, :n], Vc[-1, :n] = rnd(n, 128), rnd(n, 128)
    pos = torch.arange(cap, dtype=torch.int32, device=DEV).repeat(U, 1)
    util = torch.rand(U, cap, generator=g, device=DEV, dtype=torch.float64)
    ln = torch.full((U,), n, dtype=torch.int32, device=DEV)
    p = K.make_params(U, G, cap, n, rule=K.RULE_SINGLE)
    cache = K.make_cache(Kc, Vc, None, pos, util, ln)
    mask = torch.tensor([[1, 3, 7]], dtype=torch.int64, device=DEV)
    tree = K.make_tree(T, U, mask)
    path = K.make_path(2, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV),
                       torch.tensor([2], dtype=torch.int32, device=DEV),
                       torch.tensor([9000], dtype=torch.int32, device=DEV))
    q, k, v = rnd(U, T, G, 128), rnd(U, T, 128), rnd(U, T, 128)
    o = torch.zeros(U, T, G, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(U, T, G, device=DEV)
    S = torch.zeros(U, cap, device=DEV)
    ws = torch.zeros(K.kvc_tree_workspace_size(p, T), dtype=torch.uint8, device=DEV)
    dws = torch.empty(K.kvc_decode_workspace_size(p), dtype=torch.uint8, device=DEV)
    K.kvc_decode_workspace_init(p, dws)
    K.kvc_tree_attend(p, n, tree, q, k, v, cache, None, o, lse, ws)
    K.kvc_tree_weights(p, n, tree, path, None, q, k, lse, cache, S, ws)
    ne = torch.zeros(U, dtype=torch.int32, device=DEV)
    rk, rv = f64(Kc[-1, :n]), f64(Vc[-1, :n])
    K.kvc_tree_commit(p, n, tree, path, k, v, S, cache, None, 2, None, None, ne, dws)
    assert K.kvc_get_device_status(ws) == 0 and K.kvc_get_device_status(dws) == 0
    ro, rl, bo, bl = R.attend(f64(q[-1]), rk, rv, None, n, f64(k[-1]), f64(v[-1]), [1, 3, 7], T,
                              None, False, False)
    assert (np.abs(f64(o[-1]) - ro) <= bo).all() and (np.abs(f64(lse[-1]) - rl) <= bl).all()
    rs, bs = R.weights(f64(q[-1]), rk, None, n, f64(k[-1]), [1, 3, 7], [0, 1], np.ones(2), f64(lse[-1]))
    assert (np.abs(f64(S[-1, :n + 2]) - rs) <= bs).all()
    ref = R.commit(rk, rv, None, np.arange(n), np.zeros(n), n, n, "single", 0, f64(S[-1, :n + 2]),
                   f64(k[-1]), f64(v[-1]), [0, 1], 9000, None)
    assert np.array_equal(f64(Kc[-1, :n]), ref["K"]) and np.array_equal(f64(Vc[-1, :n]), ref["V"])
    assert ne.tolist() == [2] * U


# ------------------------------------------------------- one unit does not reach another

@pytest.mark.parametrize("correction", [K.CORR_FIRST_ORDER, K.CORR_ZERO_ORDER])
@pytest.mark.parametrize("n", [NAN, -3.0, 0.0])
def test_attend_moment_count_stays_in_its_unit(n, correction):
    """A count of evicted tokens that is NaN (or not above zero) is its unit's
    own matter: three units of a CTA's list have it, the others are as they
    were to the bit.  NaN gives NaN as in the one-token correction; without
    evicted tokens the output is the attention's."""
    U, odd = 480, [3, 156, 307]
    c = Case(61, 4, 2, 5, [10 + i % 7 for i in range(U)], moments=True, correction=correction)
    c.t["mom"][0].copy_(1 + torch.arange(U, device=DEV) % 9)
    o, lse = (x.clone() for x in c.run_attend())
    c.t["mom"][0][odd] = n
    got, got_lse = c.run_attend()
    assert K.kvc_get_device_status(c.ws) == 0
    rest = [u for u in range(U) if u not in odd]
    assert torch.equal(got[rest], o[rest]) and torch.equal(got_lse, lse)
    if n != n:
        assert torch.isnan(got[odd]).all()
        return
    c.p.correction = K.CORR_OFF
    plain = c.run_attend()[0]
    # the groups' sums are normalised before or after they are added: a few half steps of
    # fp32 on values of order 1 (2^-20), then bf16 roundings that are at most a step apart
    assert torch.allclose(got[odd].double(), plain[odd].double(), rtol=2.0 ** -7, atol=2.0 ** -20)


@pytest.mark.parametrize("call", ["attend", "weights", "step"])
def test_first_call_of_a_host_thread(call):
    """The first thing a host thread does is a call: it is not refused (the
    thread has no context of its own yet), gives the bits that it gives
    elsewhere, and a one-token step takes the same kernels (their bits)."""
    lib, ref = K.load(), ctypes.byref
    c = Case(73, 1, 4, 6, [300, 64], kind="chain", moments=True, L=300)
    c.path([3, 2], 3)
    c.run_attend()
    S = torch.zeros(c.U, c.cap, device=DEV)
    at = {n: x.data_ptr() for n, x in c.t.items() if isinstance(x, torch.Tensor)}
    st, rnd = _stream(4, 2, 4, 65, 70, 64, 1)
    st.step_calls(1, 65, rnd(2, 4, 128).bfloat16(), rnd(2, 128).bfloat16(), rnd(2, 128).bfloat16(), 66)
    st.set_kmax(1)
    q, k, v = rnd(2, 4, 128).bfloat16(), rnd(2, 128).bfloat16(), rnd(2, 128).bfloat16()
    out, state, args = {
        "attend": ([c.o, c.lse], [],
                   (ref(c.p), c.max_len, ref(c.tree), at["q"], at["kt"], at["vt"], ref(c.cache),
                    ref(c.moments), c.o.data_ptr(), c.lse.data_ptr(), c.ws.data_ptr(), c.ws.numel(), None)),
        "weights": ([S], [],
                    (ref(c.p), c.max_len, ref(c.tree), ref(c.accept), None, at["q"], at["kt"],
                     c.lse.data_ptr(), ref(c.cache), S.data_ptr(), c.ws.data_ptr(), c.ws.numel(), None)),
        "step": ([st.o, st.util, st.C], [st.K, st.V, st.pos, st.util, st.len, st.n, st.mu_k, st.mu_v, st.C],
                 (ref(st.params), 2, 66, 65, q.data_ptr(), k.data_ptr(), v.data_ptr(), ref(st.cache),
                  ref(st.moments), st.o.data_ptr(), None, 1, st.evict_idx.data_ptr(), None,
                  st.n_evict.data_ptr(), st.ws.data_ptr(), st.ws.numel(), None)),
    }[call]
    name = {"attend": "kvc_tree_attend", "weights": "kvc_tree_weights", "step": "kvc_decode_step"}[call]
    first = [x.clone() for x in state]
    torch.cuda.synchronize()
    assert getattr(lib, name)(*args) == 0
    torch.cuda.synchronize()
    want = [x.clone() for x in out]
    for x, y in zip(state, first):
        x.copy_(y)
    for x in out if not state else [st.o]:
        x.zero_()
    torch.cuda.synchronize()
    got = []

    def run():
        got.append((getattr(lib, name)(*args), K.kvc_last_error()))

    thread = threading.Thread(target=run)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert got[0][0] == 0, got
    for x, y in zip(out, want):
        assert torch.equal(x, y)


def test_calls_of_two_host_threads():
    """Two host threads with a stream, a state and sizes of their own (one
    accepted token and no moments; 64 and moments, 512 rows of q) call at
    once, as fast as they can: no call is refused, and what they leave is what
    the same calls leave one thread after the other."""
    lib, ref, calls = K.load(), ctypes.byref, 3000

    def make(seed, G, T, A, moments):
        c = Case(seed, 1, G, T, [300, 200], kind="chain", moments=moments, budget=[300, 200], L=300)
        c.path([A, A], A)
        c.run_attend()
        c.S = torch.zeros(c.U, c.cap, device=DEV)
        ne = torch.zeros(c.U, dtype=torch.int32, device=DEV)
        c.stream = torch.cuda.Stream()
        at = {n: x.data_ptr() for n, x in c.t.items() if isinstance(x, torch.Tensor)}
        mom = ref(c.moments) if moments else None
        side = ctypes.c_void_p(c.stream.cuda_stream)
        c.weights = (ref(c.p), c.max_len, ref(c.tree), ref(c.accept), None, at["q"], at["kt"],
                     c.lse.data_ptr(), ref(c.cache), c.S.data_ptr(), c.ws.data_ptr(), c.ws.numel(), side)
        c.commit = (ref(c.p), c.max_len, ref(c.tree), ref(c.accept), at["kt"], at["vt"], c.S.data_ptr(),
                    ref(c.cache), mom, A, None, None, ne.data_ptr(), c.dws.data_ptr(), c.dws.numel(), side)
        c.state = [c.t[n] for n in ("K", "V", "pos", "util", "len")] + (c.t["mom"] or []) + [c.S, ne]
        return c

    cases = [make(71, 1, 4, 1, False), make(72, 8, 64, 64, True)]
    first = [[x.clone() for x in c.state] for c in cases]
    refused = []

    def loop(c):
        for _ in range(calls):
            status = lib.kvc_tree_weights(*c.weights) or lib.kvc_tree_commit(*c.commit)
            if status:
                refused.append((status, K.kvc_last_error()))     # (the thread's own message)
                return

    torch.cuda.synchronize()
    want = []
    for c, f in zip(cases, first):
        loop(c)
        torch.cuda.synchronize()
        want.append([x.clone() for x in c.state])
        for x, y in zip(c.state, f):
            x.copy_(y)
    torch.cuda.synchronize()
    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=loop, args=(c,)) for c in cases]
        for x in threads:
            x.start()
        for x in threads:
            x.join()
    finally:
        sys.setswitchinterval(before)
    torch.cuda.synchronize()
    assert not refused, refused
    for c, w in zip(cases, want):
        assert K.kvc_get_device_status(c.ws) == 0 and K.kvc_get_device_status(c.dws) == 0
        for x, y in zip(c.state, w):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


# ------------------------------------------------------------------ the state's calls

def _chain(T, U, tok, count, pos):
    """A chain of T tokens of one sequence, and a path of it."""
    mask = torch.tensor([[(2 << i) - 1 for i in range(T)]], dtype=torch.int64, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    return K.make_tree(T, U, mask), K.make_path(len(tok), i32([tok]), i32([count]), i32([pos]))


@pytest.mark.parametrize("refused", ["a dead token", "too many victims", "too few scored"])
def test_state_reports_what_only_the_commit_refuses(refused):
    """Without a refresh only the commit looks at the path, and only it
    counts victims: tree_status() has its refusal, once."""
    U, G, L, T = 4, 2, 80, 5
    st, rnd = _stream(6, U, G, L, L + 80, L, 1)
    tree, path = _chain(T, U, [0, 5 if refused == "a dead token" else 1], 2, 500)
    args = rnd(U, T, G, 128).bfloat16(), rnd(U, T, 128).bfloat16(), rnd(U, T, 128).bfloat16()
    if refused == "too many victims":
        st.len.fill_(L + 70)                           # 70 slots over the budget
    if refused != "too few scored":
        st.util.fill_(1.0)
    max_len = int(st.len[0])
    st.verify(tree, *args, max_len)
    st.accept(tree, path, *args, max_len, refresh=False)
    assert st.n_evict.tolist() == [0] * U and st.len.tolist() == [max_len] * U
    assert st.tree_status() == (2 if refused == "too many victims" else 1)
    assert st.tree_status() == 0 and st.device_status() == 0


@pytest.mark.parametrize("handle", [False, True, "default"])
def test_first_verify_on_another_stream(handle):
    """The first call with a T makes its buffers: a call on another stream
    than the current one, which is busy, does not run ahead of their fills."""
    U, G, L, T = 4, 4, 3000, 9
    st, rnd = _stream(7, U, G, L, L + 20, L, 1)
    tree, path = _chain(T, U, [0, 1], 2, 5000)
    args = rnd(U, T, G, 128).bfloat16(), rnd(U, T, 128).bfloat16(), rnd(U, T, 128).bfloat16()
    st.util.copy_(torch.rand(U, L + 20, device=DEV, dtype=torch.float64))
    side = torch.cuda.Stream()
    room = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    del room                                           # the buffers come without a device call
    torch.cuda.synchronize()
    # (the default stream's handle is 0: the current one is another then)
    on = 0 if handle == "default" else side.cuda_stream if handle else side
    with torch.cuda.stream(side if handle == "default" else torch.cuda.current_stream()):
        torch.cuda._sleep(200_000_000)                 # about 0.1 s of the current stream
        o, lse = st.verify(tree, *args, L, stream=on)
        st.accept(tree, path, *args, L, stream=on)
    torch.cuda.synchronize()
    S, got = st.tree_S.clone(), (o.clone(), lse.clone())
    ev = st.tree_evict.clone()
    again, _ = _stream(7, U, G, L, L + 20, L, 1)
    again.util.copy_(st.util)
    want = again.verify(tree, *args, L)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    again.accept(tree, path, *args, L)
    assert torch.equal(S, again.tree_S) and (ev[0] >= 0).all()


# ------------------------------------------------------- weights below fp32's range

def wide_weights(c, u, w):
    """R.weights' sums and their bound without what fp32's range takes: every
    error is relative to its term (the logit's, the logarithms', and 16 half
    steps for the powers of two that the sum is held in)."""
    b, a, n, G = u // c.per, c.counts[u // c.per], c.lens[u], c.G
    path = [int(x) for x in c.tok[b, :a]]
    S, e_S = np.zeros(n + a), np.zeros(n + a)
    keys, lse = np.concatenate([c.K[u, :n], c.kt[u, path]]), f64(c.lse[u])
    for j, t in enumerate(path):
        see = [int(c.mask[b, t]) >> r & 1 for r in path]
        for h in range(G):
            if lse[t, h] == -np.inf:
                continue
            x = keys @ c.q[u, t, h] * R.SCALE
            e = np.exp(x - lse[t, h])
            if c.votes is not None:
                e[:n] *= c.votes[u, :n]
            e[n:] = np.where(see, e[n:], 0.0)
            e *= w[j] / G
            S += e
            e_S += e * (R.logit_error(c.q[u, t, h], keys) + 8 * R.E32 * (
                np.abs(x) + abs(lse[t, h]) + 2 + abs(np.log(w[j] / G))))
    return S, e_S + (a * G + 32) * R.E32 * S


WIDE = [
    # per, G, T, lens, counts, A, keywords
    (1, 1, 1, [0, 1, 2], [1, 1, 0], 1, {}),
    (2, 4, 7, [127, 128, 129, 0], [3, 2], 3, dict(q_scale=30.0)),
    (2, 8, 5, [255, 256, 257, 300], [5, 1], 5, dict(votes=True, q_scale=25.0)),
    (1, 2, 64, [130, 1, 400], [64, 64, 7], 64, dict(kind="chain", q_scale=12.0)),
    (1, 8, 64, [200, 129], [64, 30], 64, dict(kind="chain", q_scale=40.0)),
    (1, 4, 6, [0, 0, 5], [2, 3, 1], 3, dict(kind="none")),
    (4, 1, 24, [100, 200, 300, 400] * 45, [i % 7 for i in range(45)], 6, dict(q_scale=60.0)),
    (1, 4, 9, [700], [5], 5, dict(q_scale=90.0, votes=True)),
]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("i", range(len(WIDE)))
def test_weights_f64(i, given):
    """Logits up to several hundred apart: every weight down to 2^-1000 is
    there, to fp32's precision of its logit."""
    per, G, T, lens, counts, A, kw = WIDE[i]
    c = Case(500 + i, per, G, T, lens, **kw)
    c.path(counts, A)
    c.run_attend()
    w = (2.0 ** c.rng.uniform(-40, 1, (c.B, A))).astype(np.float32) if given else np.ones((c.B, A), np.float32)
    S = torch.full((c.U, c.cap), -3.0, device=DEV, dtype=torch.float64)
    K.kvc_tree_weights(c.p, c.max_len, c.tree, c.accept, torch.from_numpy(w).to(DEV) if given else None,
                       c.t["q"], c.t["kt"], c.lse, c.cache, S, c.ws)
    assert K.kvc_get_device_status(c.ws) == 0
    S = f64(S)
    for u in range(c.U):
        b = u // per
        n = lens[u] + counts[b]
        ref, bound = wide_weights(c, u, w[b].astype(np.float64))
        there = ref > 2.0 ** -1000
        assert (np.abs(S[u, :n] - ref)[there] <= bound[there]).all(), (
            u, (np.abs(S[u, :n] - ref)[there] / bound[there]).max())
        assert (S[u, :n][~there] <= 2.0 ** -999).all() and (S[u, :n][~there] >= 0).all()
        assert (S[u, n:] == -3).all()
    if kw.get("q_scale", 0) >= 60:
        assert (S[(S > 0)] < 2.0 ** -150).any()


def test_weights_f64_are_the_fp32_ones_where_those_hold():
    c = Case(520, 2, 4, 9, [700, 90, 33, 400], votes=True)
    c.path([4, 2], 4)
    c.run_attend()
    S = [torch.full((c.U, c.cap), -3.0, device=DEV, dtype=t) for t in (torch.float32, torch.float64)]
    for x in S:
        K.kvc_tree_weights(c.p, c.max_len, c.tree, c.accept, None, c.t["q"], c.t["kt"], c.lse, c.cache,
                           x, c.ws)
    assert (S[0] != 0).all() and torch.equal(S[0].double(), S[1])


@pytest.mark.parametrize("n,U", [(300, 2), (9000, 2), (5000, 1), (257, 400), (8300, 160)])
@pytest.mark.parametrize("rule", ["single", "cumulative", "ema"])
def test_commit_f64(rule, n, U):
    """Weights all over fp64's range, every way the work is cut: utilities as
    IEEE arithmetic gives them, and the victims that follow from them."""
    rng = np.random.default_rng(530)
    cap = n + 6
    S = np.exp2(rng.uniform(-800, 4, (U, cap)))
    old = np.exp2(rng.uniform(-800, 4, (U, cap)))
    old[rng.random(old.shape) < 0.1] = np.inf
    odd = [(0.0, 0.0), (0.0, 1.5), (0.25, 0.0), (5e-324, 5e-324), (1e-310, 1e-320), (1e300, 1.0),
           (-1.5, 1.5), (-1.5, 0.25), (1.0, 5e-324), (1.0, 3e38), (1.0, 2.0 ** -53),
           (1 + 2.0 ** -52, 2.0 ** -53), (2 - 2.0 ** -52, 2.0 ** -53), (2.0 ** -53, 2.0 ** 60)]
    for i, (x, y) in enumerate(odd):
        old[:, 200 + i], S[:, 200 + i] = x, y
    pos = np.stack([rng.permutation(cap) for _ in range(U)]).astype(np.int32)
    util, dpos = torch.from_numpy(old).to(DEV), torch.from_numpy(pos).to(DEV)
    rows = torch.zeros(U, cap, 128, dtype=torch.bfloat16, device=DEV)
    length = torch.full((U,), n, dtype=torch.int32, device=DEV)
    code = {"single": K.RULE_SINGLE, "cumulative": K.RULE_CUMULATIVE, "ema": K.RULE_EMA}[rule]
    p = K.make_params(U, 1, cap, n, rule=code, alpha=0.75)
    tree, path = _chain(4, U, [0, 1, 2], 3, cap)
    new = torch.zeros(U, 4, 128, dtype=torch.bfloat16, device=DEV)
    ei, ep = (torch.full((U, 3), -9, dtype=torch.int32, device=DEV) for _ in range(2))
    ne = torch.full((U,), -9, dtype=torch.int32, device=DEV)
    dws = torch.empty(K.kvc_decode_workspace_size(p), dtype=torch.uint8, device=DEV)
    K.kvc_decode_workspace_init(p, dws)
    K.kvc_tree_commit(p, n, tree, path, new, new, torch.from_numpy(S).to(DEV),
                      K.make_cache(rows, rows, None, dpos, util, length), None, 3, ei, ep, ne, dws)
    assert K.kvc_get_device_status(dws) == 0 and (ne == 3).all() and (length == n).all()
    m, s, R_ = old[:, :n], S[:, :n], U
    with np.errstate(invalid="ignore"):
        if rule == "ema":
            # alpha and 1 - alpha are exact: the product of the weight is rounded, then the whole
            R_ = min(U, 2)
            upd = np.array([[float(Fraction(0.75) * Fraction(x) + Fraction(0.25 * y)) if np.isfinite(x)
                             else y for x, y in zip(a, b)] for a, b in zip(m[:R_], s[:R_])])
        else:
            upd = s if rule == "single" else np.where(np.isinf(m), s, m + s)
    every = np.concatenate([upd, S[:R_, n:n + 3]], 1)
    where = np.concatenate([pos[:R_, :n], np.tile(cap + np.arange(3), (R_, 1))], 1)
    low = np.sort(np.lexsort((where, every))[:, :3], 1)
    assert np.array_equal(low, ei[:R_].cpu().numpy())
    assert np.array_equal(np.take_along_axis(where, low, 1), ep[:R_].cpu().numpy())
    keep = np.ones((R_, n + 3), dtype=bool)
    np.put_along_axis(keep, low, False, 1)                 # a victim's place is another's now
    keep = keep[:, :n]
    assert np.array_equal(f64(util)[:R_, :n][keep], upd[keep])


@pytest.mark.parametrize("rule", [K.RULE_SINGLE, K.RULE_CUMULATIVE, K.RULE_EMA])
def test_sharp_attention_evicts_what_decode_steps_evict(rule):
    """Logits some hundred apart: the weights of most slots are far below
    fp32's range, and verify / accept of one token at a time evict the same
    positions as the one-token calls, which order them."""
    U, G, n, L = 6, 4, 300, 280
    a, rnd = _stream(8, U, G, n, n + 4, L, 8)
    b, _ = _stream(8, U, G, n, n + 4, L, 8)
    a.params.rule = b.params.rule = rule
    one = torch.ones(1, 1, dtype=torch.int64, device=DEV)
    zero = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    low = 0
    for t in range(1, 13):
        q, k, v = (60 * rnd(U, G, 128)).bfloat16(), rnd(U, 128).bfloat16(), rnd(U, 128).bfloat16()
        max_len = n + 1 if t == 1 else L + 1
        b.step_calls(t, n + t - 1, q, k, v, max_len)
        if t == 1:
            a.step_calls(t, n + t - 1, q, k, v, max_len)
            continue
        tree = K.make_tree(1, U, one)
        path = K.make_path(1, zero, torch.ones(1, dtype=torch.int32, device=DEV),
                           torch.full((1,), n + t - 1, dtype=torch.int32, device=DEV))
        a.verify(tree, q, k, v, L)
        a.accept(tree, path, q, k, v, L)
        assert a.tree_status() == 0 and a.device_status() == 0
        low += int((b.probs[:, :L] < 2.0 ** -150).sum())
        assert torch.equal(a.tree_evict[1][:, 0], b.evict_pos[:, 0]), t
    assert low > U * L                                     # one in eleven of the weights at least


# ---------------------------------------------------- ways of the work seldom taken

LAYOUTS = {
    "whole, both groups": (2, 4, 9, [300, 45, 128, 700] * 2, dict(live=[9, 4, 9, 2])),
    "whole, moments": (2, 4, 9, [300, 45, 128, 700] * 2, dict(live=[9, 4, 9, 2], moments=True, votes=True)),
    "two halves of rows": (1, 4, 63, [300, 0, 130], {}),
    "two halves, moments": (1, 4, 63, [300, 0, 130], dict(moments=True)),
    "parts of a unit": (1, 2, 12, [4000, 130, 5, 0, 2050], {}),
    "parts of a unit, moments": (1, 2, 12, [4000, 130, 5, 0, 2050], dict(votes=True, moments=True)),
    "parts, two halves, two blocks": (1, 8, 40, [2900, 1, 260], dict(moments=True)),
    "line": (4, 2, 12, [(37 * i * i) % 2100 for i in range(160)], {}),
    "line, moments": (4, 2, 12, [(37 * i * i) % 2100 for i in range(160)], dict(votes=True, moments=True)),
}


@pytest.mark.parametrize("value", [NAN, float("inf"), -float("inf")])
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_attend_masked_branch_in_every_layout(layout, value):
    """One value (then one key) of every tree's token 1 is not finite: what a
    row that sees the token gets is not finite in that dimension (for a key,
    in any), everything else is as it was to the bit."""
    per, G, T, lens, kw = LAYOUTS[layout]
    c = Case(600, per, G, T, lens, kind="tree", **kw)
    o, lse = (x.clone() for x in c.run_attend())
    see = torch.zeros(c.U, T, dtype=torch.bool, device=DEV)
    for u in range(c.U):
        for t in range(c.live[u // per]):
            see[u, t] = bool(int(c.mask[u // per, t]) >> 1 & 1)
    assert see.any() and not see.all()
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[..., 5] = see[:, :, None]
    keep = c.t["vt"][:, 1, 5].clone()
    c.t["vt"][:, 1, 5] = value
    got, got_lse = c.run_attend()
    assert K.kvc_get_device_status(c.ws) == 0
    assert torch.equal(got_lse, lse) and torch.equal(got[~hit], o[~hit])
    assert not torch.isfinite(got[hit]).any()
    c.t["vt"][:, 1, 5] = keep
    c.t["kt"][:, 1, 5] = NAN
    got, got_lse = c.run_attend()
    assert K.kvc_get_device_status(c.ws) == 0
    assert torch.equal(got[~see], o[~see]) and torch.equal(got_lse[~see], lse[~see])
    assert torch.isnan(got[see]).all() and torch.isnan(got_lse[see]).all()


@pytest.mark.parametrize("n,U", [(20000, 2), (20000, 60), (1500, 160), (9000, 160), (20000, 153)])
@pytest.mark.parametrize("ties", ["zero", "few", "stride", "one group"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
def test_commit_ties_of_long_and_of_many_units(ties, n, U, dtype):
    """More slots at the bound than there are places for, in long units and
    where a unit has half the threads: the lowest (weight, position, slot)."""
    rng = np.random.default_rng(640)
    k, cap = 40, n + 41
    S = np.zeros((U, cap))
    if ties == "few":
        S = rng.integers(0, 3, S.shape).astype(np.float64)
    elif ties == "stride":
        S = 1 + rng.integers(0, 1000, S.shape) / 1024
        S[:, ::512] = 0.25
        S[:, 1:3000:3] = 0.5
    elif ties == "one group":                              # the lowest sit side by side
        S = 1 + rng.integers(0, 1000, S.shape) / 1024
        S[:, 256:290] = 0.25
        S[:, 1000:1003] = 0.125
    pos = np.stack([rng.permutation(cap) for _ in range(U)]).astype(np.int32)
    pos[:, 5] = pos[:, 3]                                  # a tie of the positions too
    util = torch.zeros(U, cap, dtype=torch.float64, device=DEV)
    rows = torch.zeros(U, cap, 128, dtype=torch.bfloat16, device=DEV)
    length = torch.full((U,), n, dtype=torch.int32, device=DEV)
    p = K.make_params(U, 1, cap, n, rule=K.RULE_SINGLE)
    tree, path = _chain(k, U, list(range(k)), k, cap)
    new = torch.zeros(U, k, 128, dtype=torch.bfloat16, device=DEV)
    ei, ep = (torch.full((U, k), -9, dtype=torch.int32, device=DEV) for _ in range(2))
    ne = torch.full((U,), -9, dtype=torch.int32, device=DEV)
    dws = torch.empty(K.kvc_decode_workspace_size(p), dtype=torch.uint8, device=DEV)
    K.kvc_decode_workspace_init(p, dws)
    K.kvc_tree_commit(p, n, tree, path, new, new, torch.from_numpy(S).to(DEV, dtype),
                      K.make_cache(rows, rows, None, torch.from_numpy(pos).to(DEV), util, length), None,
                      k, ei, ep, ne, dws)
    assert K.kvc_get_device_status(dws) == 0 and (ne == k).all() and (length == n).all()
    where = np.concatenate([pos[:, :n], np.tile(cap + np.arange(k), (U, 1))], 1)
    low = np.sort(np.lexsort((where, S[:, :n + k]))[:, :k], 1)
    assert np.array_equal(low, ei.cpu().numpy())
    assert np.array_equal(np.take_along_axis(where, low, 1), ep.cpu().numpy())


def test_lazy_steps_around_a_commit():
    """Between lazy steps a commit moves the lowest slots about: the victims
    that the refresh step queued are dropped, and the fused step takes the
    ones that the call sequence takes."""
    U, G, n, L, T = 6, 4, 90, 64, 6
    a, rnd = _stream(9, U, G, n, n + 12, L, 8)
    b, _ = _stream(9, U, G, n, n + 12, L, 8)
    a.params.refresh_period = b.params.refresh_period = 6
    pos = n
    for t in range(1, 25):
        q, k, v = rnd(U, G, 128).bfloat16(), rnd(U, 128).bfloat16(), rnd(U, 128).bfloat16()
        max_len = n + 1 if t == 1 else L + 1
        (a.step_calls if t == 1 else a.step)(t, pos, q, k, v, max_len)
        b.step_calls(t, pos, q, k, v, max_len)
        pos += 1
        assert torch.equal(a.n_evict, b.n_evict)
        assert torch.equal(a.evict_pos, b.evict_pos), t
        if t % 3 == 0:
            tree, path = _chain(T, U, [0, 1, 2], 1 + t % 2, pos)
            args = rnd(U, T, G, 128).bfloat16(), rnd(U, T, 128).bfloat16(), rnd(U, T, 128).bfloat16()
            for x in (a, b):
                x.verify(tree, *args, L)
                x.accept(tree, path, *args, L, refresh=t % 2 == 0)
                assert x.tree_status() == 0
            pos += 1 + t % 2
            assert torch.equal(a.tree_evict, b.tree_evict)
        assert a.device_status() == 0 and b.device_status() == 0
        assert torch.equal(a.pos[:, :L].sort(1)[0], b.pos[:, :L].sort(1)[0])


@pytest.mark.parametrize("budgets", [False, True])
def test_state_run_in_a_graph(budgets):
    """verify and accept captured once, replayed over new inputs and new
    paths: what the calls give outside a graph, with a budget of the state
    and with one per unit."""
    U, per, G, L, T, A = 8, 4, 4, 200, 7, 4
    rng = np.random.default_rng(3)

    def make():
        st, rnd = _stream(10, U, G, L, L + 12, L, 1, budgets=budgets)
        if budgets:
            lens = torch.tensor([L, 150, 3, 77, L - 1, 128, 129, 1], dtype=torch.int32, device=DEV)
            st.len.copy_(lens)
            st.budget.copy_(lens)
        st.util.copy_(torch.rand(U, L + 12, dtype=torch.float64, device=DEV,
                                 generator=torch.Generator(device=DEV).manual_seed(5)))
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
        ins = dict(q=torch.zeros(U, T, G, 128, dtype=torch.bfloat16, device=DEV),
                   k=torch.zeros(U, T, 128, dtype=torch.bfloat16, device=DEV),
                   v=torch.zeros(U, T, 128, dtype=torch.bfloat16, device=DEV),
                   mask=torch.zeros(2, T, dtype=torch.int64, device=DEV), tok=i32(2, A), n=i32(2),
                   pos=i32(2), live=i32(2), w=torch.zeros(2, A, device=DEV))
        tree = K.make_tree(T, per, ins["mask"], ins["live"])
        path = K.make_path(A, ins["tok"], ins["n"], ins["pos"])
        return st, ins, tree, path, rnd

    def call(st, ins, tree, path):
        st.verify(tree, ins["q"], ins["k"], ins["v"], L)
        st.accept(tree, path, ins["q"], ins["k"], ins["v"], L, row_weight=ins["w"])

    def state(st):
        o, lse = st._trees[T]["o"], st._trees[T]["lse"]
        return [st.K, st.V, st.pos, st.util, st.len, st.n, st.mu_k, st.mu_v, st.C, st.n_evict, o, lse, st.tree_S]

    a, b = make(), make()
    a[0].verify(a[2], a[1]["q"], a[1]["k"], a[1]["v"], L)      # (no live token: makes the buffers)
    b[0].verify(b[2], b[1]["q"], b[1]["k"], b[1]["v"], L)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(*b[:4])
    for step in range(5):
        rnd = a[4]
        new = dict(q=rnd(U, T, G, 128).bfloat16(), k=rnd(U, T, 128).bfloat16(), v=rnd(U, T, 128).bfloat16(),
                   mask=torch.from_numpy(tree_masks(rng, 2, T, "chain").view(np.int64)).to(DEV),
                   tok=torch.from_numpy(np.tile(np.arange(A, dtype=np.int32), (2, 1))).to(DEV),
                   n=torch.tensor([step % (A + 1), 3], dtype=torch.int32, device=DEV),
                   pos=torch.full((2,), 1000 + 10 * step, dtype=torch.int32, device=DEV),
                   live=torch.tensor([T, 5], dtype=torch.int32, device=DEV),
                   w=torch.rand(2, A, device=DEV))
        for s in (a, b):
            for name, x in new.items():
                s[1][name].copy_(x)
        call(*a[:4])
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(state(a[0]), state(b[0])):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
        for s in (a, b):
            assert s[0].tree_status() == 0
            assert torch.equal(s[0].len, s[0].budget if budgets else torch.full_like(s[0].len, L))


def test_steps_of_two_host_threads():
    """One-token steps of two states from two host threads at once, whose
    caches differ in size (and so the kernel's shared memory): no step is
    refused."""
    lib, ref, calls = K.load(), ctypes.byref, 4000

    def make(seed, L):
        st, rnd = _stream(seed, 2, 4, L + 1, L + 4, L, 1)
        q, k, v = rnd(2, 4, 128).bfloat16(), rnd(2, 128).bfloat16(), rnd(2, 128).bfloat16()
        st.step_calls(1, L + 1, q, k, v, L + 2)
        st.set_kmax(1)
        stream = torch.cuda.Stream()
        args = (L + 1, q.data_ptr(), k.data_ptr(), v.data_ptr(), ref(st.cache), ref(st.moments),
                st.o.data_ptr(), None, 1, st.evict_idx.data_ptr(), None, st.n_evict.data_ptr(),
                st.ws.data_ptr(), st.ws.numel(), ctypes.c_void_p(stream.cuda_stream))
        return st, args, (q, k, v, stream)

    states = [make(81, 64), make(82, 15000)]
    refused = []

    def loop(st, args):
        for i in range(calls):
            status = lib.kvc_decode_step(ref(st.params), 2 + i, 20000 + i, *args)
            if status:
                refused.append((status, K.kvc_last_error()))
                return

    torch.cuda.synchronize()
    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=loop, args=x[:2]) for x in states]
        for x in threads:
            x.start()
        for x in threads:
            x.join()
    finally:
        sys.setswitchinterval(before)
    torch.cuda.synchronize()
    assert not refused, refused
    for st, _, _ in states:
        assert st.device_status() == 0 and st.n_evict.tolist() == [1, 1]
