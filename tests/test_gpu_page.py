"""GPU tests of the cache in pages (kvc_page_write, kvc_page_read,
kvc_page_attend) and of the norms and rotation in front of it
(kvc_qk_norm_rope) against their definitions in 64 bits (page_ref.py): types,
head layouts, tables, lengths from zero on, what lies behind a sequence, what
the device refuses; then runs of them together and with the budgeted cache,
streams, graphs, threads and a pool past 2^31 bytes."""
import threading

import numpy as np
import pytest
import torch

import page_ref as R
from kv_cache_eviction_kvc_gb300 import kvc as K
from kv_cache_eviction_kvc_gb300.state import DecodeState, PagedState

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

DEV, D, NAN = "cuda", 128, float("nan")


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().to(torch.float32).numpy().astype(np.float64)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Pool:
    """A pool with a random table for the given lengths (room for `more` slots behind them), rows
    drawn, everything that belongs to nobody NaN; the same on the host in 64 bits."""

    def __init__(self, seed, heads, lens, page, e4m3, more=0, k_scale=1.0, v_scale=1.0, extra=2):
        rng = self.rng = np.random.default_rng(seed)
        S = self.S = len(lens)
        self.heads, self.lens, self.page, self.e4m3, self.U = heads, list(lens), page, e4m3, S * heads
        need = [-(-(n + more) // page) for n in lens]
        self.n_pages, stride = max(1, sum(need) + extra), max(need) + 1
        order = rng.permutation(self.n_pages)
        self.tab = np.full((S, stride), np.iinfo(np.int32).min, np.int32)
        at = 0
        for s, m in enumerate(need):
            self.tab[s, :m] = order[at:at + m]
            at += m
        shape = (self.n_pages, heads, page, D)
        self.rows = {}
        for name, factor in (("K", k_scale), ("V", v_scale)):
            x = np.full(shape, NAN)
            for s, n in enumerate(lens):
                i = np.arange(n)
                off = 0.5 * rng.standard_normal((heads, 1, D))
                y = f64(bf(factor * (off + rng.standard_normal((heads, n, D)))))
                x[self.tab[s, i // page], :, i % page] = y.transpose(1, 0, 2)
            self.rows[name] = x
        self.t, self.scale = {}, {"K": None, "V": None}
        for name, x in self.rows.items():
            if e4m3:
                v, sc = R.quantise(x)
                self.t[name], self.scale[name] = v.to(DEV), torch.from_numpy(sc).to(DEV)
            else:
                self.t[name] = bf(x).to(DEV)
        self.t["table"], self.t["len"] = torch.from_numpy(self.tab).to(DEV), i32(self.lens)
        self.make()

    def make(self):
        self.pages = K.make_pages(self.t["K"], self.t["V"], self.scale["K"], self.scale["V"],
                                  self.t["table"], self.t["len"])
        self.ws = torch.zeros(max(256, K.kvc_page_workspace_size(self.pages, 8)), dtype=torch.uint8,
                              device=DEV)

    def held(self, name, u, slots):
        """The rows of unit u as they are held now, fp64."""
        s, h = u // self.heads, u % self.heads
        slots = np.asarray(slots, dtype=np.int64)
        b, r = torch.from_numpy(self.tab[s][slots // self.page]).long(), torch.from_numpy(slots % self.page)
        x = f64(self.t[name].view(torch.uint8 if self.e4m3 else torch.bfloat16).cpu()[b, h, r]
                .view(self.t[name].dtype))
        if self.e4m3:
            with np.errstate(invalid="ignore"):
                x = x * self.scale[name].cpu()[b, h, r].numpy().astype(np.float64)[:, None]
        return x

    def status(self):
        return K.kvc_get_device_status(self.ws)

    def bits(self):
        return [self.t[n].view(torch.uint8).clone() for n in "KV"] + [
            None if x is None else x.view(torch.int32).clone() for x in self.scale.values()]


def attend(p, G, append=True, max_len=None, q=None, o=None, lse=None, k=None, v=None, q_scale=1.5):
    rng = p.rng
    q = bf(q_scale * rng.standard_normal((p.U, G, D))).to(DEV) if q is None else q
    if append and k is None:
        k, v = (bf(rng.standard_normal((p.U, D))).to(DEV) for _ in range(2))
    o = torch.full((p.U, G, D), 7.0, dtype=torch.bfloat16, device=DEV) if o is None else o
    lse = torch.full((p.U, G), 7.0, device=DEV) if lse is None else lse
    K.kvc_page_attend(p.pages, max_len or max(1, max(p.lens) + bool(append)), q, k, v, o, lse, p.ws)
    return q, k, v, o, lse


def check_attend(p, G, append=True, units=None, **kw):
    q, k, v, o, lse = attend(p, G, append, **kw)
    assert p.status() == 0
    qh, oh, lh = f64(q), f64(o), lse.cpu().numpy().astype(np.float64)
    for u in range(p.U) if units is None else units:
        n = p.lens[u // p.heads]
        if append:
            for name, x in (("K", k), ("V", v)):
                row = f64(x[u])
                if p.e4m3:
                    val, sc = R.quantise(row)
                    row = f64(val) * np.float64(sc)
                assert np.array_equal(p.held(name, u, [n])[0], row), (u, name)
        m = n + bool(append)
        ro, rl, bo, bl = R.attend(qh[u], p.held("K", u, range(m)), p.held("V", u, range(m)))
        assert (np.abs(oh[u] - ro) <= bo).all(), (u, m, np.abs(oh[u] - ro).max(), bo.max())
        if m:
            assert (np.abs(lh[u] - rl) <= bl).all(), (u, m, lh[u], rl)
        else:
            assert (lh[u] == -np.inf).all()
    return q, k, v, o, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 511, 513]


# ---------------------------------------------------------------------- attend

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("heads,page", [(1, 16), (8, 16), (2, 32), (1, 64), (3, 128)])
def test_attend(e4m3, G, heads, page):
    check_attend(Pool(G * 100 + page + heads, heads, LENS, page, e4m3, more=1), G)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_attend_without_append(e4m3, G):
    p = Pool(7 + G, 2, LENS, 16, e4m3)
    before = p.bits()
    check_attend(p, G, append=False)
    for a, b in zip(before, p.bits()):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_touches_its_rows_only(e4m3):
    p = Pool(3, 2, [5, 16, 0, 31], 16, e4m3, more=1)
    before = p.bits()
    check_attend(p, 4)
    rows = set()
    for s, n in enumerate(p.lens):
        for h in range(p.heads):
            rows.add((int(p.tab[s, n // p.page]) * p.heads + h) * p.page + n % p.page)
    for a, b, wide in zip(before, p.bits(), (1, 1, 0, 0)):
        if a is None:
            continue
        a, b = (x.reshape(p.n_pages * p.heads * p.page, -1) for x in (a, b))
        changed = {int(i) for i in (a != b).any(1).nonzero().flatten()}
        assert changed <= rows and (not wide or changed == rows)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [4096, 20011, 131071])
def test_attend_long(e4m3, n):
    check_attend(Pool(n, 2, [n, n // 3], 64, e4m3, more=1), 4)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G", [2, 8])
def test_attend_many_ragged_units(e4m3, G):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 700, 333)]
    p = Pool(11, 1, lens, 16, e4m3, more=1)
    check_attend(p, G, units=range(0, 333, 7))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kw", [dict(k_scale=30.0), dict(k_scale=1e-3), dict(v_scale=1e4),
                                dict(v_scale=1e-30), dict(v_scale=1e30), dict(k_scale=0.0),
                                dict(v_scale=0.0)])
def test_attend_magnitudes(e4m3, kw):
    """Sharp and flat attention, large, tiny and zero values."""
    check_attend(Pool(23, 2, [1, 40, 333, 1200], 32, e4m3, more=1, **kw), 4)


@pytest.mark.parametrize("e4m3", [False, True])
def test_attend_rows_of_very_different_magnitude(e4m3):
    """A row that weighs nothing may hold values 2^40 times those of the rows that weigh."""
    p = Pool(29, 1, [200, 200], 16, e4m3, more=1)
    for u, (big, small) in enumerate(((2.0 ** 40, 1.0), (1.0, 2.0 ** -40))):
        i = np.arange(200)
        x = f64(bf(p.rng.standard_normal((200, D)) * np.where(i % 50 == 3, big, small)[:, None]))
        y = f64(bf(p.rng.standard_normal((200, D))))
        at = (p.tab[u, i // 16], 0, i % 16)
        for name, z in (("V", x), ("K", y)):
            zt = R.quantise(z) if e4m3 else (bf(z), None)
            idx = (torch.from_numpy(at[0]).long().to(DEV), 0, torch.from_numpy(at[2]).to(DEV))
            if e4m3:
                p.t[name].view(torch.uint8)[idx] = zt[0].view(torch.uint8).to(DEV)
                p.scale[name][idx] = torch.from_numpy(zt[1]).to(DEV)
            else:
                p.t[name][idx] = zt[0].to(DEV)
    q = bf(6 * p.rng.standard_normal((2, 4, D)))
    check_attend(p, 4, q=q.to(DEV))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -20, 2.0 ** 10, 0.0])
def test_attend_queries_of_any_magnitude(e4m3, scale):
    p = Pool(31, 2, [70, 300], 16, e4m3, more=1, k_scale=1.0 if scale <= 1 else 2.0 ** -10)
    check_attend(p, 4, q_scale=scale)


@pytest.mark.parametrize("e4m3", [False, True])
def test_heads_of_one_unit_with_very_different_queries(e4m3):
    p = Pool(37, 1, [100, 257], 16, e4m3, more=1)
    q = p.rng.standard_normal((2, 8, D)) * (2.0 ** np.array([-60, -30, -8, 0, 1, 2, 3, 0]))[:, None]
    check_attend(p, 8, q=bf(q).to(DEV))


@pytest.mark.parametrize("e4m3", [False, True])
def test_nan_stays_in_its_unit(e4m3):
    """A NaN in a live row reaches its unit alone; NaN behind a sequence reaches nobody."""
    p = Pool(41, 2, [300, 300], 16, e4m3, more=1)
    q, k, v, o, _ = check_attend(p, 4)
    ref = o.clone()
    b = int(p.tab[0, 10])
    if e4m3:
        p.scale["V"][b, 1, 3] = NAN
    else:
        p.t["V"][b, 1, 3] = NAN
    _, _, _, o, _ = attend(p, 4, q=q, k=k, v=v)
    assert o[1].isnan().all() and torch.equal(o[[0, 2, 3]], ref[[0, 2, 3]])


def test_append_of_a_row_with_nan_or_infinity():
    for e4m3 in (False, True):
        p = Pool(43, 1, [20, 20, 20], 16, e4m3, more=1)
        k, v = (bf(p.rng.standard_normal((3, D))) for _ in range(2))
        v[0, 5], k[1, 5] = NAN, float("inf")
        _, _, _, o, _ = attend(p, 2, k=k.to(DEV), v=v.to(DEV))
        assert o[0, :, 5].isnan().all() and not o[2].isnan().any()
        if e4m3:
            assert np.isnan(p.held("V", 0, [20])).all() and np.isnan(p.held("K", 1, [20])).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [40, 5000])
def test_device_side_refusals(e4m3, n):
    """A bad length or page leaves its sequence's outputs; the others are right."""
    for bad, code in (("long", 2), ("negative", 2), ("page", 1), ("page_high", 1), ("new_page", 1)):
        p = Pool(47, 2, [n, n, n], 16, e4m3, more=1)
        if bad == "long":
            p.t["len"][1] = n + 1
        elif bad == "negative":
            p.t["len"][1] = -1
        elif bad == "page":
            p.t["table"][1, 1] = -1
        elif bad == "page_high":
            p.t["table"][1, 0] = p.n_pages
        else:
            p.t["table"][1, n // 16] = 1 << 30
        q, k, v, o, lse = attend(p, 4, max_len=n + 1)
        assert p.status() == code and p.status() == 0, bad
        assert (o[2:4] == 7).all() and (lse[2:4] == 7).all(), bad
        for u in (0, 1, 4, 5):
            ro, rl, bo, bl = R.attend(f64(q[u]), p.held("K", u, range(n + 1)), p.held("V", u, range(n + 1)))
            assert (np.abs(f64(o[u]) - ro) <= bo).all() and (np.abs(f64(lse[u]) - rl) <= bl).all(), (bad, u)
        # the workspace is as it was: the next call is right
        p.t["len"].copy_(i32(p.lens))
        p.t["table"].copy_(torch.from_numpy(p.tab))
        check_attend(p, 4)


@pytest.mark.parametrize("e4m3", [False, True])
def test_bound_above_the_lengths_changes_nothing(e4m3):
    """max_len bounds the lengths, however far below it they are."""
    p = Pool(53, 2, [3, 700, 129], 16, e4m3, more=1)
    p2 = torch.full((3, 9000), -5, dtype=torch.int32, device=DEV)
    p2[:, :p.tab.shape[1]] = p.t["table"]
    q, k, v, o, lse = check_attend(p, 4)
    p.t["table"] = p2
    p.make()
    for most in (701, 5000, 9000 * 16):
        _, _, _, o2, lse2 = attend(p, 4, max_len=most, q=q, k=k, v=v)
        assert p.status() == 0
        for u in range(p.U):
            n = p.lens[u // 2] + 1
            ro, rl, bo, bl = R.attend(f64(q[u]), p.held("K", u, range(n)), p.held("V", u, range(n)))
            assert (np.abs(f64(o2[u]) - ro) <= bo).all() and (np.abs(f64(lse2[u]) - rl) <= bl).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,lens", [(8, [131071]), (1, [60001]), (8, [20000, 9, 0]), (8, [4000, 3999] * 40),
                                    (1, [700] * 700), (4, [511] * 456), (4, [640] * 456), (4, [511] * 457),
                                    (4, [300, 17] * 456), (4, [300] * 913), (2, [200, 3, 126] * 608), (2, [100] * 1824),
                                    (2, [0] * 500), (4, [513, 0]), (8, [4094, 100, 0, 2049] * 2), (1, [4095]),
                                    (4, [8190, 1]), (4, [10239, 1]), (4, [10241, 1]), (2, [5119, 60]), (2, [5121, 60]), (2, [1023, 7] * 16), (8, [30, 40]),
                                    (4, [70000] + [5, 0, 33] * 100), (1, [1] * 700 + [40000, 3000]),
                                    (4, [260] * 77), (4, [1023, 300, 0] * 50)])
def test_attend_every_way_the_work_is_cut(e4m3, G, lens):
    """One unit over all warps, units of many and of few parts, whole units in clusters of every
    size, up to the number and the length that go so and one more, empty units only."""
    p = Pool(len(lens) + G, 1, lens, 64 if max(lens) > 1000 else 16, e4m3, more=1)
    some = sorted({0, 1, len(lens) // 2, len(lens) - 2, len(lens) - 1} & set(range(len(lens))))
    # (a long unit among many short ones is joined by a block)
    check_attend(p, G, units=some)
    check_attend(p, G, append=False, units=some)


@pytest.mark.parametrize("e4m3", [False, True])
def test_every_sequence_refused(e4m3):
    for n in (20, 5000):
        p = Pool(67, 2, [n, n], 16, e4m3, more=1)
        p.t["len"].fill_(n + 1)
        _, _, _, o, lse = attend(p, 4, max_len=n + 1)
        assert p.status() == 2 and (o == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_long_unit_of_zeros(e4m3):
    """Values (and then keys) of zeros, whose e4m3 scale is the least there is: the sums stay in range."""
    p = Pool(69, 1, [100000, 3], 128, e4m3, more=1, v_scale=0.0)
    check_attend(p, 4, v=torch.zeros(2, D, dtype=torch.bfloat16, device=DEV),
                 k=bf(p.rng.standard_normal((2, D))).to(DEV))
    p = Pool(70, 1, [100000, 3], 128, e4m3, more=1, v_scale=0.0, k_scale=0.0)
    check_attend(p, 4)


@pytest.mark.parametrize("e4m3", [False, True])
def test_same_call_same_bits(e4m3):
    p = Pool(59, 2, [9000, 100, 33], 16, e4m3, more=1)
    q, k, v, o, lse = attend(p, 4)
    for _ in range(5):
        _, _, _, o2, lse2 = attend(p, 4, q=q, k=k, v=v)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_shared_pages():
    """Sequences may share the pages of a common prefix."""
    p = Pool(61, 2, [64, 64], 16, True, more=1)
    p.tab[1, :4] = p.tab[0, :4]
    p.t["table"].copy_(torch.from_numpy(p.tab))
    check_attend(p, 4)


@pytest.mark.parametrize("e4m3", [False, True])
def test_pool_past_2_31_bytes(e4m3):
    """Rows at the end of a pool of more than 2^31 bytes (and elements)."""
    heads, page = 8, 128
    n_pages = (1 << 31) // (heads * page * D) + 40
    K_, V_ = (torch.zeros(n_pages, heads, page, D, device=DEV,
                          dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16) for _ in range(2))
    ks, vs = ((torch.full((n_pages, heads, page), 1.0, device=DEV) for _ in range(2)) if e4m3
              else (None, None))
    lens = [200, 129]
    tab = torch.full((2, 4), -1, dtype=torch.int32)
    tab[0, :2], tab[1, :2] = torch.tensor([n_pages - 1, 3]), torch.tensor([n_pages - 7, n_pages - 2])
    pg = K.make_pages(K_, V_, ks, vs, tab.to(DEV), i32([0, 0]))
    ws = torch.zeros(K.kvc_page_workspace_size(pg, 4), dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(67)
    k, v = (bf(rng.standard_normal((16, 200, D))).to(DEV) for _ in range(2))
    K.kvc_page_write(pg, None, i32(lens), k, v, ws)
    pg.keep[5].copy_(i32(lens))
    ko, vo = (torch.zeros(16, 200, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    K.kvc_page_read(pg, None, None, ko, vo, ws)
    q = bf(rng.standard_normal((16, 4, D))).to(DEV)
    o, lse = torch.zeros(16, 4, D, dtype=torch.bfloat16, device=DEV), torch.zeros(16, 4, device=DEV)
    kn, vn = (bf(rng.standard_normal((16, D))).to(DEV) for _ in range(2))
    K.kvc_page_attend(pg, 201, q, kn, vn, o, lse, ws)
    assert K.kvc_get_device_status(ws) == 0
    for u in range(16):
        n = lens[u // 8]
        rows = []
        for x, new, out in ((k, kn, ko), (v, vn, vo)):
            y = np.concatenate([f64(x[u, :n]), f64(new[u])[None]])
            if e4m3:
                val, sc = R.quantise(y)
                y = f64(val) * sc.astype(np.float64)[:, None]
            rows.append(y)
            assert np.array_equal(f64(out[u, :n]), f64(bf(y[:n])))
            assert (out[u, n:] == 0).all()
        ro, rl, bo, bl = R.attend(f64(q[u]), *rows)
        assert (np.abs(f64(o[u]) - ro) <= bo).all() and (np.abs(f64(lse[u]) - rl) <= bl).all()


# ---------------------------------------------------------------------- write, read

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,page", [(1, 16), (4, 16), (2, 64), (1, 128)])
@pytest.mark.parametrize("T", [1, 6, 37, 300])
def test_write_then_read(e4m3, heads, page, T):
    firsts, counts = [0, 5, 16, 31, 100], [T, T, max(0, T - 1), 0, T // 2]
    p = Pool(71 + T, heads, firsts, page, e4m3, more=T)
    before = p.bits()
    k, v = (bf(p.rng.standard_normal((p.U, T, D)) * np.exp(3 * p.rng.standard_normal((p.U, T, 1))))
            for _ in range(2))
    k[0, 0], v[p.U - 1, 0] = 0.0, 0.0                      # a row of zeros
    k[0, T - 1, 3], v[0, 0] = -3e38, 1e-40                 # the largest, subnormal
    K.kvc_page_write(p.pages, p.t["len"], i32(counts), k.to(DEV), v.to(DEV), p.ws)
    assert p.status() == 0
    written = torch.zeros(p.n_pages, heads, page, dtype=torch.bool)
    for u in range(p.U):
        s, h = u // heads, u % heads
        for t in range(counts[s]):
            at = (int(p.tab[s, (firsts[s] + t) // page]), h, (firsts[s] + t) % page)
            written[at] = True
    for name, x in (("K", k), ("V", v)):
        for u in range(p.U):
            s = u // heads
            if not counts[s]:
                continue
            row = f64(x[u, :counts[s]])
            if e4m3:
                val, sc = R.quantise(row)
                row = f64(val) * sc.astype(np.float64)[:, None]
            got = p.held(name, u, range(firsts[s], firsts[s] + counts[s]))
            assert np.array_equal(got, row), (name, u)
    for a, b in zip(before, p.bits()):                     # everything else as it was
        if a is not None:
            a, b = a.cpu(), b.cpu()
            keep = ~written if a.dim() == 3 else ~written.unsqueeze(-1).expand_as(a)
            assert torch.equal(a[keep], b[keep])
    # read back: whole, and lists in any order with repeats
    p.t["len"].add_(i32(counts))
    n = [f + c for f, c in zip(firsts, counts)]
    for m, lists in ((max(n), False), (50, True)):
        ld = m + 3
        ko, vo = (torch.full((p.U, ld, D), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        slots = cnt = None
        if lists:
            cnt = [0 if n[u // heads] == 0 else int(p.rng.integers(0, m + 1)) for u in range(p.U)]
            slots = np.full((p.U, m), -9, np.int32)
            for u in range(p.U):
                slots[u, :cnt[u]] = p.rng.integers(0, max(1, n[u // heads]), cnt[u])
        K.kvc_page_read(p.pages, None if slots is None else i32(slots.tolist()),
                        None if cnt is None else i32(cnt), ko, vo, p.ws, M=m)
        assert p.status() == 0
        for name, out in (("K", ko), ("V", vo)):
            for u in range(p.U):
                c = cnt[u] if lists else n[u // heads]
                at = slots[u, :c] if lists else range(c)
                if c:
                    want = f64(bf(p.held(name, u, at)))
                    assert np.array_equal(f64(out[u, :c]), want), (name, u)
                assert (out[u, c:] == 5).all()


def test_read_of_a_row_rounds_once():
    """value * scale has up to 28 bits: the product is exact in fp64, fp32 rounds it, bf16 again; the
    definition is the product in fp32, as torch forms it."""
    p = Pool(73, 1, [4000], 16, True)
    val = p.t["K"].float() * p.scale["K"].unsqueeze(-1)
    ko, vo = (torch.zeros(1, 4000, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    K.kvc_page_read(p.pages, None, None, ko, vo, p.ws)
    i = torch.arange(4000, device=DEV)
    want = val[p.t["table"][0][i // 16].long(), 0, i % 16].to(torch.bfloat16)
    assert torch.equal(ko[0], want)


@pytest.mark.parametrize("e4m3", [False, True])
def test_write_defaults(e4m3):
    """first and count NULL: slot 0 on, T rows."""
    p = Pool(79, 2, [0, 0], 16, e4m3, more=40)
    k, v = (bf(p.rng.standard_normal((4, 40, D))).to(DEV) for _ in range(2))
    K.kvc_page_write(p.pages, None, None, k, v, p.ws)
    p.t["len"].fill_(40)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    K.kvc_page_read(p.pages, None, None, ko, vo, p.ws)
    assert p.status() == 0
    for x, out in ((k, ko), (v, vo)):
        row = f64(x)
        if e4m3:
            val, sc = R.quantise(row)
            row = f64(bf(f64(val) * sc.astype(np.float64)[..., None]))
        assert np.array_equal(f64(out), row)


@pytest.mark.parametrize("e4m3", [False, True])
def test_write_refusals(e4m3):
    for bad, code in (((-1, 5), 2), ((0, 41), 2), ((1 << 30, 5), 2), ((-3, 3), 2), ((2147483647, 40), 2)):
        p = Pool(83, 2, [0, 0, 0], 16, e4m3, more=40)
        first, count = i32([0, bad[0], 2]), i32([40, bad[1], 30])
        if bad == (-1, 5):
            first, count = i32([0, 0, 2]), i32([40, -1, 30])
        before = p.held("K", 2, range(40)).copy()
        k, v = (bf(p.rng.standard_normal((6, 40, D))).to(DEV) for _ in range(2))
        K.kvc_page_write(p.pages, first, count, k, v, p.ws)
        assert p.status() == code, bad
        assert np.array_equal(p.held("K", 2, range(40)), before, equal_nan=True)
        for u, f, c in ((0, 0, 40), (1, 0, 40), (4, 2, 30), (5, 2, 30)):
            row = f64(k[u, :c])
            if e4m3:
                val, sc = R.quantise(row)
                row = f64(val) * sc.astype(np.float64)[:, None]
            assert np.array_equal(p.held("K", u, range(f, f + c)), row)
    p = Pool(89, 1, [0], 16, e4m3, more=40)
    p.t["table"][0, 1] = p.n_pages
    K.kvc_page_write(p.pages, None, None, k[:1], v[:1], p.ws)
    assert p.status() == 1
    assert not np.isnan(p.held("V", 0, list(range(16)) + list(range(32, 40)))).any()


def test_read_refusals():
    p = Pool(97, 1, [50, 50, 50], 16, True)
    slots = torch.arange(20, dtype=torch.int32, device=DEV).repeat(3, 1)
    for what, code in (("count", 2), ("negative", 2), ("slot", 2), ("below", 2), ("page", 1)):
        s, c = slots.clone(), i32([20, 20, 20])
        p.t["table"].copy_(torch.from_numpy(p.tab))
        if what == "count":
            c[1] = 21
        elif what == "negative":
            c[1] = -1
        elif what == "slot":
            s[1, 4] = 50
        elif what == "below":
            s[1, 4] = -1
        else:
            p.t["table"][1, 0] = -1
        ko, vo = (torch.full((3, 20, D), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        K.kvc_page_read(p.pages, s, c, ko, vo, p.ws)
        assert p.status() == code and p.status() == 0
        left = {"count": range(20), "negative": range(20), "slot": [4], "below": [4], "page": range(16)}[what]
        for u in range(3):
            for i in range(20):
                untouched = bool((ko[u, i] == 5).all())
                assert untouched == (u == 1 and i in left), (what, u, i)


# ---------------------------------------------------------------------- norms and rotation

def rope_case(seed, B, T, Hkv, G, rot=128, interleaved=False, normed=(True, True), units=None,
              first_unit=0, n=None, row=None, scale=1.0, far=5000, base=1e6, eps=1e-6, x_scale=2.0,
              pos=None, live=("q", "k", "v")):
    rng = np.random.default_rng(seed)
    heads = Hkv * (G + 2)
    row = row or heads * D
    x = np.full((B, T, row), NAN)
    x[..., :heads * D] = x_scale * rng.standard_normal((B, T, heads * D))
    for b in range(B):
        if n is not None:
            x[b, n[b]:] = NAN
    qkv = bf(x).to(DEV)
    x = f64(qkv)
    pos = rng.integers(0, far, (B, T)) if pos is None else np.asarray(pos).reshape(B, T)
    qw, kw = (bf(1 + 0.3 * rng.standard_normal(D)).to(DEV) if on else None for on in normed)
    f = base ** (-2.0 * np.arange(rot // 2) / rot) if rot else None
    freq = None if f is None else torch.from_numpy(f).to(DEV)
    units = units or Hkv
    r = K.make_rope(Hkv * G, Hkv, freq, qw, kw, eps=eps, interleaved=interleaved, scale=scale,
                    units=units, first_unit=first_unit)
    U = B * units
    out = {"q": torch.full((U, T, G, D), 5.0, dtype=torch.bfloat16, device=DEV),
           "k": torch.full((U, T, D), 5.0, dtype=torch.bfloat16, device=DEV),
           "v": torch.full((U, T, D), 5.0, dtype=torch.bfloat16, device=DEV)}
    K.kvc_qk_norm_rope(r, qkv, i32(pos.tolist()), None if n is None else i32(n),
                       *(out[name] if name in live else None for name in ("q", "k", "v")))
    got = {name: f64(t) for name, t in out.items()}
    eps = float(np.float32(eps))
    scale = float(np.float32(scale))
    fr = [] if f is None else f
    for u in range(U):
        b, g = u // units, u % units - first_unit
        mine = 0 <= g < Hkv
        for t in range(T):
            alive = mine and (n is None or t < n[b])
            for name, heads_of in (("q", range(G)), ("k", [0]), ("v", [0])):
                for j in heads_of:
                    have = got[name][u, t, j] if name == "q" else got[name][u, t]
                    if not alive or name not in live:
                        assert (have == 5).all(), (name, u, t)
                        continue
                    at = {"q": g * G + j, "k": Hkv * G + g, "v": Hkv * (G + 1) + g}[name]
                    src = x[b, t, at * D:(at + 1) * D]
                    if name == "v":
                        assert np.array_equal(have, src)
                        continue
                    w = qw if name == "q" else kw
                    want, bound = R.norm_rope(src, None if w is None else f64(w), int(pos[b, t]), fr, eps,
                                              interleaved, scale)
                    bound = bound + R.BF * np.abs(want) + 1e-37
                    assert (np.abs(have - want) <= bound).all(), (name, u, t, j,
                                                                  np.abs(have - want).max(), bound.max())


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_rope_head_layouts(G, Hkv):
    rope_case(G * 10 + Hkv, 2, 3, Hkv, G)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32, 48, 96, 112, 128])
@pytest.mark.parametrize("normed", [(True, True), (False, False), (True, False), (False, True)])
def test_rope_forms(interleaved, rot, normed):
    rope_case(rot + 3, 1, 4, 2, 2, rot=rot, interleaved=interleaved, normed=normed)


@pytest.mark.parametrize("B,T", [(1, 1), (5, 1), (1, 7), (3, 25), (2, 130)])
def test_rope_tokens(B, T):
    rope_case(B * T, B, T, 2, 2, n=[max(0, T - 3 * b) for b in range(B)] if B > 1 else None)


def test_rope_many_tokens():
    """Enough tokens that the work is cut the other way."""
    B, T, Hkv, G = 3, 1700, 1, 1
    rope_case(17, B, T, Hkv, G, n=[1700, 1699, 1], rot=64)


@pytest.mark.parametrize("Hkv,G,B,T", [(1, 1, 2, 1100), (1, 4, 1, 2100), (8, 1, 1, 1030), (2, 8, 3, 700)])
def test_rope_tiles_of_every_size(Hkv, G, B, T):
    """Tiles of 16, 8 and 4 tokens, more of them than blocks and a last one that is not full: every
    row against a call of single tokens, which has tiles of 4, and some against the definition."""
    rng = np.random.default_rng(T)
    x = bf(2 * rng.standard_normal((B, T, Hkv * (G + 2) * D))).to(DEV)
    w = bf(1 + 0.3 * rng.standard_normal(D)).to(DEV)
    f = torch.from_numpy(1e4 ** (-np.arange(64) / 64)).to(DEV)
    r = K.make_rope(Hkv * G, Hkv, f, w, w)
    pos = i32(rng.integers(0, 5000, (B, T)).tolist())
    big, small = ([torch.zeros(B * Hkv, T, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((G,), (), ())]
                  for _ in range(2))
    K.kvc_qk_norm_rope(r, x, pos, None, *big)
    step = 100
    for b in range(B):
        for t in range(0, T, step):
            m = min(step, T - t)
            part = [torch.zeros(Hkv, m, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((G,), (), ())]
            K.kvc_qk_norm_rope(r, x[b:b + 1, t:t + m], pos[b:b + 1, t:t + m].contiguous(), None, *part)
            for a, p in zip(small, part):
                a[b * Hkv:(b + 1) * Hkv, t:t + m] = p
    for a, b in zip(big, small):
        assert torch.equal(a, b)
    for t in (0, T // 2, T - 1):
        for name, at, out in (("q", 0, big[0][(B - 1) * Hkv, t, 0]), ("k", Hkv * G, big[1][(B - 1) * Hkv, t])):
            want, bound = R.norm_rope(f64(x[B - 1, t, at * D:(at + 1) * D]), f64(w), int(pos[B - 1, t]),
                                      f.cpu().tolist(), float(np.float32(1e-6)), False, 1.0)
            assert (np.abs(f64(out) - want) <= bound + R.BF * np.abs(want)).all(), (name, t)


def test_rope_positions():
    far = [0, 1, -1, -7, 1000003, 2 ** 20, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 131071]
    rope_case(5, 1, len(far), 1, 2, pos=far)
    rope_case(6, 1, len(far), 1, 2, pos=far, interleaved=True, base=1e4, rot=64, scale=1.25)


def test_rope_frequencies_of_any_size():
    """Frequencies above a turn per position, negative and zero ones."""
    qkv = bf(np.random.default_rng(3).standard_normal((1, 4, 3 * D))).to(DEV)
    f = np.array([0.0, -0.5, 7.5, 100.25, 1e-9, 6.283185307179586, 1.0, -123.456])
    r = K.make_rope(1, 1, torch.from_numpy(f).to(DEV))
    q, k, v = (torch.zeros(1, 4, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((1,), (), ()))
    pos = [0, 3, 999, -12345]
    K.kvc_qk_norm_rope(r, qkv, i32([pos]), None, q, k, v)
    for t in range(4):
        for j, out in ((0, q[0, t, 0]), (1, k[0, t])):
            want, bound = R.norm_rope(f64(qkv[0, t, j * D:(j + 1) * D]), None, pos[t], f, 0, False, 1.0)
            assert (np.abs(f64(out) - want) <= bound + R.BF * np.abs(want)).all()


@pytest.mark.parametrize("kw", [dict(units=12, first_unit=5), dict(units=12, first_unit=8, n=[3, 0]),
                                dict(row=7 * D * 4 + 8), dict(x_scale=1e-12), dict(x_scale=1e15),
                                dict(eps=0.0), dict(live=("q",)), dict(live=("k", "v")), dict(live=("v",))])
def test_rope_layouts_and_magnitudes(kw):
    rope_case(23, 2, 3, 4, 2, **kw)


def test_rope_rows_further_apart():
    """A slice of wider rows, whose neighbours are NaN, and a row of zeros."""
    wide = torch.full((2, 3, 5 * D), NAN, dtype=torch.bfloat16, device=DEV)
    x = bf(np.random.default_rng(1).standard_normal((2, 3, 3 * D))).to(DEV)
    x[0, 0] = 0
    wide[..., D:4 * D] = x
    w = bf(np.ones(D)).to(DEV)
    f = torch.from_numpy(1e4 ** (-np.arange(64) / 64)).to(DEV)
    r = K.make_rope(1, 1, f, w, w)
    outs = []
    for src in (x, wide[..., D:4 * D]):
        q, k, v = (torch.zeros(2, 3, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((1,), (), ()))
        K.kvc_qk_norm_rope(r, src, i32([[0, 1, 2], [7, 8, 9]]), None, q, k, v)
        outs.append((q, k, v))
    for a, b in zip(*outs):
        assert torch.equal(a, b) and not a.isnan().any()
    with pytest.raises(ValueError):
        K.kvc_qk_norm_rope(r, wide[..., :2 * D], i32([[0, 1, 2], [7, 8, 9]]), None, q, k, v)
    with pytest.raises(ValueError):
        K.kvc_qk_norm_rope(r, wide.transpose(0, 1), i32([[0, 1, 2], [7, 8, 9]]), None, q, k, v)
    with pytest.raises(ValueError):
        K.kvc_qk_norm_rope(r, wide[:, :2], i32([[0, 1], [7, 8]]), None, q, k, v)
    with pytest.raises(ValueError):
        K.kvc_qk_norm_rope(r, x[0], i32([[0, 1, 2]]), None, q, k, v)
    # one token each of sequences further apart, and one token alone
    for src, at in ((wide[:, 1:2, D:4 * D], [[1], [8]]), (wide[1:, 1:2, D:4 * D], [[8]])):
        B = len(at)
        q1, k1, v1 = (torch.zeros(B, 1, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((1,), (), ()))
        K.kvc_qk_norm_rope(r, src, i32(at), None, q1, k1, v1)
        for have, all_ in ((q1, q), (k1, k), (v1, v)):
            assert torch.equal(have[:, 0], all_[2 - B:, 1])


# ---------------------------------------------------------------------- together

def _step_inputs(rng, B, T, Hkv, G):
    return bf(1.5 * rng.standard_normal((B, T, Hkv * (G + 2) * D))).to(DEV)


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_steps_and_selection(e4m3):
    """Projection rows -> norms and rotation -> pages; steps over the pages; the kept rows go to the
    budgeted cache, whose steps go on.  In bf16 the budgeted cache's first step gives what a cache
    filled without pages gives, to the bit."""
    rng = np.random.default_rng(101)
    B, Hkv, G, L, cap = 3, 2, 4, 40, 48
    U, lens = B * Hkv, [150, 97, 41]
    w = bf(1 + 0.2 * rng.standard_normal(D)).to(DEV)
    f = torch.from_numpy(1e6 ** (-np.arange(64) / 64)).to(DEV)
    r = K.make_rope(Hkv * G, Hkv, f, w, w)
    T = max(lens)
    st = PagedState(B, Hkv, G, 200, page=16, e4m3=e4m3, n_pages=33)
    with pytest.raises(RuntimeError):
        st.reserve([200, 200, 200])
    st.reserve(lens)
    q, k, v = (torch.zeros(U, T, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((G,), (), ()))
    pos = torch.arange(T, dtype=torch.int32, device=DEV).repeat(B, 1)
    K.kvc_qk_norm_rope(r, _step_inputs(rng, B, T, Hkv, G), pos, i32(lens), q, k, v)
    st.write(k, v, i32(lens))
    held = [(f64(k[u, :lens[u // Hkv]]), f64(v[u, :lens[u // Hkv]])) for u in range(U)]

    def store(x):
        if not e4m3:
            return x
        val, sc = R.quantise(x)
        return f64(val) * sc.astype(np.float64)[:, None]

    held = [[store(a), store(b)] for a, b in held]
    n = list(lens)
    for step in range(4):
        st.reserve([x + 1 for x in n])
        qs, ks, vs = (torch.zeros(U, 1, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((G,), (), ()))
        K.kvc_qk_norm_rope(r, _step_inputs(rng, B, 1, Hkv, G), i32([[x] for x in n]), None, qs, ks, vs)
        n = [x + 1 for x in n]
        o, lse = st.step(qs.view(U, G, D), ks.view(U, D), vs.view(U, D), max(n))
        for u in range(U):
            for i, x in enumerate((ks, vs)):
                held[u][i] = np.concatenate([held[u][i], store(f64(x[u]))])
            ro, rl, bo, bl = R.attend(f64(qs[u, 0]), *held[u])
            assert (np.abs(f64(o[u]) - ro) <= bo).all() and (np.abs(f64(lse[u]) - rl) <= bl).all()
    assert st.status() == 0 and st.len.tolist() == n
    # the whole of it
    k2, v2 = st.read(max(n))
    for u in range(U):
        m = n[u // Hkv]
        assert np.array_equal(f64(k2[u, :m]), f64(bf(held[u][0]))) and (k2[u, m:] == 0).all()
        assert np.array_equal(f64(v2[u, :m]), f64(bf(held[u][1])))
    # a selection, to the budgeted cache
    slots = np.stack([np.sort(rng.permutation(n[u // Hkv])[:L]) for u in range(U)]).astype(np.int32)
    outs = []
    for way in ("pages", "direct"):
        ds = DecodeState(U, G, cap, L, rule=K.RULE_CUMULATIVE)
        if way == "pages":
            st.hand_over(ds, i32(slots.tolist()), i32([L] * U))
        else:
            idx = torch.from_numpy(slots).long().to(DEV).unsqueeze(-1).expand(-1, -1, D)
            ds.load_prefill(torch.gather(k2, 1, idx), torch.gather(v2, 1, idx), None, i32(slots.tolist()),
                            i32([L] * U))
        for t in range(1, 4):
            gen = torch.Generator(device=DEV).manual_seed(t)
            qn, kn, vn = (torch.randn(*s, generator=gen, device=DEV).bfloat16()
                          for s in ((U, G, D), (U, D), (U, D)))
            ds.step(t, 500 + t, qn, kn, vn, L + 1)
        assert ds.device_status() == 0
        outs.append([ds.o, ds.len, ds.K[:, :L], ds.pos[:, :L], ds.util[:, :L], ds.C])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert st.status() == 0
    # a sequence ends, another takes its pages
    st.release(-1)
    assert st.len.tolist()[-1] == 0 and (st.table[-1] == -1).all()
    st.reserve([n[0], n[1], 3])
    st.release(0)
    assert st.len.tolist()[0] == 0
    st.reserve([120, n[1], n[2]])
    assert len({int(x) for x in st.table.flatten() if x >= 0}) == int((st.table >= 0).sum())


def test_drafted_tokens_take_the_layouts():
    """Trees of drafted tokens: normed and rotated rows go to verify as they are."""
    rng = np.random.default_rng(103)
    B, Hkv, G, T, L = 2, 2, 4, 5, 60
    U = B * Hkv
    r = K.make_rope(Hkv * G, Hkv, torch.from_numpy(1e4 ** (-np.arange(64) / 64)).to(DEV))
    q, k, v = (torch.zeros(U, T, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((G,), (), ()))
    qkv = _step_inputs(rng, B, T, Hkv, G)
    K.kvc_qk_norm_rope(r, qkv, i32([[L + i for i in range(T)]] * B), None, q, k, v)
    st = DecodeState(U, G, L + 10, L)
    st.load_prefill(*(bf(rng.standard_normal((U, L, D))).to(DEV) for _ in range(2)), None,
                    torch.arange(L, dtype=torch.int32, device=DEV).repeat(U, 1), i32([L] * U))
    tree = K.make_tree(T, Hkv, torch.tensor([[1, 3, 7, 15, 31]] * B, device=DEV))
    o, lse = st.verify(tree, q, k, v, L)
    assert st.tree_status() == 0
    # the last of the chain sees everything: the same as one token over pages of the same rows
    ps = PagedState(B, Hkv, G, 80, page=16, e4m3=False)
    ps.reserve([L + T] * B)
    ps.write(st.K[:, :L].contiguous(), st.V[:, :L].contiguous())
    ps.write(k[:, :T - 1].contiguous(), v[:, :T - 1].contiguous())
    o1, lse1 = ps.step(q[:, T - 1].contiguous(), k[:, T - 1].contiguous(), v[:, T - 1].contiguous(), L + T)
    for u in range(U):
        rows = [torch.cat([a[u, :L], b[u]]) for a, b in ((st.K, k), (st.V, v))]
        ro, rl, bo, bl = R.attend(f64(q[u, T - 1]), *(f64(x) for x in rows))
        assert (np.abs(f64(o1[u]) - ro) <= bo).all() and (np.abs(f64(lse1[u]) - rl) <= bl).all()
        # the tree's weights are bf16: each off by 2^-8 of itself at most, and they sum to one
        assert (np.abs(f64(o[u, T - 1]) - ro) <= bo + R.BF * f64(rows[1].abs()).max()).all()
        assert (np.abs(f64(lse[u, T - 1]) - rl) <= bl).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_graph_advances_with_the_lengths(e4m3):
    """One captured step (rotation, append, attention, lengths) replayed gives what calls give."""
    rng = np.random.default_rng(107)
    B, Hkv, G, n0, steps = 2, 2, 4, 1000, 20
    U = B * Hkv
    r = K.make_rope(Hkv * G, Hkv, torch.from_numpy(1e4 ** (-np.arange(64) / 64)).to(DEV))
    kp, vp = (bf(rng.standard_normal((U, n0, D))).to(DEV) for _ in range(2))
    inputs = [_step_inputs(rng, B, 1, Hkv, G) for _ in range(steps)]
    outs = []
    for graphed in (False, True):
        st = PagedState(B, Hkv, G, 1100, page=16, e4m3=e4m3)
        st.reserve([n0 + steps] * B)
        st.write(kp, vp)
        x = torch.zeros_like(inputs[0])
        q, k, v = (torch.zeros(U, 1, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((G,), (), ()))

        def call():
            K.kvc_qk_norm_rope(r, x, st.len.view(B, 1), None, q, k, v)
            st.step(q.view(U, G, D), k.view(U, D), v.view(U, D), n0 + steps)
        if graphed:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                call()
        got = []
        for i in range(steps):
            x.copy_(inputs[i])
            g.replay() if graphed else call()
            got.append((st.o.clone(), st.lse.clone()))
        assert st.status() == 0 and st.len.tolist() == [n0 + steps] * B
        outs.append(got)
    for (a, b), (c, d) in zip(*outs):
        assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("e4m3", [False, True])
def test_write_and_read_in_a_graph(e4m3):
    """Captured on a side stream and replayed with other rows, places and counts."""
    p = Pool(108, 2, [0, 0], 16, e4m3, more=90)
    k, v = (torch.zeros(4, 40, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ko, vo = (torch.zeros(4, 90, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    count, s = i32([40, 40]), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        K.kvc_page_write(p.pages, p.t["len"], count, k, v, p.ws)
        p.t["len"].add_(count)
        K.kvc_page_read(p.pages, None, None, ko, vo, p.ws)
    held = [[np.zeros((0, D)), np.zeros((0, D))] for _ in range(4)]
    for counts in ([40, 3], [0, 40], [17, 1]):
        count.copy_(i32(counts))
        for i, x in enumerate((k, v)):
            x.copy_(bf(p.rng.standard_normal((4, 40, D))))
            for u in range(4):
                row = f64(x[u, :counts[u // 2]])
                if e4m3 and len(row):
                    val, sc = R.quantise(row)
                    row = f64(bf(f64(val) * sc.astype(np.float64)[:, None]))
                held[u][i] = np.concatenate([held[u][i], row])
        g.replay()
        for u in range(4):
            n = len(held[u][0])
            assert np.array_equal(f64(ko[u, :n]), held[u][0]) and np.array_equal(f64(vo[u, :n]), held[u][1])
    assert p.status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_two_graphs_share_a_workspace(e4m3):
    """Calls of different sizes captured with one workspace, replayed in turn and out of turn."""
    ps = [Pool(109 + i, h, lens, 16, e4m3, more=1) for i, (h, lens) in enumerate(
        (((2, [9000, 700])), (1, [40, 3, 5000, 600, 1]), (4, [300])))]
    ws = torch.zeros(max(p.ws.numel() for p in ps), dtype=torch.uint8, device=DEV)
    graphs, want = [], []
    for p in ps:
        p.ws = ws
        q, k, v, o, lse = check_attend(p, 4)
        o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            attend(p, 4, q=q, k=k, v=v, o=o2, lse=lse2)
        graphs.append(g)
        want.append((o, lse, o2, lse2, q, k, v))       # the graph reads q, k, v again
    for i in (0, 1, 2, 2, 0, 1, 0):
        want[i][2].zero_()
        graphs[i].replay()
        assert torch.equal(want[i][0], want[i][2]) and torch.equal(want[i][1], want[i][3]), i


def test_streams_and_threads():
    """Calls of several host threads, each with a stream, a cache and a workspace of its own."""
    ps = [Pool(113 + i, 2, [900 + 50 * i, 30], 16, bool(i % 2), more=1) for i in range(4)]
    want = [check_attend(p, 4) for p in ps]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            q, k, v, o, lse = want[i]
            with torch.cuda.stream(s):
                for _ in range(20):
                    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
                    K.kvc_page_attend(ps[i].pages, 1200, q, k, v, o2, lse2, ps[i].ws)
                    K.kvc_page_attend(ps[i].pages, max(ps[i].lens) + 1, q, k, v, o2, lse2, ps[i].ws,
                                      stream=s)
                    s.synchronize()
                    if not (torch.equal(o, o2) and torch.equal(lse, lse2)):
                        bad.append(i)
        except Exception as e:                                 # noqa: BLE001
            bad.append(e)

    for p in ps:                                               # room for a bound of 1200
        t = torch.full((2, 80), -1, dtype=torch.int32, device=DEV)
        t[:, :p.tab.shape[1]] = p.t["table"]
        p.t["table"] = t
        p.make()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad, bad


def test_calls_of_another_stream_overlap_nothing():
    """A call on a side stream behind an event, its outputs read there."""
    p = Pool(127, 2, [5000, 64], 64, True, more=1)
    q, k, v, o, lse = check_attend(p, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    s.wait_stream(torch.cuda.current_stream())
    K.kvc_page_attend(p.pages, 5001, q, k, v, o2, lse2, p.ws, stream=s)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_workspace_too_small_is_refused():
    p = Pool(131, 2, [5000, 64], 64, True, more=1)
    need = K.kvc_page_workspace_size(p.pages, 4)
    q, k, v, o, lse = check_attend(p, 4)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    with pytest.raises(K.KvcError):
        K.kvc_page_attend(p.pages, 5001, q, k, v, o, lse, ws[:need - 256])


def test_binding_checks():
    p = Pool(137, 2, [50], 16, True, more=1)
    q, k, v, o, lse = check_attend(p, 4)
    for args in ((q[:1], k, v, o, lse), (q, k[:1], v, o, lse), (q, k, v, o[:1], lse), (q, k, v, o, lse[:1]),
                 (q.float(), k, v, o, lse), (q, None, v[:1], o, lse), (q.transpose(1, 2), k, v, o, lse)):
        with pytest.raises((ValueError, TypeError)):
            K.kvc_page_attend(p.pages, 51, *args, p.ws)
    with pytest.raises(K.KvcError):
        K.kvc_page_attend(p.pages, 51, q, None, v, o, lse, p.ws)
    with pytest.raises(ValueError):
        K.kvc_page_write(p.pages, None, i32([1, 1])[:0], k.view(2, 1, D), v.view(2, 1, D), p.ws)
    with pytest.raises(ValueError):
        K.kvc_page_read(p.pages, i32([[1]]), None, k.view(2, 1, D), v.view(2, 1, D), p.ws)
    assert p.status() == 0
