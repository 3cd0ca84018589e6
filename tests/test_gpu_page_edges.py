"""GPU tests of the cache in pages, and of the norms and rotation in front of it,
where the numbers are at an edge: contributions far apart, values that are not
finite or near the ends of fp32, lengths at which a tile could be lost, places of
a batch that are free.  Against the definitions in 64 bits (page_ref.py)."""
import numpy as np
import pytest
import torch

import page_ref as R
from kv_cache_eviction_kvc_gb300.state import DecodeState, PagedState
from test_gpu_page import DEV, D, NAN, K, Pool, attend, bf, check_attend, f64, i32

pytestmark = pytest.mark.gpu


def put(p, name, u, slots, x):
    """Rows x [len(slots)][D] of a unit of the pool."""
    s, h = u // p.heads, u % p.heads
    slots = np.asarray(slots)
    b = torch.from_numpy(p.tab[s][slots // p.page].astype(np.int64)).to(DEV)
    r = torch.from_numpy(slots % p.page).to(DEV)
    if p.e4m3:
        v, sc = R.quantise(f64(bf(x)))
        p.t[name].view(torch.uint8)[b, h, r] = v.view(torch.uint8).to(DEV)
        p.scale[name][b, h, r] = torch.from_numpy(sc).to(DEV)
    else:
        p.t[name][b, h, r] = bf(x).to(DEV)


def spike(at, width=1):
    """A row of ones in dimensions [at, at + width), zeros elsewhere."""
    x = np.zeros(D)
    x[at:at + width] = 1.0
    return x


# ---------------------------------------------------------------------- contributions far apart

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens", [[200, 40], [2000] * 130])
def test_small_contributions_beside_a_large_one(e4m3, lens):
    """One slot has nearly all of the weight and values in half of the dimensions; the others weigh
    2^-18 to 2^-21 of it and have the other half to themselves, where each of them counts in full."""
    p = Pool(211, 1, lens, 16, e4m3)
    q = p.rng.standard_normal((p.U, 4, D))
    q[:, :, 0] = 4 * np.array([18, 19, 20, 21]) / 18
    b = -18 * np.log(2) * np.sqrt(D) / 4                   # logits of -18 octaves for the first head
    some = [0, 1, p.U - 1]
    for u in range(p.U) if p.U < 10 else some:
        n = p.lens[u]
        at = 5 + 11 * u % (n - 5)
        put(p, "K", u, range(n), np.tile(b * spike(0), (n, 1)))
        put(p, "K", u, [at], np.zeros((1, D)))
        put(p, "V", u, range(n), np.tile(0.8 * spike(64, 64), (n, 1)))
        put(p, "V", u, [at], spike(0, 64)[None])
    check_attend(p, 4, append=False, q=bf(q).to(DEV), units=some)


# ---------------------------------------------------------------------- values that are not finite

def lse_of(q, k):
    """log sum exp of the logits of q [G][D] over k [n][D], and the bound of page_ref.attend."""
    _, lse, _, bl = R.attend(q, k, np.zeros_like(k))
    return lse, bl


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens", [[300, 300, 20], [40000, 3, 700], [500] * 1000])
@pytest.mark.parametrize("bad", [NAN, -NAN, np.inf, -np.inf])
def test_lse_beside_values_that_are_not_finite(e4m3, lens, bad):
    """lse goes by the keys alone: a value row with a NaN or an infinity makes o NaN (in e4m3 the whole
    row is NaN, in bf16 the dimension), and leaves lse and the other units."""
    p = Pool(223, 1, lens, 16, e4m3)
    x = p.rng.standard_normal((1, D))
    x[0, 7] = bad
    put(p, "V", 0, [len(lens) % 7 + 9], x)
    q, _, _, o, lse = attend(p, 4, append=False)
    assert p.status() == 0
    for u in (0, 1, p.U - 1):
        want, bound = lse_of(f64(q[u]), p.held("K", u, range(lens[u])))
        assert (np.abs(f64(lse[u]) - want) <= bound).all(), (u, f64(lse[u]), want)
    assert (o[0].isnan() if e4m3 else ~o[0, :, 7].isfinite()).all()
    assert not o[1:].isnan().any() and (e4m3 or not o[0, :, 8:].isnan().any())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [20, 4000])
def test_lse_with_an_appended_value_that_is_not_finite(e4m3, n):
    p = Pool(227, 1, [n, n, n], 16, e4m3, more=1)
    k, v = (bf(p.rng.standard_normal((3, D))) for _ in range(2))
    v[0, 5], v[1, 5] = NAN, np.inf
    q, _, _, o, lse = attend(p, 2, k=k.to(DEV), v=v.to(DEV))
    assert p.status() == 0
    for u in range(3):
        want, bound = lse_of(f64(q[u]), p.held("K", u, range(n + 1)))
        assert (np.abs(f64(lse[u]) - want) <= bound).all(), (u, f64(lse[u]), want)
    assert not o[0, :, 5].isfinite().any() and not o[1, :, 5].isfinite().any() and o[2].isfinite().all()


# ---------------------------------------------------------------------- values of any magnitude

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("first,then", [(0.0, 1e12), (1e12, 0.0), (1e-30, 1e25), (1e25, 1e-30)])
@pytest.mark.parametrize("lens", [[300, 40], [9000, 70, 700], [600] * 1000, [70000]])
def test_weights_do_not_depend_on_the_order_of_values(e4m3, first, then, lens):
    """A run of slots with small or no values before (behind) one with large ones: all have the same
    weight, in one warp and across parts."""
    p = Pool(229, 1, lens, 16, e4m3)
    some = sorted({0, p.U // 2, p.U - 1})
    for u in some:
        n = lens[u]
        i = np.arange(n)[:, None] >= n // 2
        put(p, "V", u, range(n), np.where(i, then, first) * (1 + p.rng.random((n, D))))
    check_attend(p, 4, append=False, q_scale=0.0, units=some)
    check_attend(p, 4, append=False, q_scale=0.5, units=some)


@pytest.mark.parametrize("lens", [[300, 40], [9000, 70, 700], [600] * 1000])
@pytest.mark.parametrize("v_scale", [1e-36, 1e33, 4e37])
def test_sharp_attention_over_values_near_the_ends_of_fp32(lens, v_scale):
    """Values in e4m3 up to the largest fp32 holds: weights far below the largest count all the same
    (their contributions, and their sum).  The least values are multiples of the least scale."""
    p = Pool(233, 1, lens, 16, True, v_scale=v_scale, k_scale=2.0)
    check_attend(p, 4, append=False, units=sorted({0, p.U // 2, p.U - 1}))
    # one slot 20 octaves above all others, whose values have dimensions to themselves
    n, some = lens[0], [0]
    put(p, "K", 0, range(n), np.tile(-20 * np.log(2) * np.sqrt(D) / 4 * spike(0), (n, 1)))
    put(p, "K", 0, [n // 2], np.zeros((1, D)))
    put(p, "V", 0, range(n), np.tile(v_scale * spike(64, 64), (n, 1)))
    put(p, "V", 0, [n // 2], v_scale * spike(0, 64)[None])
    q = np.zeros((p.U, 4, D))
    q[:, :, 0] = 4
    check_attend(p, 4, append=False, q=bf(q).to(DEV), units=some)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G", [4, 8])
def test_long_sums_are_rounded_not_cut_off(e4m3, G):
    """Equal weights over runs of 8192 slots of values of 1.5 at most, and as many of the same negated: o is 0.
    A sum that grows to 8192 and back is off by half its step (2^-11 at most) in each of 1024 additions
    at most; rounded, these are either way alike, and 8 standard deviations of their sum are
    8 2^-10 sqrt(1024 / 12) over 16384 slots, with parts (sums of 1/2, rounded to 2^-25) joined besides.
    Cut off, they add up to 1024 2^-12 (2^-11 on the average, half of it as the sum grows)."""
    page, runs = 128, 1824
    x = 1 + (np.random.default_rng(5).random((page, D)) - 0.5)
    x[1::2] /= 64                                          # bits below those that sums of the others keep
    p = Pool(239, 1, [page, page], page, e4m3)
    put(p, "V", 0, range(page), x)
    put(p, "V", 1, range(page), x)
    a, b = int(p.tab[0, 0]), int(p.tab[1, 0])
    if e4m3:
        p.t["V"].view(torch.uint8)[b] ^= 128
    else:
        p.t["V"][b].neg_()
    n = runs * 128 * page
    tab = torch.tensor(([a] * 64 + [b] * 64) * runs, dtype=torch.int32, device=DEV).view(1, -1)
    p.t["table"], p.t["len"] = tab, i32([n])
    p.U = 1
    p.make()
    _, _, _, o, lse = attend(p, G, append=False, max_len=n, q_scale=0.0)
    assert p.status() == 0
    assert np.abs(f64(o)).max() <= 8 * 2.0 ** -10 * np.sqrt(1024 / 12) / 16384 + 8 * 2.0 ** -24
    assert np.abs(f64(lse) - np.log(n)).max() <= 8 * 2.0 ** -24 * np.log(n)


# ---------------------------------------------------------------------- logits of any magnitude

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens", [[300, 40], [9000, 70], [600] * 1000])
def test_large_queries_and_keys_that_do_not_meet(e4m3, lens):
    """A query and keys near the ends of fp32 whose products are all zero: every logit is zero."""
    p = Pool(241, 1, lens, 16, e4m3, more=1)
    some = sorted({0, p.U // 2, p.U - 1})
    for u in some:
        put(p, "K", u, range(lens[u]), 3e37 * (1 + p.rng.random((lens[u], 1))) * spike(64, 64))
    q = np.zeros((p.U, 4, D))
    q[:, :, :64] = 1e38 * np.array([1, 2, 3, -3])[:, None]
    k = bf(np.zeros((p.U, D))).to(DEV)
    _, _, _, _, lse = check_attend(p, 4, q=bf(q).to(DEV), units=some, k=k, v=k + 1)
    for u in some:
        assert np.abs(f64(lse[u]) - np.log(lens[u] + 1)).max() <= 8 * 2.0 ** -24 * np.log(lens[u] + 1)


# ---------------------------------------------------------------------- norms and rotation

def rotated(x, w=None, pos=3, rot=128, interleaved=False, eps=1e-6, base=1e4, freq=None):
    """One token's query and key head of x [D] through the call: [2][D], and the frequencies."""
    f = base ** (-2.0 * np.arange(rot // 2) / rot) if rot else None
    f = f if freq is None else np.asarray(freq, dtype=np.float64)
    w = None if w is None else bf(w).to(DEV)
    r = K.make_rope(1, 1, None if f is None else torch.from_numpy(f).to(DEV), w, w, eps=eps,
                    interleaved=interleaved)
    qkv = bf(np.concatenate([x, x, x]))[None, None].to(DEV)
    q, k, v = (torch.zeros(1, 1, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((1,), (), ()))
    K.kvc_qk_norm_rope(r, qkv, i32([[pos]]), None, q, k, v)
    assert torch.equal(v[0, 0].view(torch.int16), qkv[0, 0, 2 * D:].view(torch.int16))
    return f64(torch.stack([q[0, 0, 0], k[0, 0]])), [] if f is None else f


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 32, 64, 112])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("bad", [NAN, np.inf, -np.inf])
def test_rope_of_a_row_that_is_not_finite(interleaved, rot, normed, bad):
    """A dimension that is not turned is its own affair: y = x without a norm; with one, an infinity
    leaves zeros elsewhere (its own place is NaN), a NaN makes the row NaN."""
    rng = np.random.default_rng(rot)
    w = 1 + 0.3 * rng.standard_normal(D) if normed else None
    for at in sorted({rot, rot + 1, rot + 4, 120, 127}):
        x = f64(bf(rng.standard_normal(D)))
        x[at] = bad
        got, f = rotated(x, w, rot=rot, interleaved=interleaved)
        others = np.arange(D) != at
        for y in got:
            if not normed:
                assert np.array_equal(y[at], bad, equal_nan=True)
                clean = np.where(others, x, 0.0)
                want, bound = R.norm_rope(clean, None, 3, f, 1e-6, interleaved, 1.0)
                assert (np.abs(y - want)[others] <= (bound + R.BF * np.abs(want))[others]).all(), at
                assert np.array_equal(y[rot:][others[rot:]], x[rot:][others[rot:]])
            elif np.isnan(bad):
                assert np.isnan(y).all()
            else:
                assert np.isnan(y[at]) and (y[others] == 0).all(), at


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-30, 1e-6])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-23, 1e-20, 1e-16, 1e-3, 1e18])
def test_rope_norm_of_any_magnitude(interleaved, eps, scale):
    """Rows whose squares are below fp32's range, beside rows of its middle and of its upper end."""
    rng = np.random.default_rng(31)
    Hkv, G, T = 2, 4, 5
    x = rng.standard_normal((T, Hkv * (G + 2), D)) * np.where(rng.random((T, Hkv * (G + 2), 1)) < 0.5, scale, 1.0)
    qkv = bf(x).view(1, T, -1).to(DEV)
    x = f64(qkv).reshape(T, -1, D)
    w = bf(1 + 0.3 * rng.standard_normal(D))
    f = 1e4 ** (-np.arange(64) / 64)
    r = K.make_rope(Hkv * G, Hkv, torch.from_numpy(f).to(DEV), w.to(DEV), w.to(DEV), eps=eps,
                    interleaved=interleaved)
    q, k, v = (torch.zeros(Hkv, T, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((G,), (), ()))
    K.kvc_qk_norm_rope(r, qkv, i32([list(range(T))]), None, q, k, v)
    for t in range(T):
        for h in range(Hkv * (G + 2)):
            y = (q[h // G, t, h % G] if h < Hkv * G else k[h - Hkv * G, t] if h < Hkv * (G + 1)
                 else v[h - Hkv * (G + 1), t])
            if h >= Hkv * (G + 1):
                assert np.array_equal(f64(y), x[t, h])
                continue
            want, bound = R.norm_rope(x[t, h], f64(w), t, f, float(np.float32(eps)), interleaved, 1.0)
            assert (np.abs(f64(y) - want) <= bound + R.BF * np.abs(want) + 1e-37).all(), (t, h)


def test_rope_small_negative_frequencies():
    """A negative frequency has the bits of the positive one: far positions at little angle."""
    f = np.array([1e-13, 1e-11, 3e-10, 1e-9, 0.5, 7.5, 100.25, 1e-14])
    x = np.zeros(D)
    x[:len(f)] = 1.0                                       # y_2 of the pairs is then the sine
    for pos in (2 ** 31 - 1, 123456789, -2 ** 31, 1):
        up, _ = rotated(x, freq=f, pos=pos)
        down, _ = rotated(x, freq=-f, pos=pos)
        for y, sign in ((up, 1), (down, -1)):
            want, bound = R.norm_rope(x, None, pos, sign * f, 0, False, 1.0)
            for z in y:
                small = np.abs(pos * f) < 1e-2             # where the angle is the sine: its own relative error
                i = len(f) + np.arange(len(f))[small]
                assert (np.abs(z - want)[i] <= (R.BF + 2.0 ** -20) * np.abs(want)[i]).all(), (pos, z[i], want[i])
                assert (np.abs(z - want) <= bound + R.BF * np.abs(want)).all()


# ---------------------------------------------------------------------- lengths, free places

class Held:
    """What the sequences of a PagedState hold, on the host, and steps against the definition."""

    def __init__(self, st, seed):
        self.st, self.rng = st, np.random.default_rng(seed)
        self.U = st.seqs * st.heads
        self.rows = [([], []) for _ in range(self.U)]
        self.o, self.lse = st.o.clone(), st.lse.clone()

    def store(self, x):
        if self.st.K.dtype is torch.bfloat16:
            return x
        v, sc = R.quantise(x)
        return f64(v) * sc.astype(np.float64)[..., None]

    def write(self, T, count, taken):
        k, v = (bf(self.rng.standard_normal((self.U, T, D))) for _ in range(2))
        self.st.write(k.to(DEV), v.to(DEV), None if count is None else i32(count))
        for u in range(self.U):
            s = u // self.st.heads
            if s in taken:
                for have, x in zip(self.rows[u], (k, v)):
                    have.extend(self.store(f64(x[u, :T if count is None else count[s]])))

    def step(self, max_len, taken, call=None):
        G = self.st.G
        q = bf(self.rng.standard_normal((self.U, G, D))).to(DEV)
        k, v = (bf(self.rng.standard_normal((self.U, D))).to(DEV) for _ in range(2))
        o, lse = self.st.step(q, k, v, max_len) if call is None else call(q, k, v)
        for u in range(self.U):
            if u // self.st.heads not in taken:                # as it was, to the bit
                assert torch.equal(o[u], self.o[u]) and torch.equal(lse[u], self.lse[u]), u
                continue
            for have, x in zip(self.rows[u], (k, v)):
                have.append(self.store(f64(x[u])))
            ro, rl, bo, bl = R.attend(f64(q[u]), *(np.array(x) for x in self.rows[u]))
            assert (np.abs(f64(o[u]) - ro) <= bo).all() and (np.abs(f64(lse[u]) - rl) <= bl).all(), u
        self.o, self.lse = o.clone(), lse.clone()
        assert self.st.len.tolist() == self.lengths()

    def release(self, s):
        self.st.release(s)
        for u in range(s * self.st.heads, (s + 1) * self.st.heads):
            self.rows[u] = ([], [])

    def lengths(self):
        return [len(self.rows[s * self.st.heads][0]) for s in range(self.st.seqs)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens", [[40, 25, 33], [3000, 2500, 700], [17] * 500])
def test_a_place_is_released_and_taken_again(e4m3, lens):
    """The others step on; a free place records nothing, its outputs stay, and who takes it starts at
    slot 0, over pages that held other rows."""
    S, mine = len(lens), [0, 1, 2]
    st = PagedState(S, 2, 4, max(lens) + 64, page=16, e4m3=e4m3)
    h = Held(st, 251)
    st.reserve([n + 20 for n in lens])
    h.write(max(lens), lens, range(S))
    every = set(range(S))
    most = max(lens) + 40
    h.step(most, every)
    for s in (1, 2):
        h.release(s)
        every -= {s}
        for _ in range(3):
            h.step(most, every)
            assert st.status() == 0
    st.reserve([st.page * len(p) for p in st._held[:1]] + [22] + [0] * (S - 2))
    h.write(20, [0, 20] + [0] * (S - 2), {1})
    every |= {1}
    assert st.status() == 0 and st.len.tolist()[1:3] == [20, 0]
    h.step(most, every)
    h.step(most, every)
    assert st.status() == 0
    k, v = st.read(most)
    for u in (0, 2, 3, 4):
        for out, rows in ((k, h.rows[u][0]), (v, h.rows[u][1])):
            n = len(rows)
            assert n == 0 or np.array_equal(f64(out[u, :n]), f64(bf(np.array(rows))))
            assert (out[u, n:] == 0).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_refused_rows_do_not_count(e4m3):
    """Past the pages, past max_len, and with counts that are none: lengths stay, the error is told,
    and the next calls are right, rows that were written before it over the ones refused."""
    st = PagedState(3, 2, 2, 128, page=16, e4m3=e4m3)
    h = Held(st, 257)
    st.reserve([32, 16, 48])
    h.write(30, [30, 15, 30], {0, 1, 2})
    h.step(64, {0, 1, 2})
    assert st.status() == 0
    h.step(64, {0, 2})                                     # sequence 1 has no slot left
    assert st.status() == 1
    h.step(64, {2})                                        # nor has 0
    assert st.status() == 1
    st.reserve([48, 32, 48])
    h.step(33, {0, 1})                                     # 2 holds 33 already
    assert st.status() == 2
    h.step(64, {0, 1, 2})
    assert st.status() == 0
    h.write(14, [14, -1, 15], {0})
    assert st.status() == 2 and st.len.tolist() == h.lengths()
    h.write(15, [1, 15, 15], set())                        # they hold 48 of 48, 18 of 32 and 34 of 48
    assert st.status() == 1 and st.len.tolist() == h.lengths()
    h.write(15, [1, 14, 15], {1})
    assert st.status() == 1 and st.len.tolist() == h.lengths()
    st.reserve([64, 64, 64])
    h.write(2, None, {0, 1, 2})
    h.step(128, {0, 1, 2})
    assert st.status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_captured_step_follows_the_places(e4m3):
    """A graph captured with every place taken, replayed with places free and taken again."""
    lens = [900, 60, 300]
    st = PagedState(3, 2, 4, 1024, page=16, e4m3=e4m3)
    h = Held(st, 263)
    st.reserve([n + 20 for n in lens])
    h.write(max(lens), lens, {0, 1, 2})
    h.step(1000, {0, 1, 2})
    q, k, v = (torch.zeros(6, *s, D, dtype=torch.bfloat16, device=DEV) for s in ((4,), (), ()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        st.step(q, k, v, 1000)

    def call(*new):
        for to, x in zip((q, k, v), new):
            to.copy_(x)
        g.replay()
        return st.o, st.lse

    h.step(1000, {0, 1, 2}, call)
    h.release(0)
    h.step(1000, {1, 2}, call)
    h.step(1000, {1, 2}, call)
    st.reserve([30, 0, 0])
    h.write(10, [10, 0, 0], {0})
    h.step(1000, {0, 1, 2}, call)
    assert st.status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [50, 300, 4000, 20000])
def test_free_places_among_others(e4m3, n):
    """However the work is cut: free places behind what another call left in the workspace."""
    p = Pool(269, 2, [n, n, n, n, n], 16, e4m3, more=1)
    check_attend(p, 4, units=[0, 9])
    for free in ([0], [2, 3], [4], [0, 4], [0, 1, 2, 3, 4]):
        tab = p.t["table"].clone()
        lens = i32(p.lens)
        for s in free:
            p.t["len"][s] = 0
            p.t["table"][s, 0] = -1
        q, k, v, o, lse = attend(p, 4, max_len=n + 1)
        assert p.status() == 0
        for u in range(p.U):
            if u // 2 in free:
                assert (o[u] == 7).all() and (lse[u] == 7).all()
            elif u in (1, 5, 8):
                ro, rl, bo, bl = R.attend(f64(q[u]), p.held("K", u, range(n + 1)), p.held("V", u, range(n + 1)))
                assert (np.abs(f64(o[u]) - ro) <= bo).all() and (np.abs(f64(lse[u]) - rl) <= bl).all(), (free, u)
        # without a token to append, length 0 is nothing to attend over
        _, _, _, o, lse = attend(p, 4, append=False, max_len=n + 1, q=q)
        assert p.status() == 0
        for s in free:
            assert (o[2 * s] == 0).all() and (lse[2 * s] == -np.inf).all()
        p.t["table"].copy_(tab)
        p.t["len"].copy_(lens)


def test_a_refused_selection_is_not_handed_over():
    """Units whose count or slots the read refuses are empty in the budgeted cache, the others whole."""
    lens = [40, 25, 33]
    st = PagedState(3, 2, 4, 64, page=16, e4m3=False)
    h = Held(st, 271)
    st.reserve(lens)
    h.write(40, lens, {0, 1, 2})
    slots = torch.arange(20, dtype=torch.int32, device=DEV).repeat(6, 1)
    ds = DecodeState(6, 4, 32, 24)
    for bad in ("none", "long", "negative", "slot", "below", "behind"):
        sl, count = slots.clone(), i32([20, 15, 0, 20, 1, 20])
        if bad == "long":
            count[1] = 21
        elif bad == "negative":
            count[1] = -1
        elif bad == "slot":
            sl[1, 14] = 40
        elif bad == "below":
            sl[1, 0] = -1
        elif bad == "behind":                              # nobody asks for it
            sl[1, 15] = 1 << 30
        ds.K.fill_(7.0)
        ds.len.fill_(5)
        st.hand_over(ds, sl, count)
        refused = bad in ("long", "negative", "slot", "below")
        assert st.status() == (2 if refused else 0)
        assert ds.len.tolist() == [20, 0 if refused else 15, 0, 20, 1, 20], bad
        for u in range(6):
            n = int(ds.len[u])
            assert n == 0 or np.array_equal(f64(ds.K[u, :n]), f64(bf(np.array(h.rows[u][0][:n]))))


# ---------------------------------------------------------------------- long units

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens", [[131070], [131070, 65536], [100003] * 3, [70001] * 20, [65600, 3, 0] * 60])
def test_every_slot_counts_once_in_a_long_unit(e4m3, lens):
    """Equal weights: lse is log n to a fraction of 1/n, so no slot is missing or there twice.  The
    values are zero but in slots around the places where the line of tiles is cut for the warps, each
    with a dimension of its own: o is their value over n."""
    p = Pool(277, 1, lens, 64, e4m3, more=1)
    tile = 32 if e4m3 else 16
    tiles = [-(-(n + 1) // tile) for n in lens]
    total, warps = sum(tiles), 152 * 3 * 4
    cuts = [c * (total // warps) + min(c, total % warps) for c in range(warps)]
    some, want = sorted({0, len(lens) // 2, len(lens) - 1}), {}
    v_new = np.zeros((p.U, D))
    for u in some:
        n, first = lens[u], sum(tiles[:u])
        edges = [(c - first) * tile for c in cuts if first < c < first + tiles[u]]
        at = {0, n - 1, 63, 64} | {int(e) + d for e in p.rng.permutation(edges)[:40] for d in (-1, 0)}
        at |= {int(x) for x in p.rng.integers(0, max(n, 1), 30)}
        at = sorted(x for x in at if 0 <= x < n)[:D - 1]
        x = np.zeros((n, D))
        x[at, range(len(at))] = 1000.0 + np.arange(len(at))
        v_new[u, D - 1] = 555.0
        if n:
            put(p, "V", u, range(n), x)
        want[u] = at
    zero = bf(np.zeros((p.U, D))).to(DEV)
    _, _, _, o, lse = attend(p, 4, q_scale=0.0, k=zero, v=bf(v_new).to(DEV))
    assert p.status() == 0
    for u, at in want.items():
        n = lens[u] + 1
        expect = np.zeros(D)
        if at:
            expect[:len(at)] = p.held("V", u, at)[range(len(at)), range(len(at))]
        expect[D - 1] = p.held("V", u, [n - 1])[0, D - 1]
        expect /= n
        # the weights are 1 and their sum is exact: a quotient (2 ulp) and the rounding to bf16
        assert (np.abs(f64(o[u]) - expect) <= (R.BF + 2.0 ** -20) * np.abs(expect)).all(), u
        # a logarithm to base 2 to an ulp, its product with ln 2 (rounded to 2^-25 of itself)
        y = np.log(n)
        bound = np.spacing(np.float32(np.log2(n))) * np.log(2) + 2.0 ** -25 * y + np.spacing(np.float32(y)) / 2
        assert n < 1000 or bound < 0.5 / n
        assert np.abs(f64(lse[u]) - y).max() <= bound, u


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("n,k_scale", [(131071, 4.0), (20011, 10.0), (131071, 30.0)])
def test_sharp_attention_over_long_units(e4m3, G, n, k_scale):
    """A few slots have nearly all of the weight, wherever they are; each head has others."""
    p = Pool(n + G, 1, [n, n // 3, 40], 64, e4m3, more=1, k_scale=k_scale)
    check_attend(p, G)
    check_attend(p, G, append=False, units=[0])


@pytest.mark.parametrize("G", [4, 8])
@pytest.mark.parametrize("n", [20, 300, 9000])
@pytest.mark.parametrize("octaves,ratio", [(100, 2.0 ** 100), (125, 2.0 ** 124), (138, 2.0 ** 138), (150, 2.0 ** 150),
                                           (300, 2.0 ** 200), (2000, 2.0 ** 200)])
def test_a_large_value_of_a_weight_below_fp32(G, n, octaves, ratio):
    """In e4m3 a value 2^100 and more above the others counts by its contribution, whether or not its
    weight is one that fp32 holds, and leaves the others theirs where it has none."""
    p = Pool(281, 1, [n, n], 16, True)
    q = np.zeros((2, G, D))
    q[:, :, 0] = 4
    low = 2.0 ** -100
    for u, at in ((0, n // 3), (1, n - 1)):
        put(p, "K", u, range(n), np.zeros((n, D)))
        put(p, "K", u, [at], -octaves * np.log(2) * np.sqrt(D) / 4 * spike(0)[None])
        put(p, "V", u, range(n), low * (1 + p.rng.random((n, D))))
        put(p, "V", u, [at], low * ratio * spike(0, 64)[None])
    check_attend(p, G, append=False, q=bf(q).to(DEV))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,lens", [(4, [300, 40]), (8, [9000, 70]), (4, [600] * 1000)])
@pytest.mark.parametrize("size", [1e9, 1e15, 1e30])
@pytest.mark.parametrize("v_scale", [1e-20, 1.0, 1e30])
def test_logits_of_any_size(e4m3, G, lens, size, v_scale):
    """Logits of plus and minus `size`: the slots of the larger one share the weight, whatever their
    values' scale, and lse is that logit and the logarithm of their number.  Slots of the smaller one
    with the largest values weigh nothing."""
    p = Pool(283, 1, lens, 16, e4m3)
    some = sorted({0, p.U // 2, p.U - 1})
    q = np.zeros((p.U, G, D))
    q[:, :, 0] = np.sqrt(size)
    first = {}
    for u in some:
        n = lens[u]
        up = p.rng.random(n) < 0.3
        up[p.rng.integers(n)] = True
        first[u] = up
        put(p, "K", u, range(n), np.where(up, 1.0, -1.0)[:, None] * np.sqrt(size) * spike(0))
        put(p, "V", u, range(n), v_scale * np.where(up, 1.0, 1e3)[:, None] * (1 + p.rng.random((n, D))))
    _, _, _, o, lse = attend(p, G, append=False, q=bf(q).to(DEV))
    assert p.status() == 0
    qh = f64(bf(q))
    for u in some:
        rows = np.nonzero(first[u])[0]
        want = p.held("V", u, rows).mean(0)
        # equal weights of 1: their sums of n terms, a quotient and the rounding to bf16
        assert (np.abs(f64(o[u]) - want) <= (R.BF + (len(rows) + 16) * 2.0 ** -24) * want).all(), u
        x = qh[u, 0, 0] * p.held("K", u, rows[:1])[0, 0] / np.sqrt(D)
        assert (np.abs(f64(lse[u]) - (x + np.log(len(rows)))) <= 16 * 2.0 ** -24 * x).all(), u


@pytest.mark.parametrize("lens", [[300, 40], [9000, 70, 700], [600] * 1000])
def test_infinite_keys(lens):
    """Keys with an infinity, in bf16: a logit of -inf weighs nothing, all of them are no slots at all,
    one of +inf or a NaN makes lse and o of its head NaN."""
    p = Pool(293, 1, lens, 16, False)
    u, n = 1, lens[1]
    q = p.rng.standard_normal((p.U, 4, D))
    q[:, :, 0] = [1, -1, 0, -2]
    q = bf(q)
    k = p.rng.standard_normal((n, D))
    k[:, 0] = 0.5
    k[n // 2, 0] = np.inf
    put(p, "K", u, range(n), k)
    _, _, _, o, lse = attend(p, 4, append=False, q=q.to(DEV))
    rest = [i for i in range(n) if i != n // 2]
    for h in (1, 3):
        ro, rl, bo, bl = R.attend(f64(q[u, h])[None], p.held("K", u, rest), p.held("V", u, rest))
        assert (np.abs(f64(o[u, h]) - ro[0]) <= bo[0]).all() and abs(float(lse[u, h]) - rl[0]) <= bl[0]
    for h in (0, 2):
        assert o[u, h].isnan().all() and lse[u, h].isnan()
    k[:, 0] = np.inf
    put(p, "K", u, range(n), k)
    _, _, _, o, lse = attend(p, 4, append=False, q=q.to(DEV))
    for h in (1, 3):
        assert (o[u, h] == 0).all() and lse[u, h] == -np.inf
    for h in (0, 2):
        assert o[u, h].isnan().all() and lse[u, h].isnan()
    assert not o[0].isnan().any() and not lse[0].isnan().any() and p.status() == 0
