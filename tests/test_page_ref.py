"""The definitions that the GPU tests of the cache in pages, and of the norms and
rotation, are held against (page_ref.py), against independent forms (CPU)."""
import math

import numpy as np
import pytest
import torch

import page_ref as R


def rows(seed, *shape):
    x = np.random.default_rng(seed).standard_normal(shape)
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("factor", [1.0, 1e-20, 1e20])
def test_quantised_rows(factor):
    """Every value within half a step of e4m3 (2^-4 of it, 2^-10 of the scale among the subnormal
    ones; the two roundings of the quotient besides), the largest at 448 scales."""
    x = rows(1, 50, R.D)
    x = torch.from_numpy(x * factor * np.exp(rows(2, 50, 1))).to(torch.bfloat16).double().numpy()
    v, s = R.quantise(x)
    v, s = v.double().numpy(), s.astype(np.float64)[:, None]
    assert (np.abs(v * s - x) <= np.abs(x) * (2.0 ** -4 + 2.0 ** -22) + s * 2.0 ** -10).all()
    assert (np.abs(v).max(1) == 448).all()
    assert (np.abs(s[:, 0] * 448 - np.abs(x).max(1)) <= 2.0 ** -23 * np.abs(x).max(1)).all()


def test_quantised_rows_at_the_ends():
    x = np.zeros((4, R.D))
    x[1, 3], x[2, 5], x[3, 7] = np.nan, np.inf, 1e-40
    v, s = R.quantise(x)
    with np.errstate(invalid="ignore"):
        back = v.float().numpy() * s[:, None]
    assert (back[0] == 0).all() and s[0] == R.TINY
    assert np.isnan(back[1]).all() and np.isnan(back[2]).all()
    assert s[3] == R.TINY and np.isfinite(back[3]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    x, w = rows(3, R.D), 1 + 0.2 * rows(4, R.D)
    f = 1e4 ** (-np.arange(32) / 32)
    for pos in (0, 1, -3, 77777):
        got, bound = R.norm_rope(x, w, pos, f, 1e-6, interleaved, 1.5)
        y = x * w / np.sqrt(np.mean(x * x) + 1e-6)
        pairs = y[:64].reshape(32, 2) if interleaved else y[:64].reshape(2, 32).T
        z = (pairs[:, 0] + 1j * pairs[:, 1]) * 1.5 * np.exp(1j * pos * f)
        want = np.concatenate([np.stack([z.real, z.imag], 1).reshape(-1) if interleaved else
                               np.concatenate([z.real, z.imag]), y[64:]])
        assert np.abs(got - want).max() < 1e-9 and (bound > 0).all()
        assert math.isclose(np.linalg.norm(got[:64]), 1.5 * np.linalg.norm(y[:64]), rel_tol=1e-12)


def test_far_positions_need_no_reduction():
    """Whole turns do not count: a frequency of a 2^k-th turn comes back after 2^k positions."""
    x = rows(5, R.D)
    f = [2 * math.pi / 1024]
    a, _ = R.norm_rope(x, None, 5, f, 0, False, 1.0)
    b, _ = R.norm_rope(x, None, 5 + 1024 * 1000000, f, 0, False, 1.0)
    # 2 pi / 1024 is rounded to 53 bits: 1e9 positions of it are off by up to 1e9 f 2^-53
    assert np.abs(a - b).max() <= 8 * 1.1e9 * f[0] * 2.0 ** -53 * np.abs(x).max()


@pytest.mark.parametrize("n", [1, 2, 33, 500])
def test_attention_is_softmax(n):
    q, k, v = rows(6, 4, R.D), rows(7, n, R.D), rows(8, n, R.D)
    o, lse, bo, bl = R.attend(q, k, v)
    x = torch.from_numpy(q) @ torch.from_numpy(k).T / math.sqrt(R.D)
    assert np.allclose(o, (torch.softmax(x, 1) @ torch.from_numpy(v)).numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(lse, torch.logsumexp(x, 1).numpy(), rtol=1e-13)
    # the bounds are about a bf16 step of the outputs and well below the outputs themselves
    assert (bo >= 2.0 ** -9 * np.abs(o)).all() and bo.max() < 0.05 * np.abs(v).max() and bl.max() < 1e-2


def test_attention_over_nothing():
    o, lse, _, _ = R.attend(rows(9, 2, R.D), np.zeros((0, R.D)), np.zeros((0, R.D)))
    assert (o == 0).all() and (lse == -np.inf).all()


def test_plain_forms_of_the_cases_quantise_alike():
    from perf import more_operators as M
    x = torch.from_numpy(rows(10, 200, R.D)).to(torch.bfloat16)
    v, s = M._quantise(x)
    rv, rs = R.quantise(x.double().numpy())
    assert torch.equal(v.view(torch.uint8), rv.view(torch.uint8)) and np.array_equal(s.numpy(), rs)
