"""Pins of the paged-cache oracle: its codes against torch's 8-bit casts, its
attention against the dense oracle on the decoded cache, its append and
eviction against closed forms on small inputs."""
import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import paged as P

TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_codes_match_torch(kind):
    vals = P.code_values(kind)
    got = torch.arange(256, dtype=torch.uint8).view(TORCH[kind]).double().numpy()
    assert np.array_equal(np.nan_to_num(vals, nan=1e9), np.nan_to_num(got, nan=1e9))
    x = np.random.default_rng(1).standard_normal(20000) * np.exp2(np.random.default_rng(2).uniform(-20, 8, 20000))
    x = np.concatenate([x, vals[np.isfinite(vals)], [0.0, -0.0]])
    # halfway cases: the mean of neighbouring codes
    grid = np.sort(np.unique(vals[np.isfinite(vals)]))
    x = np.concatenate([x, (grid[1:] + grid[:-1]) / 2]).astype(np.float32)
    x = np.clip(x, -P.LARGEST[kind], P.LARGEST[kind])
    want = torch.from_numpy(x).to(TORCH[kind]).view(torch.uint8).numpy()
    assert np.array_equal(P.encode(x, kind), want)


def test_codes_beyond_the_range():
    for kind in ("e4m3", "e5m2"):
        top = P.LARGEST[kind]
        c = P.encode(np.array([top * 1.5, -top * 4, np.nan]), kind)
        v = P.code_values(kind)[c]
        assert v[0] == top and v[1] == -top and np.isnan(v[2])
    assert np.isinf(P.code_values("e5m2")[P.encode(np.array([np.inf]), "e5m2")][0])
    assert np.isnan(P.code_values("e4m3")[P.encode(np.array([np.inf]), "e4m3")][0])


def test_attention_equals_the_dense_oracle():
    rng = np.random.default_rng(3)
    pages, Hkv, ps, d, B, T, Nq, g = 9, 2, 16, 64, 2, 4, 3, 2
    kp, vp = (rng.integers(0, 0x7F, (pages, Hkv, ps, d)).astype(np.uint8) for _ in range(2))
    ks, vs = rng.uniform(1e-3, 1e-2, (2, pages, Hkv))
    table = rng.permutation(pages)[:B * T].reshape(B, T)
    lens = np.array([50, 17])
    q = rng.standard_normal((B, g * Hkv, Nq, d))
    o, lse, w, mass = P.attention(q, (kp, vp, ks, vs), "e4m3", table, lens, 0.1, True)
    for b in range(B):
        for hq in range(g * Hkv):
            n = lens[b]
            k = P.slots(kp, ks, table[b], n, hq // g, "e4m3")
            v = P.slots(vp, vs, table[b], n, hq // g, "e4m3")
            ro, rl = A.forward_head(q[b, hq], k, v, 0.1, True)
            assert np.abs(o[b, hq] - ro).max() < 1e-12 and np.abs(lse[b, hq] - rl).max() < 1e-12
    # the weights of a head's rows sum to the number of its rows
    assert np.allclose(w.sum(axis=2), g * Nq)


def test_append_scale_is_the_smallest():
    for kind in ("e4m3", "e5m2"):
        for amax in (1.0, 447.9, 448.0, 448.1, 57344.0, 1e-20, 3.5, 3.51):
            s = P.append_scale(amax, kind)
            assert amax <= P.LARGEST[kind] * s and amax > P.LARGEST[kind] * s / 2
        assert P.append_scale(0.0, kind) == 2.0 ** -100


def test_eviction_by_hand():
    w = np.array([5.0, 1.0, 4.0, 1.0, 3.0, 2.0, 0.0, 9.0])
    pos = np.arange(8)
    assert P.evict_plan(w, pos, 8, 8, 2) == ([], [])
    # the last two stay, then 5, 4, 3: slots 0, 2, 4 stay, 6 and 7 move into 1 and 3
    assert P.evict_plan(w, pos, 8, 5, 2) == ([1, 3], [6, 7])
    # equal weights: the lowest slots stay
    assert P.evict_plan(np.ones(6), np.zeros(6), 6, 4, 0) == ([], [])
    assert P.evict_plan(np.array([0.0, np.nan, 1.0, 2.0]), np.arange(4), 4, 2, 0) == ([0], [3])


def test_eviction_moves_values():
    rng = np.random.default_rng(5)
    pages, ps, d = 4, 16, 64
    cache = [rng.integers(0, 0x70, (pages, 1, ps, d)).astype(np.uint8) for _ in range(2)]
    cache += [2.0 ** rng.integers(-4, 1, (pages, 1)).astype(np.float32) for _ in range(2)]
    table = np.array([[2, 0, 3]])
    w, pos = rng.random((1, 1, 48)), np.arange(48).reshape(1, 1, 48)
    kp, vp, ks, vs, w2, p2, n2 = P.evict(cache, "e4m3", table, w, pos, np.array([40]), 21, 5)
    before = P.slots(cache[0], cache[2], table[0], 40, 0, "e4m3")
    after = P.slots(kp, ks, table[0], 21, 0, "e4m3")
    assert n2[0] == 21 and set(range(35, 40)) <= set(p2[0, 0, :21])
    for j in range(21):  # each slot holds its token's values, up to one rounding at the page's scale
        assert w2[0, 0, j] == w[0, 0, p2[0, 0, j]]
        assert np.abs(after[j] - before[p2[0, 0, j]]).max() <= 2.0 ** -10 * ks[table[0, j // ps], 0] + 1e-12
    old = w2[0, 0, :21][p2[0, 0, :21] < 35]  # the 16 that are not protected: the heaviest of 35
    assert np.array_equal(np.sort(old), np.sort(w[0, 0, :35])[-16:])
