"""The 8-bit paged K/V cache on the GPU against the float64 oracle: attention
(every head width, row count, page size and type; ragged, empty and
masked-out sequences), append, eviction, and a run of them together."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_forward_gb300 as fa
from oracle import paged as P

from paged_util import DT, TORCH, Cache, check_attention, values16

pytestmark = pytest.mark.gpu


def _lens(lens):
    return torch.tensor(lens, dtype=torch.int32, device="cuda")


def _q(B, Hq, Nq, d, dtype, seed):
    return values16(np.random.default_rng(seed).standard_normal((B, Hq, Nq, d)) * 1.3, dtype)


ATTEND = [  # Hq, Hkv, Nq, d, lens, ps, dtype, kind, causal, splits
    (1, 1, 1, 128, [1], 16, "bf16", "e4m3", True, 1),
    (2, 1, 1, 128, [128], 128, "bf16", "e4m3", True, 1),
    (4, 2, 1, 128, [300, 0, 1, 129], 64, "bf16", "e4m3", True, 1),
    (4, 2, 1, 128, [300, 0, 1, 129], 64, "bf16", "e4m3", True, 3),
    (8, 2, 1, 64, [257], 16, "bf16", "e4m3", True, 0),
    (8, 1, 1, 256, [515, 77], 32, "bf16", "e4m3", False, 0),
    (8, 2, 2, 128, [700, 31], 16, "fp16", "e4m3", True, 0),
    (8, 1, 2, 64, [400, 16], 16, "bf16", "e5m2", True, 2),
    (14, 2, 2, 64, [1000, 999], 128, "fp16", "e5m2", True, 0),
    (16, 1, 1, 128, [650], 32, "bf16", "e4m3", True, 2),
    (16, 1, 1, 256, [650, 3], 64, "fp16", "e4m3", True, 2),
    (8, 1, 4, 128, [333, 2], 16, "bf16", "e4m3", True, 1),
    (8, 1, 4, 64, [333, 2], 32, "fp16", "e4m3", True, 1),
    (8, 1, 4, 256, [333, 5], 64, "bf16", "e5m2", True, 3),
    (16, 2, 5, 256, [900, 131], 32, "fp16", "e5m2", True, 0),
    (6, 2, 13, 128, [500, 7, 0], 64, "bf16", "e4m3", True, 0),   # 39 rows: two row tiles
    (4, 1, 25, 128, [140, 99], 16, "fp16", "e4m3", True, 1),     # 100 rows
    (4, 1, 25, 256, [140, 20], 128, "bf16", "e4m3", False, 2),
    (3, 3, 1, 128, [5000, 4999], 64, "bf16", "e4m3", True, 0),
    (3, 3, 7, 64, [2049, 1], 16, "bf16", "e4m3", True, 1024),    # a chunk a tile
    (32, 8, 1, 128, [2100] * 3, 128, "bf16", "e4m3", True, 0),
]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention_matches_oracle(case, weights):
    Hq, Hkv, Nq, d, lens, ps, dtype, kind, causal, splits = ATTEND[case]
    B = len(lens)
    T = (max(lens) + ps - 1) // ps + 1
    c = Cache(B, Hkv, T, ps, d, kind, seed=case)
    handle = c.to("cuda")
    qf, q = _q(B, Hq, Nq, d, dtype, 100 + case)
    acc = torch.full((B, Hkv, T * ps), 2.5, device="cuda") if weights else None
    o, lse = fa.forward_paged(handle, q.cuda(), _lens(lens), causal=causal, weight_acc=acc, num_splits=splits)
    fa.fa_device_status()
    check_attention(qf, c, lens, 1 / math.sqrt(d), causal, dtype, o, lse, acc, added=2.5)


SHARED = [  # B, Hq, Hkv, Nq, d, longest, ps, dtype, kind: many sequences, several a CTA
    (40, 16, 8, 1, 128, 900, 16, "bf16", "e4m3"),
    (1000, 2, 2, 1, 64, 120, 64, "bf16", "e4m3"),       # one tile each
    (300, 4, 2, 2, 64, 260, 32, "fp16", "e5m2"),
    (90, 4, 2, 10, 128, 500, 128, "bf16", "e4m3"),       # 20 rows: three groups
    (30, 10, 2, 8, 256, 700, 32, "fp16", "e4m3"),        # 40 rows: five groups
    (30, 12, 2, 8, 64, 700, 32, "bf16", "e4m3"),         # 48 rows: two row tiles of 24
    (1100, 1, 1, 1, 64, 300, 16, "bf16", "e4m3"),        # too many to share out: one head a CTA
    (3, 4, 2, 1, 128, 4000, 16, "bf16", "e4m3"),
]


@pytest.mark.parametrize("case", range(len(SHARED)))
def test_ragged_batches_match_oracle(case):
    """Lengths of all kinds (a third of them 0, 1, or whole tiles): the CTAs' shares begin and end anywhere."""
    B, Hq, Hkv, Nq, d, longest, ps, dtype, kind = SHARED[case]
    rng = np.random.default_rng(200 + case)
    lens = rng.integers(2, longest + 1, B)
    odd = rng.integers(0, 3, B) == 0
    lens[odd] = rng.choice([0, 1, 127, 128, 129, 256], B)[odd]
    lens = np.minimum(lens, longest)
    lens[-1], lens[0] = 0, longest
    T = (longest + ps - 1) // ps
    c = Cache(B, Hkv, T, ps, d, kind, seed=210 + case)
    qf, q = _q(B, Hq, Nq, d, dtype, 220 + case)
    acc = torch.zeros(B, Hkv, T * ps, device="cuda")
    handle = c.to("cuda")
    if T * ps <= 512:  # shared out from 513 slots on
        handle = fa.PagedCache(*c.t[:4], torch.cat([c.t[4], torch.full((B, 512 // ps), -1, dtype=torch.int32,
                                                                      device="cuda")], 1))
        acc = torch.zeros(B, Hkv, handle.slots, device="cuda")
    o, lse = fa.forward_paged(handle, q.cuda(), _lens(lens.tolist()), causal=True, weight_acc=acc)
    fa.fa_device_status()
    check_attention(qf, c, lens.tolist(), 1 / math.sqrt(d), True, dtype, o, lse, acc[..., :T * ps], added=0.0)
    # chunks by num_splits: the same numbers up to rounding, and the same bits whatever the batch is
    acc1 = torch.zeros_like(acc)
    o1, lse1 = fa.forward_paged(handle, q.cuda(), _lens(lens.tolist()), causal=True, weight_acc=acc1, num_splits=2)
    fa.fa_device_status()
    check_attention(qf, c, lens.tolist(), 1 / math.sqrt(d), True, dtype, o1, lse1, acc1[..., :T * ps], added=0.0)
    one = fa.PagedCache(*handle.tensors[:4], handle.tensors[4][:1].contiguous())
    o2, lse2 = fa.forward_paged(one, q[:1].cuda(), _lens(lens[:1].tolist()), causal=True, num_splits=2)
    fa.fa_device_status()
    assert torch.equal(o1[:1], o2) and torch.equal(lse1[:1], lse2)


def test_scales_far_apart():
    """Pages whose scales differ by 2^40 in K (scores near 0 beside ordinary ones) and by 10^6 in V."""
    c = Cache(2, 2, 9, 64, 128, seed=3)
    c.np[2][::2] *= np.float32(2.0 ** -40)
    c.np[3][::3] *= np.float32(1e6)
    c.np[3][1::3] *= np.float32(1e-6)
    qf, q = _q(2, 8, 1, 128, "bf16", 4)
    o, lse = fa.forward_paged(c.to("cuda"), q.cuda(), _lens([570, 64]), num_splits=2)
    fa.fa_device_status()
    check_attention(qf, c, [570, 64], 1 / math.sqrt(128), False, "bf16", o, lse)


def test_large_scales_behind_a_small_weight():
    """The page of large V scale gets next to no weight: the others' precision is their own."""
    c = Cache(1, 1, 3, 64, 128, seed=5, spread=0.0)
    c.np[3][c.table[0, 1]] *= np.float32(1e4)
    c.np[0][c.table[0, 1], 0] = P.encode(np.tile(np.sign(np.linspace(-1, 1, 128)) * -100, (64, 1)), "e4m3")
    c.np[0][c.table[0, 0], 0] = P.encode(np.tile(np.sign(np.linspace(-1, 1, 128)) * 2, (64, 1)), "e4m3")
    qf, q = values16(np.tile(np.sign(np.linspace(-1, 1, 128)) * 1.5, (1, 1, 1, 1)), "bf16")
    o, lse = fa.forward_paged(c.to("cuda"), q.cuda(), _lens([128]), num_splits=1)
    fa.fa_device_status()
    ro, rl, _, mass = P.attention(qf, c.np, "e4m3", c.table, [128], 1 / math.sqrt(128), False)
    # no term for lost weights here: the page's own largest value bounds it
    assert (np.abs(o.cpu().double().numpy() - ro) <= 2.0 ** -8 * np.abs(ro) + 1.1 * 2.0 ** -8 * mass).all()
    assert abs(lse.item() - rl.item()) < 1e-4


def test_many_small_weights_are_kept():
    """One slot outweighs each of 16000 others by 2^16; together they still count."""
    n, ps = 16001, 128
    c = Cache(1, 1, 126, ps, 64, seed=6, spread=0.0)
    c.np[0][...] = 0
    c.np[0][c.table[0, 0], 0, 0, 0] = 0x78  # 256
    c.np[1][...] = P.encode(np.float64(64.0), "e4m3")
    c.np[1][c.table[0, 0], 0, 0] = P.encode(np.float64(-64.0), "e4m3")
    x = np.zeros((1, 1, 1, 64))
    x[..., 0] = 1.0
    qf, q = values16(x, "bf16")
    scale = 16 * math.log(2) / (256 * float(c.np[2][c.table[0, 0], 0]))
    o, lse = fa.forward_paged(c.to("cuda"), q.cuda(), _lens([n]), scale=scale, num_splits=1)
    fa.fa_device_status()
    check_attention(qf, c, [n], scale, False, "bf16", o, lse)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("splits", [1, 2])
def test_bytes_behind_the_length_do_not_matter(kind, splits):
    """NaN codes, NaN scales and wrong page numbers behind the filled slots."""
    c = Cache(2, 2, 6, 64, 128, kind, seed=7)
    lens = [131, 64]
    for b, n in enumerate(lens):
        for t in range(6):
            p = c.table[b, t]
            for x in c.np[:2]:
                x[p, :, max(0, min(64, n - t * 64)):] = 0x7F
            if t * 64 >= n:
                c.np[2][p], c.np[3][p] = np.nan, np.inf
    clean = [x.copy() for x in c.np]
    c.table[0, 3:] = -7
    c.table[1, 1:] = 1 << 30
    qf, q = _q(2, 4, 1, 128, "bf16", 8)
    acc = torch.zeros(2, 2, 384, device="cuda")
    o, lse = fa.forward_paged(c.to("cuda"), q.cuda(), _lens(lens), weight_acc=acc, num_splits=splits)
    fa.fa_device_status()  # entries that are not needed are not looked at
    clean[2], clean[3] = np.nan_to_num(clean[2], nan=0.01), np.nan_to_num(clean[3], posinf=0.01)
    check_attention(qf, c, lens, 1 / math.sqrt(128), False, "bf16", o, lse, acc, kv=clean)
    assert float(acc[0, :, 131:].abs().max()) == 0 and float(acc[1, :, 64:].abs().max()) == 0


def test_bad_page_and_bad_length_are_reported():
    c = Cache(3, 2, 6, 32, 64, seed=9)
    c.table[0, 2] = len(c.np[0])  # one past the pool: its slots are not seen
    qf, q = _q(3, 2, 1, 64, "bf16", 10)
    handle = c.to("cuda")
    lens = [180, 100, 50]
    o, lse = fa.forward_paged(handle, q.cuda(), _lens(lens), num_splits=1)
    with pytest.raises(fa.FAError) as e:
        fa.fa_device_status()
    assert e.value.code == 8
    check_attention(qf, c, lens, 1 / 8, False, "bf16", o, lse)
    for bad in (-1, 193):
        for splits in (1, 2):
            acc = torch.zeros(3, 2, 192, device="cuda")
            o, lse = fa.forward_paged(handle, q.cuda(), _lens([100, bad, 50]), weight_acc=acc, num_splits=splits)
            with pytest.raises(fa.FAError) as e:
                fa.fa_device_status()
            assert e.value.code in (7, 8)
            assert torch.isinf(lse[1]).all() and not o[1].any() and not acc[1].any()
            assert torch.isfinite(lse[0]).all() and torch.isfinite(lse[2]).all()
    fa.fa_device_status()


def test_not_finite_queries_stay_in_their_row():
    c = Cache(1, 1, 4, 64, 128, seed=11)
    qf, q = _q(1, 4, 2, 128, "fp16", 12)
    q[0, 1, 0, 5] = float("nan")
    q[0, 2, 1, 7] = float("inf")
    for splits in (1, 2):
        o, lse = fa.forward_paged(c.to("cuda"), q.cuda(), _lens([200]), causal=True, num_splits=splits)
        fa.fa_device_status()
        assert torch.isnan(o[0, 1, 0]).all() and torch.isnan(o[0, 2, 1]).all()
        assert torch.isnan(lse[0, 1, 0]) and torch.isnan(lse[0, 2, 1])
        good = np.ones((1, 4, 2), bool)
        good[0, 1, 0] = good[0, 2, 1] = False
        ro, rl, _, _ = P.attention(np.nan_to_num(qf, posinf=0.0), c.np, "e4m3", c.table, [200], 1 / math.sqrt(128), True)
        assert np.abs(o.cpu().double().numpy() - ro)[good].max() < 2e-2
        assert np.abs(lse.cpu().double().numpy() - rl)[good].max() < 1e-3


@pytest.mark.parametrize("splits", [0, 1, 3])
def test_scores_far_below_zero(splits):
    """Scores of about -1e33 to -1e37: all keys equal, and one slot's score half of the others'.

    Equal scores: every weight is a power of two (the V scales are), O is V's mean; its 700 terms are rounded in 32-bit
    sums (2^-23 each, 2^-13 of the largest |V|), and once to bf16, 2^-8.  LSE: seven roundings of 2^-24 (log2 e, scale
    and their product, times the page's scale, times the row's, ln 2, the result); ln 700 is far below one of them, so
    that parts of a row joined by their LSE weigh alike whatever they hold: that O is looked at where there is one."""
    n, d = 700, 64
    c = Cache(2, 1, 11, 64, d, "e4m3", seed=90, powers=True)
    c.np[0][:] = P.encode(np.array([1.0]), "e4m3")[0]
    c.np[3][:] = 0.25
    c.np[0][c.table[1, 7], 0, 13] = P.encode(np.array([0.5]), "e4m3")[0]
    q = torch.full((2, 2, 1, d), -1.0).bfloat16()
    q[:, 1] = -1000.0
    for ks in (1e32, 1e34):
        c.np[2][:] = np.float32(ks)
        o, lse = fa.forward_paged(c.to("cuda"), q.cuda(), _lens([n, n]), scale=0.125, num_splits=splits)
        fa.fa_device_status()
        ro, rl, _, _ = P.attention(q.double().numpy(), c.np, "e4m3", c.table, [n, n], 0.125, False)
        o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
        assert np.isfinite(rl).all() and rl.max() < -1e32
        assert (np.abs(lse - rl) <= 7 * 2.0 ** -24 * np.abs(rl)).all()
        if splits == 1:
            assert (np.abs(o - ro)[0] <= 2.0 ** -13 * 448 * 0.25 + 2.0 ** -8 * np.abs(ro[0])).all()
        one = P.code_values("e4m3")[c.np[1][c.table[1, 7], 0, 13]] * 0.25  # the one slot's V, all of O
        assert np.array_equal(o[1, 0, 0], one) and np.array_equal(o[1, 1, 0], one)


def test_zero_and_tiny_rows():
    """A query of zeros, one of subnormal numbers, pages of zeros with the smallest scale."""
    c = Cache(1, 1, 3, 64, 64, seed=13)
    p = c.table[0, 1]
    c.np[0][p] = c.np[1][p] = 0
    c.np[2][p] = c.np[3][p] = np.float32(2.0 ** -100)
    c.np[2][c.table[0, 2]] = 0.0
    c.np[3][c.table[0, 2]] = 0.0
    qf, q = _q(1, 4, 1, 64, "bf16", 14)
    q[0, 0] = 0
    q[0, 1] = 1e-39
    o, lse = fa.forward_paged(c.to("cuda"), q.cuda(), _lens([170]))
    fa.fa_device_status()
    check_attention(q.double().numpy(), c, [170], 1 / 8, False, "bf16", o, lse)


def test_results_do_not_depend_on_the_rest_of_the_batch_or_the_run():
    c = Cache(3, 2, 40, 64, 128, seed=15)
    handle = c.to("cuda")
    _, q = _q(3, 8, 2, 128, "bf16", 16)
    lens = _lens([2500, 2400, 17])
    first = None
    for _ in range(3):
        acc = torch.zeros(3, 2, 2560, device="cuda")
        o, lse = fa.forward_paged(handle, q.cuda(), lens, causal=True, weight_acc=acc)
        fa.fa_device_status()
        if first is None:
            first = (o, lse, acc)
        assert all(torch.equal(x, y) for x, y in zip(first, (o, lse, acc)))


def test_max_len_bounds_the_grid():
    c = Cache(2, 1, 64, 32, 128, seed=17)
    handle = c.to("cuda")
    qf, q = _q(2, 4, 1, 128, "bf16", 18)
    for max_len in (301, 384, 2048):
        o, lse = fa.forward_paged(handle, q.cuda(), _lens([301, 5]), max_len=max_len)
        fa.fa_device_status()
        check_attention(qf, c, [301, 5], 1 / math.sqrt(128), False, "bf16", o, lse)
    # a last chunk whose end is not a tile's, with weights
    acc = torch.zeros(2, 1, 2048, device="cuda")
    o, lse = fa.forward_paged(handle, q.cuda(), _lens([301, 5]), max_len=301, num_splits=2, weight_acc=acc)
    fa.fa_device_status()
    check_attention(qf, c, [301, 5], 1 / math.sqrt(128), False, "bf16", o, lse, acc)


# ---------------------------------------------------------------- append
APPEND = [  # Hkv, N, d, lens, counts, ps, dtype, kind
    (2, 1, 128, [0, 1, 15, 16, 17], None, 16, "bf16", "e4m3"),
    (1, 1, 64, [63, 64], None, 64, "fp16", "e5m2"),
    (3, 1, 256, [100], None, 128, "bf16", "e5m2"),
    (2, 70, 64, [0, 33, 5], [70, 0, 31], 16, "bf16", "e4m3"),
    (1, 200, 128, [7, 64], [200, 129], 64, "fp16", "e4m3"),
    (1, 300, 256, [100, 0], None, 128, "bf16", "e4m3"),
    (2, 17, 256, [31, 32, 33], [17, 1, 2], 32, "fp16", "e5m2"),
]


@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_matches_oracle(case, powers):
    Hkv, N, d, lens, counts, ps, dtype, kind = APPEND[case]
    B = len(lens)
    T = (max(lens) + N + ps - 1) // ps
    c = Cache(B, Hkv, T, ps, d, kind, seed=20 + case, powers=powers)
    handle = c.to("cuda")
    rng = np.random.default_rng(40 + case)
    # some heads much larger than what the page holds, some much smaller
    size = np.exp2(rng.integers(-6, 7, (B, Hkv, 1, 1)))
    kf, k = values16(rng.standard_normal((B, Hkv, N, d)) * size, dtype)
    vf, v = values16(rng.standard_normal((B, Hkv, N, d)) / size, dtype)
    k[0, 0, 0, 3] = 0.0
    kf[0, 0, 0, 3] = 0.0
    acc = torch.full((B, Hkv, T * ps), 3.0, device="cuda")
    pos = torch.full((B, Hkv, T * ps), -5, device="cuda", dtype=torch.int32)
    first = torch.arange(1000, 1000 + B, device="cuda", dtype=torch.int32) if case % 2 else None
    new_lens = torch.full((B,), -1, device="cuda", dtype=torch.int32)
    fa.fa_paged_append(handle, k.cuda(), v.cuda(), _lens(lens), new_lens, None if counts is None else _lens(counts),
                       acc, pos, first)
    fa.fa_device_status()
    cnt = [N] * B if counts is None else counts
    assert new_lens.tolist() == [n + x for n, x in zip(lens, cnt)]
    kp, ks = P.append(c.np[0], c.np[2], kind, c.table, kf, lens, cnt)
    vp, vs = P.append(c.np[1], c.np[3], kind, c.table, vf, lens, cnt)
    got = c.read()
    for name, x, y in (("ks", got[2], ks), ("vs", got[3], vs), ("k", got[0], kp), ("v", got[1], vp)):
        assert np.array_equal(x, y), (name, np.argwhere(x != y)[:5], (x != y).sum())
    for b in range(B):
        new = slice(lens[b], lens[b] + cnt[b])
        base = 1000 + b if case % 2 else lens[b]
        assert (acc[b, :, new] == 0).all() and (acc[b, :, :lens[b]] == 3).all() and (acc[b, :, new.stop:] == 3).all()
        assert (pos[b, :, new].cpu() == torch.arange(base, base + cnt[b])).all()
        assert (pos[b, :, :lens[b]] == -5).all() and (pos[b, :, new.stop:] == -5).all()


def test_append_of_zeros_and_of_what_is_not_finite():
    c = Cache(2, 1, 2, 16, 64, "e4m3", seed=30)
    handle = c.to("cuda")
    k = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    v = torch.ones(2, 1, 2, 64, dtype=torch.bfloat16) * 3
    v[0, 0, 0, 0], v[0, 0, 1, 1], v[1, 0, 0, 2] = float("nan"), float("inf"), -float("inf")
    new_lens = torch.zeros(2, device="cuda", dtype=torch.int32)
    fa.fa_paged_append(handle, k.cuda(), v.cuda(), _lens([0, 16]), new_lens)
    fa.fa_device_status()
    got = c.read()
    for b, t in ((0, 0), (1, 1)):
        p = c.table[b, t]
        assert got[2][p, 0] == 2.0 ** -100 and not got[0][p, 0, :2].any()
        assert got[3][p, 0] == 2.0 ** -7  # 3 <= 448 / 2^7
    vals = P.code_values("e4m3")[got[1]]
    assert np.isnan(vals[c.table[0, 0], 0, 0, 0]) and np.isnan(vals[c.table[0, 0], 0, 1, 1])
    assert np.isnan(vals[c.table[1, 1], 0, 0, 2]) and vals[c.table[1, 1], 0, 0, 3] == 384.0
    # largest and smallest 16-bit numbers
    for dt, big, small in ((torch.bfloat16, 3.3895313892515355e38, 9.2e-41), (torch.float16, 65504.0, 6e-8)):
        for kind in ("e4m3", "e5m2"):
            c = Cache(1, 1, 1, 16, 64, kind, seed=31)
            handle = c.to("cuda")
            k = torch.full((1, 1, 1, 64), big, dtype=dt)
            v = torch.full((1, 1, 1, 64), small, dtype=dt)
            fa.fa_paged_append(handle, k.cuda(), v.cuda(), _lens([0]), new_lens[:1])
            fa.fa_device_status()
            got, p = c.read(), c.table[0, 0]
            for pages, scale, x in ((got[0], got[2], k), (got[1], got[3], v)):
                s = P.append_scale(float(x[0, 0, 0, 0].double()), kind)
                assert scale[p, 0] == s
                assert (pages[p, 0, 0] == P.encode(x[0, 0, 0].double().numpy() / s, kind)).all()


def test_append_refuses_on_the_device():
    """A sequence that would not fit, bad counts, bad lengths: left as they are and reported; a wrong page: not written."""
    c = Cache(5, 1, 2, 16, 64, seed=32)
    before = [x.copy() for x in c.np]
    handle = c.to("cuda")
    k = torch.randn(5, 1, 4, 64).bfloat16().cuda()
    new_lens = torch.zeros(5, device="cuda", dtype=torch.int32)
    fa.fa_paged_append(handle, k, k, _lens([29, -1, 33, 5, 5]), new_lens, _lens([4, 1, 0, 5, -1]))
    with pytest.raises(fa.FAError) as e:
        fa.fa_device_status()
    assert e.value.code == 7
    assert new_lens.tolist() == [29, -1, 33, 5, 5]
    assert all(np.array_equal(x, y) for x, y in zip(before, c.read()))
    c.table[:, 1] = [-1, 10 ** 6, 0, 0, 0]
    handle = c.to("cuda")
    fa.fa_paged_append(handle, k, k, _lens([16, 20, 0, 0, 0]), new_lens, _lens([2, 2, 0, 0, 0]))
    with pytest.raises(fa.FAError) as e:
        fa.fa_device_status()
    assert e.value.code == 8 and new_lens.tolist() == [18, 22, 0, 0, 0]
    assert all(np.array_equal(x, y) for x, y in zip(before, c.read()))


# ---------------------------------------------------------------- evict
EVICT = [  # Hkv, d, lens, keep, recent, ps, kind, powers
    (2, 128, [200, 77, 78, 0], 77, 20, 16, "e4m3", True),
    (1, 64, [333, 1], 300, 0, 64, "e4m3", False),
    (3, 256, [150, 149], 33, 33, 32, "e5m2", False),
    (1, 128, [1000], 1, 0, 128, "e4m3", True),
    (2, 64, [1000, 513], 512, 100, 128, "e5m2", True),
    (1, 128, [1025], 1024, 1, 16, "e4m3", False),
    (1, 64, [5000], 2047, 301, 16, "e4m3", False),
]


def _evict_case(case, ties=False, big=None):
    Hkv, d, lens, keep, recent, ps, kind, powers = EVICT[case]
    B = len(lens)
    T = max((max(lens) + ps - 1) // ps, (keep + ps - 1) // ps) + 1
    c = Cache(B, Hkv, T, ps, d, kind, seed=50 + case, powers=powers)
    rng = np.random.default_rng(60 + case)
    w = rng.random((B, Hkv, T * ps)).astype(np.float32)
    if ties:
        w = np.round(w * 3).astype(np.float32) * np.where(rng.random(w.shape) < 0.5, 1, -1).astype(np.float32)
    pos = np.stack([rng.permutation(T * ps) for _ in range(B * Hkv)]).reshape(B, Hkv, T * ps).astype(np.int32)
    return c, w, pos, lens, keep, recent, kind


def _run_evict(c, w, pos, lens, keep, recent):
    handle = c.to("cuda")
    acc, position = torch.from_numpy(w.copy()).cuda(), torch.from_numpy(pos.copy()).cuda()
    new_lens = torch.full((len(lens),), -1, device="cuda", dtype=torch.int32)
    ws = torch.full((fa.fa_paged_evict_workspace_size(handle, keep),), 0xA5, device="cuda", dtype=torch.uint8)
    fa.fa_paged_evict(handle, _lens(lens), new_lens, acc, position, ws, keep, recent)
    return acc, position, new_lens


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict_matches_oracle(case, ties):
    c, w, pos, lens, keep, recent, kind = _evict_case(case, ties)
    acc, position, new_lens = _run_evict(c, w, pos, lens, keep, recent)
    fa.fa_device_status()
    want = P.evict(c.np, kind, c.table, w, pos, np.array(lens), keep, recent)
    got = c.read() + [acc.cpu().numpy(), position.cpu().numpy(), new_lens.cpu().numpy()]
    for name, x, y in zip(("k", "v", "ks", "vs", "weight", "position", "lens"), got, want):
        assert np.array_equal(x, y), (name, np.argwhere(x != y)[:5], (x != y).sum())


def test_evict_odd_weights():
    """NaN, infinities, zeros of both signs, negative weights; equal positions."""
    c, w, pos, lens, keep, recent, kind = _evict_case(0)
    w[0, :, 5:40:7], w[0, :, 6:60:9], w[0, :, 100:130], w[0, :, 130:150] = np.nan, np.inf, 0.0, -0.0
    w[0, :, 8:50:11] = -np.inf
    pos[0, 1] = 4
    for rec in (0, 20):
        acc, position, new_lens = _run_evict(c, w, pos, lens, keep, rec)
        fa.fa_device_status()
        want = P.evict(c.np, kind, c.table, w, pos, np.array(lens), keep, rec)
        got = c.read() + [acc.cpu().numpy(), position.cpu().numpy(), new_lens.cpu().numpy()]
        for name, x, y in zip(("k", "v", "ks", "vs", "weight", "position", "lens"), got, want):
            assert np.array_equal(x, y, equal_nan=x.dtype.kind == "f"), name


@pytest.mark.parametrize("n,ps,kind", [(20400, 16, "many"), (60000, 128, "many"), (60000, 128, "few"),
                                       (170000, 128, "many"), (40000, 64, "zeros")])
def test_evict_long_heads(n, ps, kind):
    """Heads that take one large CTA, a cluster, and more than a cluster holds in registers; many different
    weights, a few, mostly zeros."""
    T = (n + ps - 1) // ps + 1
    c = Cache(1, 1, T, ps, 64, seed=70)
    rng = np.random.default_rng(71)
    w = rng.integers(0, 3 if kind == "few" else 30000, (1, 1, T * ps)).astype(np.float32)
    if kind == "zeros":
        w *= rng.random(w.shape) < 0.1
    pos = np.arange(T * ps, dtype=np.int32).reshape(1, 1, -1)
    keep = n // 3 + 1
    acc, position, new_lens = _run_evict(c, w, pos, [n], keep, 700)
    fa.fa_device_status()
    want = P.evict(c.np, "e4m3", c.table, w, pos, np.array([n]), keep, 700)
    got = c.read() + [acc.cpu().numpy(), position.cpu().numpy(), new_lens.cpu().numpy()]
    assert all(np.array_equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("kind", ["nan", "inf", "huge"])
@pytest.mark.parametrize("n,ps", [(600, 64), (30000, 128)])
def test_evict_many_of_the_largest(kind, n, ps):
    """More slots than stay with NaN, infinite or very large weights over small, and over negative, others."""
    rng = np.random.default_rng(77)
    T = (n + ps - 1) // ps
    for low in (1e-38, 1e-3, -1e-3, -1e30, -3e38):
        c = Cache(1, 2, T, ps, 64, seed=76)
        w = (rng.random((1, 2, T * ps)) * low).astype(np.float32)
        top = rng.random(w.shape) < 0.6
        w[top] = {"nan": np.nan, "inf": np.inf, "huge": 1.0}[kind]
        if kind == "huge":
            w[top] = 3e38 * rng.random(int(top.sum()))
        pos = np.broadcast_to(np.arange(T * ps, dtype=np.int32), w.shape).copy()
        for keep in (n // 2 - 3, n // 5) if n < 1000 else (n // 50,):
            acc, position, new_lens = _run_evict(c, w, pos, [n], keep, 9)
            fa.fa_device_status()
            want = P.evict(c.np, "e4m3", c.table, w, pos, np.array([n]), keep, 9)
            got = c.read() + [acc.cpu().numpy(), position.cpu().numpy(), new_lens.cpu().numpy()]
            assert all(np.array_equal(x, y, equal_nan=x.dtype.kind == "f") for x, y in zip(got, want)), (low, keep)


def test_evict_when_all_weights_are_equal():
    for value in (0.0, -0.0, np.inf, np.nan, -3.0):
        c = Cache(2, 1, 10, 64, 64, seed=72)
        w = np.full((2, 1, 640), value, np.float32)
        pos = np.zeros((2, 1, 640), np.int32)
        pos[:, :, 600:] = 9
        for recent in (0, 5):
            acc, position, new_lens = _run_evict(c, w, pos, [640, 500], 321, recent)
            fa.fa_device_status()
            want = P.evict(c.np, "e4m3", c.table, w, pos, np.array([640, 500]), 321, recent)
            got = c.read() + [acc.cpu().numpy(), position.cpu().numpy(), new_lens.cpu().numpy()]
            assert all(np.array_equal(x, y, equal_nan=x.dtype.kind == "f") for x, y in zip(got, want)), (value, recent)


def test_evict_refuses_on_the_device():
    c, w, pos, lens, keep, recent, kind = _evict_case(0)
    before = [x.copy() for x in c.np]
    acc, position, new_lens = _run_evict(c, w, pos, [-3, 10 ** 6, 70, 0], keep, recent)
    with pytest.raises(fa.FAError) as e:
        fa.fa_device_status()
    assert e.value.code == 7 and new_lens.tolist() == [-3, 10 ** 6, 70, 0]
    c.table[0, 3] = -1
    acc, position, new_lens = _run_evict(c, w, pos, [200, 77, 3, 0], keep, recent)
    with pytest.raises(fa.FAError) as e:
        fa.fa_device_status()
    assert e.value.code == 8 and new_lens.tolist() == [200, 77, 3, 0]
    assert all(np.array_equal(x, y) for x, y in zip(before, c.read()))
    assert np.array_equal(acc.cpu().numpy(), w) and np.array_equal(position.cpu().numpy(), pos)


# ---------------------------------------------------------------- together
def test_a_run_of_them_together():
    """Prompt, decoding steps that count weights, eviction to a budget, more steps: the cache holds at every
    step what the oracle makes of the same calls, and attention is exact on what it holds."""
    B, Hkv, g, d, ps, T, kind = 2, 2, 4, 64, 16, 12, "e4m3"
    c = Cache(B, Hkv, T, ps, d, kind, seed=80)
    handle = c.to("cuda")
    rng = np.random.default_rng(81)
    acc = torch.zeros(B, Hkv, T * ps, device="cuda")
    pos = torch.zeros(B, Hkv, T * ps, device="cuda", dtype=torch.int32)
    a, bb = _lens([0, 0]), _lens([0, 0])
    ws_e = torch.empty(fa.fa_paged_evict_workspace_size(handle, 96), dtype=torch.uint8, device="cuda")
    state = [x.copy() for x in c.np]
    n, seen = [0, 0], [0, 0]
    for step in range(40):
        N = 100 if step == 0 else 1 + step % 3
        cnt = [N, max(1, N - 30)] if step == 0 else [N, 1]
        kf, k = values16(rng.standard_normal((B, Hkv, N, d)) * (1 + step % 5), "bf16")
        vf, v = values16(rng.standard_normal((B, Hkv, N, d)), "bf16")
        fa.fa_paged_append(handle, k.cuda(), v.cuda(), a, bb, _lens(cnt), acc, pos, _lens(seen))
        state[0], state[2] = P.append(state[0], state[2], kind, c.table, kf, n, cnt)
        state[1], state[3] = P.append(state[1], state[3], kind, c.table, vf, n, cnt)
        n, seen = [x + y for x, y in zip(n, cnt)], [x + y for x, y in zip(seen, cnt)]
        qf, q = values16(rng.standard_normal((B, g * Hkv, 1, d)), "bf16")
        before = acc.cpu().double().numpy()
        o, lse = fa.forward_paged(handle, q.cuda(), bb, causal=True, weight_acc=acc)
        fa.fa_device_status()
        assert bb.tolist() == n
        assert all(np.array_equal(x, y) for x, y in zip(c.read(), state)), step
        check_attention(qf, c, n, 1 / 8, True, "bf16", o, lse, acc, kv=state, added=before)
        w, p = acc.cpu().numpy(), pos.cpu().numpy()
        fa.fa_paged_evict(handle, bb, a, acc, pos, ws_e, 96, 24)
        fa.fa_device_status()
        want = P.evict(state, kind, c.table, w, p, np.array(n), 96, 24)
        got = c.read() + [acc.cpu().numpy(), pos.cpu().numpy(), a.cpu().numpy()]
        assert all(np.array_equal(x, y) for x, y in zip(got, want)), step
        state, n = list(want[:4]), want[6].tolist()
    assert n == [96, 96]


def test_steps_in_a_graph_and_on_another_stream():
    """Append, attention with weights and eviction captured on a side stream: replays equal the same calls made eagerly."""
    B, Hkv, g, d, ps, T = 2, 1, 2, 128, 32, 5
    rng = np.random.default_rng(90)
    k, v = (torch.from_numpy(rng.standard_normal((B, Hkv, 2, d))).bfloat16().cuda() for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((B, g, 1, d))).bfloat16().cuda()

    def fresh():
        c = Cache(B, Hkv, T, ps, d, seed=91)
        h = c.to("cuda")
        s = dict(c=c, h=h, acc=torch.ones(B, Hkv, T * ps, device="cuda"),
                 pos=torch.arange(T * ps, device="cuda", dtype=torch.int32).repeat(B, Hkv, 1), a=_lens([128, 128]),
                 b=_lens([0, 0]), o=torch.zeros(B, g, 1, d, device="cuda", dtype=torch.bfloat16),
                 lse=torch.zeros(B, g, 1, device="cuda"), first=_lens([T * ps, T * ps]))
        s["ws"] = torch.empty(fa.fa_paged_workspace_size(h, g, 1, weights=True), dtype=torch.uint8, device="cuda")
        s["wse"] = torch.empty(fa.fa_paged_evict_workspace_size(h, 128), dtype=torch.uint8, device="cuda")
        return s

    def step(s):
        fa.fa_paged_append(s["h"], k, v, s["a"], s["b"], None, s["acc"], s["pos"], s["first"])
        fa.fa_forward_paged(s["h"], q, s["b"], s["o"], s["lse"], s["ws"], causal=True, weight_acc=s["acc"])
        fa.fa_paged_evict(s["h"], s["b"], s["a"], s["acc"], s["pos"], s["wse"], 128, 10)
        s["first"].add_(2)

    eager, graphed = fresh(), fresh()
    for _ in range(5):
        step(eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(graphed)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(graphed)
        for _ in range(4):
            graph.replay()
    torch.cuda.current_stream().wait_stream(side)
    fa.fa_device_status()
    for name in ("acc", "pos", "a", "b", "o", "lse"):
        assert torch.equal(eager[name], graphed[name]), name
    assert all(np.array_equal(x, y) for x, y in zip(eager["c"].read(), graphed["c"].read()))


def test_python_refusals():
    c = Cache(2, 2, 4, 32, 64, seed=95)
    h = c.to("cuda")
    k, v, ks, vs, table = c.t
    with pytest.raises(TypeError):
        fa.PagedCache(k.view(torch.uint8), v, ks, vs, table)
    with pytest.raises(TypeError):
        fa.PagedCache(k, v, ks, vs, table.long())
    with pytest.raises(ValueError):
        fa.PagedCache(k, v, ks[:, :1].contiguous(), vs, table)
    with pytest.raises(ValueError):
        fa.PagedCache(k.transpose(1, 2), v, ks, vs, table)
    with pytest.raises(TypeError):
        fa.PagedCache(k.cpu(), v, ks, vs, table)
    q = torch.zeros(2, 4, 1, 64, device="cuda", dtype=torch.bfloat16)
    lens = _lens([3, 3])
    for bad in (q[:, :, :, :32], q[:1], q.transpose(0, 1), q.cpu()):
        with pytest.raises((ValueError, TypeError)):
            fa.forward_paged(h, bad, lens)
    with pytest.raises(TypeError):
        fa.forward_paged(h, q.float(), lens)
    with pytest.raises(ValueError):
        fa.forward_paged(h, q, lens.long())
    with pytest.raises(ValueError):
        fa.forward_paged(h, q, lens, weight_acc=torch.zeros(2, 2, 64, device="cuda"))
    with pytest.raises(fa.FAError):
        fa.forward_paged(h, q[:, :3].contiguous(), lens)
    for kw in (dict(max_len=1 << 32), dict(num_splits=(1 << 32) + 1)):
        with pytest.raises(ValueError):
            fa.forward_paged(h, q, lens, **kw)
    with pytest.raises(ValueError):
        fa.fa_paged_evict_workspace_size(h, (1 << 32) + 5)
    acc, pos = torch.zeros(2, 2, 128, device="cuda"), torch.zeros(2, 2, 128, device="cuda", dtype=torch.int32)
    ws = torch.empty(1 << 20, device="cuda", dtype=torch.uint8)
    for keep, recent in (((1 << 32) + 5, 1), (5, 1 << 32)):
        with pytest.raises(ValueError):
            fa.fa_paged_evict(h, lens, lens.clone(), acc, pos, ws, keep, recent)
    new = torch.zeros(2, 2, 1, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(fa.FAError):
        fa.fa_paged_append(h, new, new, lens, lens)
    with pytest.raises(ValueError):
        fa.fa_paged_append(h, new, new.half(), lens, lens.clone())
    fa.fa_device_status()


# ---------------------------------------------------------------- large pools, streams, the example
def test_pools_beyond_32_bits():
    """Pages whose codes lie past 2^31 and 2^32 bytes: the same bits as from a small pool."""
    B, Hkv, ps, d, T = 2, 8, 128, 256, 5
    c = Cache(B, Hkv, T, ps, d, seed=300)
    n = len(c.np[0])
    small = c.to("cuda")
    page = Hkv * ps * d  # bytes
    P = (1 << 32) // page + n + 3
    far = (torch.arange(n) * 1 + P - n).tolist()
    far[::2] = [(1 << 31) // page + i for i in range(len(far[::2]))]  # some past 2^31, some past 2^32
    far = torch.tensor(far)
    k, v = (torch.empty(P, Hkv, ps, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(P, Hkv, device="cuda") for _ in range(2))
    for big, x in ((k, c.t[0].view(torch.uint8)), (v, c.t[1].view(torch.uint8)), (ks, c.t[2]), (vs, c.t[3])):
        big[far.cuda()] = x
    table = far.to(torch.int32).cuda()[c.t[4].long()].contiguous()
    large = fa.PagedCache(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs, table)
    _, q = _q(B, 16, 1, d, "bf16", 301)
    got = []
    for cache in (small, large):
        lens, now = _lens([600, 577]), _lens([0, 0])
        acc = torch.zeros(B, Hkv, T * ps, device="cuda")
        pos = torch.zeros_like(acc, dtype=torch.int32)
        new = torch.randn(B, Hkv, 3, d, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
        fa.fa_paged_append(cache, new, new * 2, lens, now, None, acc, pos)
        pos.copy_(torch.arange(T * ps, device="cuda"))
        o, lse = fa.forward_paged(cache, q.cuda(), now, weight_acc=acc)
        ws = torch.empty(fa.fa_paged_evict_workspace_size(cache, 500), dtype=torch.uint8, device="cuda")
        fa.fa_paged_evict(cache, now, lens, acc, pos, ws, 500, 50)
        o2, lse2 = fa.forward_paged(cache, q.cuda(), lens)
        fa.fa_device_status()
        got.append((o, lse, acc, pos, lens, o2, lse2))
    assert all(torch.equal(x, y) for x, y in zip(*got))
    for big, x in ((k, c.t[0].view(torch.uint8)), (ks, c.t[2])):
        assert torch.equal(big[far.cuda()], x)


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace, on streams other than the tensors' own."""
    runs = []
    for i, (B, Hq, Hkv, Nq, d, n) in enumerate([(3, 8, 2, 1, 128, 9000), (2, 16, 2, 4, 256, 5000), (4, 4, 4, 1, 64, 7000)]):
        c = Cache(B, Hkv, (n + 63) // 64, 64, d, seed=310 + i)
        _, q = _q(B, Hq, Nq, d, "bf16", 320 + i)
        runs.append((c.to("cuda"), q.cuda(), _lens([n, n - 777, 5, 300][:B]), c))
    alone = [fa.forward_paged(h, q, lens, causal=True) for h, q, lens, _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        streams = [torch.cuda.Stream() for _ in runs]
        got = [fa.forward_paged(h, q, lens, causal=True, stream=s) for (h, q, lens, _), s in zip(runs, streams)]
        for s in streams:
            s.synchronize()
        fa.fa_device_status()
        assert all(torch.equal(x, y) for a, b in zip(alone, got) for x, y in zip(a, b))
    o, lse = fa.forward_paged(*runs[0][:3], causal=True, stream=streams[0].cuda_stream)  # a raw handle
    streams[0].synchronize()
    assert torch.equal(o, alone[0][0])


def test_the_loop_of_the_documentation():
    P, Hkv, ps, d, B, T = 128, 8, 64, 128, 4, 16
    k, v = (torch.zeros(P, Hkv, ps, d, device="cuda", dtype=torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(P, Hkv, device="cuda") for _ in range(2))
    table = torch.randperm(P, device="cuda")[:B * T].view(B, T).int()
    cache = fa.PagedCache(k, v, ks, vs, table)
    lens, now = (torch.zeros(B, device="cuda", dtype=torch.int32) for _ in range(2))
    weight = torch.zeros(B, Hkv, cache.slots, device="cuda")
    pos, first = torch.zeros_like(weight, dtype=torch.int32), torch.zeros_like(lens)
    ws = torch.empty(fa.fa_paged_evict_workspace_size(cache, 512), device="cuda", dtype=torch.uint8)
    for N in (500, 1, 30, 1, 1):
        k_new, v_new = (torch.randn(B, Hkv, N, d, device="cuda").bfloat16() for _ in range(2))
        q = torch.randn(B, 32, N if N > 1 else 1, d, device="cuda").bfloat16()
        fa.fa_paged_append(cache, k_new, v_new, lens, now, weight_acc=weight, positions=pos, first_position=first)
        o, lse = fa.forward_paged(cache, q, now, causal=True, weight_acc=weight)
        fa.fa_paged_evict(cache, now, lens, weight, pos, ws, keep=512, recent=256)
        first += N
        fa.fa_device_status()
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert lens.tolist() == [512] * B and first.tolist() == [533] * B
    # the last 256 tokens are all there, in every head
    for b in range(B):
        for h in range(Hkv):
            assert set(range(533 - 256, 533)) <= set(pos[b, h, :512].tolist())
