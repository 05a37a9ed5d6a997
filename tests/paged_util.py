"""Inputs for the paged-cache tests and the bounds that results are held to."""
import numpy as np
import torch

import exact_io_aware_forward_gb300 as fa
from oracle import paged as P

TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
# half a step of the 16-bit types, relative to the value
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
# a softmax weight split into e4m3 terms: 4 significant bits each (a code is off by at most 2^-4), two or three terms
WEIGHT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -12}
# what of a weight may be lost, relative to the chunk's largest: half the smallest code (2^-10) of the last
# term, which is scaled by 16 (256), of weights scaled by 256 over the reference
LOST = {"bf16": 2.0 ** -22, "fp16": 2.0 ** -26}


def values16(x, dtype):
    """numpy float64 of x rounded to the 16-bit type, and the CPU tensor."""
    t = torch.from_numpy(np.asarray(x, dtype=np.float32)).to(DT[dtype])
    return t.double().numpy(), t


class Cache:
    """A pool with random contents (float64 codes by the oracle's encoder), its numpy arrays and its device tensors."""

    def __init__(self, B, Hkv, T, ps, d, kind="e4m3", seed=0, spread=1.0, spare=3, powers=False):
        rng = np.random.default_rng(seed)
        n = B * T + spare
        self.kind, self.ps, self.T, self.B, self.Hkv, self.d = kind, ps, T, B, Hkv, d
        self.np = []
        scales = []
        for _ in range(2):
            s = np.exp2(rng.uniform(-spread, spread, (n, Hkv)) - 6).astype(np.float32)
            if powers:
                s = np.exp2(np.round(np.log2(s))).astype(np.float32)
            x = rng.standard_normal((n, Hkv, ps, d))
            top = P.LARGEST[kind]
            self.np.append(P.encode(np.clip(x * 64 * (1 if kind == "e4m3" else 64), -top, top), kind))
            scales.append(s if kind == "e4m3" else s / 64)
        self.np += scales
        self.table = rng.permutation(n)[:B * T].reshape(B, T).astype(np.int32)

    def to(self, dev):
        k, v, ks, vs = (torch.from_numpy(x.copy()) for x in self.np)
        self.t = [k.to(dev).view(TORCH[self.kind]), v.to(dev).view(TORCH[self.kind]), ks.to(dev), vs.to(dev),
                  torch.from_numpy(self.table.copy()).to(dev)]
        return fa.PagedCache(*self.t)

    def read(self):
        """The device's pages and scales as numpy arrays."""
        return [self.t[0].view(torch.uint8).cpu().numpy(), self.t[1].view(torch.uint8).cpu().numpy(),
                self.t[2].cpu().numpy(), self.t[3].cpu().numpy()]


def check_attention(q, cache, lens, scale, causal, dtype, o, lse, weights=None, kv=None, added=0.0):
    """Holds O, LSE and the added weights against the oracle on the same codes, element by element."""
    kv = cache.np if kv is None else kv
    ro, rl, rw, mass = P.attention(q, kv, cache.kind, cache.table, lens, scale, causal)
    of, lf = o.cpu().double().numpy(), lse.cpu().double().numpy()
    assert np.array_equal(np.isfinite(lf), np.isfinite(rl))
    seen = np.isfinite(rl)
    # scores: d products and sums in float32 (each off by 2^-24 of the sum of magnitudes, d + 8 of them at most), and
    # the parts of q below 2^-22 of its row's largest
    top_k = P.LARGEST[cache.kind] * float(np.abs(kv[2]).max())
    vals = np.nan_to_num(P.code_values(cache.kind), nan=0.0, posinf=0.0, neginf=0.0)
    k_abs = float((np.abs(vals[kv[0]]).max(axis=(2,)) * kv[2][..., None]).sum(axis=2).max())  # sum over d of max |k|
    q_top = float(np.abs(q).max())
    size = scale * q_top * min(k_abs, top_k * q.shape[3])
    ds = size * ((q.shape[3] + 8) * 2.0 ** -24 + 2.0 ** -22)
    # exponentials and sums: ex2 and its argument (2^-22 each of up to 2 log2 units a doubling), the sums' rounding
    tol_lse = ds + 2.0 ** -20 * (1.0 + np.abs(np.where(seen, rl, 0.0)))
    off_lse = np.abs(np.where(seen, lf, 0.0) - np.where(seen, rl, 0.0))
    assert (off_lse <= tol_lse).all(), off_lse.max()
    n = min(int(max(lens)), 16384)
    v_top = P.LARGEST[cache.kind] * float(np.abs(kv[3]).max())
    tol = HALF_STEP[dtype] * np.abs(ro) + (WEIGHT[dtype] + 2 * ds + 2.0 ** -18) * mass + n * LOST[dtype] * v_top + 1e-30
    off = np.abs(of - ro) - tol
    assert (off <= 0).all(), (float(np.abs(of - ro).max()), float(off.max()), np.argwhere(off > 0)[:5])
    if weights is not None:
        wf = weights.cpu().double().numpy()
        tol_w = (rw * (2 * ds + 2.0 ** -18)) + 2.0 ** -23 * np.abs(added + rw) * (q.shape[1] * q.shape[2]) + 1e-30
        # slots that are not seen are not touched
        bad = np.abs(wf - (added + rw)) - tol_w
        assert (bad <= 0).all(), (float(bad.max()), np.argwhere(bad > 0)[:5])
    return float(np.abs(of - ro).max()), float(off_lse.max())
