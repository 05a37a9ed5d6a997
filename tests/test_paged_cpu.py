"""Refusals of the paged-cache entry points: every bad argument is answered
with its status before any CUDA work (no GPU needed)."""
import ctypes

import pytest

from exact_io_aware_forward_gb300 import build as fa_build

PTR = 1 << 20  # aligned, never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    from exact_io_aware_forward_gb300 import _lib
    return _lib.lib()


def cache(**kw):
    from exact_io_aware_forward_gb300._lib import PagedCacheStruct
    a = dict(k_pages=PTR, v_pages=PTR, k_scale=PTR, v_scale=PTR, page_table=PTR, num_pages=40, pages_per_seq=8, B=2,
             Hkv=4, page_size=64, d=128, cache_dtype=0)
    a.update(kw)
    return ctypes.byref(PagedCacheStruct(**a))


BAD_CACHES = [(dict(num_pages=0), INVALID), (dict(B=0), INVALID), (dict(Hkv=-1), INVALID),
              (dict(pages_per_seq=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
              (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
              (dict(cache_dtype=2), UNSUPPORTED), (dict(num_pages=1 << 30), UNSUPPORTED),
              (dict(pages_per_seq=1 << 25), UNSUPPORTED), (dict(B=20000), UNSUPPORTED),
              (dict(k_pages=None), INVALID), (dict(v_pages=PTR + 8), INVALID), (dict(k_scale=PTR + 4), INVALID),
              (dict(v_scale=None), INVALID), (dict(page_table=PTR + 4), INVALID)]


def attend(lib, c, q=PTR, lens=PTR, o=PTR, lse=PTR, acc=None, Hq=8, Nq=1, dt=1, scale=0.1, max_len=0, splits=0, ws=PTR,
           ws_bytes=1 << 40):
    return lib.fa_forward_paged(c, q, lens, o, lse, acc, Hq, Nq, dt, 1, scale, max_len, splits, ws, ws_bytes, None)


def append(lib, c, k=PTR, v=PTR, lens=PTR, counts=None, new_lens=2 * PTR, acc=None, pos=None, first=None, N=3, dt=1):
    return lib.fa_paged_append(c, k, v, lens, counts, new_lens, acc, pos, first, N, dt, None)


def evict(lib, c, lens=PTR, new_lens=2 * PTR, acc=PTR, pos=PTR, keep=100, recent=10, ws=PTR, ws_bytes=1 << 40):
    return lib.fa_paged_evict(c, lens, new_lens, acc, pos, keep, recent, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches(lib, kw, want):
    assert attend(lib, cache(**kw)) == want
    assert append(lib, cache(**kw)) == want
    assert evict(lib, cache(**kw)) == want
    if not any("pages" == k[2:] or "scale" in k or "table" in k for k in kw):
        assert lib.fa_paged_workspace_size(cache(**kw), 8, 1, 0, 0, 1) == 0
        assert lib.fa_paged_evict_workspace_size(cache(**kw), 10) == 0


def test_null_cache(lib):
    assert attend(lib, None) == INVALID and append(lib, None) == INVALID and evict(lib, None) == INVALID
    assert lib.fa_paged_workspace_size(None, 8, 1, 0, 0, 0) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(q=PTR + 2), INVALID), (dict(lens=None), INVALID), (dict(lens=PTR + 2), INVALID),
    (dict(o=PTR + 8), INVALID), (dict(lse=None), INVALID), (dict(acc=PTR + 4), INVALID), (dict(Hq=6), INVALID),
    (dict(Hq=0), INVALID), (dict(Nq=0), INVALID), (dict(dt=2), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=3e38), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(max_len=513), INVALID),
    (dict(max_len=-1), INVALID), (dict(splits=-1), INVALID), (dict(splits=1025), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=PTR + 16), WORKSPACE), (dict(splits=4, ws_bytes=100), WORKSPACE), (dict(acc=PTR, ws_bytes=100), WORKSPACE),
    (dict(Nq=1 << 22), UNSUPPORTED)])
def test_bad_attention_arguments(lib, kw, want):
    assert attend(lib, cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(v=PTR + 2), INVALID), (dict(lens=None), INVALID), (dict(new_lens=None), INVALID),
    (dict(new_lens=PTR), INVALID), (dict(new_lens=PTR + 4), INVALID), (dict(counts=PTR + 1), INVALID),
    (dict(counts=2 * PTR), INVALID), (dict(first=2 * PTR + 4), INVALID), (dict(acc=PTR + 4), INVALID),
    (dict(pos=PTR + 4), INVALID), (dict(first=PTR + 3), INVALID), (dict(N=0), INVALID), (dict(dt=5), UNSUPPORTED)])
def test_bad_append_arguments(lib, kw, want):
    assert append(lib, cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(lens=None), INVALID), (dict(new_lens=PTR), INVALID), (dict(new_lens=PTR - 4), INVALID),
    (dict(acc=None), INVALID), (dict(pos=None), INVALID), (dict(acc=PTR + 4), INVALID), (dict(keep=0), INVALID),
    (dict(keep=513), INVALID), (dict(recent=-1), INVALID), (dict(recent=101), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=PTR + 128), WORKSPACE), (dict(ws_bytes=64), WORKSPACE)])
def test_bad_evict_arguments(lib, kw, want):
    assert evict(lib, cache(), **kw) == want


def test_workspace_sizes(lib):
    """O and LSE of two parts a CTA, 8 G rows each; scores of every row and slot for the weights."""
    size = lib.fa_paged_workspace_size

    def parts(n, rows, d=128):
        return n * rows * d * 4 + (n * rows * 4 + 255) // 256 * 256

    # one chunk, or at most 512 slots: nothing to merge
    assert size(cache(), 8, 1, 0, 1, 0) == 256 and size(cache(), 8, 1, 512, 0, 0) == 256
    # 2 x 4 heads, 6 rows (a tile of 8), four chunks
    assert size(cache(), 8, 3, 512, 4, 0) == parts(2 * 8 * 4, 8)
    assert size(cache(), 8, 3, 512, 4, 1) == parts(2 * 8 * 4, 8) + 8 * 8 * 512 * 4
    assert size(cache(), 4, 3, 512, 4, 1) == parts(2 * 8 * 4, 8) + 8 * 4 * 512 * 4
    # 50 rows: two tiles of 32
    assert size(cache(), 8, 25, 512, 2, 0) == parts(2 * 8 * 2 * 2, 32)
    # a count that leaves a last chunk empty is lowered
    assert size(cache(), 8, 1, 300, 1000, 0) == parts(2 * 8 * 3, 8)
    # a chunk has at most 16384 slots
    big = cache(pages_per_seq=1 << 11, num_pages=1 << 12)
    assert size(big, 8, 1, 0, 1, 0) == parts(2 * 8 * 8, 8)
    # shared out evenly: a CTA for a head's start and two tiles at least, no more CTAs than fit (152 SMs without a GPU) ...
    mid = cache(pages_per_seq=16)
    assert size(mid, 8, 1, 0, 0, 0) == parts(2 * 8 * (8 + 4) // 6, 8) + 256
    assert size(big, 8, 1, 0, 0, 0) == parts(2 * 304, 8) + 256
    assert size(big, 80, 2, 0, 0, 0) == parts(2 * 152, 40) + 256
    # ... unless one would get more than 127 tiles
    huge = cache(pages_per_seq=1 << 15, num_pages=1 << 17)
    assert size(huge, 8, 1, 0, 0, 0) == parts(2 * -(-8 * ((1 << 14) + 4) // 127), 8) + 256
    # slots that cannot be merged
    assert size(cache(pages_per_seq=1 << 20, num_pages=1 << 21), 8, 1, 0, 0, 0) == 0
    ev = lib.fa_paged_evict_workspace_size
    assert ev(cache(), 100) == 256 + 256 + 2 * 3328 + 256 and ev(cache(), 0) == 0 and ev(cache(), 513) == 0


def test_status_has_a_name(lib):
    from exact_io_aware_forward_gb300._lib import status_string
    assert status_string(8).startswith("FA_ERR_PAGES")
