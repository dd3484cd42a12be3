"""kvq8_paged_copy and kvq8_paged_compact: every byte of the planes against the same moves on the host."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._paged import i32, masks64, starts_of, tree_words  # noqa: E402

pytestmark = pytest.mark.gpu


def _cache(seed, pages, hkv, page, hd):
    """A cache of random bits, and its planes on the host."""
    from speculative_verify_attention_gb300 import KVPagedCacheQ8
    rng = np.random.default_rng(seed)
    codes = [rng.integers(-128, 128, (pages, hkv, page, hd)).astype(np.int8) for _ in range(2)]
    scales = [rng.integers(0, 1 << 16, (pages, hkv, page, hd // 32)).astype(np.uint16) for _ in range(2)]
    t = [torch.from_numpy(c).cuda() for c in codes] + [torch.from_numpy(s.view(np.float16)).cuda() for s in scales]
    return KVPagedCacheQ8.from_planes(t[0], t[2], t[1], t[3]), codes + scales


def _same(cache, planes):
    torch.cuda.synchronize()
    for t, w in zip((cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales), planes):
        g = t.cpu().numpy()
        assert np.array_equal(g.view(np.uint16) if g.dtype == np.float16 else g, w)


SHAPES = [(4, 256, 16), (1, 256, 128), (2, 128, 32), (8, 128, 16), (3, 128, 64), (1, 128, 1024)]


@pytest.mark.parametrize("hkv,hd,page", SHAPES)
def test_copies_of_some_rows(lib, hkv, hd, page):
    from speculative_verify_attention_gb300 import kvq8_paged_copy
    rng = np.random.default_rng(page)
    for n in (1, 5, 40):
        pages = 3 * n + 4
        cache, planes = _cache(n, pages, hkv, page, hd)
        order = rng.permutation(pages)
        src, dst = order[:n].copy(), order[n:2 * n].copy()
        src[n // 2:] = src[0]                                        # one page to several
        rows = rng.integers(0, page + 1, n)
        rows[0] = page
        if n > 4:
            src[1], dst[2], rows[3], rows[4] = -1, pages, -3, page + 9
            dst[n - 1] = src[n - 1]                                  # onto itself
            src[n - 2] = 2 ** 31 - 1
        kvq8_paged_copy(cache, i32(src), i32(dst), i32(rows))
        for a, b, r in zip(src, dst, rows):
            if 0 <= a < pages and 0 <= b < pages and a != b:
                for p in planes:
                    p[b, :, :max(0, min(r, page))] = p[a, :, :max(0, min(r, page))]
        _same(cache, planes)
        a, b = order[2 * n], order[2 * n + 1]
        kvq8_paged_copy(cache, i32([a]), i32([b]))                   # whole pages
        for p in planes:
            p[b] = p[a]
        _same(cache, planes)


def _compact(seed, lens, rows, kept, hkv, hd, page, table=None, out=True, width=None):
    """One call over a cache of random bits, checked."""
    from speculative_verify_attention_gb300 import kvq8_paged_compact
    rng = np.random.default_rng(seed)
    n = len(lens)
    held = [max(0, -(-x // page)) for x in lens]
    pages = sum(held) + 3
    width = width or max(held + [1])
    if table is None:
        table, order, at = np.full((n, width), -9, np.int32), rng.permutation(pages), 0
        for b, h in enumerate(held):
            table[b, :min(h, width)] = order[at:at + h][:width]
            at += h
    cache, planes = _cache(seed, pages, hkv, page, hd)
    lens_out = torch.full((n,), -5, dtype=torch.int32, device="cuda")
    kvq8_paged_compact(cache, i32(table), i32(lens), i32(starts_of(rows)), masks64(kept), lens_out=lens_out if out else None)
    want = list(lens)
    for b in range(n):
        t = rows[b]
        if not 0 <= t <= 64 or t > lens[b] or lens[b] > width * page:
            continue
        places = [j for j in range(t) if kept[b] >> j & 1]
        want[b] = lens[b] - t + len(places)
        moves = []
        for k, j in enumerate(places):
            a, d = lens[b] - t + j, lens[b] - t + k
            pa, pd = int(table[b, a // page]), int(table[b, d // page])
            if 0 <= pa < pages and 0 <= pd < pages:
                moves.append((pd, d % page, [p[pa, :, a % page].copy() for p in planes]))
        for pd, off, values in moves:
            for p, v in zip(planes, values):
                p[pd, :, off] = v
    _same(cache, planes)
    assert not out or lens_out.tolist() == want


@pytest.mark.parametrize("hkv,hd,page", SHAPES)
def test_kept_rows_move_together(lib, hkv, hd, page):
    rng = np.random.default_rng(page + hd)
    rows = [1, 2, 7, 16, 33, 63, 64, 64, 64, 12]
    lens = [t + int(rng.integers(0, 3 * page)) for t in rows]
    for k in range(3):
        kept = [int(rng.integers(0, 1 << 62)) | int(rng.integers(0, 4)) << 62 for _ in rows]
        kept[7], kept[8] = (2 ** 64 - 1, 1 << 63) if k else (2 ** 64 - 2, 0)
        kept[9] |= (2 ** 64 - 1) << 12 & (2 ** 64 - 1)                # bits behind the window
        _compact(k, lens, rows, kept, hkv, hd, page, out=k != 1)


def test_paths_of_trees_and_windows_alone(lib):
    rng = np.random.default_rng(4)
    rows = [int(x) for x in rng.integers(1, 65, 60)]
    kept = [tree_words(t, rng)[int(rng.integers(t))] for t in rows]
    _compact(7, rows, rows, kept, 2, 128, 16)                         # no context before the window
    _compact(8, [t + 100 for t in rows], rows, kept, 2, 128, 16)


def test_malformed_requests_and_pages_are_left(lib):
    lens, rows = [40, 5, 30, 20, 0, 70, 90], [8, 9, 0, 3, 0, 65, 64]
    kept = [0b10110010] * 7
    _compact(1, lens, rows, kept, 2, 128, 16)
    _compact(2, lens, rows, kept, 2, 128, 16, width=3)                # longer than the table is wide
    table = np.array([[3, -1, 99], [0, 1, 2], [4, 5, 6]], np.int32)
    _compact(3, [40, 36, 40], [20, 9, 20], [0x8fff3, 0x1f0, 0xf0f0a], 2, 128, 16, table=table)


def test_thousands_of_requests(lib):
    rng = np.random.default_rng(5)
    rows = [int(x) for x in rng.integers(0, 6, 4096)]
    _compact(9, [t + int(rng.integers(0, 9)) for t in rows], rows, [int(x) for x in rng.integers(0, 64, 4096)], 1, 128, 16)


def test_rows_far_into_a_large_pool(lib):
    """Element offsets past 2^32: 5.4 GB of codes a plane, and the last pages are the ones that move."""
    from speculative_verify_attention_gb300 import KVPagedCacheQ8, kvq8_paged_append, kvq8_paged_append_rope, kvq8_paged_compact, kvq8_paged_copy, rope_turns
    pages, hkv, page, hd = 20500, 8, 128, 256
    cache = KVPagedCacheQ8(hkv, hd, page, pages)
    assert cache.k_codes.numel() > 2 ** 32
    x = torch.randn((8, hkv, hd), device="cuda")
    last = (pages - 1) * page
    kvq8_paged_append(x, 2 * x, cache, torch.arange(last, last + 8, device="cuda"))
    kvq8_paged_copy(cache, i32([pages - 1]), i32([pages - 3]), i32([8]))
    for p in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        assert torch.equal(p[pages - 1, :, :8], p[pages - 3, :, :8]) and p[pages - 3, :, :8].abs().sum() > 0
    kvq8_paged_compact(cache, i32([[pages - 3]]), i32([8]), i32([0, 8]), masks64([0b10100001]))
    for p in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        assert torch.equal(p[pages - 3, :, :3], p[pages - 1, :, [0, 5, 7]])
    kvq8_paged_append_rope(x.repeat(1, 2, 1), x, 2 * x, cache, torch.arange(last - 2 * page, last - 2 * page + 8, device="cuda") + page,
                           i32([0] * 8), rope_turns(torch.ones(64)).cuda())
    for p in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        assert torch.equal(p[pages - 2, :, :8], p[pages - 1, :, :8])
