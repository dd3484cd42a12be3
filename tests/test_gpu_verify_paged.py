"""attn_verify_paged_q8 against its definition in 64 bits, with a bound derived element by element (Batch.expect)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._paged import Batch, i32  # noqa: E402

pytestmark = pytest.mark.gpu


def _clean():
    from speculative_verify_attention_gb300 import kvq8_device_error
    assert kvq8_device_error(reset=True) == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,hd", [(4, 4, 128), (8, 2, 128), (6, 1, 256), (24, 4, 256)])
@pytest.mark.parametrize("tree", [False, True])
def test_small_ragged_batches(lib, dtype, hq, hkv, hd, tree):
    b = Batch(hq + hd, hq, hkv, hd, 16, [1, 70, 17, 3, 129, 64], [1, 5, 2, 3, 1, 4], dtype, tree, pad_rows=2)
    b.check(b.call())
    _clean()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("hd", [128, 256])
def test_pages_end_inside_and_outside_tiles(lib, page, hd):
    lens = [page - 1, page, page + 1, 2 * page + 5, 63, 64, 65, 128, 129]
    b = Batch(page + hd, 4, 2, hd, page, lens, [1, 2, 3, 4, 5, 1, 2, 3, 4])
    b.check(b.call())
    _clean()


@pytest.mark.parametrize("rows,hq,hkv,hd", [(1, 64, 1, 128), (33, 4, 1, 128), (64, 6, 1, 256), (64, 64, 1, 128), (43, 12, 4, 256),
                                            (16, 8, 1, 128), (17, 8, 1, 128)])
def test_row_counts_around_the_row_tile(lib, rows, hq, hkv, hd):
    b = Batch(rows, hq, hkv, hd, 32, [rows, rows + 131], [rows, rows], torch.float16, tree=True)
    b.check(b.call())
    _clean()


@pytest.mark.parametrize("hd", [128, 256])
def test_empty_windows_empty_masks_and_no_context(lib, hd):
    """Requests without rows, rows that see nothing (zeros), and windows with nothing before them."""
    b = Batch(5, 8, 2, hd, 16, [40, 3, 0, 80, 4, 0], [0, 3, 0, 2, 4, 0], tree=True)
    s = b.starts
    b.words[s[1]] = 0               # no context, no key: zeros
    b.words[s[1] + 1] = 0b100       # sees only a later key of its window
    b.words[s[3]] = 0               # context only
    b.words[s[4] + 3] = 2 ** 64 - 1  # bits behind the window count for nothing
    out = b.call()
    b.check(out)
    assert not out[s[1]].any()
    _clean()


def test_all_requests_empty_leave_the_output(lib):
    b = Batch(6, 4, 1, 128, 16, [9, 5], [0, 0], pad_rows=3)
    out = b.call(max_rows=4)
    assert torch.all(out == 77.0)
    _clean()


def test_malformed_requests_are_left_alone(lib):
    b = Batch(7, 8, 2, 128, 16, [40, 50, 30, 20], [3, 2, 4, 1])
    expected = b.expect()
    b.lens[1] = 1                       # more rows than tokens
    b.lens[3] = b.table.shape[1] * 16 + 1  # more tokens than the table holds
    out = b.call(max_rows=3)            # request 2 has four
    got = out.double().cpu().numpy()
    for (r, h), (o, off) in expected.items():
        if r < 3:
            assert np.all(np.abs(got[r, h] - o) <= off)
    assert torch.all(out[3:] == 77.0)
    _clean()


def test_row_starts_out_of_range_are_left_alone(lib):
    b = Batch(8, 4, 2, 128, 16, [40, 50, 30], [2, 2, 2])
    from speculative_verify_attention_gb300 import attn_verify_paged_q8
    for starts in ([0, 2, 4, 900], [-5, 2, 4, 6], [4, 2, 6, 1]):
        out = torch.full(b.q.shape, 77.0, dtype=b.dtype, device="cuda")
        attn_verify_paged_q8(b.q.cuda(), b.cache(), i32(b.table), i32(b.lens), i32(starts), 2, b.scale, out=out)
        torch.cuda.synchronize()
        for k in range(3):
            a, e = starts[k], starts[k + 1]
            if not (0 <= a <= e <= 6 and e - a <= 2):
                rows = [r for r in range(6) if not any(0 <= starts[m] <= r < starts[m + 1] <= 6 and
                                                       starts[m + 1] - starts[m] <= 2 for m in range(3))]
                assert torch.all(out[rows] == 77.0)
    _clean()


@pytest.mark.parametrize("hd", [128, 256])
def test_pages_outside_the_pool_count_as_masked(lib, hd):
    b = Batch(9, 8, 2, hd, 16, [100, 300, 20], [2, 3, 2])
    pages = len(b.codes[0])
    b.table[0, 1], b.table[1, 0], b.table[1, 9], b.table[1, 18] = -1, pages, 2 ** 31 - 1, -2 ** 31
    b.table[2, :2] = [pages + 5, -3]   # nothing left: zeros
    out = b.call()
    b.check(out)
    assert not out[int(b.starts[2]):].any()
    _clean()


@pytest.mark.parametrize("hd", [128, 256])
def test_long_contexts_are_split_and_joined(lib, hd):
    b = Batch(10, 4, 1, hd, 64, [5000, 9, 2111], [4, 1, 7], torch.float16, tree=True)
    b.check(b.call())
    _clean()


def test_many_requests_and_pages(lib):
    rng = np.random.default_rng(11)
    lens = rng.integers(1, 60, 700).tolist()
    b = Batch(11, 2, 1, 128, 16, lens, [1 + i % min(3, n) for i, n in enumerate(lens)])
    rows = set(range(0, int(b.starts[-1]), 7)) | {int(b.starts[-1]) - 1}
    b.check(b.call(), b.expect(rows=rows))
    _clean()


@pytest.mark.parametrize("gain", [1e-6, 1e3, 1e30])
def test_queries_of_any_size(lib, gain):
    """bf16 queries outside the fp16 range: the scores are scaled back by the softmax scale."""
    b = Batch(12, 8, 2, 128, 16, [200, 33], [3, 2], torch.bfloat16, q_gain=gain)
    s = b.scale / gain
    b.check(b.call(softmax_scale=s), b.expect(scale=s))
    _clean()


def test_one_key_far_above_the_rest(lib):
    """Scores that jump by hundreds in the middle of the context: the running maximum has to follow."""
    b = Batch(13, 4, 1, 256, 16, [700], [3], torch.float16)
    for key in (100, 350, 600):
        pg, off = b.table[0, key // 16], key % 16
        q = b.q[1, 2].double().numpy()
        b.codes[0][pg, 0, off] = np.clip(np.rint(127 * q / np.abs(q).max()), -127, 127)
        b.scales[0][pg, 0, off] = np.float16(0.02 + key / 20000)
    b.check(b.call())
    _clean()


def test_strided_queries_other_stream_and_graph(lib):
    b = Batch(14, 8, 2, 128, 32, [90, 200], [3, 2], torch.bfloat16, tree=True)
    expected, cache = b.expect(), b.cache()
    wide = torch.zeros((5, 3, 8, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = b.q.cuda()
    b.check(b.call(cache, q=wide[:, 1]), expected)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.full(b.q.shape, 77.0, dtype=b.dtype, device="cuda")
    torch.cuda.synchronize()
    b.call(cache, out=out, stream=side)
    side.synchronize()
    b.check(out, expected)

    # captured once, replayed after lengths, pages and queries changed in place
    from speculative_verify_attention_gb300 import attn_verify_paged_q8, attn_verify_paged_q8_workspace_bytes
    c = Batch(15, 8, 2, 128, 32, [211, 64], [1, 4], torch.bfloat16, tree=True, spare=0)
    d = Batch(14, 8, 2, 128, 32, [90, 200], [3, 2], torch.bfloat16, tree=True)
    wide_table = np.zeros((2, 7), np.int32)
    q, lens, starts = b.q.cuda(), i32(b.lens), i32(b.starts)
    wide_table[:, :b.table.shape[1]] = b.table
    table, mask = i32(wide_table), torch.as_tensor(np.array(b.words, np.uint64).view(np.int64), device="cuda")
    ws = torch.empty(attn_verify_paged_q8_workspace_bytes(8, 2, 128, 4), dtype=torch.uint8, device="cuda")
    pool = b.cache()
    args = (q, pool, table, lens, starts, 4, b.scale)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        attn_verify_paged_q8(*args, window_mask=mask, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn_verify_paged_q8(*args, window_mask=mask, out=out, workspace=ws)
    # the same planes under another batch: request order turned round, one token fewer each
    d.table, d.lens, d.n_new = b.table[::-1].copy(), [199, 89], [1, 4]
    d.starts = np.array([0, 1, 5], np.int32)
    d.q, d.words = c.q, c.words
    q.copy_(d.q.cuda())
    lens.copy_(i32(d.lens))
    starts.copy_(i32(d.starts))
    wide_table[:, :d.table.shape[1]] = d.table
    table.copy_(i32(wide_table))
    mask.copy_(torch.as_tensor(np.array(d.words, np.uint64).view(np.int64), device="cuda"))
    for _ in range(2):
        out.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        d.check(out)
    _clean()


def test_repeated_calls_give_the_same_bits(lib):
    b = Batch(16, 24, 4, 256, 16, [900, 33, 1500], [4, 2, 5], torch.bfloat16)
    cache = b.cache()
    one = b.call(cache)
    for _ in range(3):
        assert torch.equal(b.call(cache), one)
    _clean()


def test_one_page_of_a_large_pool_past_32_bits(lib):
    """Element offsets past 2^32: the pages of a 4.6 GB code plane's far end."""
    pages = 2 ** 32 // (8 * 64 * 128) + 4500
    from speculative_verify_attention_gb300 import KVPagedCacheQ8, attn_verify_paged_q8
    b = Batch(17, 8, 8, 128, 64, [150, 64], [2, 1], torch.float16, spare=0)
    cache = KVPagedCacheQ8.from_planes(*(torch.empty((pages, 8, 64, w), dtype=t, device="cuda")
                                         for w, t in ((128, torch.int8), (4, torch.float16)) * 2))
    n = len(b.codes[0])
    for k, dst, ds in ((0, cache.k_codes, cache.k_scales), (1, cache.v_codes, cache.v_scales)):
        dst[pages - n:] = torch.from_numpy(b.codes[k]).cuda()
        ds[pages - n:] = torch.from_numpy(b.scales[k]).cuda()
    out = torch.full(b.q.shape, 77.0, dtype=b.dtype, device="cuda")
    attn_verify_paged_q8(b.q.cuda(), cache, i32(np.where(b.table >= 0, b.table + pages - n, 0)), i32(b.lens), i32(b.starts), 2,
                         b.scale, out=out)
    b.check(out)
    _clean()


def test_single_window_agrees_with_the_contiguous_call(lib):
    """One request in order of its pages is attn_verify_tree_q8 over the same bytes."""
    from speculative_verify_attention_gb300 import KVCacheQ8, attn_verify_tree_q8
    b = Batch(18, 24, 4, 256, 16, [800], [8], torch.float16, tree=True)
    out = b.call()
    c = KVCacheQ8(4, 256, 800)
    for k, dst, ds in ((0, c.k_codes, c.k_scales), (1, c.v_codes, c.v_scales)):
        dst.copy_(torch.from_numpy(b.codes[k][b.table[0]].transpose(1, 0, 2, 3).reshape(4, -1, 256)))
        ds.copy_(torch.from_numpy(b.scales[k][b.table[0]].transpose(1, 0, 2, 3).reshape(4, -1, 8)))
    ref = attn_verify_tree_q8(b.q.cuda().float(), c, 800, 792, i32(np.array(b.words, np.uint32).view(np.int32)), b.scale)
    for (r, h), (o, off) in b.expect().items():
        assert np.all(np.abs(out[r, h].double().cpu().numpy() - ref[r, h].double().cpu().numpy()) <= off + 1e-4 * np.abs(o).max())
    _clean()
