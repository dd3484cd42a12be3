"""attn_verify_paged_q8 by each of its kernels: which one runs follows the window's rows and the table's capacity, so
the same kinds of batch run here under a narrow and a wide table (columns that no request uses hold no page)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._paged import Batch  # noqa: E402

pytestmark = pytest.mark.gpu


def _widened(b, tiles=64 * 512):
    """A table with room for this many tiles of 64 keys over the batch's KV heads."""
    cols = -(-tiles * 64 // (b.page * len(b.lens) * b.hkv))
    b.table = np.pad(b.table, ((0, 0), (0, max(0, cols - b.table.shape[1]))), constant_values=-7)
    return b


def _clean():
    from speculative_verify_attention_gb300 import kvq8_device_error
    assert kvq8_device_error(reset=True) == 0


SHAPES = [(4, 1, 128, 13), (8, 1, 128, 8), (24, 4, 256, 5), (6, 1, 256, 9), (2, 1, 256, 8), (3, 1, 256, 3)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("hq,hkv,hd,rows", SHAPES)
def test_ragged_batches_under_a_wide_table(lib, dtype, page, hq, hkv, hd, rows):
    lens = [rows, 70 + rows, 17 + rows, 127, 128, 129, 256 + rows, 700]
    b = _widened(Batch(hd + rows + page, hq, hkv, hd, page, lens, [rows, 1, rows, 2, rows, 3, 1, rows], dtype, tree=True,
                       pad_rows=2))
    out = b.call()
    b.check(out)
    assert torch.equal(b.call(), out)
    _clean()


@pytest.mark.parametrize("hq,hd,rows", [(4, 128, 16), (6, 256, 4)])
def test_empty_masks_and_bad_pages_under_a_wide_table(lib, hq, hd, rows):
    b = _widened(Batch(hd + 1, hq, 1, hd, 16, [rows, 300, 0, 500], [rows, rows, 0, 2], tree=True))
    s, pages = b.starts, len(b.codes[0])
    b.words[s[0]] = 0               # no key: zeros
    b.words[s[1]] = 0               # context only
    b.words[s[1] + 3] = 2 ** 64 - 1
    b.table[1, 0], b.table[1, 9], b.table[3, 17] = -1, pages, 2 ** 31 - 1
    out = b.call()
    b.check(out)
    assert not out[s[0]].any()
    _clean()


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("hq,hkv,hd,rows,dtype", [(4, 1, 128, 7, torch.float16), (4, 1, 128, 15, torch.bfloat16),
                                                  (6, 1, 256, 5, torch.bfloat16), (6, 1, 256, 10, torch.float16)])
def test_many_tiles_under_a_wide_table(lib, page, hq, hkv, hd, rows, dtype):
    lens = [30000 if hd == 128 else 20000, 37, 11000, 9999]
    b = _widened(Batch(hd + rows, hq, hkv, hd, page, lens, [rows, max(1, rows - 1), 1, rows], dtype, tree=True))
    sample = {0, int(b.starts[1]) - 1, int(b.starts[1]), int(b.starts[2]), int(b.starts[4]) - 1}
    out = b.call()
    b.check(out, b.expect(rows=sample))
    assert torch.equal(b.call(), out)
    _clean()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("hq,hd,rows,row,head", [(4, 128, 2, 1, 2), (4, 128, 9, 8, 3), (6, 256, 9, 3, 1), (6, 256, 32, 2, 5),
                                                 (6, 256, 32, 20, 0), (6, 256, 32, 31, 5), (6, 128, 27, 24, 2), (6, 256, 64, 63, 1)])
def test_scores_that_jump_for_one_row(lib, wide, hq, hd, rows, row, head):
    """The reference of one row has to follow its scores, again and again, in whichever warps and lanes its sums lie: one
    key in each of many tiles is that row's query, ever longer."""
    b = Batch(hd + rows + row, hq, 1, hd, 16, [1500 + rows, 900 + rows], [rows, rows], torch.float16, tree=True)
    if wide:
        _widened(b)
    for at, key in enumerate(range(70, 1500, 110)):
        pg, off = b.table[0, key // 16], key % 16
        q = b.q[row, head].double().numpy()
        b.codes[0][pg, 0, off] = np.clip(np.rint(127 * q / np.abs(q).max()), -127, 127)
        b.scales[0][pg, 0, off] = np.float16(0.003 * (at + 1))
    out = b.call()
    near = {0, row, max(0, row - 1), min(rows - 1, row + 1), rows, rows + row}
    b.check(out, b.expect(rows=near))
    assert torch.equal(b.call(), out)
    _clean()


def test_shares_of_single_tiles(lib):
    """Many short requests of wide windows: segments of one tile, one after another."""
    lens = [40 + 7 * (i % 9) for i in range(90)]
    for rows, hq in ((32, 6), (9, 6)):
        b = Batch(rows, hq, 1, 256, 16, lens, [rows - i % 5 for i in range(90)], torch.bfloat16, tree=True)
        picked = set(range(0, int(b.starts[-1]), 61)) | {int(b.starts[-1]) - 1}
        expected = b.expect(rows=picked)
        b.check(b.call(), expected)
        if rows == 9:
            _widened(b)
            b.check(b.call(), expected)
    _clean()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("hq,hd,rows,row,head", [(4, 128, 2, 1, 2), (6, 256, 1, 0, 3), (6, 256, 4, 2, 1), (6, 256, 9, 8, 0), (6, 256, 32, 30, 5),
                                                 (6, 256, 32, 3, 4)])
@pytest.mark.parametrize("n", [40, 3000])
def test_a_query_that_is_not_a_number_stays_one_and_alone(lib, wide, hq, hd, rows, row, head, n):
    b = Batch(hd + rows, hq, 1, hd, 16, [n + rows, 300 + rows], [rows, rows], torch.float16, tree=True)
    if wide:
        _widened(b)
    expected = {k: v for k, v in b.expect(rows={0, row, rows}).items() if k != (row, head)}
    b.q[row, head, 5] = float("nan")
    out = b.call()
    assert torch.isnan(out[row, head]).all()
    b.check(torch.nan_to_num(out, nan=77.0), expected)
    _clean()
