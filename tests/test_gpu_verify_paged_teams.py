"""attn_verify_paged_q8 where several CTAs share a window's rows (more than 192 a KV head) and the batch's windows differ: a
short window has rows for some CTAs of a team only, and every row of every request has to come out, cut items too."""
import pytest

torch = pytest.importorskip("torch")

from ._paged import Batch  # noqa: E402

pytestmark = pytest.mark.gpu

# query heads, KV heads, head_dim, windows, lengths: of these the last CTAs of a team have no row of a window of one token
BATCHES = [(19, 1, 128, [53, 1, 2, 2, 1], [1757, 1896, 610, 1500, 2460]),
           (38, 2, 128, [55, 1, 55, 1], [3348, 2234, 1931, 1596]),
           (32, 1, 128, [55, 1, 55, 1], [900, 20000, 900, 9000]),
           (32, 1, 256, [60, 1, 33, 1], [4000, 9000, 3000, 8000]),
           (40, 1, 128, [62, 1, 62, 1, 21], [3493, 1864, 1004, 1491, 806]),
           (48, 1, 128, [41, 1], [2000, 5000]),
           (96, 2, 256, [59, 1, 1, 12, 1], [3444, 3952, 171, 1757, 3485]),
           (64, 1, 128, [34, 1], [2000, 5000]),
           (64, 1, 256, [60, 1, 60, 2], [8192, 8192, 700, 64]),
           (64, 1, 128, [63, 10, 1, 63, 1], [1945, 855, 1543, 409, 2009]),
           (128, 2, 128, [63, 1, 12, 1], [1661, 1475, 1155, 3654])]


@pytest.mark.parametrize("hq,hkv,hd,windows,lens", BATCHES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_short_windows_beside_long_ones(lib, dtype, hq, hkv, hd, windows, lens):
    from speculative_verify_attention_gb300 import kvq8_device_error
    b = Batch(hq + hd, hq, hkv, hd, 32, lens, windows, dtype, tree=True, pad_rows=1)
    out = b.call()
    # the first and last row of each window, of all heads
    picked = {int(r) for s, n in zip(b.starts, windows) for r in (s, s + n - 1)}
    b.check(out, b.expect(rows=picked))
    assert not (out[:int(b.starts[-1])] == 77.0).any()  # what the output held before
    assert torch.equal(b.call(), out)
    assert kvq8_device_error(reset=True) == 0
