"""A mean of equal values is that value: with the same V at every key, attn_verify_paged_q8 gives it back exactly, whatever the
weights, because their sum is taken of what the products use.

One key outweighs the others by 2^7 to 2^7.4 in a later tile than the first of them, so that its weight is not a power of two
times the reference and is rounded, and is most of the sum; the value is an fp16 number v, weights and their sum add up in fp32 to within (keys + 4) 2^-24 of v <= 2^-15
v, far less than the half step 2^-12 v that would give another fp16 number."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._paged import Batch  # noqa: E402
from .test_gpu_verify_paged_routes import _widened  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("hq,hd,rows", [(4, 128, 1), (4, 128, 4), (6, 256, 1), (6, 256, 4), (6, 128, 9), (6, 256, 9), (6, 256, 20), (6, 256, 32),
                                        (32, 128, 20)])
def test_equal_values_come_back(lib, wide, hq, hd, rows):
    rng = np.random.default_rng(hq + hd + rows)
    n = 400  # so many that a thread block takes several tiles of a request in turn
    b = Batch(hd + rows, hq, 1, hd, 16, [80 + rows] * n, [rows] * n, torch.float16)
    if wide:
        _widened(b)
    q = rng.choice([-1.0, 1.0], hd)
    b.codes[0][:] = 0
    for r in range(n):
        b.table[r, 1:4] = -1  # few other keys
        key = 70
        pg, off = b.table[r, key // 16], key % 16
        b.codes[0][pg, 0, off] = (127 * q).astype(np.int8)
        b.scales[0][pg, 0, off] = np.float16(0.01)
    row = rng.integers(-127, 128, hd).astype(np.int8)
    scale = (0.02 * np.exp(0.4 * rng.standard_normal(hd // 32))).astype(np.float16)
    b.codes[1][:], b.scales[1][:] = row, scale
    # scores in units of log2 between 7 and 7.4, the others 0
    gain = rng.uniform(7.0, 7.4, (n * rows, hq, 1)) * np.log(2) / (b.scale * 127 * float(np.float16(0.01)) * hd)
    b.q = torch.from_numpy((q * gain).astype(np.float32)).half()
    out = b.call()
    value = torch.from_numpy((row.astype(np.float32) * np.repeat(scale, 32).astype(np.float32))).half().cuda()
    wrong = (out != value).any(-1)
    assert not wrong.any(), float(wrong.double().mean())
