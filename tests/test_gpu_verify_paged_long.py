"""attn_verify_paged_q8 over many tiles of every kernel shape: the rings of its pipeline go round many times, against
the definition in 64 bits for sampled rows."""
import pytest

torch = pytest.importorskip("torch")

from ._paged import Batch  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("hq,hkv,hd,rows,dtype", [(8, 2, 128, 3, torch.float16), (4, 1, 128, 13, torch.bfloat16), (4, 1, 128, 33, torch.float16),
                                                  (6, 1, 256, 5, torch.bfloat16), (6, 1, 256, 9, torch.float16), (12, 2, 256, 32, torch.bfloat16)])
def test_many_tiles_per_share(lib, page, hq, hkv, hd, rows, dtype):
    lens = [30000 if hd == 128 else 20000, 37, 11000, 9999]
    b = Batch(hd + rows, hq, hkv, hd, page, lens, [rows, max(1, rows - 1), 1, rows], dtype, tree=True)
    sample = {0, int(b.starts[1]) - 1, int(b.starts[1]), int(b.starts[2]), int(b.starts[4]) - 1}
    out = b.call()
    b.check(out, b.expect(rows=sample))
    from speculative_verify_attention_gb300 import kvq8_device_error
    assert kvq8_device_error(reset=True) == 0
    assert torch.equal(b.call(), out)
