"""bf16 queries that are not finite: attn_verify_paged_q8 scales the rows that it holds together by one power of two, which
a NaN or an infinity in one of them must not change, whatever the size of the others."""
import pytest

torch = pytest.importorskip("torch")

from ._paged import Batch  # noqa: E402
from .test_gpu_verify_paged_routes import _widened  # noqa: E402

pytestmark = pytest.mark.gpu

# query heads, head_dim, window, row and head of the query: each kernel, and each group of its rows
WHERE = [(4, 128, 2, 1, 2), (4, 128, 4, 0, 3), (6, 256, 1, 0, 3), (6, 256, 4, 2, 1), (6, 256, 9, 8, 0), (6, 256, 32, 30, 5), (32, 128, 12, 7, 9)]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("gain", [1e-6, 1.0, 1e6])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("hq,hd,rows,row,head", WHERE)
def test_a_bf16_query_that_is_not_finite_changes_no_other(lib, value, gain, wide, hq, hd, rows, row, head):
    from speculative_verify_attention_gb300 import kvq8_device_error
    b = Batch(hd + rows, hq, 1, hd, 16, [700 + rows, 300 + rows], [rows, rows], torch.bfloat16, tree=True, q_gain=gain)
    if wide:
        _widened(b)
    scale = b.scale / gain
    near = {0, row, max(0, row - 1), rows - 1, rows}
    expected = {k: v for k, v in b.expect(scale=scale, rows=near).items() if k != (row, head)}
    b.q[row, head, 5] = value
    out = b.call(softmax_scale=scale)
    assert torch.isnan(out[row, head]).all()  # an infinity's scores are infinite of both signs, or 0 times it
    b.check(torch.nan_to_num(out, nan=77.0), expected)
    assert kvq8_device_error(reset=True) == 0
