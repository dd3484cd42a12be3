"""logits_adjust rounds as its description says: the same bits as its operations one by one in fp32, for rows that see a window token
beside a value and for rows that do not."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._paged import i32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [4096, 4099])
def test_each_operation_is_rounded_once(lib, vocab, dtype):
    from speculative_verify_attention_gb300 import logits_adjust
    rng = np.random.default_rng(vocab)
    rows = 6
    x = -torch.from_numpy(np.abs(rng.standard_normal((rows, vocab))).astype(np.float32) * 7).to(dtype)  # below 0: times the repetition
    counts = rng.integers(0, 9, (2, vocab)).astype(np.int32)
    pen = np.array([[1.3, 0.37, 0.29], [0.7, 0.11, -0.53]], np.float32)
    bias_tokens = np.tile(np.arange(vocab, dtype=np.int32), 2)
    bias = rng.standard_normal((2, vocab)).astype(np.float32)
    tokens = rng.integers(0, vocab, rows).astype(np.int32)
    out = logits_adjust(x.cuda(), i32([0, 3, rows]), penalties=torch.from_numpy(pen).cuda(), counts=i32(counts), window_tokens=i32(tokens),
                        bias_starts=i32([0, vocab, 2 * vocab]), bias_tokens=i32(bias_tokens), bias_values=torch.from_numpy(bias.ravel()).cuda())
    got = out.cpu().numpy()
    for r in range(rows):
        b = r // 3
        c = counts[b].copy()
        np.add.at(c, tokens[3 * b:r + 1], 1)
        f = np.float32
        y = x[r].float().numpy()
        y = np.where(c > 0, (y * pen[b, 0]).astype(f), y)
        penalty = np.where(c > 0, ((pen[b, 1] * c.astype(f)).astype(f) + pen[b, 2]).astype(f), f(0))
        shift = (bias[b] - penalty).astype(f)
        assert np.array_equal(got[r], (y + shift).astype(f)), r
