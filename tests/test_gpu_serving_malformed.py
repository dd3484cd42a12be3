"""Row starts, lists and penalties that make no sense or lie at the ends of their types: nothing of them is read or
written, and the requests beside them are served."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._paged import i32  # noqa: E402
from .test_gpu_logits_adjust import _call, _case, _check  # noqa: E402

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("starts", [[5, LOW], [HIGH, LOW], [HIGH, HIGH], [LOW, HIGH], [1, LOW, 3], [7, 3]])
def test_adjust_leaves_the_rows_of_malformed_requests(lib, starts):
    c = _case(31, [2, 3], 300, pad=2)
    c["starts"] = np.array(starts, np.int64).astype(np.int32)
    n = len(starts) - 1
    c["state_of"], c["penalties"], c["bias"] = c["state_of"][:n], c["penalties"][:n], c["bias"][:n]
    c["tokens"] = None
    out = _call(c)
    assert torch.all(out == 55.0)


def test_adjust_ignores_malformed_bias_lists(lib):
    from speculative_verify_attention_gb300 import logits_adjust
    x = torch.randn((4, 64), device="cuda")
    tokens, values = i32([1, 2, 3]), torch.ones(3, device="cuda")
    for starts in ([5, LOW, 3, 9, 2], [HIGH, HIGH, LOW, LOW, 1], [-1, 2, -5, 1, 4]):
        out = logits_adjust(x, i32([0, 1, 2, 3, 4]), bias_starts=i32(starts), bias_tokens=tokens, bias_values=values)
        want = x.clone()
        for b in range(4):
            if 0 <= starts[b] <= starts[b + 1] <= 3:
                want[b, tokens[starts[b]:starts[b + 1]].long()] += 1
        assert torch.equal(out, want)


@pytest.mark.parametrize("repetition", [2.0 ** -120, 2.0 ** -100, 2.0 ** 100, 2.0 ** 120, 1.0])
@pytest.mark.parametrize("vocab", [64, 67])
def test_adjust_at_the_ends_of_the_repetition_penalty(lib, repetition, vocab):
    c = _case(32, [3, 2], vocab, bias=0, grammar=False)
    c["logits"] *= 2.0 ** -10
    c["penalties"][:, 0] = repetition
    c["penalties"][:, 1:] = 0.0
    _check(c, _call(c))


def test_infinite_logits_under_a_repetition_penalty(lib):
    c = _case(33, [4], 40, grammar=False)
    c["logits"][0, ::3] = float("inf")
    c["logits"][1, ::3] = -float("inf")
    c["logits"][2, ::5] = 3.4e38
    c["penalties"][:, 0] = 1.5
    _check(c, _call(c))


@pytest.mark.parametrize("starts", [[HIGH, HIGH], [HIGH - 9, 3], [HIGH, LOW], [5, LOW], [LOW, 3]])
def test_counts_of_malformed_lists(lib, starts):
    from speculative_verify_attention_gb300 import token_counts
    t = torch.full((1, 40), 3, dtype=torch.int32, device="cuda")
    token_counts(i32([1, 2, 3]), i32(np.array(starts, np.int64).astype(np.int32)), t, i32([HIGH]))
    assert torch.all(t == 3)


def test_counts_with_prompts_at_the_ends_of_their_type(lib):
    from speculative_verify_attention_gb300 import token_counts
    t = torch.zeros((2, 8), dtype=torch.int32, device="cuda")
    token_counts(i32([1, 1, 2, 3]), i32([0, 2, 4]), t, i32([HIGH, LOW]))
    want = torch.zeros_like(t)
    want[0, 1] = LOW
    want[1, 2], want[1, 3] = 1, 1
    assert torch.equal(t, want)
