"""beam_select's rows at their end: every value of `ended` below zero means that the row goes on, by whichever kernels the sizes choose."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._beams import check_selection  # noqa: E402
from ._paged import i32, starts_of  # noqa: E402

pytestmark = pytest.mark.gpu
GOES_ON = (-1, -2, -3, -7, -100, -2 ** 31)
AT_END = (0, 2, 2 ** 31 - 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vocab,requests,n_out", [(1001, 5, 6),      # a row read as a whole: a small vocabulary,
                                                  (2048, 3, 64),
                                                  (9000, 90, 12),    # or some hundreds of rows
                                                  (12000, 200, 32),  # too few groups for so many continuations
                                                  (32504, 200, 9),   # a warp a row behind the scan
                                                  (20003, 4, 5)])    # a block a row
def test_all_below_zero_go_on(lib, dtype, vocab, requests, n_out):
    from speculative_verify_attention_gb300 import beam_select
    rng = np.random.default_rng(vocab + n_out)
    starts = starts_of([4] * requests)
    n = int(starts[-1])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(vocab)
    x = torch.randn((n, vocab), generator=gen, device="cuda").mul_(3.0).to(dtype)
    ended = rng.choice(GOES_ON + AT_END, n).astype(np.int64)
    ended[:len(GOES_ON) + len(AT_END)] = GOES_ON + AT_END
    ended[-4:] = -100                                                # nothing of this request is at its end
    scores = torch.from_numpy((-20 - 3 * rng.random(n)).astype(np.float32)).cuda()
    got = beam_select(x, i32(starts), n_out, scores=scores, ended=i32(ended))
    same = beam_select(x, i32(starts), n_out, scores=scores, ended=i32(np.maximum(ended, -1)))
    for a, b in zip(got, same):
        assert torch.equal(a, b)
    assert torch.all(got[0][-1] >= n - 4)
    few = min(requests, 20)                                          # the definition, of some
    check_selection(x[:4 * few].float().cpu().numpy(), starts[:few + 1], n_out, [t[:few] for t in got],
                    scores.cpu().numpy()[:4 * few], None, ended[:4 * few])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,requests,n_out", [(5, 3, 6), (1001, 5, 6), (2048, 3, 64), (9001, 90, 12), (32504, 200, 9), (20003, 4, 5)])
def test_logits_of_rows_at_their_end_count_for_nothing(lib, dtype, vocab, requests, n_out):
    """Whatever they hold, the outputs are the same bits; requests whose rows are all at their end among them."""
    from speculative_verify_attention_gb300 import beam_select
    rng = np.random.default_rng(vocab)
    starts = starts_of([4] * requests)
    n = int(starts[-1])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(vocab + 1)
    x = torch.randn((n, vocab), generator=gen, device="cuda").mul_(3.0).to(dtype)
    ended = np.where(rng.random(n) < 0.5, 3, -1)
    ended[4:8] = vocab - 1
    at_end = torch.from_numpy(ended >= 0).cuda()
    scores = torch.from_numpy((-20 - 3 * rng.random(n)).astype(np.float32)).cuda()
    first = None
    for held in (0.0, float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).max):
        x[at_end] = held
        got = beam_select(x, i32(starts), n_out, scores=scores, ended=i32(ended))
        first = first or got
        for a, b in zip(got, first):
            assert torch.equal(a, b), held
    assert first[1][1, :4].tolist() == [vocab - 1] * 4 and torch.all(first[0][1, 4:] == -1)
