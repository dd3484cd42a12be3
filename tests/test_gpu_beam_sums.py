"""beam_select's log sum exp against 64 bits, as closely as its roundings allow: every route and type, near zero and far from it.

How far it may be off, all relative to the sum, for V values x with maximum m and softmax p (E is the mean by p; E[m - x] <= H, the entropy,
<= ln V, as m - x_i <= -ln p_i):
  2^-22                 the hardware's exponential
  n 2^-24               the additions that a value goes through: 7 of a lane's eight, 2 of its four loads, one a chunk that its lane takes (two
                        at most behind the scan, a row's thousands where it is read as a whole), 5 between lanes
  2^-24 (H + 1/2)       the exponents, x log2 e less a whole number within 0.6 of m log2 e, rounded once
  1.4e-8 H              log2 e as fp32: sums are of 2^(k x), their log2 is divided by the same k, and the derivative of
                        (1/t) log sum exp(t x) by t at 1 is -H
  1.5 V 2^-43           parts, one for 1024 values, rounded to 2^-33 of a sum that is 2^-1/2 at least
  2^-28                 the sum's log2
From |m| = 2^20 on the exponents are differences to m, rounded twice (2^-23 E[m - x]).  What follows is in 64 bits: 2^-51 of the
numbers' size.  Scores bring the totals near zero here, so their rounding to fp32 is next to nothing."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._paged import i32  # noqa: E402

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
SIZES = [(7, 5, 1), (1000, 40, 4), (2048, 9, 64), (9000, 400, 8), (19000, 800, 32), (32504, 800, 8), (20003, 40, 8), (248320, 24, 16)]


def _bound(vocab, entropy, size):
    whole = vocab <= 2048 or vocab in (9000, 19000)        # the sizes above that are read as wholes
    adds = 9 + 5 + (-(-vocab // 1024) if whole else 2)
    return 1.001 * (2.0 ** -22 + adds * 2.0 ** -24 + 2.0 ** -23 * (entropy + 0.5) + 1.4e-8 * entropy + 1.5 * vocab * 2.0 ** -43 + 2.0 ** -28) + size * 2.0 ** -51


def _check(x, n_out):
    """Every row a request of its own, and the same rows in requests of four."""
    from speculative_verify_attention_gb300 import beam_select
    n, vocab = x.shape
    best, entropy, size = (torch.empty(n, dtype=torch.float64, device="cuda") for _ in range(3))
    for r in range(n):
        row = x[r].double()
        row = row - row.max()                              # exact where it counts: what is far below the maximum adds nothing
        norm = row.exp().sum().log()
        p = (row - norm).exp()
        best[r], entropy[r], size[r] = -norm, norm - (p * row.clamp(min=-800)).sum(), x[r].double().abs().max()
    score = (-best).float()
    want = best + score.double()
    tol = torch.tensor([_bound(vocab, float(h), float(s)) for h, s in zip(entropy, size)], device="cuda") + want.abs() * 2.0 ** -24 + 2.0 ** -40
    parents, _, totals = beam_select(x, i32(list(range(n + 1))), n_out, scores=score)
    assert torch.equal(parents[:, 0], i32(list(range(n))))
    off = (totals[:, 0].double() - want).abs()
    assert torch.all(off <= tol), (float((off / tol).max()), float(off.max()))
    starts = list(range(0, n, 4)) + [n]
    parents, _, totals = beam_select(x, i32(starts), n_out, scores=score)
    assert torch.all((totals[:, 0].double() - want[parents[:, 0].long()]).abs() <= tol[parents[:, 0].long()])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab,rows,n_out", SIZES)
def test_sums_are_as_good_as_their_roundings(lib, dtype, vocab, rows, n_out):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(vocab)
    spread = torch.logspace(-3, 1.5, rows, device="cuda").unsqueeze(1)
    x = (torch.randn((rows, vocab), generator=gen, device="cuda") * spread).to(dtype)
    x[1::5] += torch.arange(vocab, device="cuda").div(vocab).mul(40).to(dtype)      # chunk after chunk a larger maximum
    x[2::5] -= torch.arange(vocab, device="cuda").div(vocab).mul(40).to(dtype)
    _check(x, n_out)


@pytest.mark.parametrize("offset", [1e4, -1e4, 1e6, -1e6, 2.0 ** 20, -2.0 ** 20, 1e9, -1e9])
@pytest.mark.parametrize("vocab,rows,n_out", SIZES[1:6])
def test_sums_far_from_zero(lib, offset, vocab, rows, n_out):
    """Rows of one value, whose log sum exp is that value and ln V, and rows of values around it."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(vocab)
    x = torch.randn((rows, vocab), generator=gen, device="cuda").mul_(3.0)
    x[::3] = 0.0
    x += offset
    _check(x, n_out)
    from speculative_verify_attention_gb300 import beam_select
    same = x[:1]
    score = np.float32(math.log(vocab))
    _, tokens, totals = beam_select(same, i32([0, 1]), 1, scores=torch.tensor([score], device="cuda"))
    assert tokens.item() == 0
    assert abs(totals.item() - (float(score) - math.log(vocab))) <= _bound(vocab, math.log(vocab), abs(offset)) + 2.0 ** -40
