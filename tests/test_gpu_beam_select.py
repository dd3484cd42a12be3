"""beam_select against its definition in 64 bits: every type and route, ties, masks, rows without anything, ragged requests."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._beams import check_selection  # noqa: E402
from ._paged import i32, starts_of  # noqa: E402

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _f32(v):
    return None if v is None else torch.as_tensor(np.asarray(v, np.float32), device="cuda")


def _run(x, starts, n_out, scores=None, weights=None, ended=None):
    """x: a tensor on the GPU.  The call's outputs, checked against the definition."""
    from speculative_verify_attention_gb300 import beam_select
    scores, weights = (None if v is None else np.asarray(v, np.float32) for v in (scores, weights))
    got = beam_select(x, i32(starts), n_out, scores=_f32(scores), weights=_f32(weights), ended=None if ended is None else i32(ended))
    host = x.float().cpu().numpy()
    check_selection(host, starts, n_out, got, scores, weights, ended)
    return got


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 255, 256, 257, 1000, 1024, 4097, 32008, 106299])
def test_types_and_vocabularies(lib, dtype, vocab):
    rng = np.random.default_rng(vocab)
    for n_out, beams in ((1, [1]), (8, [4, 1, 3]), (64, [5, 64 if vocab < 2000 else 7])):
        starts = starts_of(beams)
        x = torch.from_numpy(rng.standard_normal((starts[-1], vocab)).astype(np.float32) * 3).to(dtype).cuda()
        _run(x, starts, n_out, scores=-20 - 3 * rng.random(starts[-1]))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("shift", [0, 1, 3, 8])
def test_strided_rows_that_start_anywhere(lib, dtype, shift):
    rng = np.random.default_rng(5)
    whole = torch.from_numpy(rng.standard_normal((9, 5000 + 24)).astype(np.float32) * 3).to(dtype).cuda()
    _run(whole[:, shift:shift + 5000], [0, 4, 9], 10, scores=-rng.random(9))
    _run(whole[::2, shift:shift + 4993], [0, 5], 10)


def test_many_rows_of_one_large_vocabulary(lib):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn((40, 248320), generator=gen, device="cuda").mul_(3.0)
    _run(x.bfloat16(), list(range(0, 41, 8)), 16, scores=-20 - np.random.default_rng(1).random(40))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [300001, 2000008])
def test_vocabularies_of_more_groups_than_a_block_keeps(lib, dtype, vocab):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(vocab)
    x = torch.randn((5, vocab), generator=gen, device="cuda").mul_(3.0).to(dtype)
    x[3] = x[3].round()            # many equal values
    x[4] = 1.0
    _run(x, [0, 3, 5], 12, scores=[-1.0, -1.5, -0.5, -2.0, -2.0])
    _run(x, [0, 5], 64)


def test_equal_values_go_to_the_lowest_token_and_row(lib):
    """Rows of a few levels: most values tie.  Equal rows tie as wholes: the lower row first."""
    rng = np.random.default_rng(6)
    for vocab, n_out in ((300, 7), (5000, 64), (100003, 64)):
        levels = rng.integers(0, 3, (6, vocab)).astype(np.float32)
        levels[3] = levels[1]
        levels[4] = 2.0                                    # one level: tokens 0, 1, 2, ...
        levels[5] = 0.0
        levels[5, ::2] = -0.0                              # -0 equals 0
        x = torch.from_numpy(levels).cuda()
        for dtype in (F32, BF16):
            parents, tokens, _ = _run(x[4:5].to(dtype), [0, 1], n_out)
            assert tokens[0].tolist() == list(range(min(n_out, vocab)))
            _, tokens, _ = _run(x[5:6].to(dtype), [0, 1], n_out)
            assert tokens[0].tolist() == list(range(n_out))
            parents, tokens, _ = _run(x[1:4:2].contiguous().to(dtype), [0, 2], n_out)   # the same row twice
            twos = np.nonzero(levels[1] == 2.0)[0]
            want = [(0, v) for v in twos] + [(1, v) for v in twos]
            n = min(n_out, len(want))
            assert list(zip(parents[0].tolist(), tokens[0].tolist()))[:n] == want[:n]
            _run(x[:4].to(dtype), [0, 4], n_out, scores=[-1.0, -2.0, -1.5, -2.0])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_masks(lib, dtype):
    """Rows of -inf but for a few values, of nothing else, and of the type's lowest value."""
    rng = np.random.default_rng(7)
    vocab, low = 3001, torch.finfo(dtype).min
    x = np.full((7, vocab), -np.inf, np.float32)
    x[0, 2900:] = rng.standard_normal(101)
    x[2, 17] = 1.0
    x[3] = low
    x[4] = low
    x[4, [5, 77]] = [0.25, 3.0]
    x[5] = rng.standard_normal(vocab)
    x[5, rng.random(vocab) < 0.9] = -np.inf
    t = torch.from_numpy(x).to(dtype).cuda()
    for r in range(7):
        parents, _, _ = _run(t[r:r + 1], [0, 1], 20)
        assert (parents >= 0).sum() == min(20, int((x[r] > -np.inf).sum()))
    _run(t, [0, 7], 64)
    _run(t, [0, 2, 4, 7], 12, scores=[-1, -2, -3, -4, -5, -6, -7])


def test_numbers_that_are_none(lib):
    """NaN and +inf in a row, scores and weights that are not finite or not positive: the row has no continuation."""
    rng = np.random.default_rng(8)
    for vocab in (1000, 30007):
        x = rng.standard_normal((8, vocab)).astype(np.float32)
        x[1, vocab - 1] = np.nan
        x[2, 500] = np.inf
        x[3] = np.nan
        _run(torch.from_numpy(x).cuda(), [0, 8], 30, scores=[-1, -1, -1, -1, np.nan, -np.inf, np.inf, -1])
        _run(torch.from_numpy(x).cuda(), [0, 1, 2, 4, 8], 30, weights=[1, 1, 1, 1, 0, -1, np.nan, np.inf])
        parents, _, _ = _run(torch.from_numpy(x[1:4].copy()).cuda(), [0, 3], 5)
        assert torch.all(parents == -1)


@pytest.mark.parametrize("size", [1e4, 1e6, 1e9, 1e25, 3e38])
def test_logits_of_any_size(lib, size):
    rng = np.random.default_rng(9)
    x = (rng.random((3, 2000)).astype(np.float32) * 2 - 1) * np.float32(size)
    _run(torch.from_numpy(x).cuda(), [0, 3], 9)
    x[1] = -np.float32(size)
    x[2] = np.float32(size)
    _run(torch.from_numpy(x).cuda(), [0, 1, 2, 3], 9)


def test_beams_at_their_end_and_weights(lib):
    rng = np.random.default_rng(10)
    beams = [4, 8, 1, 3, 5]
    starts, vocab = starts_of(beams), 4003
    x = rng.standard_normal((21, vocab)).astype(np.float32) * 3
    scores, weights = -3 - 2 * rng.random(21), 0.05 + 0.05 * rng.random(21)
    ended = np.where(rng.random(21) < 0.4, 2, -1)
    ended[12] = 9       # the third request's only beam
    x[ended >= 0] = np.nan  # not read
    parents, tokens, totals = _run(torch.from_numpy(x).cuda(), starts, 10, scores, weights, ended)
    assert tokens[2, 0] == 9 and parents[2, 0] == 12 and torch.all(parents[2, 1:] == -1)
    assert float(totals[2, 0]) == np.float32(scores[12])
    _run(torch.from_numpy(x).cuda(), starts, 6, scores.astype(np.float32), None, ended)


def test_ragged_requests_and_rows_of_none(lib):
    """Empty requests, one of 65 rows, rows behind the last, starts outside."""
    from speculative_verify_attention_gb300 import beam_select
    rng = np.random.default_rng(11)
    x = rng.standard_normal((80, 700)).astype(np.float32)
    x[76:] = np.nan
    t = torch.from_numpy(x).cuda()
    got = beam_select(t, i32([0, 0, 3, 3, 11, 76, 76]), 5)
    check_selection(x, [0, 0, 3, 3, 11], 5, [g[:4] for g in got])
    assert torch.all(got[0][4:] == -1) and torch.all(got[1][4:] == -1) and torch.all(torch.isinf(got[2][4:]))
    got = beam_select(t, i32([0, 64]), 64)
    check_selection(x, [0, 64], 64, got)
    got = beam_select(t, i32([-2, 3, 81]), 5)
    assert torch.all(got[0] == -1)


def test_thousands_of_requests(lib):
    rng = np.random.default_rng(12)
    beams = rng.integers(0, 4, 4096)
    starts = starts_of(beams)
    x = torch.from_numpy(rng.standard_normal((int(starts[-1]), 257)).astype(np.float32)).cuda()
    _run(x, starts.tolist(), 3, scores=-rng.random(int(starts[-1])))


def test_the_same_call_gives_the_same_bits_and_can_be_captured(lib):
    from speculative_verify_attention_gb300 import beam_select, beam_select_workspace_bytes
    rng = np.random.default_rng(13)
    x = torch.from_numpy(rng.standard_normal((12, 50001)).astype(np.float32)).half().cuda()
    starts = i32([0, 4, 8, 12])
    out = dict(parents=i32(np.zeros((3, 8))), tokens=i32(np.zeros((3, 8))), totals=torch.zeros((3, 8), device="cuda"))
    ws = torch.full((beam_select_workspace_bytes(12, 50001, 3, 8),), 0x5a, dtype=torch.uint8, device="cuda")
    beam_select(x, starts, 8, workspace=ws, **out)
    first = {k: v.clone() for k, v in out.items()}
    for _ in range(5):
        beam_select(x, starts, 8, workspace=ws, **out)
    for k in out:
        assert torch.equal(out[k], first[k])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        beam_select(x, starts, 8, workspace=ws, **out)
    x.copy_(torch.from_numpy(rng.standard_normal((12, 50001)).astype(np.float32)).half())
    starts.copy_(i32([0, 5, 5, 12]))
    g.replay()
    torch.cuda.synchronize()
    check_selection(x.float().cpu().numpy(), [0, 5, 5, 12], 8, tuple(out.values()))


def test_calls_that_overlap_on_two_streams(lib):
    from speculative_verify_attention_gb300 import beam_select
    rng = np.random.default_rng(14)
    x = torch.from_numpy(rng.standard_normal((64, 60000)).astype(np.float32)).cuda()
    starts = i32(list(range(0, 65, 8)))
    one = beam_select(x, starts, 12)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [beam_select(x, starts, 12, stream=s if k % 4 < 2 else s.cuda_stream) for k in range(8) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, one))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab,n_out", [(1001, 16), (2500, 16), (9000, 12), (10240, 16), (10250, 16), (15000, 32), (25001, 32), (32501, 1), (32504, 9)])
def test_many_rows(lib, dtype, vocab, n_out):
    """Rows of every kind by the hundreds: normal, of few levels, of one, masked by -inf and by the type's lowest value, NaN, +inf, -inf
    alone, at their end; requests of no rows and of 65."""
    from speculative_verify_attention_gb300 import beam_select as lib_select
    rng = np.random.default_rng(vocab + n_out)
    beams = [8] * 60 + [0, 65, 1, 33] + list(rng.integers(0, 12, 60))
    starts = starts_of(beams)
    n = int(starts[-1])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(vocab)
    x = torch.randn((n, vocab), generator=gen, device="cuda").mul_(3.0)
    low = torch.finfo(dtype).min
    x[1::9] = x[1::9].round()
    x[2::27] = 1.0
    x[3::27, 40:] = low
    x[4::27, :vocab - 5] = -float("inf")
    x[5::27, vocab // 2] = float("nan")
    x[6::27, vocab - 1] = float("inf")
    x[7::27] = -float("inf")
    x[8::27] = x[9::27][:len(x[8::27])].round().clamp_(min=0) if len(x[9::27]) == len(x[8::27]) else 0.0
    x = x.to(dtype)
    scores, weights = (-20 - 3 * rng.random(n)).astype(np.float32), (0.5 + rng.random(n)).astype(np.float32)
    ended = np.where(rng.random(n) < 0.1, 2, -1)
    host = x.float().cpu().numpy()
    for more in ((scores, weights, ended), (None, None, None)):
        got = lib_select(x, i32(starts), n_out, scores=_f32(more[0]), weights=_f32(more[1]), ended=None if more[2] is None else i32(ended))
        assert torch.all(got[0][61] == -1) and torch.all(got[1][61] == -1) and torch.all(got[2][61] == -float("inf"))    # of 65 rows
        check_selection(host, starts[:62], n_out, [t[:61] for t in got], *more)
        check_selection(host, starts[62:], n_out, [t[62:] for t in got], *more)


def test_many_rows_of_requests_of_one(lib):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    for vocab in (3, 1000, 4096, 12345):
        x = torch.randn((1000, vocab), generator=gen, device="cuda").bfloat16()
        _run(x, list(range(1001)), 16)


@pytest.mark.parametrize("vocab,n_out", [(2049, 64), (20003, 64), (41000, 33), (98000, 64), (700, 64)])
def test_requests_of_many_beams(lib, vocab, n_out):
    """Vocabularies of fewer groups than continuations, and of a few more; equal totals across rows."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(vocab)
    beams = [64, 32, 17, 1, 40]
    x = torch.randn((sum(beams), vocab), generator=gen, device="cuda").mul_(3.0)
    x[70:80] = x[70]
    scores = -torch.rand(sum(beams), generator=gen, device="cuda").cpu().numpy()
    scores[70:80] = scores[70]
    for dtype in (F32, BF16):
        _run(x.to(dtype), starts_of(beams), n_out, scores=scores)
