"""logits_adjust and token_counts against their definitions: -inf and rows left alone exact, values within six half steps."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._paged import adjusted, i32, masks64, starts_of, tree_words  # noqa: E402

pytestmark = pytest.mark.gpu
PROMPT = -2 ** 31


def _case(seed, n_new, vocab, dtype=torch.float32, tree=False, bias=5, grammar=True, pad=0):
    rng = np.random.default_rng(seed)
    n, rows = len(n_new), int(sum(n_new)) + pad
    c = {"starts": starts_of(n_new), "logits": torch.from_numpy(rng.standard_normal((rows, vocab)).astype(np.float32) * 4).to(dtype)}
    counts = rng.integers(0, 4, (n + 1, vocab)) * (rng.random((n + 1, vocab)) < 0.3)
    c["counts"] = (counts + np.where(rng.random((n + 1, vocab)) < 0.2, PROMPT, 0)).astype(np.int32)
    c["state_of"] = rng.permutation(n + 1)[:n].astype(np.int32)
    c["penalties"] = (rng.random((n, 3)) * [0.5, 1, 1] + [0.9, -0.2, -0.2]).astype(np.float32)
    c["tokens"] = rng.integers(0, min(vocab, 5) if tree else vocab, rows).astype(np.int32)
    c["words"] = sum((tree_words(k, rng) for k in n_new), []) + [0] * pad if tree else None
    c["bias"] = [[(int(v), float(np.float32(x))) for v, x in zip(rng.integers(0, vocab, bias), rng.standard_normal(bias) * 3)]
                 for _ in range(n)] if bias else None
    c["grammar"] = rng.integers(-2 ** 31, 2 ** 31, (max(rows // 2, 1), -(-vocab // 32))).astype(np.int32) if grammar else None
    c["grammar_of"] = rng.integers(-1, max(rows // 2, 1), rows).astype(np.int32) if grammar else None
    return c


def _call(c, out=None, **more):
    from speculative_verify_attention_gb300 import logits_adjust
    kw = {}
    for k, name in (("counts", "counts"), ("state_of", "state_of"), ("tokens", "window_tokens"), ("grammar", "grammar"),
                    ("grammar_of", "grammar_of")):
        if c.get(k) is not None:
            kw[name] = i32(c[k])
    if c.get("penalties") is not None:
        kw["penalties"] = torch.from_numpy(c["penalties"]).cuda()
    if c.get("words") is not None:
        kw["window_mask"] = masks64(c["words"])
    if c.get("bias") is not None:
        kw["bias_starts"] = i32(starts_of([len(x) for x in c["bias"]]))
        flat = sum(c["bias"], [])
        kw["bias_tokens"] = i32([v for v, _ in flat])
        kw["bias_values"] = torch.tensor([x for _, x in flat], dtype=torch.float32, device="cuda")
    logits = more.pop("logits", None)
    logits = c["logits"].cuda() if logits is None else logits
    if out is None:
        out = torch.full(c["logits"].shape, 55.0, dtype=torch.float32, device="cuda")
    return logits_adjust(logits, i32(c["starts"]), out=out, **kw, **more)


def _check(c, out, left=55.0):
    x, off = adjusted(c["logits"], c["starts"], **{k: c.get(k) for k in ("penalties", "counts", "state_of", "tokens", "words",
                                                                        "bias", "grammar", "grammar_of")})
    got = out.double().cpu().numpy()
    alone = np.isnan(x) & ~np.isnan(c["logits"].double().numpy())
    if left is not None:
        assert np.all(got[alone] == left)
    fine = np.isfinite(x)
    assert np.array_equal(got[~fine & ~alone], x[~fine & ~alone], equal_nan=True)
    assert np.all(np.abs(got[fine] - x[fine]) <= off[fine])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 7, 8, 33, 2047, 2048, 2056, 4099, 10000])
@pytest.mark.parametrize("tree", [False, True])
def test_everything_at_once(lib, dtype, vocab, tree):
    c = _case(vocab, [3, 1, 0, 6, 1, 1, 1, 9], vocab, dtype, tree, pad=3)
    _check(c, _call(c))


@pytest.mark.parametrize("drop", [("counts", "state_of"), ("tokens", "words"), ("bias",), ("grammar", "grammar_of"), ("grammar_of",),
                                  ("state_of",), ("words",), ("penalties", "counts", "state_of", "tokens", "words"),
                                  ("penalties", "counts", "state_of", "tokens", "words", "bias", "grammar", "grammar_of")])
def test_each_part_may_be_left_out(lib, drop):
    c = _case(3, [2, 5, 1], 5000, torch.bfloat16, tree=True)
    for k in drop:
        c[k] = None
    if drop == ("grammar_of",):
        c["grammar"] = np.random.default_rng(0).integers(-2 ** 31, 2 ** 31, (8, 157)).astype(np.int32)
    _check(c, _call(c))


def test_windows_of_64_rows_of_one_token(lib):
    """Every window token the same: a row counts as many as it sees; and one window longer than a mask is left alone."""
    c = _case(5, [64, 65, 2], 300, tree=False, pad=0)
    c["tokens"][:] = 17
    out = _call(c)
    want = adjusted(c["logits"], c["starts"], **{k: c[k] for k in ("penalties", "counts", "state_of", "tokens", "words", "bias",
                                                                   "grammar", "grammar_of")})
    got = out.double().cpu().numpy()
    for rows in (slice(0, 64), slice(129, 131)):
        fine = np.isfinite(want[0][rows])
        assert np.array_equal(np.isfinite(got[rows]), fine)
        assert np.all(np.abs(got[rows] - want[0][rows])[fine] <= want[1][rows][fine])
    assert np.all(got[64:129] == 55.0)
    c["tokens"] = c["words"] = None   # without window tokens a window may be of any length
    _check(c, _call(c))


def test_ids_and_states_out_of_range_are_ignored(lib):
    c = _case(6, [3, 4], 1000, tree=True)
    c["tokens"][[0, 4]] = [-1, 1000]
    c["tokens"][5] = 2 ** 31 - 1
    c["state_of"][:] = [-3, 99]
    c["bias"] = [[(1000, 3.0), (-1, 2.0), (999, 1.0)], [(2 ** 31 - 1, 1.0)]]
    c["grammar_of"][:4] = [-2 ** 31, 2 ** 31 - 1, 3, 0]
    _check(c, _call(c))


def test_last_bias_entry_of_a_token_holds(lib):
    c = _case(7, [2, 2], 6000, bias=0, grammar=False)
    c["bias"] = [[(5, 1.0), (4000, 2.0), (5, -3.0), (5, 0.25)] + [(v, 1.0) for v in range(100, 700)] + [(300, 9.0)], []]
    _check(c, _call(c))


def test_special_values(lib):
    c = _case(8, [4], 4096, bias=0)
    c["logits"][0, :50] = float("nan")
    c["logits"][1, 20:70] = float("inf")
    c["logits"][2, :] = -float("inf")
    c["logits"][3, ::3] = torch.finfo(torch.float32).min / 4
    c["bias"] = [[(30, -float("inf")), (31, 1e30)]]
    c["grammar_of"][:] = [0, 1, -1, 0]
    c["grammar"][1] = 0                 # nothing allowed: all -inf, whatever stood there
    out = _call(c)
    assert torch.all(out[1] == -float("inf"))
    with np.errstate(invalid="ignore"):
        _check(c, out, left=None)


@pytest.mark.parametrize("vocab", [4096, 4099])
def test_in_place_and_strided(lib, vocab):
    c = _case(9, [3, 2, 6], vocab, tree=True)
    rows = len(c["logits"])
    wide = torch.full((rows, vocab + 13), 55.0, device="cuda")
    wide[:, :vocab] = c["logits"].cuda()
    _call(c, logits=wide[:, :vocab], out=wide[:, :vocab])
    _check(c, wide[:, :vocab])
    assert torch.all(wide[:, vocab:] == 55.0)
    half = dict(c, logits=c["logits"].half())
    wide = torch.zeros((rows, vocab + 3), dtype=torch.float16, device="cuda")
    wide[:, 3:] = half["logits"].cuda()
    _check(half, _call(half, logits=wide[:, 3:]))


def test_full_vocabulary_then_argmax(lib):
    """The head's order: adjust, then argmax_rows_top_prob, against the same two steps in 64 bits."""
    from speculative_verify_attention_gb300 import argmax_rows_top_prob
    c = _case(10, [4, 8], 248320, torch.bfloat16, tree=True, bias=300)
    out = _call(c)
    _check(c, out)
    idx, top = argmax_rows_top_prob(out)
    x = out.double()
    assert torch.equal(idx.long(), x.argmax(1))
    want = torch.softmax(x, 1).amax(1)
    assert torch.all((top.double() - want).abs() <= 1e-5 * want)


# ---------------------------------------------------------------- counts

def _counted(tokens, starts, prompts, state_of, counts, clear):
    counts = counts.astype(np.int64) & 0xffffffff
    n = len(starts) - 1
    if clear:
        for i in range(n):
            if 0 <= state_of[i] < len(counts):
                counts[state_of[i]] = 0
    for i in range(n):
        if not 0 <= state_of[i] < len(counts):
            continue
        for k in range(starts[i], starts[i + 1]):
            if 0 <= tokens[k] < counts.shape[1]:
                if k - starts[i] < prompts[i]:
                    counts[state_of[i], tokens[k]] |= 1 << 31
                else:
                    counts[state_of[i], tokens[k]] += 1
    return counts.astype(np.uint32).view(np.int32)


@pytest.mark.parametrize("clear", [False, True])
@pytest.mark.parametrize("vocab", [1, 31, 5000, 106299])
def test_counts(lib, clear, vocab):
    from speculative_verify_attention_gb300 import token_counts
    rng = np.random.default_rng(vocab)
    lens = [0, 1, 700, 3, 0, 4000, 33]
    starts = starts_of(lens)
    tokens = (rng.random(starts[-1]) ** 3 * vocab).astype(np.int32)
    tokens[::97] = rng.integers(-3, 0, len(tokens[::97]))
    tokens[50::301] = vocab
    prompts = np.array([2, 0, 500, 9, 1, 4000, -4])
    state_of = np.array([0, 3, 5, 3, 8, 1, -1])   # two lists on one row, two skipped
    counts = rng.integers(-2 ** 31, 100, (7, vocab)).astype(np.int32)
    counts &= PROMPT | 127
    want = _counted(tokens, starts, prompts, state_of, counts, clear)
    got = token_counts(i32(tokens), i32(starts), t := i32(counts), i32(prompts), i32(state_of), clear)
    assert got is t and np.array_equal(t.cpu().numpy(), want)


def test_counts_without_lists_tokens_or_prompts(lib):
    from speculative_verify_attention_gb300 import token_counts
    t = torch.full((2, 40), 3, dtype=torch.int32, device="cuda")
    token_counts(i32([]), i32([0, 0]), t, clear=True)
    assert not t[0].any() and torch.all(t[1] == 3)
    token_counts(i32([]), i32([0]), t)
    token_counts(i32([7, 7, 7]), i32([1, 3]), t)
    assert t[0].sum() == 2 and t[0, 7] == 2
    for starts in ([-1, 2], [0, 4], [3, 1]):   # outside the tokens: nothing
        token_counts(i32([1, 2, 3]), i32(starts), t)
    assert t[0].sum() == 2 and torch.all(t[1] == 3)
