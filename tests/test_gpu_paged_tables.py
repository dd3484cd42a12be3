"""kvq8_paged_tables against the same bookkeeping done request by request on the host: every value equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._paged import i32, tables  # noqa: E402

pytestmark = pytest.mark.gpu


def _state(seed, n, page, max_len, grow=0.5, width=None, spare=5, head=None):
    """Requests that hold pages of a shuffled pool, and lengths that grow, shrink, stay and end."""
    rng = np.random.default_rng(seed)
    held = rng.integers(0, max_len // page + 1, n)
    lens = np.where(rng.random(n) < grow, held * page + rng.integers(0, 3 * page, n), rng.integers(0, max_len + 1, n))
    lens[rng.random(n) < 0.15] = 0
    n_new = np.minimum(lens, rng.integers(0, 9, n))
    n_new[rng.random(n) < 0.1] = 0
    need = -(-lens // page)
    width = width or int(max(need.max(), held.max(), 1))
    take = int(np.maximum(need - held, 0).sum())
    pages = int(held.sum()) + take + spare
    order = rng.permutation(pages).astype(np.int32)
    table = rng.integers(-50, 0, (n, width)).astype(np.int32)
    at = 0
    for b in range(n):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    head = int(rng.integers(pages)) if head is None else head
    ring = np.full(pages, -9, np.int32)
    ring[(head + np.arange(pages - at)) % pages] = order[at:]
    return lens, n_new, held, table, ring, np.array([head, pages - at]), page


def _run(s, n_rows, in_place=False):
    from speculative_verify_attention_gb300 import kvq8_paged_tables
    lens, n_new, held, table, ring, state, page = s
    t = [i32(x) for x in (lens, n_new, held, table, ring, state)]
    n = len(lens)
    starts, status = torch.full((n + 1,), -5, dtype=torch.int32, device="cuda"), i32([-1])
    slots = torch.full((n_rows,), -5, dtype=torch.int64, device="cuda")
    positions = torch.full((n_rows,), -5, dtype=torch.int32, device="cuda")
    held_out = t[2] if in_place else torch.full_like(t[2], -5)
    ring_out = t[5] if in_place else torch.full_like(t[5], -5)
    kvq8_paged_tables(t[0], t[1], t[2], t[3], t[4], t[5], page, starts, slots, positions, status, held_out=held_out,
                      ring_out=ring_out)
    torch.cuda.synchronize()
    return t, (t[3], t[4], held_out, ring_out, starts, slots, positions, status)


def _check(s, n_rows, in_place=False):
    want = tables(*s[:6], s[6], n_rows)
    t, got = _run(s, n_rows, in_place)
    for name, g, w in zip(("table", "ring", "held", "ring_state", "row_starts", "slots", "positions", "status"), got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
    if not in_place:
        for k in (0, 1, 2, 5):
            assert np.array_equal(t[k].cpu().numpy(), np.asarray(s[k]))
    return want[-1]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n", [1, 2, 31, 33, 1023, 1024, 1025, 2500, 4096])
def test_steps_of_many_sizes(lib, n, in_place):
    s = _state(n, n, 16, 90)
    assert _check(s, int(s[1].sum()) + 5, in_place) == 0
    assert _check(s, int(s[1].sum()), in_place) == 0


@pytest.mark.parametrize("page", [16, 64, 1024])
def test_prompts_of_thousands_of_tokens(lib, page):
    lens, n_new = np.array([20000, 5, 0, 9001, 17]), np.array([20000, 1, 0, 9001, 17])
    held = np.array([0, 1, 3, 0, 1])
    need = -(-lens // page)
    pages = int(held.sum() + np.maximum(need - held, 0).sum()) + 2
    order = np.random.default_rng(3).permutation(pages).astype(np.int32)
    table = np.zeros((5, int(max(need.max(), 3))), np.int32)
    table[1, 0], table[2, :3], table[4, 0] = order[0], order[1:4], order[4]
    ring = np.zeros(pages, np.int32)
    ring[(pages - 3 + np.arange(pages - 5)) % pages] = order[5:]
    assert _check((lens, n_new, held, table, ring, np.array([pages - 3, pages - 5]), page), 29023 + 7) == 0


def test_no_rows_and_nothing_to_do(lib):
    s = _state(4, 9, 16, 60, grow=1.0)
    s = (s[2] * 16, s[1] * 0) + s[2:]
    assert _check(s, 0) == 0 and _check(s, 4, True) == 0


def test_steps_follow_one_another_until_the_pages_come_back(lib):
    """Grow by windows, drop rejected tokens, end: the ring goes round and every page comes home."""
    rng = np.random.default_rng(8)
    n, page, width, pages = 37, 16, 12, 37 * 12 // 2
    held, table = np.zeros(n, np.int64), np.zeros((n, width), np.int32)
    ring, state = np.arange(pages, dtype=np.int32), np.array([0, pages])
    lens = np.zeros(n, np.int64)
    for step in range(40):
        new = rng.integers(0, 9, n)
        wish = np.minimum(np.where(rng.random(n) < 0.1, 0, lens - rng.integers(0, 5, n)).clip(0) + new, width * page)
        new = np.minimum(new, wish)
        if step == 39:
            wish, new = wish * 0, new * 0
        s = (wish, new, held, table, ring, state, page)
        status = _check(s, 37 * 9, True)
        if status == 0:
            lens = wish
        table, ring, held, state = (np.asarray(x) for x in tables(*s[:6], page, 37 * 9)[:4])
        seen = np.concatenate([table[b, :held[b]] for b in range(n)] + [ring[(state[0] + np.arange(state[1])) % pages]])
        assert np.array_equal(np.sort(seen), np.arange(pages))
    assert state[1] == pages


def test_too_few_pages_and_malformed_input_change_nothing(lib):
    base = _state(12, 50, 16, 200, spare=0, head=3)
    rows = int(base[1].sum()) + 2

    def but(k, i, v):
        s = [np.array(x) for x in base[:6]]
        s[k][i] = v
        return tuple(s) + (16,)

    take = int(np.maximum(-(-base[0] // 16) - base[2], 0).sum())
    assert _check(but(5, 1, take), rows) == 0
    assert _check(but(5, 1, take - 1), rows, True) == 1
    width = base[3].shape[1]
    for s in (but(0, 7, -1), but(1, 7, -1), but(1, 7, 2 ** 31 - 1), but(2, 7, -1), but(2, 7, width + 1), but(0, 7, width * 16 + 1),
              but(0, 7, 2 ** 31 - 1), but(5, 0, -1), but(5, 0, len(base[4])), but(5, 1, -1), but(5, 1, len(base[4]) + 1)):
        assert _check(s, rows) == 2 and _check(s, rows, True) == 2
    assert _check(base, int(base[1].sum()) - 1) == 2
    huge = (np.full(50, 10 ** 9), np.full(50, 10 ** 9)) + base[2:]  # sums past 2^31
    assert _check(huge, rows) == 2


def test_a_captured_step_replays_on_new_lengths(lib):
    from speculative_verify_attention_gb300 import kvq8_paged_tables
    s = _state(5, 20, 16, 100, spare=60)
    t = [i32(x) for x in s[:6]]
    starts, status = i32(np.zeros(21)), i32([0])
    slots, pos = torch.zeros(300, dtype=torch.int64, device="cuda"), i32(np.zeros(300))
    saved = [x.clone() for x in t]
    args = (t[0], t[1], t[2], t[3], t[4], t[5], 16, starts, slots, pos, status)
    kvq8_paged_tables(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq8_paged_tables(*args)
    for x, y in zip(t, saved):
        x.copy_(y)
    cur = [np.asarray(x) for x in s[:6]]
    for step in range(3):
        want = tables(*cur, 16, 300)
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip((t[3], t[4], t[2], t[5], starts, slots, pos, status), want):
            assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
        cur = [np.minimum(cur[0] + 3, s[3].shape[1] * 16), np.minimum(cur[0] + 3, 3), want[2], want[0], want[1], want[3]]
        t[0].copy_(i32(cur[0]))
        t[1].copy_(i32(cur[1]))
