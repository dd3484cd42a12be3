"""token_counts_fork and kvq8_paged_fork against the same bookkeeping done sequence by sequence on the host: every value equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._beams import fork_counts, fork_pages  # noqa: E402
from ._paged import i32, tables  # noqa: E402

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- counts

def _counts(parents, state_of, counts, in_place=False, null=False):
    from speculative_verify_attention_gb300 import token_counts_fork
    c, st = i32(counts), i32(state_of)
    out = st if in_place else torch.full((len(parents),), -7, dtype=torch.int32, device="cuda")
    status = i32([-1])
    token_counts_fork(i32(parents), None if null else st, c, out, status, n_seqs=len(state_of))
    want = fork_counts(list(parents), list(state_of), np.asarray(counts, np.int32))
    assert int(status) == want[2]
    assert np.array_equal(out.cpu().numpy(), want[0])
    assert np.array_equal(c.cpu().numpy(), want[1])
    return want


@pytest.mark.parametrize("vocab", [1, 3, 8, 1000, 4099, 33000])
@pytest.mark.parametrize("n,m,states", [(1, 1, 1), (1, 8, 8), (4, 4, 4), (37, 50, 60), (50, 37, 51)])
def test_counts_follow(lib, vocab, n, m, states):
    rng = np.random.default_rng(vocab + n)
    counts = rng.integers(-2 ** 31, 2 ** 31, (states, vocab))
    for k in range(3):
        parents = rng.integers(0, n, m)
        parents[rng.random(m) < 0.2 * k] = -1 - k
        _counts(parents, rng.permutation(states)[:n], counts)
    if n == m:
        _counts(parents, rng.permutation(states)[:n], counts, in_place=True)


def test_counts_without_rows_and_too_few(lib):
    rng = np.random.default_rng(1)
    counts = rng.integers(0, 99, (5, 40))
    assert _counts([0, 0, 1, 2], [3, 9, -1], counts)[2] == 0        # sequences without a row have children without one
    assert _counts([0, 0, 0, 0, 0], [2], counts)[2] == 0
    assert _counts([0, 0, 0, 0, 0, 0], [2], counts)[2] == 1         # six rows are wanted
    assert _counts([0, 1], [2, 2], counts)[2] == 2                  # one row, gone on from twice
    assert _counts([0, 0], [2, 2], counts)[2] == 0                  # the second one ends
    assert _counts([0, 3], [2, 1], counts)[2] == 2
    assert _counts([-1, -5], [2, 1], counts)[2] == 0
    assert _counts([2, 0, 0], [0, 1, 2], counts, null=True)[2] == 0
    assert _counts([1, 1, 0, 0], [0, 1, 2, 3], counts, in_place=True)[2] == 0


def test_thousands_of_counts_rows(lib):
    rng = np.random.default_rng(2)
    counts = rng.integers(0, 99, (9001, 12))
    for _ in range(3):
        _counts(rng.integers(-1, 4096, 4096), rng.permutation(9001)[:4096], counts)
    big = np.zeros((65536, 1), np.int32)
    big[:, 0] = np.arange(65536)
    _counts(np.zeros(4096, int), [65535], big)


# ---------------------------------------------------------------- pages

def _state(seed, n, page, width, share=0.5, spare=20, extra_held=True):
    """Sequences that share pages at random, and the ring of the others."""
    rng = np.random.default_rng(seed)
    held = rng.integers(0, width + 1, n)
    table = np.full((n, width), -3, np.int32)
    holders, used = [], 0
    for k in range(width):
        for q in range(n):
            if k >= held[q]:
                continue
            if q and k < held[q - 1] and rng.random() < share:
                table[q, k] = table[q - 1, k]
                holders[table[q, k]] += 1
            else:
                table[q, k] = used
                holders.append(0)
                used += 1
    pages = used + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.where(table >= 0, order[table], table).astype(np.int32)
    shares = np.zeros(pages, np.int32)
    shares[order[:used]] = holders
    head = int(rng.integers(pages))
    ring = np.full(pages, -9, np.int32)
    ring[(head + np.arange(spare)) % pages] = order[used:]
    lens = np.array([int(rng.integers(0, h * page + 1)) if extra_held or not h else int(rng.integers((h - 1) * page + 1, h * page + 1))
                     for h in held])
    return lens, held, page, table, shares, ring, np.array([head, spare])


def _pages(parents, s, in_place=False, width_out=None):
    from speculative_verify_attention_gb300 import kvq8_paged_fork
    lens, held, page, table, shares, ring, state = s
    m = len(parents)
    t = [i32(x) for x in (lens, held, table, shares, ring, state)]
    old = np.full((m, table.shape[1]), -5, np.int32)
    new, rest = i32(old), [torch.full((m,), -5, dtype=torch.int32, device="cuda") for _ in range(5)]
    status = i32([-1])
    shares_out, ring_out = (t[3], t[5]) if in_place else (torch.full_like(t[3], -5), torch.full_like(t[5], -5))
    kvq8_paged_fork(i32(parents), t[0], t[1], page, t[2], t[3], t[4], t[5], new, *rest, status, shares_out=shares_out, ring_out=ring_out)
    want = fork_pages(list(parents), lens, held, page, table, shares, ring, state, old)
    got = (new, rest[0], rest[1], shares_out, t[4], ring_out, rest[2], rest[3], rest[4], status)
    for name, g, w in zip(("table", "lens", "held", "shares", "ring", "ring_state", "copy_src", "copy_dst", "copy_rows", "status"), got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
    for k, x in ((0, lens), (1, held), (2, table)):
        assert np.array_equal(t[k].cpu().numpy(), x)
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,m,width", [(1, 1, 1), (1, 7, 5), (6, 6, 9), (33, 40, 30), (40, 9, 12), (300, 300, 7), (5, 5, 1500), (4096, 4096, 2)])
def test_pages_follow(lib, n, m, width, in_place):
    rng = np.random.default_rng(n + m)
    for k, page in enumerate((16, 64, 1024)):
        s = _state(n * 7 + k, n, page, width, spare=m + 3)
        parents = rng.integers(0, n, m)
        parents[rng.random(m) < 0.15 * k] = -1
        assert _pages(parents, s, in_place)[-1] == 0


@pytest.mark.parametrize("n,width,spare", [(64, 600, 100), (40, 12, 200000), (9, 5, 20000), (700, 40, 800)])
def test_long_tables_and_large_pools(lib, n, width, spare):
    rng = np.random.default_rng(spare)
    s = _state(spare, n, 16, width, share=0.8, spare=spare)
    for k in range(2):
        parents = rng.integers(0, n, n)
        parents[rng.random(n) < 0.5 * k] = -1
        assert _pages(parents, s, bool(k))[-1] == 0


def test_full_pages_and_lengths_of_nothing(lib):
    s = list(_state(3, 12, 16, 6, spare=30))
    s[0] = s[1] * 16                                        # every last page is full: nothing is copied
    got = _pages([0, 0, 5, 5, 5, 11, 3], tuple(s))
    assert np.all(got[6] == -1) and got[-1] == 0
    s[0] = s[0] * 0                                         # nothing is taken over
    assert np.all(_pages([0, 0, 5, 5, 5, 11, 3], tuple(s))[2] == 0)
    assert _pages([-1] * 5, tuple(s))[-1] == 0              # all end
    s[0] = np.minimum(s[1] * 16, 5)                         # cut into a page that others share: everybody copies
    _pages(list(range(12)) + [3, 3], tuple(s))


def test_too_few_pages_and_malformed_input_change_nothing(lib):
    base = _state(5, 20, 16, 8, share=0.0, spare=25)
    parents = [0, 0, 4, 4, 4, 7, 7, 19]
    takes = int((_pages(parents, base)[6] >= 0).sum())
    assert takes >= 2

    def but(k, i, v):
        s = [np.array(x) for x in base]
        s[k][i] = v
        return (s[0], s[1], 16) + tuple(s[3:])

    ring = but(6, 1, takes - 1)
    assert _pages(parents, ring)[-1] == 1 and _pages(parents, ring, True)[-1] == 1
    assert _pages(parents, but(6, 1, takes))[-1] == 0
    for s in (but(0, 4, -1), but(0, 4, int(base[1][4]) * 16 + 1), but(0, 4, 2 ** 31 - 1), but(1, 9, -1), but(1, 9, 9), but(6, 0, -1),
              but(6, 0, len(base[5])), but(6, 1, -1), but(6, 1, len(base[5]) + 1)):
        assert _pages(parents, s)[-1] == 2 and _pages(parents, s, True)[-1] == 2
    assert _pages(parents + [20], base)[-1] == 2
    assert _pages(parents, but(0, 9, -77))[-1] == 0         # the length of a sequence that ends is not looked at


def test_page_ids_outside_the_pool_are_passed_on(lib):
    s = list(_state(6, 4, 16, 5, share=0.0))
    for q in range(4):
        if s[1][q] > 1:
            s[3][q, 0] = len(s[5]) + 7 if q % 2 else -4
    parents = [0, 0, 1, 2, 2, 3]
    assert _pages(parents, tuple(s))[-1] == 0


def test_steps_of_beams_until_every_page_comes_home(lib):
    """Forks and growth in turn: no page is lost, held by more sequences than its share says, or in the ring while it is held."""
    rng = np.random.default_rng(9)
    n, page, width, pages = 12, 16, 10, 80
    ring, state, shares = np.arange(pages, dtype=np.int32), np.array([5, pages]), np.zeros(pages, np.int32)
    held, lens, table = np.zeros(n, np.int64), np.zeros(n, np.int64), np.zeros((n, width), np.int32)
    live = np.zeros(n, bool)
    live[:3] = True
    for step in range(60):
        new = np.where(live, rng.integers(1, 9, n), 0)
        new = np.minimum(new, width * page - lens)
        got = tables(lens + new, new, held, table, ring, state, page, n * 9)
        if got[-1] == 0:
            lens, table, ring, held, state = lens + new, got[0], got[1], np.asarray(got[2]), np.asarray(got[3])
        alive = np.nonzero(live)[0]
        parents = rng.choice(alive, n) if len(alive) and step < 58 else np.full(n, -1)
        parents = np.where(rng.random(n) < 0.2, -1, parents)
        if step % 17 == 11:
            lens = np.maximum(lens - rng.integers(0, 20, n), 0)      # rejected tokens
        want = _pages(parents.tolist(), (lens, held, page, table, shares, ring, state), bool(step % 2))
        if want[-1]:
            continue
        table, lens, held, shares, ring, state = (np.asarray(x) for x in want[:6])
        table = np.where(table == -5, 0, table)
        live = parents >= 0
        if not live.any() and step < 55:
            live[0] = True
        holders = np.zeros(pages, int)
        for q in range(n):
            assert len(set(table[q, :held[q]].tolist())) == held[q]
            np.add.at(holders, table[q, :held[q]], 1)
        free = ring[(state[0] + np.arange(state[1])) % pages]
        assert len(set(free.tolist())) == len(free) and np.all(holders[free] == 0) and (holders > 0).sum() + len(free) == pages
        assert np.array_equal(np.maximum(holders - 1, 0), shares)
        part = np.nonzero(lens % page)[0]
        for q in part:
            assert holders[table[q, held[q] - 1]] == 1               # what a sequence writes next is its own
    assert state[1] == pages


def test_a_captured_fork_replays_on_new_parents(lib):
    from speculative_verify_attention_gb300 import kvq8_paged_fork, kvq8_paged_fork_workspace_bytes
    s = _state(10, 16, 16, 12, spare=40)
    lens, held, page, table, shares, ring, state = s
    t = [i32(x) for x in (lens, held, table, shares, ring, state)]
    parents = i32(np.arange(16))
    old = np.full((16, 12), -5, np.int32)
    new, rest, status = i32(old), [i32(np.zeros(16)) for _ in range(5)], i32([0])
    so, ro = torch.empty_like(t[3]), torch.empty_like(t[5])
    ws = torch.full((kvq8_paged_fork_workspace_bytes(16, 16, len(ring)),), 0x77, dtype=torch.uint8, device="cuda")

    def call():
        kvq8_paged_fork(parents, t[0], t[1], page, t[2], t[3], t[4], t[5], new, *rest, status, shares_out=so, ring_out=ro, workspace=ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    rng = np.random.default_rng(2)
    for _ in range(4):
        p = rng.integers(-1, 16, 16)
        parents.copy_(i32(p))
        new.fill_(-5)
        t[4].copy_(i32(ring))
        g.replay()
        torch.cuda.synchronize()
        want = fork_pages(p.tolist(), lens, held, page, table, shares, ring, state, old)
        for a, w in zip((new, rest[0], rest[1], so, t[4], ro, rest[2], rest[3], rest[4], status), want):
            assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))


@pytest.mark.parametrize("vocab", [1, 2, 5, 1000, 1001, 1002, 1003, 20001])
@pytest.mark.parametrize("first", [1, 2, 3])
def test_counts_that_start_anywhere(lib, vocab, first):
    """Rows at every distance from 16 bytes to rows at every other; values beside the counts stay."""
    from speculative_verify_attention_gb300 import token_counts_fork
    rng = np.random.default_rng(vocab + first)
    states = 19
    whole = rng.integers(-2 ** 31, 2 ** 31, states * vocab + 8).astype(np.int32)
    on = torch.from_numpy(whole).cuda()
    counts = on[first:first + states * vocab].view(states, vocab)
    assert counts.data_ptr() % 16 == 4 * first
    parents, state_of = rng.integers(0, 9, 17), rng.permutation(states)[:9]
    out, status = i32(np.full(17, -7)), i32([-1])
    token_counts_fork(i32(parents), i32(state_of), counts, out, status, n_seqs=9)
    want = fork_counts(list(parents), list(state_of), whole[first:first + states * vocab].reshape(states, vocab))
    assert int(status) == want[2] == 0 and np.array_equal(out.cpu().numpy(), want[0])
    whole[first:first + states * vocab] = want[1].reshape(-1)
    assert np.array_equal(on.cpu().numpy(), whole)


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 1023, 2 ** 31 - 1024])
def test_lengths_at_the_end_of_their_type(lib, length):
    """Rounded up to pages such a length passes 31 bits.  Two million entries of a table, all but the first and last of no page."""
    width = 2 ** 21
    table = np.full((1, width), -3, np.int32)
    table[0, [0, (length - 1) // 1024]] = 4, 6
    ring = np.array([1, 2, 3, 5, 7, 0, -9, -9], np.int32)
    s = (np.array([length]), np.array([width]), 1024, table, np.zeros(8, np.int32), ring, np.array([0, 6]))
    want = _pages([0, 0], s)
    assert want[2].tolist() == [-(-length // 1024)] * 2 and want[-1] == 0
