"""Outputs over inputs, or over one another: refused by status before any launch, without a GPU."""
import pytest

from .test_beam_refusals import COMPACT, COUNTS, FORK, INVALID, ROPE, SELECT, WORKSPACE, A, _call

# bytes of each array as tests/test_beam_refusals.py has the call: 4 children of 3 sequences, tables of 5 pages, a pool of 9
READ = dict(parents=16, lens=12, held=12, page_table=60, shares=36, ring_state=8)
WRITTEN = dict(free_ring=36, page_table_out=80, lens_out=16, held_out=16, shares_out=36, ring_out=8, copy_src=16, copy_dst=16, copy_rows=16,
               status=4)
IN_PLACE = {("shares", "shares_out"), ("ring_state", "ring_out")}


def _refused(name, over, at):
    assert _call("kvq8_paged_fork", FORK, {name: FORK[over] + at}) == INVALID, (name, over, at)


@pytest.mark.parametrize("name", WRITTEN)
def test_fork_writes_over_nothing_that_it_reads(name):
    for over, size in READ.items():
        for at in (0, 4, size - 4, 4 - WRITTEN[name]):
            if at == 0 and (over, name) in IN_PLACE:
                continue
            _refused(name, over, at)


@pytest.mark.parametrize("name", WRITTEN)
def test_fork_has_no_two_outputs_in_one_place(name):
    for over, size in WRITTEN.items():
        for at in (0, size - 4, 4 - WRITTEN[name]):
            if over != name:
                _refused(name, over, at)


def test_fork_takes_arrays_side_by_side_and_in_place():
    """Behind one another in one buffer, and shares and the ring's state updated in place: what is refused then is the workspace."""
    at, but = A, {}
    for name, size in {**READ, **WRITTEN}.items():
        but[name] = at
        at += size
    assert _call("kvq8_paged_fork", FORK, {**but, "workspace": None}) == WORKSPACE
    assert _call("kvq8_paged_fork", FORK, {**but, "shares_out": but["shares"], "ring_out": but["ring_state"], "workspace": None}) == WORKSPACE


@pytest.mark.parametrize("over,size", [("lens", 12), ("row_starts", 16), ("kept", 24), ("page_table", 48)])
def test_compact_writes_over_nothing_that_it_reads(over, size):
    apart = dict(COMPACT, page_table=A, lens=2 * A, row_starts=3 * A, kept=4 * A, lens_out=5 * A)
    for at in (0, 4, size - 4, -8):
        assert _call("kvq8_paged_compact", apart, {"lens_out": apart[over] + at}) == INVALID, (over, at)


@pytest.mark.parametrize("name", ["parents", "tokens", "totals"])
def test_select_writes_over_nothing_at_all(name):
    """Logits of 4 rows of 1000 values, 1100 apart: over their first, last or any row, the workspace, another output."""
    apart = dict(SELECT, logits=A, logits_stride=1100, row_starts=2 * A, scores=3 * A, weights=4 * A, ended=5 * A, parents=6 * A, tokens=7 * A,
                 totals=8 * A, workspace=9 * A)
    for at in (-36, 0, 3996, 4400 - 36, 4400, 2 * 4400 + 2000, 3 * 4400 - 36, 3 * 4400 + 3996):
        assert _call("beam_select", apart, {name: A + at}) == INVALID, at
    for at in (-36, 0, 16):
        assert _call("beam_select", apart, {name: apart["workspace"] + at}) == INVALID, at
    for other in {"parents", "tokens", "totals"} - {name}:
        for at in (-36, 0, 36):
            assert _call("beam_select", apart, {name: apart[other] + at}) == INVALID, (other, at)


@pytest.mark.parametrize("name,size", [("counts", 2000), ("state_of_out", 16), ("status", 4), ("workspace", 32)])
def test_counts_fork_writes_over_nothing_that_it_reads(name, size):
    """4 children of 3 sequences, 5 rows of 100 counts; state_of_out in place of state_of, with status over it."""
    sizes = dict(parents=16, state_of=12, counts=2000, state_of_out=16, status=4, workspace=32)
    apart = {**COUNTS, **{k: (i + 1) * A for i, k in enumerate(sizes)}}
    for over in sizes:
        for at in (0, 16 if name == "workspace" else 4, sizes[over] - 4, 4 - size):
            there = apart[over] + at
            if over == name or not there < apart[over] + sizes[over] or (over, name, at) == ("state_of", "state_of_out", 0):
                continue
            if name == "workspace":
                there -= there % 16
            if there + size > apart[over]:
                assert _call("token_counts_fork", apart, {name: there}) == INVALID, (over, at)
    if name == "status":
        assert _call("token_counts_fork", apart, {"state_of_out": apart["state_of"], name: apart["state_of"] + 8}) == INVALID


@pytest.mark.parametrize("name,size", [("positions", 48), ("turns", 512), ("axis_of", 256), ("slots", 48)])
def test_rope_turns_no_queries_over_what_says_how(name, size):
    """6 tokens on 2 axes, 128 dims turned; rows of q_out of 2048 bytes, as they are and 2400 apart."""
    apart = dict(ROPE, q=A, k=2 * A, v=3 * A, q_out=4 * A, positions=5 * A, turns=6 * A, axis_of=7 * A, slots=8 * A)
    for stride in (1024, 1200):
        for at in (8 - size, 0, 2040, 2 * stride * 5, 2 * stride * 5 + 2040):
            assert _call("kvq8_paged_append_rope", apart, {"out_stride": stride, name: apart["q_out"] + at}) == INVALID, at
