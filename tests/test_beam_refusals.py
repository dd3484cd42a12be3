"""What the calls around beams, trees and rotary positions refuse, by status code, without a GPU: before any launch."""
import pytest

from speculative_verify_attention_gb300 import kvq8_paged_cache, load_library

A = 1 << 20            # an aligned address that nothing reads
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)
BIG = 1 << 40


def _cache(**but):
    f = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, n_kv_heads=2, head_dim=128, page_size=16, n_pages=9)
    f.update(but)
    return kvq8_paged_cache(**f)


def _call(name, args, but):
    a = dict(args)
    a.update(but)
    return getattr(load_library(), name)(*a.values())


SELECT = dict(logits=A, dtype=0, logits_stride=1000, n_rows=4, vocab=1000, row_starts=A, n_seqs=2, scores=A, weights=A, ended=A, n_out=5,
              parents=A, tokens=A, totals=A, workspace=A, workspace_bytes=BIG, stream=None)


@pytest.mark.parametrize("but,status", [
    *[({k: None}, INVALID) for k in ("logits", "row_starts", "parents", "tokens", "totals")], ({"workspace": None}, WORKSPACE),
    ({"dtype": 3}, INVALID), ({"n_rows": -1}, INVALID), ({"n_rows": 0}, INVALID), ({"n_seqs": -1}, INVALID), ({"vocab": 0}, INVALID),
    ({"n_out": 0}, INVALID), ({"logits_stride": 999}, INVALID), ({"n_rows": 65536}, UNSUPPORTED), ({"n_seqs": 4097}, UNSUPPORTED),
    ({"n_out": 65}, UNSUPPORTED), ({"vocab": 2 ** 30 + 1, "logits_stride": 2 ** 31}, UNSUPPORTED), ({"workspace_bytes": 64}, WORKSPACE),
    ({"logits": A + 2}, MISALIGNED), ({"dtype": 2, "logits": A + 1}, MISALIGNED), ({"workspace": A + 8}, MISALIGNED),
    *[({k: A + 2}, MISALIGNED) for k in ("row_starts", "scores", "weights", "ended", "parents", "tokens", "totals")],
    ({"n_seqs": 0, "logits": None}, OK)])
def test_select(but, status):
    assert _call("beam_select", SELECT, but) == status


@pytest.mark.parametrize("name", ["parents", "tokens", "totals"])
@pytest.mark.parametrize("over,at", [("row_starts", 8), ("scores", 0), ("scores", -36), ("scores", 12), ("weights", 12), ("ended", -36)])
def test_select_writes_over_nothing_that_it_reads(name, over, at):
    apart = dict(SELECT, row_starts=2 * A, scores=3 * A, weights=4 * A, ended=5 * A, parents=6 * A, tokens=7 * A, totals=8 * A)
    assert _call("beam_select", apart, {name: apart[over] + at}) == INVALID


def test_workspaces_are_asked_for_as_the_calls_want_them():
    lib = load_library()
    need = lib.beam_select_workspace_bytes(4, 1000, 2, 5)
    assert need > 0 and _call("beam_select", SELECT, {"workspace_bytes": need - 1}) == WORKSPACE
    for a in ((0, 1000, 2, 5), (4, 0, 2, 5), (4, 1000, 0, 5), (4, 1000, 2, 0), (4, 1000, 2, 65), (65536, 1000, 2, 5), (4, 1000, 4097, 5)):
        assert lib.beam_select_workspace_bytes(*a) == 0
    assert lib.beam_select_workspace_bytes(65535, 1 << 30, 4096, 64) > 65535 * (1 << 22) * 4
    assert lib.token_counts_fork_workspace_bytes(0) == lib.token_counts_fork_workspace_bytes(4097) == 0
    for a in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (4097, 1, 1), (1, 4097, 1), (1, 1, 2 ** 30 + 1)):
        assert lib.kvq8_paged_fork_workspace_bytes(*a) == 0
    assert _call("token_counts_fork", COUNTS, {"workspace_bytes": lib.token_counts_fork_workspace_bytes(4) - 1}) == WORKSPACE
    assert _call("kvq8_paged_fork", FORK, {"workspace_bytes": lib.kvq8_paged_fork_workspace_bytes(3, 4, 9) - 1}) == WORKSPACE


COUNTS = dict(parents=A, n_children=4, state_of=2 * A, n_seqs=3, counts=A, n_states=5, vocab=100, state_of_out=3 * A, status=A, workspace=A,
              workspace_bytes=BIG, stream=None)


@pytest.mark.parametrize("but,status", [
    *[({k: None}, INVALID) for k in ("parents", "counts", "state_of_out", "status")], *[({k: 0}, INVALID) for k in ("n_children", "n_seqs",
                                                                                                                 "n_states", "vocab")],
    ({"state_of_out": A}, INVALID), ({"state_of_out": A + 12}, INVALID), ({"state_of_out": 2 * A + 4}, INVALID),
    ({"n_children": 4097}, UNSUPPORTED), ({"n_seqs": 4097}, UNSUPPORTED), ({"n_states": 65537}, UNSUPPORTED), ({"vocab": 2 ** 30 + 1}, UNSUPPORTED),
    ({"workspace": None}, WORKSPACE), ({"workspace_bytes": 8}, WORKSPACE), ({"workspace": A + 8}, MISALIGNED),
    *[({k: 5 * A + 2}, MISALIGNED) for k in ("parents", "state_of", "counts", "state_of_out", "status")]])
def test_counts(but, status):
    assert _call("token_counts_fork", COUNTS, but) == status


FORK = dict(parents=A, n_children=4, lens=2 * A, held=3 * A, n_seqs=3, page_size=16, page_table=4 * A, max_pages=5, shares=5 * A,
            free_ring=6 * A, n_pages=9, ring_state=7 * A, page_table_out=8 * A, lens_out=9 * A, held_out=10 * A, shares_out=11 * A,
            ring_out=12 * A, copy_src=13 * A, copy_dst=14 * A, copy_rows=15 * A, status=16 * A, workspace=17 * A, workspace_bytes=BIG, stream=None)
_ARRAYS = [k for k, v in FORK.items() if isinstance(v, int) and v >= A and k not in ("workspace", "workspace_bytes")]


@pytest.mark.parametrize("but,status", [
    *[({k: None}, INVALID) for k in _ARRAYS], *[({k: 0}, INVALID) for k in ("n_children", "n_seqs", "max_pages", "n_pages")],
    *[({"page_size": p}, UNSUPPORTED) for p in (8, 17, 48, 2048, 0, -16)], ({"n_seqs": 4097}, UNSUPPORTED), ({"n_children": 4097}, UNSUPPORTED),
    ({"n_pages": 2 ** 30 + 1}, UNSUPPORTED), ({"max_pages": 2 ** 24 + 1}, UNSUPPORTED), ({"workspace": None}, WORKSPACE),
    ({"workspace_bytes": 16}, WORKSPACE), ({"workspace": A + 4}, MISALIGNED), *[({k: 20 * A + 2}, MISALIGNED) for k in _ARRAYS],
    ({"page_table_out": 4 * A}, INVALID), ({"page_table_out": 4 * A + 56}, INVALID), ({"lens_out": 2 * A}, INVALID), ({"held_out": 3 * A + 8}, INVALID),
    ({"copy_rows": A}, INVALID), ({"copy_src": 2 * A}, INVALID), ({"shares_out": 5 * A + 4}, INVALID), ({"ring_out": 7 * A + 4}, INVALID)])
def test_fork(but, status):
    assert _call("kvq8_paged_fork", FORK, but) == status


CACHES = [(dict(k_codes=None), INVALID), (dict(v_scales=None), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_pages=0), INVALID),
          (dict(page_size=0), INVALID), (dict(page_size=8), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
          (dict(head_dim=64), UNSUPPORTED), (dict(k_scales=A + 8), MISALIGNED), (dict(v_codes=A + 4), MISALIGNED)]
COPY = dict(kv=_cache(), src=A, dst=A, rows=A, n=3, stream=None)


@pytest.mark.parametrize("but,status", [
    *[({"kv": _cache(**c)}, s) for c, s in CACHES], ({"kv": None}, INVALID), ({"src": None}, INVALID), ({"dst": None}, INVALID), ({"n": -1}, INVALID),
    *[({k: A + 2}, MISALIGNED) for k in ("src", "dst", "rows")], ({"n": 0, "src": None}, OK)])
def test_copy(but, status):
    assert _call("kvq8_paged_copy", COPY, but) == status


COMPACT = dict(kv=_cache(), page_table=A, max_pages=4, lens=2 * A, row_starts=A, n_seqs=3, kept=A, lens_out=3 * A, stream=None)


@pytest.mark.parametrize("but,status", [
    *[({"kv": _cache(**c)}, s) for c, s in CACHES], *[({k: None}, INVALID) for k in ("kv", "page_table", "lens", "row_starts", "kept")],
    ({"n_seqs": -1}, INVALID), ({"max_pages": 0}, INVALID), ({"n_seqs": 4097}, UNSUPPORTED), ({"lens_out": 2 * A}, INVALID),
    ({"lens_out": 2 * A + 8}, INVALID), *[({k: 4 * A + 2}, MISALIGNED) for k in ("page_table", "lens", "row_starts", "lens_out")],
    ({"kept": A + 4}, MISALIGNED), ({"n_seqs": 0, "lens": None}, OK)])
def test_compact(but, status):
    assert _call("kvq8_paged_compact", COMPACT, but) == status


ROPE = dict(q=A, k=2 * A, v=3 * A, dtype=1, n_tok=6, n_q_heads=8, q_stride=1024, k_stride=256, v_stride=256, positions=A, n_axes=2, turns=A,
            axis_of=A, rot_dim=128, pairs=0, kv=_cache(), slots=A, q_out=4 * A, out_stride=1024, stream=None)


@pytest.mark.parametrize("but,status", [
    *[({"kv": _cache(**c)}, s) for c, s in CACHES], *[({k: None}, INVALID) for k in ("q", "k", "v", "positions", "turns", "slots", "q_out", "kv")],
    ({"dtype": 3}, INVALID), ({"n_tok": -1}, INVALID), ({"n_q_heads": 0}, INVALID), ({"n_axes": 0}, INVALID),
    *[({k: 248}, INVALID) for k in ("q_stride", "k_stride", "v_stride", "out_stride")], *[({"rot_dim": r}, UNSUPPORTED) for r in (0, 32, 96, 192, 256, -64)],
    ({"n_axes": 5}, UNSUPPORTED), ({"n_q_heads": 65537, "q": 1 << 40, "q_out": 1 << 41, "q_stride": 1 << 24, "out_stride": 1 << 24}, UNSUPPORTED),
    *[({k: 9 * A + 8}, MISALIGNED) for k in ("q", "k", "v", "q_out")], *[({k: 1028}, MISALIGNED) for k in ("q_stride", "k_stride", "v_stride", "out_stride")],
    *[({k: A + 2}, MISALIGNED) for k in ("positions", "axis_of")], *[({k: A + 4}, MISALIGNED) for k in ("turns", "slots")],
    ({"q_out": A, "out_stride": 1032}, INVALID), ({"q_out": A + 16}, INVALID), ({"q_out": 2 * A}, INVALID), ({"q_out": 3 * A - 1024 * 12}, OK),
    ({"q_out": 3 * A - 1024 * 12 + 16}, INVALID), ({"n_tok": 0, "q": None}, OK)])
def test_rope(but, status):
    if status == OK and but.get("n_tok") != 0:   # a call that would be launched: only what it refuses is asked for
        but = {**but, "rot_dim": 96}
        status = UNSUPPORTED
    assert _call("kvq8_paged_append_rope", ROPE, but) == status


@pytest.mark.parametrize("out,status", [(A, UNSUPPORTED), (A + 1024 * 2, INVALID), (A + 1280 * 2, INVALID), (A + 1536 * 2, UNSUPPORTED)])
def test_rope_on_the_rows_of_one_product(out, status):
    """q, k, v and something beside them in rows of 2560 values: q_out over q or the rest, but not over k or v.  (An n_axes that is not
    supported is refused after that, so nothing is launched.)"""
    rows = dict(q=A, k=A + 1024 * 2, v=A + 1280 * 2, q_stride=2560, k_stride=2560, v_stride=2560, q_out=out, out_stride=2560, n_tok=1000)
    assert _call("kvq8_paged_append_rope", ROPE, {**rows, "n_axes": 5}) == status


def test_the_binding_refuses_tensors_it_cannot_pass_on():
    import torch

    import speculative_verify_attention_gb300 as kv
    i32 = torch.int32
    host = kv.KVPagedCacheQ8(2, 128, 16, 3, device="cpu")
    z = torch.zeros(4, dtype=i32)
    with pytest.raises(ValueError, match="CUDA device"):
        kv.beam_select(torch.zeros((4, 10)), torch.zeros(2, dtype=i32), 3)
    with pytest.raises(ValueError, match="CUDA device"):
        kv.token_counts_fork(z, z, torch.zeros((4, 10), dtype=i32), z, z[:1])
    with pytest.raises(ValueError, match="CUDA device"):
        kv.kvq8_paged_fork(z, z, z, 16, torch.zeros((4, 2), dtype=i32), z, z, z[:2], torch.zeros((4, 2), dtype=i32), z, z, z, z, z, z[:1])
    with pytest.raises(ValueError, match="CUDA device"):
        kv.kvq8_paged_copy(host, z, z)
    with pytest.raises(ValueError, match="CUDA device"):
        kv.kvq8_paged_compact(host, torch.zeros((4, 2), dtype=i32), z, torch.zeros(5, dtype=i32), torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA device"):
        x = torch.zeros((4, 2, 128))
        kv.kvq8_paged_append_rope(x, x, x, host, torch.zeros(4, dtype=torch.int64), z, kv.rope_turns(torch.ones(64)))


def test_turns_of_frequencies():
    """To the nearest 2^-64 of a turn, modulo a turn, against whole-number arithmetic from pi's digits."""
    import math
    from fractions import Fraction

    import torch

    from speculative_verify_attention_gb300 import rope_turns
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798214808651")
    f = [1.0, 10000.0 ** -0.5, 1e-12, 0.0, -0.25, math.pi, 2 * math.pi, 100.0, 1e6 + 0.5, -1e-30]
    for x, got in zip(f, rope_turns(torch.tensor(f, dtype=torch.float64)).tolist()):
        exact = Fraction(x) / (2 * pi) * 2 ** 64
        want = math.floor(exact + Fraction(1, 2)) % 2 ** 64
        assert got % 2 ** 64 == want, x
    for bad in (float("nan"), float("inf")):
        with pytest.raises(ValueError):
            rope_turns(torch.tensor([bad]))
