"""What the paged serving calls refuse, by status code, without a GPU: every refusal comes before any launch."""
import ctypes

import pytest

from speculative_verify_attention_gb300 import kvq8_paged_cache, load_library

A = 1 << 20            # an aligned address that nothing reads
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)


def _cache(**but):
    f = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, n_kv_heads=2, head_dim=128, page_size=16, n_pages=9)
    f.update(but)
    return kvq8_paged_cache(**f)


def _call(name, args, but):
    a = dict(args)
    a.update(but)
    return getattr(load_library(), name)(*a.values())


TABLES = dict(lens=A, n_new=A, held=A, n_seqs=3, page_size=16, page_table=A, max_pages=4, free_ring=A, n_pages=9, ring_state=A,
              held_out=A, ring_out=A, row_starts=A, slots=A, positions=A, n_rows=5, status=A, stream=None)


@pytest.mark.parametrize("but,status", [
    *[({k: None}, INVALID) for k in ("lens", "n_new", "held", "page_table", "free_ring", "ring_state", "held_out", "ring_out",
                                     "row_starts", "slots", "positions", "status")],
    *[({k: 0}, INVALID) for k in ("n_seqs", "max_pages", "n_pages")], ({"n_rows": -1}, INVALID),
    *[({"page_size": p}, UNSUPPORTED) for p in (8, 17, 48, 2048, 0, -16)], ({"n_seqs": 4097}, UNSUPPORTED),
    ({"n_pages": 2 ** 30 + 1}, UNSUPPORTED), ({"n_rows": 2 ** 30 + 1}, UNSUPPORTED),
    *[({k: A + 2}, MISALIGNED) for k in ("lens", "n_new", "held", "page_table", "free_ring", "ring_state", "held_out",
                                         "ring_out", "row_starts", "positions", "status")], ({"slots": A + 4}, MISALIGNED)])
def test_tables(but, status):
    assert _call("kvq8_paged_tables", TABLES, but) == status


CACHES = [(dict(k_codes=None), INVALID), (dict(v_scales=None), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_pages=0), INVALID),
          (dict(page_size=0), INVALID), (dict(page_size=8), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
          (dict(page_size=2048), UNSUPPORTED), (dict(head_dim=64), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED),
          (dict(k_scales=A + 8), MISALIGNED), (dict(v_codes=A + 4), MISALIGNED)]
APPEND = dict(k=A, v=A, dtype=0, n_tok=4, k_stride=256, v_stride=256, kv=_cache(), slots=A, stream=None)


@pytest.mark.parametrize("but,status", [
    *[({"kv": _cache(**c)}, s) for c, s in CACHES], ({"kv": None}, INVALID), ({"k": None}, INVALID), ({"v": None}, INVALID),
    ({"slots": None}, INVALID), ({"dtype": 3}, INVALID), ({"dtype": -1}, INVALID), ({"n_tok": -1}, INVALID),
    ({"k_stride": 255}, INVALID), ({"v_stride": 0}, INVALID), ({"k_stride": 258}, MISALIGNED), ({"dtype": 2, "v_stride": 260}, MISALIGNED),
    ({"k": A + 8}, MISALIGNED), ({"slots": A + 4}, MISALIGNED), ({"n_tok": 0, "k": None}, OK)])
def test_append(but, status):
    assert _call("kvq8_paged_append", APPEND, but) == status


def _strides(*v):
    return (ctypes.c_int64 * 2)(*v)


READ = dict(kv=_cache(), slots=A, n_tok=4, dtype=1, k=A, v=A, k_strides=_strides(256, 128), v_strides=_strides(128, 4096), stream=None)


@pytest.mark.parametrize("but,status", [
    *[({"kv": _cache(**c)}, s) for c, s in CACHES], ({"k": None}, INVALID), ({"slots": None}, INVALID), ({"k_strides": None}, INVALID),
    ({"dtype": 5}, INVALID), ({"n_tok": -2}, INVALID), ({"k_strides": _strides(127, 128)}, INVALID),
    ({"v_strides": _strides(128, 0)}, INVALID), ({"v_strides": _strides(132, 128)}, MISALIGNED), ({"v": A + 8}, MISALIGNED),
    ({"slots": A + 2}, MISALIGNED), ({"n_tok": 0, "k": None}, OK)])
def test_read(but, status):
    assert _call("kvq8_paged_read", READ, but) == status


VERIFY = dict(q=A, dtype=1, q_stride=1024, n_rows=6, n_q_heads=8, kv=_cache(), page_table=A, max_pages=4, lens=A, row_starts=A,
              n_seqs=2, max_rows=3, window_mask=None, scale=0.1, out=A, workspace=A, workspace_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("but,status", [
    *[({"kv": _cache(**c)}, s) for c, s in CACHES], *[({k: None}, INVALID) for k in ("q", "out", "page_table", "lens", "row_starts", "kv")],
    ({"dtype": 0}, INVALID), ({"dtype": 9}, INVALID), ({"n_rows": -1}, INVALID), ({"n_seqs": -1}, INVALID), ({"max_pages": 0}, INVALID),
    ({"kv": _cache(k_codes=A + 16)}, MISALIGNED), ({"kv": _cache(v_codes=A + 16)}, MISALIGNED),
    ({"kv": _cache(n_pages=2 ** 30, page_size=16, n_kv_heads=1)}, UNSUPPORTED),
    ({"kv": _cache(n_pages=2 ** 16, page_size=1024, n_kv_heads=32)}, UNSUPPORTED),
    ({"n_q_heads": 0}, INVALID), ({"max_rows": 0}, INVALID), ({"q_stride": 1023}, INVALID),
    *[({"scale": x}, INVALID) for x in (0.0, -1.0, float("inf"), float("nan"))],
    ({"n_q_heads": 7, "q_stride": 4096}, UNSUPPORTED), ({"n_q_heads": 130, "q_stride": 1 << 20}, UNSUPPORTED), ({"max_rows": 65}, UNSUPPORTED),
    ({"n_seqs": 4097}, UNSUPPORTED), ({"n_rows": 2 ** 24 + 1}, UNSUPPORTED), ({"workspace": None}, WORKSPACE),
    ({"workspace_bytes": 152 * 2 * 12 * 128 * 4}, WORKSPACE), ({"q": A + 8}, MISALIGNED), ({"out": A + 2}, MISALIGNED), ({"workspace": A + 8}, MISALIGNED),
    ({"q_stride": 1028}, MISALIGNED), ({"lens": A + 1}, MISALIGNED), ({"page_table": A + 2}, MISALIGNED),
    ({"row_starts": A + 2}, MISALIGNED), ({"window_mask": A + 4}, MISALIGNED), ({"n_rows": 0, "q": None}, OK), ({"n_seqs": 0, "q": None}, OK)])
def test_verify(but, status):
    assert _call("attn_verify_paged_q8", VERIFY, but) == status


def test_verify_workspace_query_refuses_what_the_call_refuses():
    f = load_library().attn_verify_paged_q8_workspace_bytes
    assert f(8, 2, 128, 3) > 0 and f(24, 4, 256, 64) > 0
    for a in ((0, 2, 128, 3), (8, 2, 64, 3), (8, 0, 128, 3), (8, 3, 128, 3), (8, 2, 128, 0), (8, 2, 128, 65), (130, 2, 128, 3)):
        assert f(*a) == 0


ADJUST = dict(logits=A, dtype=0, logits_stride=1000, n_rows=4, vocab=1000, row_starts=A, n_seqs=2, penalties=A, counts=A, n_states=3,
              state_of=A, window_tokens=A, window_mask=A, bias_starts=A, bias_tokens=A, bias_values=A, n_bias=5, grammar=A, n_grammar=2,
              grammar_of=A, out=2 * A, out_stride=1000, stream=None)


@pytest.mark.parametrize("but,status", [
    ({"dtype": 3}, INVALID), ({"n_rows": -1}, INVALID), ({"n_seqs": -1}, INVALID), ({"vocab": 0}, INVALID), ({"n_bias": -1}, INVALID),
    *[({k: None}, INVALID) for k in ("logits", "out", "row_starts", "penalties", "bias_tokens", "bias_values")],
    ({"penalties": None, "counts": None}, INVALID), ({"n_states": 0}, INVALID), ({"window_tokens": None}, INVALID), ({"n_grammar": 0}, INVALID),
    ({"logits_stride": 999}, INVALID), ({"out_stride": 999}, INVALID), ({"out": A, "out_stride": 1004}, INVALID),
    ({"out": A, "dtype": 1}, INVALID), ({"n_seqs": 4097}, UNSUPPORTED), ({"n_rows": 262141}, UNSUPPORTED),
    ({"vocab": 2 ** 30 + 1, "logits_stride": 2 ** 31, "out_stride": 2 ** 31}, UNSUPPORTED), ({"logits": A + 2}, MISALIGNED),
    ({"window_mask": A + 4}, MISALIGNED), *[({k: 2 * A + 2}, MISALIGNED) for k in ("row_starts", "penalties", "counts", "state_of",
                                                                                  "window_tokens", "bias_starts", "bias_tokens",
                                                                                  "bias_values", "grammar", "grammar_of", "out")],
    ({"n_rows": 0, "logits": None}, OK), ({"n_seqs": 0, "logits": None}, OK)])
def test_adjust(but, status):
    assert _call("logits_adjust", ADJUST, but) == status


COUNTS = dict(tokens=A, token_starts=A, n_lists=2, n_tokens=9, prompt_lens=A, state_of=A, clear=1, counts=A, n_states=3, vocab=100, stream=None)


@pytest.mark.parametrize("but,status", [
    ({"n_lists": -1}, INVALID), ({"n_tokens": -1}, INVALID), ({"n_states": 0}, INVALID), ({"vocab": 0}, INVALID),
    *[({k: None}, INVALID) for k in ("tokens", "token_starts", "counts")], ({"n_lists": 4097}, UNSUPPORTED),
    ({"vocab": 2 ** 30 + 1}, UNSUPPORTED), ({"n_tokens": 2 ** 30 + 1}, UNSUPPORTED),
    *[({k: A + 2}, MISALIGNED) for k in ("tokens", "token_starts", "prompt_lens", "state_of", "counts")], ({"n_lists": 0, "tokens": None}, OK)])
def test_counts(but, status):
    assert _call("token_counts", COUNTS, but) == status


def test_the_binding_refuses_tensors_it_cannot_pass_on():
    import torch

    import speculative_verify_attention_gb300 as kv
    host = kv.KVPagedCacheQ8(2, 128, 16, 3, device="cpu")
    k = torch.zeros((4, 2, 128))
    with pytest.raises(ValueError):
        kv.kvq8_paged_append(k, k, host, torch.zeros(4, dtype=torch.int64))       # on the host
    with pytest.raises(ValueError):
        kv.kvq8_paged_append(k, k.half(), host, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        kv.kvq8_paged_append(k[:, :, ::2], k[:, :, ::2], host, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        kv.attn_verify_paged_q8(torch.zeros((4, 4, 128)), host, torch.zeros((1, 2), dtype=torch.int32),
                                torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 4, 0.1)
    with pytest.raises(ValueError):
        kv.logits_adjust(torch.zeros((4, 10)), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        kv.KVPagedCacheQ8.from_planes(host.k_codes, host.k_scales[:1], host.v_codes, host.v_scales)
