"""Outputs of the serving calls that lie over their inputs or over themselves are refused, before any launch."""
import pytest

from .test_paged_refusals import ADJUST, INVALID, READ, A, _cache, _call, _strides

BARE = dict(penalties=None, counts=None, state_of=None, window_tokens=None, window_mask=None)


@pytest.mark.parametrize("but", [
    dict(out=A + 4), dict(out=A - 4), dict(out=A + 4 * 999), dict(out=A + 4000), dict(out=A + 3 * 4000 + 4 * 999),  # fp32 rows over fp32 rows
    dict(out=A - 3 * 4000), dict(out=A + 4000, logits_stride=2000, out_stride=1000), dict(out=A + 4 * 1500, logits_stride=2000, out_stride=2000),
    dict(out=A, out_stride=1008, logits_stride=1008, dtype=1), dict(out=A + 2000, dtype=1), dict(out=A - 3996, dtype=2),
    dict(out=A + 2000, dtype=1, logits_stride=2000, out_stride=1000),     # a 16-bit row in each fp32 row, and the next too near
    dict(out=A + 4 * 1000, logits_stride=2000, out_stride=2003)])         # clear of the first row only
def test_adjust(but):
    assert _call("logits_adjust", ADJUST, {**BARE, **but}) == INVALID


@pytest.mark.parametrize("n_tok,heads,strides", [
    (4, 2, (128, 128)), (4, 2, (128, 384)), (4, 3, (256, 128)), (4, 3, (384, 192)), (4, 5, (512, 128)), (1000, 8, (128, 999 * 128)),
    (4, 2, (256, 192)), (2, 4096, (4095 * 128, 128))])
@pytest.mark.parametrize("plane", ["k_strides", "v_strides"])
def test_read(n_tok, heads, strides, plane):
    wide = _strides(1 << 20, 128)  # rows that lie apart
    but = dict(kv=_cache(n_kv_heads=heads), n_tok=n_tok, k_strides=wide, v_strides=wide)
    assert _call("kvq8_paged_read", READ, {**but, plane: _strides(*strides)}) == INVALID
