"""kvq8_paged_append_rope against rotations in 64 bits: types, layouts, axes, positions of any size, strides, in place, skipped tokens."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402

from ._beams import angles_of, rotated  # noqa: E402
from ._paged import HALF_STEP, i32  # noqa: E402

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16

# cos and sin: the angle's fraction of a turn to 2^-33 (2^-34 cut off, 2^-65 of a turn a position from the table, of up to 2^31
# positions), rounded to fp32 once (2^-24 of at most pi / 4 radians), the functions to 2 units in the last place of at most 1; two
# products and a sum, each rounded once.
TURN_ERR = math.pi / 4 * 2.0 ** -24 + 2 * math.pi * 2.0 ** -33 + 2 * 2.0 ** -24


def _bound(x, pairs, half):
    """|error| of each rotated value in fp32: (|a| + |b|) (TURN_ERR + 2 half steps)."""
    a = np.abs(x.astype(np.float64))
    off = np.zeros_like(a)
    i, j = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    off[..., i] = off[..., j] = (a[..., i] + a[..., j]) * (TURN_ERR + 2 * 2.0 ** -24)
    return off


def _check_k(codes, scales, k, off):
    """Codes and scales [n][heads][hd], [n][heads][hd / 32] of values k that are known to within off: a code is the rounded quotient of
    some number within, the scale the rounded maximum of some."""
    blocks, slack = k.reshape(*k.shape[:2], -1, 32), off.reshape(*k.shape[:2], -1, 32)
    top = np.abs(blocks).max(-1)
    s = scales.astype(np.float64)
    err = slack.max(-1) / 127 + top / 127 * (2.0 ** -11 + 2.0 ** -22)
    assert np.all(np.abs(s - top / 127) <= err + 2.0 ** -25)
    d = (top / 127)[..., None]
    got = codes.reshape(blocks.shape).astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        room = 0.5 + np.where(d > 0, slack / d + np.abs(blocks) / d * (slack.max(-1, keepdims=True) / (127 * d) + 2.0 ** -22), 0)
        assert np.all((np.abs(got - np.where(d > 0, blocks / d, 0)) <= room) | (d == 0))


def _case(seed, n, hq, hkv, hd, dtype, rot, pairs=False, axes=1, far=30000, page=16, positions=None, axis_of=None, freq=None,
          in_place=False, fused=False, skip=False, one_axis=False):
    from speculative_verify_attention_gb300 import KVPagedCacheQ8, kvq8_paged_append_rope, rope_turns
    rng = np.random.default_rng(seed)
    half = rot // 2
    freq = 10000.0 ** (-np.arange(half) / half) if freq is None else np.asarray(freq, np.float64)
    if positions is None:
        positions = rng.integers(0, far, (axes, n))
    if fused:  # q, k and v of a token side by side, as one product gives them
        whole = torch.from_numpy(rng.standard_normal((n, hq + 2 * hkv + 1, hd)).astype(np.float32)).to(dtype).cuda()
        q, k, v = whole[:, :hq], whole[:, hq:hq + hkv], whole[:, hq + hkv:hq + 2 * hkv]
    else:
        q, k, v = (torch.from_numpy(rng.standard_normal((n, h, hd)).astype(np.float32)).to(dtype).cuda() for h in (hq, hkv, hkv))
    xq, xk, xv = (t.float().cpu().numpy() for t in (q, k, v))
    pages = -(-n // page) + 2
    order, at = rng.permutation(pages), np.arange(n)
    slots = order[at // page] * page + at % page
    left = np.zeros(n, bool)
    if skip:
        left = rng.random(n) < 0.3
        slots = np.where(left, rng.choice([-1, -2 ** 40, pages * page, 2 ** 50], n), slots)
    cache = KVPagedCacheQ8(hkv, hd, page, pages)
    for p in (cache.k_codes, cache.v_codes):
        p.fill_(77)
    before = whole.clone() if fused else None
    out = q if in_place else torch.full(q.shape, 55.0, dtype=dtype, device="cuda")
    kvq8_paged_append_rope(q, k, v, cache, torch.from_numpy(slots).cuda(), i32(positions[0] if one_axis else positions),
                           rope_turns(torch.from_numpy(freq).cuda()), axis_of=None if axis_of is None else i32(axis_of), pairs=pairs,
                           q_out=out)
    torch.cuda.synchronize()
    ang = angles_of(np.asarray(positions), freq, axis_of)
    got, want, off = out.double().cpu().numpy(), rotated(xq, ang, pairs), _bound(xq, pairs, half)
    off = off + (np.abs(want) + off) * (0 if dtype == F32 else HALF_STEP[dtype]) + 2.0 ** -140 + (2.0 ** -25 if dtype == F16 else 0)
    assert np.all(np.abs(got - want)[~left] <= off[~left])
    assert np.all(got[left] == (xq[left] if in_place else 55.0))
    assert np.array_equal(got[~left][..., rot:], xq[~left][..., rot:])            # what is not rotated passes as it is
    if fused:                                                                     # nothing beside q is written
        assert torch.equal(whole[:, hq:], before[:, hq:])
    ok = ~left
    pg, o = slots[ok] // page, slots[ok] % page
    kc, ks = cache.k_codes.cpu().numpy()[pg, :, o], cache.k_scales.float().cpu().numpy()[pg, :, o]
    if ok.any():
        _check_k(kc, ks, rotated(xk, ang, pairs)[ok], _bound(xk, pairs, half)[ok])
    vc, vs = cache.v_codes.cpu().numpy()[pg, :, o], cache.v_scales.cpu().numpy().view(np.uint16)[pg, :, o]
    if ok.any():
        ref = oracle.Cache(hkv, hd, int(ok.sum()))
        ref.append(np.ascontiguousarray(xk[ok]), np.ascontiguousarray(xv[ok]), 0)
        assert np.array_equal(vc, ref.v_codes.transpose(1, 0, 2)) and np.array_equal(vs, ref.v_scales.transpose(1, 0, 2))
        tail = slice(rot, hd)
        assert np.array_equal(kc[..., tail], ref.k_codes.transpose(1, 0, 2)[..., tail])
    written = np.zeros((pages, page), bool)
    written[pg, o] = True
    assert np.all(cache.k_codes.cpu().numpy().transpose(0, 2, 1, 3)[~written] == 77)
    return out, cache


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("hq,hkv,hd,rot", [(24, 4, 256, 256), (12, 1, 256, 64), (8, 2, 128, 128), (5, 5, 128, 64), (3, 3, 256, 192), (1, 1, 128, 128)])
def test_types_and_layouts(lib, dtype, pairs, hq, hkv, hd, rot):
    for n in (1, 2, 37):
        _case(n, n, hq, hkv, hd, dtype, rot, pairs)


@pytest.mark.parametrize("pairs", [False, True])
def test_axes(lib, pairs):
    """Sections of the dims, dims in turn, an axis that there is not, more axes than pairs ask for."""
    rng = np.random.default_rng(1)
    half = 64
    for axes in (1, 2, 3, 4):
        for axis_of in (np.arange(half) * axes // half, np.arange(half) % axes, rng.integers(-1, axes + 1, half), None):
            _case(axes, 50, 8, 2, 128, BF16, 128, pairs, axes=axes, axis_of=axis_of)
    _case(9, 20, 8, 2, 128, F32, 128, pairs, one_axis=True)


def test_positions_of_any_size_and_frequencies(lib):
    top = 2 ** 31 - 1
    positions = np.array([[0, 1, -1, 7, -12345, 10 ** 6, 10 ** 9, top, -top - 1, top - 1, 1 << 30, 12]])
    half = 64
    rng = np.random.default_rng(2)
    for freq in (10000.0 ** (-np.arange(half) / half), np.full(half, math.pi), np.full(half, -math.pi / 2), rng.random(half) * 7 - 3.5,
                 np.where(np.arange(half) % 2, 0.0, 1e-12), (2 * math.pi) * np.arange(half) / 64):
        for pairs in (False, True):
            _case(3, 12, 2, 1, 128, F32, 128, pairs, positions=positions, freq=freq)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place_fused_rows_and_skipped_tokens(lib, dtype):
    for n in (1, 40):
        for kw in (dict(in_place=True), dict(fused=True), dict(fused=True, in_place=True), dict(skip=True), dict(skip=True, in_place=True)):
            _case(n, n, 8, 2, 128, dtype, 128, **kw)
            _case(n, n, 6, 3, 256, dtype, 128, pairs=True, **kw)


def test_prompts(lib):
    """Thousands of tokens: several a block, the last block not full."""
    for n in (2047, 2048, 4099):
        _case(n, n, 4, 1, 128, BF16, 128, axes=3, axis_of=np.arange(64) * 3 // 64, page=64)


def test_no_rotation_is_an_append(lib):
    """Positions of zero: the bytes of kvq8_paged_append."""
    from speculative_verify_attention_gb300 import KVPagedCacheQ8, kvq8_paged_append, kvq8_paged_append_rope, rope_turns
    rng = np.random.default_rng(4)
    x = [torch.from_numpy(rng.standard_normal((33, h, 128)).astype(np.float32)).cuda() for h in (8, 2, 2)]
    for t in x:
        t[3] = 0.0
        t[4] *= 1e-30
        t[5] *= 1e30
    slots = torch.arange(33, device="cuda") + 5
    a, b = KVPagedCacheQ8(2, 128, 16, 4), KVPagedCacheQ8(2, 128, 16, 4)
    kvq8_paged_append(x[1], x[2], a, slots)
    out = kvq8_paged_append_rope(*x, b, slots, i32([0] * 33), rope_turns(torch.rand(64)).cuda())
    assert torch.equal(out, x[0])
    for p, q in ((a.k_codes, b.k_codes), (a.k_scales, b.k_scales), (a.v_codes, b.v_codes), (a.v_scales, b.v_scales)):
        assert torch.equal(p, q)


def test_numbers_that_are_none_stay_in_their_pair_and_block(lib):
    from speculative_verify_attention_gb300 import KVPagedCacheQ8, kvq8_paged_append_rope, rope_turns
    x = [torch.randn((4, h, 128), device="cuda") for h in (4, 1, 1)]
    cache = KVPagedCacheQ8(1, 128, 16, 1)
    args = (cache, torch.arange(4, device="cuda"), i32([5, 6, 7, 8]), rope_turns(torch.rand(32)).cuda())
    one = kvq8_paged_append_rope(*x, *args)
    clean = cache.k_codes.clone()
    x[0][1, 2, 3], x[1][2, 0, 100] = float("nan"), float("inf")
    two = kvq8_paged_append_rope(*x, *args)
    wrong = torch.isnan(two)
    assert wrong.sum() == 2 and wrong[1, 2, 3] and wrong[1, 2, 35]
    assert torch.equal(two[~wrong], one[~wrong])
    same = torch.ones_like(clean, dtype=torch.bool)
    same[0, 0, 2, 96:] = False
    assert torch.equal(cache.k_codes[same], clean[same])


def test_a_captured_call_and_another_stream(lib):
    from speculative_verify_attention_gb300 import KVPagedCacheQ8, kvq8_paged_append_rope, rope_turns
    x = [torch.randn((9, h, 128), device="cuda").bfloat16() for h in (8, 2, 2)]
    cache, slots, pos = KVPagedCacheQ8(2, 128, 16, 3), torch.arange(9, device="cuda"), i32(np.arange(9))
    turns, out = rope_turns(torch.rand(64)).cuda(), torch.empty_like(x[0])
    kvq8_paged_append_rope(*x, cache, slots, pos, turns, q_out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq8_paged_append_rope(*x, cache, slots, pos, turns, q_out=out)
    pos.add_(1000)
    slots.add_(20)
    g.replay()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    codes = cache.k_codes.clone()
    for stream in (side, side.cuda_stream):
        other = kvq8_paged_append_rope(*x, cache, slots, pos, turns, stream=stream)
        side.synchronize()
        assert torch.equal(other, out) and torch.equal(cache.k_codes, codes)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("n,hq,hkv,hd,rot", [(1901, 8, 2, 128, 64), (1999, 1, 1, 128, 128), (1001, 12, 1, 256, 192), (923, 2, 1, 256, 256)])
def test_many_tokens_of_few_heads(lib, dtype, pairs, n, hq, hkv, hd, rot):
    """Blocks that take two groups of tokens, and come round with a part of one."""
    _case(n, n, hq, hkv, hd, dtype, rot, pairs, axes=2, axis_of=np.arange(rot // 2) % 2, skip=True)
    _case(n + 1, n + 6, hq, hkv, hd, dtype, rot, pairs, far=10 ** 6, in_place=True, fused=True)
