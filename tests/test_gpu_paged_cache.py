"""kvq8_paged_append and kvq8_paged_read: bytes equal to the oracle's quantiser, values equal to code * scale rounded once."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402

pytestmark = pytest.mark.gpu


def _pool(hkv, hd, page, pages, seed=0):
    from speculative_verify_attention_gb300 import KVPagedCacheQ8
    c = KVPagedCacheQ8(hkv, hd, page, pages)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.randint(-127, 128, t.shape, generator=gen, device="cuda"))
    for t in (c.k_scales, c.v_scales):
        t.copy_(torch.rand(t.shape, generator=gen, device="cuda"))
    return c


def _planes(c):
    """Planes as [slot][head][...], on the host."""
    return [t.cpu().numpy().transpose(0, 2, 1, 3).reshape(c.n_pages * c.page_size, c.n_kv_heads, -1).copy()
            for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]


def _values(rng, n, hkv, hd):
    x = rng.standard_normal((n, hkv, hd)).astype(np.float32)
    x[:, :, 3] *= 30.0
    x[rng.random((n, hkv)) < 0.1] = 0.0
    x[:, :, 32:64] *= 1e-4
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hkv,hd,page", [(4, 256, 16), (8, 128, 64), (1, 128, 1024), (3, 256, 32), (33, 128, 16)])
@pytest.mark.parametrize("n", [1, 2, 5, 77])
def test_appended_bytes_equal_the_oracles(lib, dtype, hkv, hd, page, n):
    from speculative_verify_attention_gb300 import kvq8_paged_append
    rng = np.random.default_rng(n * hd + page)
    c = _pool(hkv, hd, page, -(-n // page) + 2)
    total = c.n_pages * page
    before = _planes(c)
    k, v = (torch.from_numpy(_values(rng, n, hkv, hd)).to(dtype) for _ in range(2))
    slots = rng.permutation(total)[:n].astype(np.int64)
    kvq8_paged_append(k.cuda(), v.cuda(), c, torch.from_numpy(slots).cuda())
    orc = oracle.Cache(hkv, hd, n)
    orc.append(k.float().numpy(), v.float().numpy(), 0)
    want = [orc.k_codes, orc.k_scales, orc.v_codes, orc.v_scales]
    for got, old, w in zip(_planes(c), before, want):
        old.view(np.int8 if old.dtype == np.int8 else np.uint16)[slots] = w.transpose(1, 0, 2)
        assert np.array_equal(got.view(np.uint8), old.view(np.uint8))


def test_slots_outside_are_skipped_and_tokens_may_be_strided(lib):
    from speculative_verify_attention_gb300 import kvq8_paged_append
    rng = np.random.default_rng(1)
    c = _pool(2, 128, 16, 3)
    before = _planes(c)
    wide = torch.from_numpy(rng.standard_normal((9, 5, 2, 128)).astype(np.float32)).cuda().bfloat16()
    slots = np.array([-1, 48, 7, 47, -2 ** 62, 2 ** 62, 0, 2 ** 32 + 5, 20])
    kvq8_paged_append(wide[:, 1], wide[:, 4], c, torch.from_numpy(slots).cuda())
    orc = oracle.Cache(2, 128, 9)
    orc.append(wide[:, 1].float().cpu().numpy(), wide[:, 4].float().cpu().numpy(), 0)
    inside = [2, 3, 6, 8]
    for got, old, w in zip(_planes(c), before, [orc.k_codes, orc.k_scales, orc.v_codes, orc.v_scales]):
        old.view(w.dtype)[slots[inside]] = w.transpose(1, 0, 2)[inside]
        assert np.array_equal(got.view(np.uint8), old.view(np.uint8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hkv,hd,page", [(4, 256, 16), (1, 128, 64), (3, 128, 16), (8, 256, 256)])
def test_read_values_are_rounded_once(lib, dtype, hkv, hd, page):
    from speculative_verify_attention_gb300 import kvq8_paged_read
    c = _pool(hkv, hd, page, 7, seed=hd)
    total = 7 * page
    slots = np.random.default_rng(2).integers(0, total, 133)
    slots[[3, 60]] = [-1, total]
    k, v = (torch.full((133, hkv, hd), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    kvq8_paged_read(c, torch.from_numpy(slots).cuda(), k, v)
    p = _planes(c)
    ok = (slots >= 0) & (slots < total)
    for got, codes, scales in ((k, p[0], p[1]), (v, p[2], p[3])):
        want = codes.astype(np.float64) * np.repeat(scales.astype(np.float64), 32, axis=-1)
        want = np.where(ok[:, None, None], want[np.where(ok, slots, 0)], 0.0)
        assert torch.equal(got.cpu(), torch.from_numpy(want).float().to(dtype))  # the product is exact in fp32


def test_read_fills_an_fp16_pool_for_a_prompt(lib):
    """A prompt chunk behind a paged context: the pages read into an fp16 pool, then attn_prompt_f16 over it, against
    attn_prompt_q8 over the same bytes kept in one piece (both round code * scale to fp16 once: the same operands)."""
    from speculative_verify_attention_gb300 import (KVCacheF16, KVCacheQ8, attn_prompt_f16, attn_prompt_q8, kvq8_paged_append,
                                                    kvq8_paged_read)
    rng = np.random.default_rng(3)
    n, hkv, hd, page = 517, 2, 128, 16
    c = _pool(hkv, hd, page, 40)
    order = rng.permutation(40)[:-(-n // page)]
    slots = torch.from_numpy(order[np.arange(n) // page] * page + np.arange(n) % page).cuda()
    k, v = (torch.from_numpy(rng.standard_normal((n, hkv, hd)).astype(np.float32)).cuda() for _ in range(2))
    kvq8_paged_append(k, v, c, slots)
    pool = KVCacheF16(hkv, hd, 600)
    kvq8_paged_read(c, slots, pool.k.transpose(0, 1)[:n], pool.v.transpose(0, 1)[:n])
    assert not pool.k[:, n:].any() and not pool.v[:, n:].any()
    whole = KVCacheQ8(hkv, hd, 600)
    whole.append(k, v, 0)
    q = torch.from_numpy(rng.standard_normal((100, 8, hd)).astype(np.float32)).cuda().half()
    a = attn_prompt_f16(q, pool, n, n - 100, 0.09)
    b = attn_prompt_q8(q, whole, n, n - 100, 0.09)
    assert torch.equal(a, b)


def test_append_then_read_past_32_bit_offsets(lib):
    from speculative_verify_attention_gb300 import KVPagedCacheQ8, kvq8_paged_append, kvq8_paged_read
    pages = 2 ** 32 // (8 * 64 * 128) + 100
    c = KVPagedCacheQ8.from_planes(*(torch.empty((pages, 8, 64, w), dtype=t, device="cuda")
                                     for w, t in ((128, torch.int8), (4, torch.float16)) * 2))
    total = pages * 64
    slots = torch.tensor([total - 1, 0, total - 64 * 90], device="cuda")
    k, v = torch.randn((2, 3, 8, 128), device="cuda").unbind(0)
    kvq8_paged_append(k, v, c, slots)
    a, b = torch.empty_like(k), torch.empty_like(v)
    kvq8_paged_read(c, slots, a, b)
    for x, y in ((a, k), (b, v)):
        block = y.unflatten(2, (4, 32)).abs().amax(-1, keepdim=True) / 127
        # half a code step, and the scale's own rounding (2^-11 of up to 127 codes)
        assert torch.all((x - y).unflatten(2, (4, 32)).abs() <= block * (0.5 + 127 * 2.0 ** -11 + 1e-3))
