"""Blocks with values that are no numbers, through the paged appends: the bytes of kvq8_append for the same values, whatever the type they
come in.  A block's scale is that of its largest number; NaN is code -127, and a block of 32 NaN has a NaN for its scale."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def _blocks(n, rng):
    x = rng.standard_normal((n, 2, 8, 32)).astype(np.float32)
    x[0::8] = np.nan
    x[1::8, :, :, 5] = np.nan
    x[2::8, :, :, 8:16] = np.nan                # a lane's eight
    x[3::8, :, :, 31] = np.inf
    x[4::8, :, :, ::2] = -np.inf
    x[5::8, :, :, 1:] = np.nan
    x[5::8, :, :, 0] = 0.0                      # nothing but zero beside them
    x[6::8, :, :, 3], x[6::8, :, :, 4] = np.nan, np.inf
    return x.reshape(n, 2, 256)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_bytes_are_those_of_the_plain_append(lib, dtype):
    from speculative_verify_attention_gb300 import KVCacheQ8, KVPagedCacheQ8, kvq8_append, kvq8_paged_append, kvq8_paged_append_rope, rope_turns
    n = 64
    k, v = (torch.from_numpy(_blocks(n, np.random.default_rng(s))).cuda().to(dtype) for s in (1, 2))
    flat, paged, turned = KVCacheQ8(2, 256, n), KVPagedCacheQ8(2, 256, 16, 4), KVPagedCacheQ8(2, 256, 16, 4)
    slots = torch.arange(n, device="cuda")
    kvq8_append(k.float(), v.float(), flat, 0)
    kvq8_paged_append(k, v, paged, slots)
    kvq8_paged_append_rope(k, k, v, turned, slots, slots.int(), rope_turns(torch.ones(128, dtype=torch.float64)).cuda())
    for cache, names in ((paged, ("k_codes", "v_codes", "k_scales", "v_scales")), (turned, ("v_codes", "v_scales"))):
        for name in names:
            a, b = getattr(flat, name), getattr(cache, name)
            b = b.permute(1, 0, 2, 3).reshape(2, n, -1)
            a, b = a.float().cpu().numpy(), b.float().cpu().numpy()
            assert np.array_equal(a, b, equal_nan=True), name
    codes, scales = (getattr(paged, name).permute(1, 0, 2, 3).reshape(2, n, -1).cpu().numpy() for name in ("k_codes", "k_scales"))
    assert np.all(np.isnan(scales[:, 0::8])) and np.all(codes[:, 0::8] == -127)
    assert np.all(scales[:, 5::8] == 0) and np.all(codes[:, 5::8] == 0)
    assert np.all(np.isfinite(scales[:, 1::8])) and np.all(codes[:, 1::8].reshape(2, -1, 8, 32)[..., 5] == -127)
