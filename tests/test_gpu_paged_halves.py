"""The paged append's quantiser where codes are decided: values at and around the half-integers of their block's step, blocks of tiny,
huge and subnormal steps, and random ones; its bytes are kvq8_append's, which go through the IEEE division."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def _both(x):
    """x fp32 [tokens][2][256] through kvq8_append and kvq8_paged_append: the same bytes."""
    from speculative_verify_attention_gb300 import KVCacheQ8, KVPagedCacheQ8, kvq8_append, kvq8_paged_append
    n = len(x)
    t = torch.from_numpy(x).cuda()
    flat, paged = KVCacheQ8(2, 256, n), KVPagedCacheQ8(2, 256, 16, -(-n // 16))
    kvq8_append(t, t.flip(0).contiguous(), flat, 0)
    kvq8_paged_append(t, t.flip(0).contiguous(), paged, torch.arange(n, device="cuda"))
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        a, b = getattr(flat, name), getattr(paged, name)
        b = b.permute(1, 0, 2, 3).reshape(2, -1, b.shape[3])[:, :n]
        if a.dtype == torch.float16:
            a, b = a.view(torch.int16), b.contiguous().view(torch.int16)
        assert torch.equal(a, b), name


def test_values_around_the_half_integers(lib):
    rng = np.random.default_rng(1)
    n = 6000
    step = np.exp(rng.uniform(-60, 60, (n, 2, 8, 1))).astype(np.float32)
    codes = rng.integers(-127, 127, (n, 2, 8, 32)) + 0.5
    x = (codes * step).astype(np.float32)
    x[..., 0] = (127 * step[..., 0]).astype(np.float32)
    near = rng.integers(-40, 41, x.shape) * (rng.random(x.shape) < 0.7)
    bits = x.view(np.int32) + near.astype(np.int32)                   # some units in the last place to either side
    x = np.where(np.abs(x) > 0, bits.view(np.float32), x)
    _both(x.reshape(n, 2, 256))


def test_values_as_far_as_the_short_way_trusts(lib):
    """Quotients within 2^-18 .. 2^-10 of a half-integer, to both sides of where the division takes over."""
    rng = np.random.default_rng(2)
    n = 6000
    step = np.exp(rng.uniform(-3, 3, (n, 2, 8, 1))).astype(np.float32)
    off = 2.0 ** rng.uniform(-18, -10, (n, 2, 8, 32)) * rng.choice([-1, 1], (n, 2, 8, 32))
    x = ((rng.integers(-126, 126, off.shape) + 0.5 + off) * step).astype(np.float32)
    x[..., 5] = -(127 * step[..., 0]).astype(np.float32)
    _both(x.reshape(n, 2, 256))


def test_steps_of_every_size(lib):
    rng = np.random.default_rng(3)
    n = 4000
    x = rng.standard_normal((n, 2, 8, 32)).astype(np.float32) * np.exp2(rng.uniform(-150, 120, (n, 2, 8, 1))).astype(np.float32)
    x[::7, :, 3] = 0.0
    x[1::7, :, 4] = np.where(np.arange(32) == 9, 1e-45, 0.0)          # the step is zero
    x[2::7, :, 5, 1:] = 0.0
    _both(x.reshape(n, 2, 256).astype(np.float32))
