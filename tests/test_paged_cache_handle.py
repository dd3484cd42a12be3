"""KVPagedCacheQ8: the C struct that its calls pass follows the planes."""
import pytest

torch = pytest.importorskip("torch")

from speculative_verify_attention_gb300 import KVPagedCacheQ8  # noqa: E402

PLANES = ("k_codes", "k_scales", "v_codes", "v_scales")


def test_a_replaced_plane_is_the_one_that_is_passed():
    c = KVPagedCacheQ8(2, 128, 16, 5, device="cpu")
    for name in PLANES:
        new = getattr(c, name).clone()
        setattr(c, name, new)
        assert getattr(c, name) is new
        for other in PLANES:
            assert getattr(c.struct(), other) == getattr(c, other).data_ptr()
    assert (c.struct().n_pages, c.struct().n_kv_heads, c.struct().page_size, c.struct().head_dim) == (5, 2, 16, 128)


@pytest.mark.parametrize("name", PLANES)
def test_a_plane_that_does_not_fit_is_refused_and_changes_nothing(name):
    c = KVPagedCacheQ8(2, 128, 16, 5, device="cpu")
    before = {n: getattr(c, n) for n in PLANES}
    for bad in (before[name][:4].clone(), before[name].float(), before[name].transpose(1, 2)):
        with pytest.raises(ValueError):
            setattr(c, name, bad)
    assert all(getattr(c, n) is before[n] and getattr(c.struct(), n) == before[n].data_ptr() for n in PLANES)
