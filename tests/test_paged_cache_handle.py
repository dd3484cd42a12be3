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


def test_a_plane_replaced_while_a_call_runs_frees_nothing_that_the_call_reads(monkeypatch):
    """The native calls get the struct's address and let other threads run: one of them may replace a plane meanwhile.  The struct that
    the call was given, and the planes that it names, have to last until it returns."""
    import gc
    import weakref

    from speculative_verify_attention_gb300 import binding, kvq8_paged_cache
    i32, z = torch.int32, torch.zeros(4, dtype=torch.int32)
    slots, x, turns = torch.zeros(4, dtype=torch.int64), torch.zeros((4, 2, 128)), torch.zeros(64, dtype=torch.int64)
    calls = {"paged_read": lambda c: binding.kvq8_paged_read(c, slots, x, x.clone()),
             "paged_copy": lambda c: binding.kvq8_paged_copy(c, z, z),
             "paged_compact": lambda c: binding.kvq8_paged_compact(c, torch.zeros((4, 2), dtype=i32), z, torch.zeros(5, dtype=i32), slots),
             "paged_append_rope": lambda c: binding.kvq8_paged_append_rope(x, x, x, c, slots, z, turns, q_out=x)}
    monkeypatch.setattr(binding, "_launch_on", lambda device, stream: 0)
    for name, call in calls.items():
        cache = KVPagedCacheQ8(2, 128, 16, 5, device="cpu")
        struct, plane, address = weakref.ref(cache.struct()), weakref.ref(cache.k_codes), cache.k_codes.data_ptr()
        seen = []

        class Native:
            pass

        def during(at, *rest):
            cache.k_codes = cache.k_codes.clone()      # what another thread may do
            gc.collect()
            seen.append(struct() is not None and plane() is not None)
            if seen[0]:
                seen.append(kvq8_paged_cache.from_address(at).k_codes == address)
            return 0
        setattr(Native, name, staticmethod(during))
        monkeypatch.setattr(binding, "_native", lambda: Native)
        call(cache)
        assert seen == [True, True], name
        gc.collect()
        assert struct() is None and plane() is None and cache.struct().k_codes == cache.k_codes.data_ptr()  # and no longer
