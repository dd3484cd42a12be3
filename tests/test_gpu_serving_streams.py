"""The serving calls on streams that are not the current one, given as objects and as raw handles: the memory that a call takes
for itself belongs to the stream that it runs on."""
import pytest

torch = pytest.importorskip("torch")

from ._paged import Batch, i32  # noqa: E402

pytestmark = pytest.mark.gpu
CYCLES = 40_000_000  # some 20 ms


def _streams():
    side = torch.cuda.Stream()
    return [(side, side), (side, side.cuda_stream)]


@pytest.mark.parametrize("raw", [False, True])
def test_a_workspace_is_not_given_out_to_the_current_stream(lib, raw, monkeypatch):
    from speculative_verify_attention_gb300 import attn_verify_paged_q8, attn_verify_paged_q8_workspace_bytes, binding
    side, stream = _streams()[raw]
    b = Batch(21, 8, 2, 128, 16, [900, 40], [3, 2], torch.float16, tree=True)
    b.words = None
    cache, q, args = b.cache(), b.q.cuda(), (i32(b.table), i32(b.lens), i32(b.starts), 3, b.scale)
    expected = b.expect()
    size = attn_verify_paged_q8_workspace_bytes(8, 2, 128, 3)
    taken, take = [], binding._scratch
    monkeypatch.setattr(binding, "_scratch", lambda *a: taken.append(take(*a)) or taken[-1])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    out = attn_verify_paged_q8(q, cache, *args, stream=stream)
    at = {t.data_ptr() for t in taken}
    assert size in {t.numel() for t in taken}
    taken.clear()  # the call has returned and holds nothing
    new = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert new.data_ptr() not in at
    side.synchronize()
    b.check(out, expected)


@pytest.mark.parametrize("raw", [False, True])
def test_an_output_is_not_memory_that_the_current_stream_still_uses(lib, raw):
    from speculative_verify_attention_gb300 import logits_adjust
    side, stream = _streams()[raw]
    x, starts = torch.randn((64, 5000), device="cuda"), i32([0, 64])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(CYCLES)
    old = torch.full((64, 5000), 9.0, device="cuda")  # written late, and its memory free at once
    del old
    out = logits_adjust(x, starts, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(out, x)


@pytest.mark.parametrize("handle", [0, 1, 2])
def test_the_default_streams_handles(lib, handle):
    """0 and 1 are the legacy default stream, 2 the thread's."""
    b = Batch(22, 8, 2, 128, 16, [300, 40], [3, 2], torch.bfloat16)
    from speculative_verify_attention_gb300 import attn_verify_paged_q8
    args = (b.q.cuda(), b.cache(), i32(b.table), i32(b.lens), i32(b.starts), 3, b.scale)
    torch.cuda.synchronize()
    out = attn_verify_paged_q8(*args, stream=handle)
    torch.cuda.synchronize()
    b.check(out)


@pytest.mark.parametrize("rows,hq,hd,lens", [(2, 8, 128, [9000, 1200]), (5, 12, 256, [20000, 3000]), (30, 12, 256, [6000, 900])])
def test_calls_that_overlap_on_two_streams(lib, rows, hq, hd, lens):
    """Calls over one cache on two streams at once, each with a workspace and an output of its own."""
    from speculative_verify_attention_gb300 import attn_verify_paged_q8, attn_verify_paged_q8_workspace_bytes, kvq8_device_error
    b = Batch(23 + rows, hq, 2, hd, 32, lens, [rows, rows], torch.bfloat16)
    cache, q, args = b.cache(), b.q.cuda(), (i32(b.table), i32(b.lens), i32(b.starts), rows, b.scale)
    one = b.call(cache)
    b.check(one, b.expect(rows={0, rows - 1, rows, 2 * rows - 1}))
    size = attn_verify_paged_q8_workspace_bytes(hq, 2, hd, rows)
    streams = [torch.cuda.Stream() for _ in range(2)]
    space = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [[torch.full_like(one, 77.0) for _ in range(10)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(10):
        for s, w, o in zip(streams, space, outs):
            attn_verify_paged_q8(q, cache, *args, out=o[i], workspace=w, stream=s)
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert torch.equal(o, one)
    assert kvq8_device_error(reset=True) == 0
