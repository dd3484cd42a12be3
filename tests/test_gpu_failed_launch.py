"""A launch that fails on the host is that call's error and no other's.

While a blocking stream is being captured, a launch into the legacy default stream is refused by the runtime: nothing
runs, the call returns an error, and the capture is over."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_verify_attention_gb300 as kv  # noqa: E402

from ._paged import Batch, i32  # noqa: E402

pytestmark = pytest.mark.gpu
RELAXED, LEGACY = 2, 0


def _calls():
    """All tensors are made here: while the capture runs, torch itself must not use the default stream."""
    b = Batch(51, 8, 2, 128, 16, [300, 40], [3, 2], torch.float16)
    cache, q, ws = b.cache(), b.q.cuda(), torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    table, lens, starts, out = i32(b.table), i32(b.lens), i32(b.starts), torch.zeros_like(q)
    x, y, slots = torch.randn((4, 2, 128), device="cuda"), torch.randn((4, 2, 128), device="cuda"), torch.arange(4, device="cuda")
    logits, bent, counts = torch.randn((5, 640), device="cuda"), torch.zeros((5, 640), device="cuda"), i32(np.zeros((2, 640)))
    one, pair = i32([0, 0]), i32([0, 2])
    t = [i32([0, 0]), i32(np.zeros((2, 4))), i32(np.arange(9)), i32([0, 9])]
    new = [i32(np.zeros(3)), torch.zeros(3, dtype=torch.int64, device="cuda"), i32(np.zeros(3)), i32([0])]
    rows, joined = i32([0, 2, 5]), torch.zeros((8, 128), device="cuda")
    q8 = kv.KVCacheQ8(2, 128, 64)
    q32, o32 = torch.randn((4, 8, 128), device="cuda"), torch.zeros((4, 8, 128), device="cuda")
    arg, top = i32(np.zeros(5)), torch.zeros(5, device="cuda")
    part_o, part_ml = torch.zeros((3, 8, 128), device="cuda"), torch.zeros((3, 8, 2), device="cuda")
    return {
        "tables": lambda: kv.kvq8_paged_tables(one, one, *t, 16, *new, stream=LEGACY),
        "append": lambda: kv.kvq8_paged_append(x, y, cache, slots, stream=LEGACY),
        "read": lambda: kv.kvq8_paged_read(cache, slots, x, y, stream=LEGACY),
        "verify": lambda: kv.attn_verify_paged_q8(q, cache, table, lens, starts, 3, b.scale, out=out, workspace=ws, stream=LEGACY),
        "adjust": lambda: kv.logits_adjust(logits, rows, out=bent, stream=LEGACY),
        "counts": lambda: kv.token_counts(pair, pair, counts, stream=LEGACY),
        "counts anew": lambda: kv.token_counts(pair, pair, counts, clear=True, stream=LEGACY),
        "one request": lambda: kv.attn_verify_q8(q32, q8, 64, 60, 0.09, out=o32, workspace=ws, stream=LEGACY),
        "combine": lambda: kv.attn_combine(part_o, part_ml, out=joined, stream=LEGACY),
        "argmax": lambda: kv.argmax_rows_top_prob(logits, workspace=ws, argmax=arg, top_prob=top, stream=LEGACY)}


@pytest.mark.parametrize("name", ["tables", "append", "read", "verify", "adjust", "counts", "counts anew", "one request", "combine",
                                  "argmax"])
def test_the_call_after_it_succeeds(lib, name):
    call = _calls()[name]
    call()
    cache = kv.KVCacheQ8(2, 128, 64)
    k, v = torch.randn((64, 2, 128), device="cuda"), torch.randn((64, 2, 128), device="cuda")
    torch.cuda.synchronize()
    cu, stream, graph = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 0) == 0
    assert cu.cuStreamBeginCapture_v2(stream, RELAXED) == 0
    try:
        with pytest.raises(kv.KVQ8Error):
            call()
    finally:
        assert cu.cuStreamEndCapture(stream, ctypes.byref(graph)) != 0  # the refused launch has ended the capture
        assert cu.cuStreamDestroy_v2(stream) == 0
    cache.append(k, v, 0, stream=LEGACY)
    call()
    torch.cuda.synchronize()
    block = k.unflatten(2, (4, 32)).abs().amax(-1) / 127
    scales = cache.k_scales.transpose(0, 1).float()
    assert torch.all((scales - block).abs() <= block * 2.0 ** -11 + 2.0 ** -24)
