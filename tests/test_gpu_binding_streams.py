"""The calls over one request on streams that are not the current one, given as objects and as raw handles: the memory that a
call takes for itself belongs to the stream that it runs on."""
import pytest

torch = pytest.importorskip("torch")

import speculative_verify_attention_gb300 as kv  # noqa: E402

pytestmark = pytest.mark.gpu
CYCLES = 40_000_000  # some 20 ms


def _calls():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    q8, k8v4, f16 = kv.KVCacheQ8(2, 128, 700), kv.KVCacheK8V4(2, 128, 700), kv.KVCacheF16(2, 128, 700)
    k, v = rand(700, 2, 128), rand(700, 2, 128)
    for c in (q8, k8v4, f16):
        c.append(k, v, 0)
    q, new, mask = rand(4, 8, 128), rand(4, 2, 128), torch.full((4,), 15, dtype=torch.int32, device="cuda")
    chunk, logits = rand(64, 8, 128).half(), rand(4, 5000)
    return {"q8": lambda s: kv.attn_verify_q8(q, q8, 700, 696, 0.09, stream=s),
            "tree": lambda s: kv.attn_verify_tree_q8(q, q8, 700, 696, mask, 0.09, stream=s),
            "k8v4": lambda s: kv.attn_verify_k8v4(q, k8v4, 700, 696, 0.09, stream=s),
            "f16": lambda s: kv.attn_verify_f16(q, f16, 700, 696, 0.09, stream=s),
            "append": lambda s: kv.attn_verify_append_q8(q, new, new, q8, 650, 0.09, stream=s),
            "prompt": lambda s: kv.attn_prompt_q8(chunk, q8, 700, 636, 0.09, stream=s),
            "prompt k8v4": lambda s: kv.attn_prompt_k8v4(chunk, k8v4, 700, 636, 0.09, stream=s),
            "prompt f16": lambda s: kv.attn_prompt_f16(chunk, f16, 700, 636, 0.09, stream=s),
            "argmax": lambda s: kv.argmax_rows_top_prob(logits, stream=s)[1]}


class _Other:
    """A stream of another library: an object with a handle."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


FORMS = {"stream": lambda s: s, "handle": lambda s: s.cuda_stream, "other": _Other}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("name", ["q8", "tree", "k8v4", "f16", "append", "prompt", "prompt k8v4", "prompt f16", "argmax"])
def test_memory_is_not_given_out_to_the_current_stream(lib, name, form, monkeypatch):
    from speculative_verify_attention_gb300 import binding
    call, side = _calls()[name], torch.cuda.Stream()
    want = call(None)
    taken, take = [], binding._scratch
    monkeypatch.setattr(binding, "_scratch", lambda *a: taken.append(take(*a)) or taken[-1])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    out = call(FORMS[form](side))
    at, size = {t.data_ptr() for t in taken} | {out.data_ptr()}, taken[0].numel()
    taken.clear()  # the call has returned and holds nothing
    assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() not in at
    side.synchronize()
    assert torch.equal(out, want)
