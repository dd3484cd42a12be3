"""logits_adjust with the output in its input's memory: in place, one call after another, and in rows that lie between the
input's."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from .test_gpu_logits_adjust import _call, _case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [4096, 4099, 248320])
def test_calls_in_place_one_after_another(lib, vocab):
    """Each launched while the one before ends, and reading what it wrote: the same bits as by separate buffers."""
    c = _case(41, [3, 12, 6], vocab, tree=True)
    x = c["logits"].cuda()
    want = [_call(c)]
    for _ in range(3):
        want.append(_call(c, logits=want[-1]))
    for _ in range(5):
        y = x.clone()
        for _ in range(4):
            _call(c, logits=y, out=y)
        assert torch.equal(y, want[3])
    assert np.isfinite(want[3].cpu().numpy()).any()


def test_calls_in_place_in_a_graph(lib):
    from speculative_verify_attention_gb300 import logits_adjust
    from ._paged import i32
    x, starts = torch.randn((40, 8192), device="cuda"), i32([0, 7, 40])
    tokens = torch.arange(8192, dtype=torch.int32, device="cuda").repeat(2)
    values = torch.randn(2 * 8192, device="cuda")
    bias = dict(bias_starts=i32([0, 8192, 2 * 8192]), bias_tokens=tokens, bias_values=values)
    want = x.clone()
    for _ in range(6):
        want[:7] += values[:8192]
        want[7:] += values[8192:]
    y = x.clone()
    logits_adjust(y, starts, out=y, **bias)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(6):
            logits_adjust(y, starts, out=y, **bias)
    y.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [4096, 4099])
def test_rows_between_the_inputs_rows(lib, vocab, dtype):
    """Output rows in the gaps of the input's are no overlap."""
    c = _case(42, [3, 12, 6], vocab, dtype, tree=True)
    rows, want = len(c["logits"]), _call(c)
    wide = torch.zeros((rows, 2 * vocab), device="cuda")
    x = wide[:, vocab:].view(dtype)[:, :vocab] if dtype != torch.float32 else wide[:, vocab:]
    x.copy_(c["logits"].cuda())
    _call(c, logits=x, out=wide[:, :vocab].fill_(55.0))
    assert torch.equal(wide[:, :vocab], want) and torch.equal(x, c["logits"].cuda())
