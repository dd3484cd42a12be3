"""What the binding refuses of tensors on the GPU, by name, for the calls around beams, trees and rotary positions."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
I32, I64 = torch.int32, torch.int64


def _z(*shape, dtype=I32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _sets():
    import speculative_verify_attention_gb300 as kv
    cache = kv.KVPagedCacheQ8(2, 128, 16, 9)
    x = lambda h: _z(4, h, 128, dtype=torch.float16)  # noqa: E731
    return [
        (kv.beam_select, dict(logits=_z(4, 50, dtype=torch.float32), row_starts=_z(3), n_out=5, scores=_z(4, dtype=torch.float32),
                              weights=_z(4, dtype=torch.float32), ended=_z(4), parents=_z(2, 5), tokens=_z(2, 5), totals=_z(2, 5, dtype=torch.float32),
                              workspace=_z(1 << 16, dtype=torch.uint8))),
        (kv.token_counts_fork, dict(parents=_z(4) - 1, state_of=_z(3), counts=_z(6, 20), state_of_out=_z(4), status=_z(1), workspace=_z(256, dtype=torch.uint8))),
        (kv.kvq8_paged_fork, dict(parents=_z(4) - 1, lens=_z(3), held=_z(3), page_size=16, page_table=_z(3, 5), shares=_z(9), free_ring=_z(9),
                                  ring_state=_z(2), page_table_out=_z(4, 5), lens_out=_z(4), held_out=_z(4), copy_src=_z(4), copy_dst=_z(4),
                                  copy_rows=_z(4), status=_z(1), shares_out=_z(9), ring_out=_z(2), workspace=_z(4096, dtype=torch.uint8))),
        (kv.kvq8_paged_copy, dict(cache=cache, src_pages=_z(4) - 1, dst_pages=_z(4) - 1, rows=_z(4))),
        (kv.kvq8_paged_compact, dict(cache=cache, page_table=_z(3, 5), lens=_z(3), row_starts=_z(4), kept=_z(3, dtype=I64), lens_out=_z(3))),
        (kv.kvq8_paged_append_rope, dict(q=x(4), k=x(2), v=x(2), cache=cache, slots=_z(4, dtype=I64) - 1, positions=_z(2, 4), turns=_z(64, dtype=I64),
                                         axis_of=_z(64), q_out=x(4)))]


def test_calls_take_what_they_document_and_name_what_they_do_not(lib):
    import speculative_verify_attention_gb300 as kv
    for call, args in _sets():
        call(**args)
        for name, t in args.items():
            if not isinstance(t, torch.Tensor):
                continue
            wrong = [t.cpu(), t.to_sparse()]
            if name != "workspace":
                wrong += [t.double(), t[None]]
                if t.shape[-1] > 1 and name not in ("logits", "row_starts", "state_of"):
                    wrong += [t[..., :-1]]
            if t.numel() > 1 and t.dim() > 1 and name not in ("logits",):
                wrong += [t.transpose(0, 1).contiguous().transpose(0, 1)]
            for bad in wrong:
                with pytest.raises((ValueError, kv.KVQ8Error, RuntimeError)):
                    call(**{**args, name: bad})
    torch.cuda.synchronize()


def test_outputs_and_workspaces_that_are_left_out(lib):
    import speculative_verify_attention_gb300 as kv
    got = kv.beam_select(torch.randn((4, 50), device="cuda"), torch.tensor([0, 4], dtype=I32, device="cuda"), 5)
    assert [t.shape for t in got] == [(1, 5)] * 3 and [t.dtype for t in got] == [I32, I32, torch.float32]
    assert kv.beam_select(torch.randn((4, 50), device="cuda"), _z(1), 5)[0].shape == (0, 5)
    for call, args in _sets()[1:3]:
        call(**{k: v for k, v in args.items() if k not in ("workspace", "shares_out", "ring_out")})
    q = torch.randn((3, 4, 128), device="cuda")
    cache = kv.KVPagedCacheQ8(2, 128, 16, 9)
    out = kv.kvq8_paged_append_rope(q, q[:, :2], q[:, 2:], cache, torch.arange(3, device="cuda"), _z(3), _z(32, dtype=I64), pairs=True)
    assert torch.equal(out, q)
    torch.cuda.synchronize()


@pytest.mark.parametrize("but", [dict(logits=(4, 5, 10)), dict(logits=(50,)), dict(logits=()), dict(row_starts=(1, 3)), dict(row_starts=(0,)), dict(row_starts=()),
                                 dict(n_out=-3)])
@pytest.mark.parametrize("with_outputs", [False, True])
def test_select_names_sizes_that_it_does_not_take(lib, but, with_outputs):
    """Of wrong rank, empty, or fewer than nothing wanted: the binding's own error, whether it makes the outputs or is given them."""
    import speculative_verify_attention_gb300 as kv
    args = dict(logits=_z(4, 50, dtype=torch.float32), row_starts=_z(3), n_out=5)
    args.update({k: _z(*v, dtype=args[k].dtype) if isinstance(v, tuple) else v for k, v in but.items()})
    if with_outputs:
        args.update(parents=_z(2, 5), tokens=_z(2, 5), totals=_z(2, 5, dtype=torch.float32), workspace=_z(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        kv.beam_select(**args)
