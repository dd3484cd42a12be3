"""The calls of a step one after another, as a serving loop makes them: tables, append, verify, adjust, argmax, counts."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402

from ._paged import Batch, adjusted, i32, masks64, starts_of, tables, tree_words  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_a_batch(lib, graph):
    """Three requests over six steps (a prompt, windows of trees and chains, a rejection, an end), eagerly and as one
    captured step replayed with new lengths; every intermediate checked against the host's own bookkeeping."""
    import speculative_verify_attention_gb300 as kv
    rng = np.random.default_rng(1)
    hq, hkv, hd, page, pages, width, vocab, n, most = 8, 2, 128, 16, 24, 8, 3001, 3, 12
    rows = n * most
    cache = kv.KVPagedCacheQ8(hkv, hd, page, pages)
    dev = dict(lens=i32([0] * n), new=i32([0] * n), held=i32([0] * n), table=i32(np.zeros((n, width))), ring=i32(np.arange(pages)),
               state=i32([0, pages]), starts=i32([0] * (n + 1)), status=i32([0]), pos=i32([0] * rows),
               slots=torch.zeros(rows, dtype=torch.int64, device="cuda"), mask=torch.zeros(rows, dtype=torch.int64, device="cuda"),
               k=torch.zeros((rows, hkv, hd), dtype=torch.bfloat16, device="cuda"),
               v=torch.zeros((rows, hkv, hd), dtype=torch.bfloat16, device="cuda"),
               q=torch.zeros((rows, hq, hd), dtype=torch.bfloat16, device="cuda"),
               out=torch.zeros((rows, hq, hd), dtype=torch.bfloat16, device="cuda"),
               logits=torch.zeros((rows, vocab), device="cuda"), bent=torch.zeros((rows, vocab), device="cuda"),
               counts=i32(np.zeros((n, vocab))), tokens=i32([0] * rows), accepted=i32([0] * rows), accepted_starts=i32([0] * (n + 1)),
               pen=torch.tensor([[1.2, 0.3, 0.1]] * n, device="cuda"),
               ws=torch.empty(max(16, kv.attn_verify_paged_q8_workspace_bytes(hq, hkv, hd, most)), dtype=torch.uint8, device="cuda"))
    scale = 1 / math.sqrt(hd)

    def step():
        d = dev
        kv.kvq8_paged_tables(d["lens"], d["new"], d["held"], d["table"], d["ring"], d["state"], page, d["starts"], d["slots"],
                             d["pos"], d["status"])
        kv.kvq8_paged_append(d["k"], d["v"], cache, d["slots"])
        kv.attn_verify_paged_q8(d["q"], cache, d["table"], d["lens"], d["starts"], most, scale, window_mask=d["mask"],
                                out=d["out"], workspace=d["ws"])
        kv.logits_adjust(d["logits"], d["starts"], penalties=d["pen"], counts=d["counts"], window_tokens=d["tokens"],
                         window_mask=d["mask"], out=d["bent"])
        kv.token_counts(d["accepted"], d["accepted_starts"], d["counts"])

    if graph:
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    else:
        run = step

    held, table, ring, state = np.zeros(n, int), np.zeros((n, width), np.int32), np.arange(pages, dtype=np.int32), np.array([0, pages])
    texts = [[] for _ in range(n)]           # the (k, v) of every cached token, by position
    counts = np.zeros((n, vocab), np.int32)
    for new, keep in (([12, 3, 0], [12, 1, 0]), ([4, 4, 12], [2, 4, 12]), ([8, 1, 5], [0, 1, 5]), ([8, 7, 0], [8, 2, 0]),
                      ([12, 12, 12], [12, 3, 12]), ([1, 0, 9], [1, 0, 9])):
        new = np.array(new)
        if new[1] == 0:
            texts[1] = []                    # request 1 ends
        lens = np.array([len(t) for t in texts]) + new
        total = int(new.sum())
        k, v = (rng.standard_normal((rows, hkv, hd)).astype(np.float32) for _ in range(2))
        q, logits = rng.standard_normal((rows, hq, hd)).astype(np.float32), rng.standard_normal((rows, vocab)).astype(np.float32)
        words = sum((tree_words(int(x), rng) for x in new), []) + [0] * (rows - total)
        tokens = rng.integers(0, vocab, rows).astype(np.int32)
        acc = [rng.integers(0, vocab, x) for x in keep]
        acc_flat = np.zeros(rows, np.int32)
        acc_flat[:sum(keep)] = np.concatenate(acc)
        for name, x in (("lens", lens), ("new", new), ("tokens", tokens), ("accepted", acc_flat), ("accepted_starts", starts_of(keep))):
            dev[name].copy_(i32(x))
        dev["mask"].copy_(masks64(words))
        for name, x in (("k", k), ("v", v), ("q", q), ("logits", logits)):
            dev[name].copy_(torch.from_numpy(x))
        dev["out"].fill_(77.0)
        dev["bent"].fill_(55.0)
        run()
        torch.cuda.synchronize()

        want = tables(lens, new, held, table, ring, state, page, rows)
        for name, w in zip(("table", "ring", "held", "state", "starts", "slots", "pos", "status"), want):
            assert np.array_equal(dev[name].cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
        table, ring, held, state, starts, slots = want[:6]
        kb, vb = dev["k"].float().cpu().numpy(), dev["v"].float().cpu().numpy()
        for b in range(n):
            texts[b] += [(kb[r], vb[r]) for r in range(starts[b], starts[b + 1])]
        # the host's cache, quantised by the oracle
        ref = Batch.__new__(Batch)
        ref.hq, ref.hkv, ref.hd, ref.page, ref.lens, ref.n_new = hq, hkv, hd, page, lens.tolist(), new.tolist()
        ref.scale, ref.dtype, ref.table, ref.starts, ref.words, ref.q = scale, torch.bfloat16, table, starts, words, dev["q"].cpu()
        ref.codes = [np.zeros((pages, hkv, page, hd), np.int8) for _ in range(2)]
        ref.scales = [np.zeros((pages, hkv, page, hd // 32), np.float16) for _ in range(2)]
        for b in range(n):
            if not texts[b]:
                continue
            orc = oracle.Cache(hkv, hd, len(texts[b]))
            orc.append(np.stack([x for x, _ in texts[b]]), np.stack([y for _, y in texts[b]]), 0)
            p = np.arange(len(texts[b]))
            for i, (c, s) in enumerate(((orc.k_codes, orc.k_scales), (orc.v_codes, orc.v_scales))):
                ref.codes[i][table[b, p // page], :, p % page] = c.transpose(1, 0, 2)
                ref.scales[i][table[b, p // page], :, p % page] = s.view(np.float16).transpose(1, 0, 2)
        ref.check(dev["out"])
        x, off = adjusted(torch.from_numpy(logits), starts, np.array([[1.2, 0.3, 0.1]] * n, np.float32), counts, None, tokens, words)
        got = dev["bent"].double().cpu().numpy()
        assert np.all(np.abs(got - x)[:total] <= off[:total]) and np.all(got[total:] == 55.0)
        for b in range(n):
            np.add.at(counts[b], acc[b], 1)
        assert np.array_equal(dev["counts"].cpu().numpy(), counts)
        for b in range(n):                   # rejected tokens leave the text
            texts[b] = texts[b][:len(texts[b]) - int(new[b]) + min(int(new[b]), keep[b])]
    assert kv.kvq8_device_error(reset=True) == 0
