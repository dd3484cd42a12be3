"""The calls of a beam-search step one after another over two layers' caches: tables, rotary append, attention, penalties, choice of
the beams, their counts and pages, copies.  Eager, and as two captured steps that hand the tables to and fro."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ._beams import check_selection, fork_counts, fork_pages  # noqa: E402
from ._paged import Batch, i32, starts_of, tables  # noqa: E402

pytestmark = pytest.mark.gpu
HQ, HKV, HD, PAGE, PAGES, WIDTH, VOCAB = 8, 2, 128, 16, 90, 8, 2003


class Beams:
    """Two requests of four beams: what a program keeps on the device, and what the host expects of it."""

    def __init__(self, n, children):
        import speculative_verify_attention_gb300 as kv
        self.kv, self.m = kv, children
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.caches = [kv.KVPagedCacheQ8(HKV, HD, PAGE, PAGES) for _ in range(2)]
        self.ring, self.state, self.shares = i32(np.arange(PAGES)), i32([0, PAGES]), z(PAGES)
        self.counts = z(children + 1, VOCAB)
        self.turns = kv.rope_turns(torch.from_numpy(10000.0 ** (-np.arange(64) / 64)).cuda())
        self.pen = torch.tensor([[1.3, 0.2, 0.1]] * children, device="cuda")

    def buffers(self, n, m, rows, most):
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        f = lambda h: torch.zeros((rows, h, HD), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        b = dict(n=n, m=m, rows=rows, most=most, new=z(n), starts=z(n + 1), slots=torch.zeros(rows, dtype=torch.int64, device="cuda"),
                 pos=z(rows), status=z(3), q=f(HQ), k=f(HKV), v=f(HKV), turned=f(HQ), out=[f(HQ), f(HQ)],
                 logits=torch.zeros((n, VOCAB), device="cuda"), bent=torch.zeros((n, VOCAB), device="cuda"),
                 seq_starts=i32(np.arange(n + 1)), req_starts=i32([0, n // 2, n]), scores=torch.zeros(n, device="cuda"),
                 parents=z(2, m // 2), tokens=z(2, m // 2), totals=torch.zeros((2, m // 2), device="cuda"), kids=i32(np.arange(m + 1)),
                 src=z(m), dst=z(m), copied=z(m))
        return b

    def step(self, b, cur, nxt):
        """cur, nxt: (table, lens, held, state_of) of the sequences before and after."""
        kv, st = self.kv, b["status"]
        table, lens, held, state_of = cur
        lens.add_(b["new"])
        kv.kvq8_paged_tables(lens, b["new"], held, table, self.ring, self.state, PAGE, b["starts"], b["slots"], b["pos"], st[:1])
        for cache, out in zip(self.caches, b["out"]):
            kv.kvq8_paged_append_rope(b["q"], b["k"], b["v"], cache, b["slots"], b["pos"], self.turns, q_out=b["turned"])
            kv.attn_verify_paged_q8(b["turned"], cache, table, lens, b["starts"], b["most"], 1 / math.sqrt(HD), out=out)
        kv.logits_adjust(b["logits"], b["seq_starts"], penalties=self.pen[:b["n"]], counts=self.counts, state_of=state_of, out=b["bent"])
        kv.beam_select(b["bent"], b["req_starts"], b["m"] // 2, scores=b["scores"], parents=b["parents"], tokens=b["tokens"], totals=b["totals"])
        parents, tokens = b["parents"].view(-1), b["tokens"].view(-1)
        kv.token_counts_fork(parents, state_of, self.counts, nxt[3], st[1:2])
        kv.token_counts(tokens, b["kids"], self.counts, state_of=nxt[3])
        kv.kvq8_paged_fork(parents, lens, held, PAGE, table, self.shares, self.ring, self.state, nxt[0], nxt[1], nxt[2], b["src"], b["dst"],
                           b["copied"], st[2:])
        for cache in self.caches:
            kv.kvq8_paged_copy(cache, b["src"], b["dst"], b["copied"])


def _host(t):
    return t.cpu().numpy().copy()


@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_beams(lib, graph):
    rng = np.random.default_rng(5)
    n, m = 2, 8
    beams = Beams(n, m)
    sets = []
    for size in (n, m, m):
        sets.append((i32(np.full((size, WIDTH), -1)), i32([0] * size), i32([0] * size), i32(np.arange(size))))
    prompts = [21, 16]
    first, steady = beams.buffers(n, m, 40, 21), beams.buffers(m, m, 10, 1)
    first["new"].copy_(i32(prompts))
    steady["new"].fill_(1)
    runs = {}

    def fill(b):
        for name in ("q", "k", "v"):
            b[name].copy_(torch.from_numpy(rng.standard_normal(b[name].shape).astype(np.float32)))
        b["logits"].copy_(torch.from_numpy(3 * rng.standard_normal((b["n"], VOCAB)).astype(np.float32)))

    texts = [[[], []] for _ in range(n)]          # by sequence and layer: the bytes of every cached token
    cur, nxt = sets[0], sets[1]
    for step in range(34):
        b = first if step == 0 else steady
        fill(b)
        if step:
            steady["scores"].copy_((first if step == 1 else steady)["totals"].view(-1))
        before = dict(table=_host(cur[0]), lens=_host(cur[1]), held=_host(cur[2]), state_of=_host(cur[3]), ring=_host(beams.ring),
                      state=_host(beams.state), shares=_host(beams.shares), counts=_host(beams.counts), next=_host(nxt[0]))
        if graph and step > 2:
            key = step % 2
            if key not in runs:
                torch.cuda.synchronize()
                runs[key] = torch.cuda.CUDAGraph()
                with torch.cuda.graph(runs[key]):
                    beams.step(b, cur, nxt)
            runs[key].replay()
        else:
            beams.step(b, cur, nxt)
        torch.cuda.synchronize()
        assert b["status"].tolist() == [0, 0, 0]
        # tables, and the lengths that the host knows
        lens = before["lens"] + _host(b["new"])
        want = tables(lens, _host(b["new"]), before["held"], before["table"], before["ring"], before["state"], PAGE, b["rows"])
        table, ring, held, state = (np.asarray(x) for x in want[:4])
        assert np.array_equal(_host(cur[0]), table) and np.array_equal(_host(b["slots"]), want[5])
        # the choice, over the logits as adjusted
        scores = _host(b["scores"])
        check_selection(_host(b["bent"]), [0, b["n"] // 2, b["n"]], m // 2, (b["parents"], b["tokens"], b["totals"]), scores)
        parents = _host(b["parents"]).reshape(-1).tolist()
        # counts
        state_of, counts, status = fork_counts(parents, before["state_of"].tolist(), before["counts"])
        for row, v in zip(state_of, _host(b["tokens"]).reshape(-1)):
            counts[row, v] += 1
        assert status == 0 and np.array_equal(_host(nxt[3]), state_of) and np.array_equal(_host(beams.counts), counts)
        # pages
        want = fork_pages(parents, lens, held, PAGE, table, before["shares"], ring, state, before["next"])
        for g, w in zip((nxt[0], nxt[1], nxt[2], beams.shares, beams.ring, beams.state, b["src"], b["dst"], b["copied"]), want):
            assert np.array_equal(_host(g).reshape(-1), np.asarray(w).reshape(-1))
        # what every sequence holds is what it held, and what its tokens of this step were
        starts, slots = _host(b["starts"]), _host(b["slots"])
        planes = [[_host(p) for p in (c.k_codes, c.v_codes, c.k_scales.view(torch.int16), c.v_scales.view(torch.int16))] for c in beams.caches]
        for s in range(b["n"]):
            for layer in range(2):
                texts[s][layer] = texts[s][layer] + [[p[slots[r] // PAGE, :, slots[r] % PAGE].copy() for p in planes[layer]]
                                                     for r in range(starts[s], starts[s + 1])]
        ref = Batch.__new__(Batch)
        ref.hq, ref.hkv, ref.hd, ref.page, ref.lens, ref.n_new = HQ, HKV, HD, PAGE, lens.tolist(), _host(b["new"]).tolist()
        ref.scale, ref.dtype, ref.table, ref.starts, ref.words, ref.q = 1 / math.sqrt(HD), torch.bfloat16, table, starts, None, b["turned"].cpu()
        for layer in range(2):
            ref.codes, ref.scales = planes[layer][:2], [p.view(np.float16) for p in planes[layer][2:]]
            found = ref.expect(rows={int(starts[s + 1]) - 1 for s in range(b["n"])})
            got = b["out"][layer].double().cpu().numpy()
            assert all(np.all(np.abs(got[r, h] - o) <= off) for (r, h), (o, off) in found.items())
        texts = [[list(texts[q][layer]) for layer in range(2)] for q in parents]
        table, lens, held = (np.asarray(x) for x in want[:3])
        for s in range(m):
            assert lens[s] == len(texts[s][0])
            for layer in range(2):
                for pos, rows in enumerate(texts[s][layer]):
                    for p, row in zip(planes[layer], rows):
                        assert np.array_equal(p[table[s, pos // PAGE], :, pos % PAGE], row), (step, s, pos)
        cur, nxt = nxt, (sets[2] if cur is sets[0] else cur)
    # all end: every page comes home
    beams.kv.kvq8_paged_fork(i32([-1] * m), cur[1], cur[2], PAGE, cur[0], beams.shares, beams.ring, beams.state, nxt[0], nxt[1], nxt[2], steady["src"],
                             steady["dst"], steady["copied"], steady["status"][:1])
    state = beams.state.tolist()
    assert state[1] == PAGES and sorted(beams.ring.tolist()) == list(range(PAGES)) and int(beams.shares.sum()) == 0
    assert starts_of([1]).tolist() == [0, 1] and beams.kv.kvq8_device_error(reset=True) == 0


def test_a_tree_is_verified_and_its_path_kept(lib):
    """Append a tree, verify it under its masks, keep one path: attention over the compacted cache is the chain's."""
    import speculative_verify_attention_gb300 as kv
    from ._paged import masks64, tree_words
    rng = np.random.default_rng(6)
    ctx, t = [40, 7], [20, 33]
    words = [tree_words(x, rng) for x in t]
    path = [max(w, key=lambda v: bin(v).count("1")) for w in words]
    places = [[j for j in range(x) if p >> j & 1] for x, p in zip(t, path)]
    rows = sum(t)
    k, v, q = (torch.from_numpy(rng.standard_normal((sum(ctx) + rows, h, HD)).astype(np.float32)).cuda() for h in (HKV, HKV, HQ))
    lens = [c + x for c, x in zip(ctx, t)]
    table = i32(np.array([[5, 3, 9, 1, 0], [2, 8, 4, 6, 7]]))
    at = lambda b, p: int(table[b, p // PAGE]) * PAGE + p % PAGE  # noqa: E731
    slots = [at(b, p) for b in range(2) for p in range(ctx[b])] + [at(b, p) for b in range(2) for p in range(ctx[b], lens[b])]
    position = [p for b in range(2) for p in range(ctx[b])] + [ctx[b] + bin(w).count("1") - 1 for b in range(2) for w in words[b]]
    cache, turns = kv.KVPagedCacheQ8(HKV, HD, PAGE, 12), kv.rope_turns(torch.from_numpy(10000.0 ** (-np.arange(64) / 64)).cuda())
    turned = kv.kvq8_paged_append_rope(q, k, v, cache, torch.tensor(slots, device="cuda"), i32(position), turns)
    window, starts = turned[sum(ctx):].half().contiguous(), i32(starts_of(t))
    tree = kv.attn_verify_paged_q8(window, cache, table, i32(lens), starts, max(t), 0.1, window_mask=masks64(sum(words, [])))
    after = i32([0, 0])
    kv.kvq8_paged_compact(cache, table, i32(lens), starts, masks64(path), lens_out=after)
    assert after.tolist() == [c + len(p) for c, p in zip(ctx, places)]
    kept = [starts.tolist()[b] + j for b in range(2) for j in places[b]]
    chain = kv.attn_verify_paged_q8(window[kept].contiguous(), cache, table, after, i32(starts_of([len(p) for p in places])),
                                    max(len(p) for p in places), 0.1)
    # the same values, summed in another order: each within 4e-4 of the exact ones and half a step of fp16
    assert (chain.float() - tree[kept].float()).norm() <= 2 * 5e-4 * tree[kept].float().norm()
