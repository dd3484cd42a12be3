"""The operators that a step of beam search, or of trees over images and text, needs around a paged Q8_0 cache, as cases to
be measured.

The queries and keys of the new tokens are rotated by positions of one or several axes, and the keys and values quantised into the
pages (kind "rope"); the best continuations of each request's beams are chosen (kind "select"); the penalties' token counts
("states") and the pages ("fork") follow the chosen beams; the accepted path of a drafted tree moves together ("compact").
With `own` false everything is computed in elementary torch operations; with `own` true the library's entry points are called.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one user's request with a few beams: where latency counts
        dict(name="select: one request of 4 beams", kind="select", seqs=1, beams=4, vocab=248320, dtype="f32", n_out=8,
             ended=False, weighted=False, masked=False),
        # a server's batch, lengths normalised, some beams at their end, twice as many candidates as beams
        dict(name="select: 48 requests of 8 beams", kind="select", seqs=48, beams=8, vocab=248320, dtype="bf16", n_out=16,
             ended=True, weighted=True, masked=False),
        # an odd vocabulary under grammars, requests with fewer beams among them
        dict(name="select: 21 requests of up to 5", kind="select", seqs=21, beams=5, vocab=106299, dtype="f16", n_out=5,
             ended=False, weighted=False, masked=True),
        # one request's counts follow its beams
        dict(name="states: one request of 4 beams", kind="states", seqs=1, beams=4, vocab=248320),
        # a server's batch under penalties
        dict(name="states: 48 requests of 8 beams", kind="states", seqs=48, beams=8, vocab=248320),
        # one request's pages follow its beams
        dict(name="fork: one request of 4 beams", kind="fork", seqs=1, beams=4, ctx=2048, page=16, hkv=4, hd=256),
        # long prompts that all beams share, many of them
        dict(name="fork: 64 requests of 8 beams", kind="fork", seqs=64, beams=8, ctx=8192, page=16, hkv=1, hd=256),
        # small trees of a few requests
        dict(name="compact: 4 trees of 8", kind="compact", seqs=4, rows=8, ctx=100, page=16, hkv=4, hd=256),
        # a large batch of wide trees
        dict(name="compact: 200 trees of 64", kind="compact", seqs=200, rows=64, ctx=150, page=64, hkv=8, hd=128),
        # windows of a few requests: one axis, halves rotated together
        dict(name="rope: 32 tokens", kind="rope", tokens=32, hq=24, hkv=4, hd=256, page=16, dtype="bf16", axes=1, rot=256,
             pairs=False, far=20676),
        # a prompt of text and images: time, height and width
        dict(name="rope: 16401 tokens, three axes", kind="rope", tokens=16401, hq=32, hkv=8, hd=128, page=64, dtype="bf16", axes=3,
             rot=128, pairs=False, far=32768),
        # fp32 activations, neighbours rotated together, half of the dims, positions far out
        dict(name="rope: 2051 tokens fp32, half", kind="rope", tokens=2051, hq=24, hkv=4, hd=256, page=32, dtype="f32", axes=2,
             rot=128, pairs=True, far=1000003),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["select", "select", "states", "fork", "compact", "rope", "rope"])
    if kind in ("select", "states"):
        vocab = rng.choice([248320, 106299, 32000 + rng.randint(0, 999), 1000 + rng.randint(0, 99)])
        beams = _log(rng, 1, 32) if kind == "select" else rng.randint(2, 16)
        seqs = _log(rng, 1, max(1, min(256, 90_000_000 // (vocab * beams), 4000 // beams)))
        if kind == "states":
            return dict(kind=kind, seqs=seqs, beams=beams, vocab=vocab)
        return dict(kind=kind, seqs=seqs, beams=beams, vocab=vocab, dtype=rng.choice(["f32", "f16", "bf16"]) if seqs * beams < 190
                    else rng.choice(["f16", "bf16"]), n_out=rng.choice([beams, beams, min(64, 2 * beams)]),
                    ended=rng.random() < 0.4, weighted=rng.random() < 0.4, masked=rng.random() < 0.4)
    if kind == "fork":
        hkv, hd = rng.choice([(4, 256), (8, 128), (1, 256), (2, 128)])
        ctx, beams = _log(rng, 20, 8192), rng.randint(2, 16)
        most = min(512 // beams, 280_000_000 / (hkv * hd * (2 * ctx + beams * (ctx // 4 + 400))))
        return dict(kind=kind, seqs=_log(rng, 1, max(1, int(most))), beams=beams, ctx=ctx, page=rng.choice([16, 32, 64, 128]), hkv=hkv,
                    hd=hd)
    if kind == "compact":
        hkv, hd = rng.choice([(4, 256), (8, 128), (1, 256), (2, 128)])
        return dict(kind=kind, seqs=_log(rng, 1, 190), rows=_log(rng, 2, 64), ctx=_log(rng, 1, 150), page=rng.choice([16, 32, 64]),
                    hkv=hkv, hd=hd)
    hq, hkv, hd = rng.choice([(24, 4, 256), (32, 8, 128), (12, 1, 256), (8, 2, 128), (16, 16, 128)])
    dtype = rng.choice(["f32", "f16", "bf16"])
    most = 16401 * 48 * 128 * 2 // ((hq + 2 * hkv) * hd * (4 if dtype == "f32" else 2))
    return dict(kind=kind, tokens=_log(rng, 1, most), hq=hq, hkv=hkv, hd=hd, page=rng.choice([16, 32, 64, 128]), dtype=dtype,
                axes=rng.randint(1, 4), rot=rng.choice([r for r in (64, 128, 192, 256) if r <= hd]), pairs=rng.random() < 0.5,
                far=_log(rng, 100, 1000003))


def _beams(case):
    """Beams of every request, the same for every seed: most have all of them, some fewer."""
    return [case["beams"] if b % 5 != 3 else max(1, case["beams"] - 1 - b % 3) for b in range(case["seqs"])]


def _parents(case):
    """The beam (of the whole batch) that each beam follows, the same for every seed: good ones several times, some never."""
    rng, beams, parents, first = np.random.default_rng(11), case["beams"], [], 0
    for b in range(case["seqs"]):
        of = np.floor(beams * rng.random(beams) ** 1.7).astype(int)
        if b % 9 == 8:
            of[beams - 1] = -first - 1  # a request that found fewer beams
        parents += (first + of).tolist()
        first += beams
    return np.array(parents, dtype=np.int32)


def _frac(b):
    return (0.37 + 0.6180339887498949 * b) % 1.0


def _lens(case):
    n, ctx = case["seqs"], case["ctx"]
    return [max(1, ctx if b == 0 else ctx // 4 + int((ctx - ctx // 4) * _frac(b))) for b in range(n)]


def _windows(case):
    """Rows of every tree, the same for every seed, and the words of its kept rows: a path from the root down."""
    rng, rows, words = np.random.default_rng(12), [], []
    for b in range(case["seqs"]):
        t = max(1, case["rows"] - (5 * b) % (case["rows"] // 2 + 1))
        word, at = 0, 0
        while at < t and b % 7 != 6:  # every seventh tree is rejected whole
            word |= 1 << at
            at += int(rng.integers(1, 5))
        rows.append(t)
        words.append(word)
    return rows, words


def work(case):
    kind = case["kind"]
    if kind == "select":
        beams = _beams(case)
        read = sum(n - (1 if case["ended"] and n > 2 else 0) for n in beams) * case["vocab"]
        return {"bytes": read * (4 if case["dtype"] == "f32" else 2) + 12 * sum(beams) + 12 * case["seqs"] * case["n_out"], "flops": 3 * read}
    if kind == "states":
        parents = _parents(case)
        of, times = np.unique(parents[parents >= 0], return_counts=True)
        rows = int((times - 1).sum() + (times > 1).sum())
        return {"bytes": 4 * rows * case["vocab"] + 12 * len(parents), "flops": 0}
    if kind == "fork":
        parents, lens, page = _parents(case), np.repeat(_lens(case), case["beams"]), case["page"]
        live = parents[parents >= 0]
        need = -(-lens // page)
        _, times = np.unique(live[lens[live] % page > 0], return_counts=True)
        copied = int((times - 1).sum()) * (page // 2) * case["hkv"] * (case["hd"] + case["hd"] // 16) * 2
        return {"bytes": 4 * int(need.sum() + need[live].sum()) + 2 * copied + 24 * len(parents), "flops": 0}
    if kind == "compact":
        _, words = _windows(case)
        moved = sum(bin(w & (w + 1)).count("1") for w in words)  # bits above the first gap
        return {"bytes": 2 * moved * case["hkv"] * 2 * (case["hd"] + case["hd"] // 16) + 24 * case["seqs"], "flops": 0}
    n, esz = case["tokens"], 4 if case["dtype"] == "f32" else 2
    kv = 2 * n * case["hkv"] * case["hd"]
    return {"bytes": 2 * n * case["hq"] * case["hd"] * esz + kv * esz + 2 * kv * 17 // 16 + kv * 2 + n * (8 + 4 * case["axes"]),
            "flops": 3 * n * (case["hq"] + case["hkv"]) * case["rot"] + 8 * kv}


# ---------------------------------------------------------------- inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(n):
    return _i32([0] + np.cumsum(n).tolist())


def _planes(pages, hkv, page, hd, gen):
    """Codes and scales of one plane as Q8_0 quantises values of about unit spread."""
    codes = torch.empty((pages, hkv, page, hd), dtype=torch.int8, device="cuda")
    for part in codes.split(max(1, (1 << 27) // (hkv * page * hd))):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(48.0).round_().clamp_(-127, 127))
    scales = torch.randn((pages, hkv, page, hd // 32), generator=gen, device="cuda").mul_(0.25).exp_().mul_(0.021)
    return codes, scales.half()


def _prepare_select(s, case, gen, rng):
    beams, v = _beams(case), case["vocab"]
    rows = sum(beams)
    x = torch.empty((rows, v), dtype=DTYPES[case["dtype"]], device="cuda")
    for part in x.split(64):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(3.0))
    if case["masked"]:  # every other row under a grammar that allows a third of the values
        for part in x[::2].split(64):
            part.masked_fill_(torch.rand(part.shape, generator=gen, device="cuda") < 0.67, -math.inf)
    s["logits"], s["starts"], s["most"] = x, _starts(beams), max(beams)
    s["scores"] = torch.rand(rows, generator=gen, device="cuda").mul_(-3.0).sub_(20.0)
    s["weights"] = torch.rand(rows, generator=gen, device="cuda").mul_(0.01).add_(0.05) if case["weighted"] else None
    s["ended"] = None
    if case["ended"]:  # one beam of each request of three or more
        ended, first = np.full(rows, -1, dtype=np.int32), 0
        for n in beams:
            if n > 2:
                ended[first + int(rng.integers(n))] = 2
            first += n
        s["ended"] = torch.from_numpy(ended).cuda()


def _prepare_states(s, case, gen, rng):
    n, v = case["seqs"] * case["beams"], case["vocab"]
    s["parents"] = torch.from_numpy(_parents(case)).cuda()
    s["counts"] = torch.zeros((n + 1, v), dtype=torch.int32, device="cuda")
    text = (torch.rand((n + 1, 2048), generator=gen, device="cuda").pow_(3.0) * v).long().clamp_(max=v - 1)
    s["counts"].scatter_add_(1, text, torch.ones_like(text, dtype=torch.int32))
    s["state_of"] = _i32(rng.permutation(n + 1)[:n].tolist())


def _prepare_fork(s, case, gen, rng):
    """Beams that share the pages of their prompt, and of what they have written the earlier ones more than the later ones."""
    beams, page = case["beams"], case["page"]
    lens = _lens(case)
    held = [-(-n // page) for n in lens]
    table = np.zeros((case["seqs"] * beams, max(held) + 1), dtype=np.int32)
    shares, used = [], 0
    for b, n in enumerate(held):
        prompt = max(0, n - 1 - lens[b] // (4 * page))
        for k in range(n):
            distinct = 1 if k < prompt else beams if k == n - 1 else 1 + (beams - 1) * (k - prompt) // max(1, n - 1 - prompt)
            of = np.arange(beams) * distinct // beams
            table[b * beams:(b + 1) * beams, k] = used + of
            shares += (np.bincount(of, minlength=distinct) - 1).tolist()
            used += distinct
    pages = used + case["seqs"] * beams + 3
    order = rng.permutation(pages).astype(np.int32)
    width = np.repeat(held, beams)[:, None]
    table = np.where(np.arange(table.shape[1]) < width, order[table], 0).astype(np.int32)
    all_shares = np.zeros(pages, dtype=np.int32)
    all_shares[order[:used]] = shares
    head = int(rng.integers(pages))
    ring = np.zeros(pages, dtype=np.int32)
    ring[(head + np.arange(pages - used)) % pages] = order[used:]
    s["parents"] = torch.from_numpy(_parents(case)).cuda()
    s["lens"], s["held"] = _i32(np.repeat(lens, beams).tolist()), _i32(np.repeat(held, beams).tolist())
    s["table"], s["shares"], s["ring"] = torch.from_numpy(table).cuda(), torch.from_numpy(all_shares).cuda(), torch.from_numpy(ring).cuda()
    s["ring_state"] = _i32([head, pages - used])
    s["next"] = torch.zeros_like(s["table"])
    s["k_codes"], s["k_scales"] = _planes(pages, case["hkv"], page, case["hd"], gen)
    s["v_codes"], s["v_scales"] = _planes(pages, case["hkv"], page, case["hd"], gen)


def _prepare_compact(s, case, gen, rng):
    rows, words = _windows(case)
    page = case["page"]
    lens = [n + t for n, t in zip(_lens(case), rows)]
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 3
    order = rng.permutation(pages)
    table = np.zeros((case["seqs"], max(held)), dtype=np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"], s["lens"], s["starts"], s["most"] = torch.from_numpy(table).cuda(), _i32(lens), _starts(rows), max(rows)
    s["kept"] = torch.from_numpy(np.array(words, dtype=np.uint64).view(np.int64)).cuda()
    s["k_codes"], s["k_scales"] = _planes(pages, case["hkv"], page, case["hd"], gen)
    s["v_codes"], s["v_scales"] = _planes(pages, case["hkv"], page, case["hd"], gen)


def _prepare_rope(s, case, gen, rng):
    n, hq, hkv, hd, axes, half = case["tokens"], case["hq"], case["hkv"], case["hd"], case["axes"], case["rot"] // 2
    dtype = DTYPES[case["dtype"]]
    s["q"] = torch.randn((n, hq, hd), generator=gen, device="cuda").to(dtype)
    k = torch.randn((n, hkv, hd), generator=gen, device="cuda")
    k[:, :, 5] *= 4.0  # an outlier channel, as keys have
    s["k"], s["v"] = k.to(dtype), torch.randn((n, hkv, hd), generator=gen, device="cuda").to(dtype)
    # a text's positions, and in every third stretch of 64 tokens an image's rows and columns
    first = int(rng.integers(max(1, case["far"] - n)))
    pos = np.tile(first + np.arange(n), (axes, 1))
    image = (np.arange(n) // 64) % 3 == 2
    for a in range(1, axes):
        pos[a, image] = first + (np.arange(n)[image] // (8 if a == 1 else 1)) % (8 * a)
    s["positions"] = _i32(pos.tolist())
    s["inv_freq"] = torch.from_numpy(10000.0 ** (-np.arange(half) / half)).cuda()
    s["axis_of"] = _i32((np.arange(half) * axes // half).tolist())  # sections of the dims, an axis each
    page = case["page"]
    pages = -(-n // page) + 1
    order, at = torch.from_numpy(rng.permutation(pages)), torch.arange(n)
    s["slots"] = (order[at // page] * page + at % page).cuda()
    s["k_codes"], s["k_scales"] = _planes(pages, hkv, page, hd, gen)
    s["v_codes"], s["v_scales"] = _planes(pages, hkv, page, hd, gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    {"select": _prepare_select, "states": _prepare_states, "fork": _prepare_fork, "compact": _prepare_compact,
     "rope": _prepare_rope}[case["kind"]](s, case, gen, np.random.default_rng(seed))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_calls if own else _plain)[s["case"]["kind"]](s)


def _planes_of(s):
    return {"k_codes": s["k_codes"], "v_codes": s["v_codes"], "k_scales": s["k_scales"].view(torch.int16),
            "v_scales": s["v_scales"].view(torch.int16)}  # moved, not computed: their bits


def _cache(s):
    """The cache's handle, as a program keeps it beside the planes."""
    import speculative_verify_attention_gb300 as kv
    if "cache" not in s:
        s["cache"] = kv.KVPagedCacheQ8.from_planes(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    return kv, s["cache"]


def _call_select(s):
    import speculative_verify_attention_gb300 as kv
    if "out" not in s:  # the program's buffers
        shape, (rows, vocab) = (s["case"]["seqs"], s["case"]["n_out"]), s["logits"].shape
        s["out"] = dict(parents=torch.empty(shape, dtype=torch.int32, device="cuda"),
                        tokens=torch.empty(shape, dtype=torch.int32, device="cuda"), totals=torch.empty(shape, device="cuda"))
        s["workspace"] = torch.empty(kv.beam_select_workspace_bytes(rows, vocab, shape[0], shape[1]), dtype=torch.uint8, device="cuda")
    kv.beam_select(s["logits"], s["starts"], s["case"]["n_out"], scores=s["scores"], weights=s["weights"], ended=s["ended"],
                   workspace=s["workspace"], **s["out"])
    return s["out"]


def _call_states(s):
    import speculative_verify_attention_gb300 as kv
    if "out" not in s:
        s["out"], s["status"] = torch.empty_like(s["parents"]), torch.empty(1, dtype=torch.int32, device="cuda")
        s["workspace"] = torch.empty(kv.token_counts_fork_workspace_bytes(len(s["parents"])), dtype=torch.uint8, device="cuda")
    kv.token_counts_fork(s["parents"], s["state_of"], s["counts"], s["out"], s["status"], workspace=s["workspace"])
    return {"counts": s["counts"], "state_of": s["out"], "status": s["status"]}


def _call_fork(s):
    kv, cache = _cache(s)
    if "out" not in s:
        new = torch.empty_like
        s["out"] = dict(page_table_out=s["next"], lens_out=new(s["parents"]), held_out=new(s["parents"]), shares_out=new(s["shares"]),
                        ring_out=new(s["ring_state"]), copy_src=new(s["parents"]), copy_dst=new(s["parents"]),
                        copy_rows=new(s["parents"]), status=torch.empty(1, dtype=torch.int32, device="cuda"))
        s["workspace"] = torch.empty(kv.kvq8_paged_fork_workspace_bytes(len(s["lens"]), len(s["parents"]), len(s["ring"])),
                                     dtype=torch.uint8, device="cuda")
    kv.kvq8_paged_fork(s["parents"], s["lens"], s["held"], s["case"]["page"], s["table"], s["shares"], s["ring"], s["ring_state"],
                       workspace=s["workspace"], **s["out"])
    kv.kvq8_paged_copy(cache, s["out"]["copy_src"], s["out"]["copy_dst"], s["out"]["copy_rows"])
    return {"ring": s["ring"], **s["out"], **_planes_of(s)}


def _call_compact(s):
    kv, cache = _cache(s)
    if "out" not in s:
        s["out"] = torch.empty_like(s["lens"])
    kv.kvq8_paged_compact(cache, s["table"], s["lens"], s["starts"], s["kept"], lens_out=s["out"])
    return {"lens_out": s["out"], **_planes_of(s)}


def _call_rope(s):
    kv, cache = _cache(s)
    if "out" not in s:
        s["turns"] = kv.rope_turns(s["inv_freq"])  # the table that a program keeps
        shape = (len(s["slots"]), cache.n_kv_heads, cache.head_dim)
        s["out"] = [torch.empty(shape, dtype=torch.float16, device="cuda") for _ in range(2)]
        s["q_out"] = torch.empty_like(s["q"])
    kv.kvq8_paged_append_rope(s["q"], s["k"], s["v"], cache, s["slots"], s["positions"], s["turns"], axis_of=s["axis_of"],
                              pairs=s["case"]["pairs"], q_out=s["q_out"])
    kv.kvq8_paged_read(cache, s["slots"], *s["out"])
    return [s["q_out"]] + s["out"]


_calls = {"select": _call_select, "states": _call_states, "fork": _call_fork, "compact": _call_compact, "rope": _call_rope}


# ---------------------------------------------------------------- plain forms

def _rows(starts, most):
    """[requests][most]: the row of each place of a request, and whether there is one."""
    place = torch.arange(most, device="cuda")
    first = starts[:-1].long().unsqueeze(1)
    return first + place, place < starts[1:].long().unsqueeze(1) - first


def _plain_select(s):
    x, n_out = s["logits"].float() + 0.0, s["case"]["n_out"]  # + 0: no -0
    rows, vocab = x.shape
    # the first n_out of a row, in order of value and then of place: unique keys of 64 bits
    bits = x.view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7fffffff)).long()
    key = key.mul_(1 << 32).add_(vocab - 1 - torch.arange(vocab, device="cuda"))
    token = vocab - 1 - (key.topk(min(n_out, vocab), 1)[0] & 0xffffffff)
    value = x.gather(1, token).double()
    top = x.amax(1, keepdim=True).double()  # sums and totals in 64 bits: candidates of two beams may be next to one another
    norm = (x.double() - top).exp_().sum(1, keepdim=True).log_() + top
    total = s["scores"].double().unsqueeze(1) + (value - norm)
    if s["ended"] is not None:  # a beam at its end goes on as it is
        done, first = (s["ended"] >= 0).unsqueeze(1), torch.arange(token.shape[1], device="cuda") == 0
        total = torch.where(done, torch.where(first, s["scores"].double().unsqueeze(1), -math.inf), total)
        token = torch.where(done, s["ended"].long().unsqueeze(1), token)
    order = total if s["weights"] is None else total * s["weights"].double().unsqueeze(1)
    order = torch.where(total > -math.inf, order, -math.inf)
    of, there = _rows(s["starts"], s["most"])
    of = of.clamp(max=rows - 1)
    order = torch.where(there.unsqueeze(2), order[of], -math.inf).flatten(1)
    if order.shape[1] < n_out:
        order = torch.cat([order, torch.full((len(order), n_out - order.shape[1]), -math.inf, dtype=order.dtype, device="cuda")], 1)
    best, at = order.sort(dim=1, descending=True, stable=True)
    best, at = best[:, :n_out], at[:, :n_out].clamp(max=of.shape[1] * token.shape[1] - 1)
    parent = of.gather(1, at // token.shape[1])
    got = best > -math.inf
    flat = parent * token.shape[1] + at % token.shape[1]
    return {"parents": torch.where(got, parent, -1).int(), "tokens": torch.where(got, token.flatten()[flat], -1).int(),
            "totals": torch.where(got, total.flatten()[flat], -math.inf).float()}


def _families(parents, n):
    """Of each beam whether it lives, its parent (0 where it has none) and whether it is the first child; children of each parent."""
    live, of = parents >= 0, parents.long().clamp(min=0)
    i = torch.arange(len(parents), device="cuda")
    first = torch.full((n,), len(parents), device="cuda").scatter_reduce_(0, of, torch.where(live, i, len(parents)), "amin")
    return live, of, live & (first[of] == i), torch.zeros(n, dtype=torch.long, device="cuda").scatter_add_(0, of, live.long())


def _plain_states(s):
    state, counts = s["state_of"].long(), s["counts"]
    live, of, first, children = _families(s["parents"], len(state))
    taken = torch.zeros(len(counts), dtype=torch.long, device="cuda").scatter_add_(0, state, (children > 0).long())
    copied = live & ~first
    # the rows that nothing is kept in, ascending, go to the beams that are not their parent's first
    free = (taken > 0).int().sort(stable=True)[1]
    to = torch.where(copied, free[(copied.long().cumsum(0) - 1).clamp(min=0)], torch.where(live, state[of], -1))
    counts[to[copied]] = counts[state[of][copied]]
    return {"counts": counts, "state_of": to.int(), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _plain_fork(s):
    lens, held, table, page, ring = s["lens"].long(), s["held"].long(), s["table"], s["case"]["page"], s["ring"]
    head, count = s["ring_state"].long()
    pages, n = len(ring), len(lens)
    live, of, first, children = _families(s["parents"], n)
    full, part, p = lens // page, lens % page, torch.arange(table.shape[1], device="cuda")
    tail = table.gather(1, full.clamp(max=table.shape[1] - 1).unsqueeze(1)).squeeze(1)
    keep = (part > 0) & (s["shares"][tail.long()] == 0) & (children > 0)  # the first child goes on in its parent's last page
    takes = live & (part[of] > 0) & ~(first & keep[of])
    fresh = ring[(head + takes.long().cumsum(0) - 1) % pages]
    need = torch.where(live, (lens + page - 1)[of] // page, 0)
    at_tail = takes.unsqueeze(1) & (p == full[of].unsqueeze(1))
    new = torch.where(at_tail, fresh.unsqueeze(1), table[of])
    new = torch.where(p < need.unsqueeze(1), new, s["next"])
    s["next"].copy_(new)
    holders = torch.where(p < full.unsqueeze(1), children.unsqueeze(1), ((p == full.unsqueeze(1)) & keep.unsqueeze(1)).long())
    change = torch.where(p < held.unsqueeze(1), holders - 1, 0)
    shares = s["shares"].long().scatter_add(0, table.flatten().long(), change.flatten())
    freed = shares < 0
    place = torch.where(freed, (head + count + freed.long().cumsum(0) - 1) % pages, pages)
    ring.copy_(torch.cat([ring, ring[:1]]).scatter(0, place, torch.arange(pages, dtype=torch.int32, device="cuda"))[:pages])
    src, dst = tail[of[takes]].long(), fresh[takes].long()
    inside = (torch.arange(page, device="cuda") < part[of][takes].unsqueeze(1)).view(-1, 1, page, 1)
    for plane in (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]):
        plane[dst] = torch.where(inside, plane[src], plane[dst])
    return {"ring": ring, "page_table_out": s["next"], "lens_out": torch.where(live, lens[of], 0).int(), "held_out": need.int(),
            "shares_out": shares.clamp(min=0).int(), "ring_out": torch.stack([(head + takes.sum()) % pages,
                                                                              count - takes.sum() + freed.sum()]).int(),
            "copy_src": torch.where(takes, tail[of], -1).int(), "copy_dst": torch.where(takes, fresh, -1).int(),
            "copy_rows": torch.where(takes, part[of], 0).int(), "status": torch.zeros(1, dtype=torch.int32, device="cuda"),
            **_planes_of(s)}


def _plain_compact(s):
    table, lens, page = s["table"].long(), s["lens"].long(), s["case"]["page"]
    rows = (s["starts"][1:] - s["starts"][:-1]).long().unsqueeze(1)
    j = torch.arange(s["most"], device="cuda")
    kept = ((s["kept"].unsqueeze(1) >> j) & 1).bool() & (j < rows)
    to = kept.long().cumsum(1) - 1
    moved = kept & (to < j)
    first = lens.unsqueeze(1) - rows
    a, b = (first + j).clamp(min=0), (first + to).clamp(min=0)
    most = table.shape[1] - 1
    src, dst = (table.gather(1, (x // page).clamp(max=most))[moved] for x in (a, b))
    at, off = (a % page)[moved], (b % page)[moved]
    for plane in (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]):
        plane[dst, :, off] = plane[src, :, at]
    return {"lens_out": (lens - rows.squeeze(1) + kept.sum(1)).int(), **_planes_of(s)}


def _quantised(x):
    x = x.unflatten(-1, (-1, 32))
    d = x.abs().amax(-1, keepdim=True) / 127.0
    y = torch.where(d == 0, 0.0, x / d)
    a = y.abs()
    whole = a.floor()
    code = ((whole + (a - whole >= 0.5)).clamp(max=127.0) * y.sign()).flatten(-2)  # ties away from zero
    return code.to(torch.int8), d.squeeze(-1).half()


def _rotated(x, cos, sin, pairs):
    x, rot = x.float(), 2 * cos.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    c, d = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([c, d], -1).flatten(-2) if pairs else torch.cat([c, d], -1), x[..., rot:]], -1)


def _plain_rope(s):
    page, slots, pairs = s["case"]["page"], s["slots"], s["case"]["pairs"]
    angle = s["positions"].double()[s["axis_of"].long()].T * s["inv_freq"]  # in 64 bits: positions far out are many turns
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    at, off = slots // page, slots % page
    s["k_codes"][at, :, off], s["k_scales"][at, :, off] = _quantised(_rotated(s["k"], cos, sin, pairs))
    s["v_codes"][at, :, off], s["v_scales"][at, :, off] = _quantised(s["v"].float())
    k = s["k_codes"][at, :, off].float().unflatten(-1, (-1, 32)) * s["k_scales"][at, :, off].float().unsqueeze(-1)
    v = s["v_codes"][at, :, off].float().unflatten(-1, (-1, 32)) * s["v_scales"][at, :, off].float().unsqueeze(-1)
    return [_rotated(s["q"], cos, sin, pairs).to(s["q"].dtype), k.flatten(-2).half(), v.flatten(-2).half()]


_plain = {"select": _plain_select, "states": _plain_states, "fork": _plain_fork, "compact": _plain_compact, "rope": _plain_rope}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    if case["kind"] not in ("select", "rope"):
        return None  # nothing but moved bits and whole numbers
    s = prepare(case, seed)
    return _exact_select(s) if case["kind"] == "select" else _exact_rope(s)


def _exact_select(s):
    """Request by request: every continuation's total, the largest n_out of them in their order."""
    starts, n_out = s["starts"].tolist(), s["case"]["n_out"]
    ended = [-1] * starts[-1] if s["ended"] is None else s["ended"].tolist()
    out = torch.full((len(starts) - 1, n_out), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(len(starts) - 1):
        totals, orders = [], []
        for r in range(starts[b], starts[b + 1]):
            if ended[r] >= 0:
                t = s["scores"][r:r + 1].double()
            else:
                x = s["logits"][r].double()
                t = (torch.log_softmax(x, 0) + s["scores"][r].double()).topk(min(n_out, len(x)))[0]
            totals.append(t)
            orders.append(t if s["weights"] is None else t * s["weights"][r].double())
        totals, orders = torch.cat(totals), torch.cat(orders)
        best = orders.argsort(descending=True)[:n_out]
        out[b, :len(best)] = totals[best]
    return {"parents": None, "tokens": None, "totals": out}


def _exact_rope(s):
    """Each rotated pair as a complex product; the format's step and the number that is rounded are 32-bit quotients."""
    case, rot = s["case"], s["case"]["rot"]
    pos = torch.stack([s["positions"][a] for a in s["axis_of"].tolist()], 1).double()
    turn = torch.polar(torch.ones_like(pos), pos * s["inv_freq"]).unsqueeze(1)

    def turned(x):
        x = x.double().clone()
        re, im = (slice(0, rot, 2), slice(1, rot, 2)) if case["pairs"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * turn
        x[..., re], x[..., im] = z.real, z.imag
        return x

    def held(x):
        blocks = x.reshape(*x.shape[:2], -1, 32)
        step = (blocks.abs().amax(3).float() / 127.0).double()
        ratio = (blocks / step.unsqueeze(3)).float().double()
        code = torch.where(step.unsqueeze(3) > 0, torch.trunc(ratio + 0.5 * ratio.sign()), 0.0).clamp(-127, 127)
        return (code * step.half().double().unsqueeze(3)).reshape(x.shape)

    return [turned(s["q"]), held(turned(s["k"])), held(s["v"].double())]
