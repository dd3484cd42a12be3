"""The operators of a batched speculative-verify step over a paged Q8_0 cache, as cases to be measured.

A step of a program that serves many requests: the block tables and slots of the new tokens
(kind "tables"), their keys and values quantised into the pages ("cache"), the windows verified over
the pages ("verify"), the logits bent by penalties, biases and grammars ("adjust"), and the token
counts that the penalties read ("counts").  With `own` false everything is computed in elementary
torch operations; with `own` true the library's entry points are called.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PROMPT_BIT = -(1 << 31)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one request with a chain of four drafted tokens: where latency counts
        dict(name="verify: one chain of 4", kind="verify", seqs=1, rows=4, tree=False, ctx=2048, hq=24, hkv=4, hd=256,
             page=16, dtype="bf16"),
        # a batch of long chats, odd windows of up to five tokens
        dict(name="verify: 8 long chains", kind="verify", seqs=8, rows=5, tree=False, ctx=32768, hq=24, hkv=4, hd=256,
             page=64, dtype="f16"),
        # trees of up to 32 drafted tokens: many rows share each key
        dict(name="verify: 16 trees of 32", kind="verify", seqs=16, rows=32, tree=True, ctx=20676, hq=24, hkv=4, hd=256,
             page=32, dtype="bf16"),
        # plain decoding, one token a request
        dict(name="verify: 64 single tokens", kind="verify", seqs=64, rows=1, tree=False, ctx=8192, hq=32, hkv=8, hd=128,
             page=16, dtype="bf16"),
        # the tables of a small batch's step
        dict(name="tables: 4 requests", kind="tables", seqs=4, rows=4, ctx=4096, page=16, prompts=0, gone=0),
        # a large server's step: prompts enter, requests end, the rest take a few tokens each
        dict(name="tables: 1024 requests", kind="tables", seqs=1024, rows=8, ctx=8192, page=16, prompts=5, gone=31),
        # eight windows of four tokens enter the cache
        dict(name="cache: 32 tokens", kind="cache", tokens=32, hkv=4, hd=256, page=16, dtype="bf16"),
        # long prompts enter the cache, and are read back for a prompt's attention
        dict(name="cache: 16401 tokens", kind="cache", tokens=16401, hkv=8, hd=128, page=64, dtype="f32"),
        # one request's window
        dict(name="adjust: one chain of 4", kind="adjust", seqs=1, rows=4, tree=False, vocab=248320, dtype="f32", bias=8),
        # trees under penalties, biases and, every other row, a grammar
        dict(name="adjust: 12 trees of 32", kind="adjust", seqs=12, rows=32, tree=True, vocab=248320, dtype="bf16",
             bias=300),
        # a few requests enter the batch, an odd vocabulary
        dict(name="counts: 3 prompts", kind="counts", seqs=3, tokens=2048, vocab=106299),
        # a batch is rebuilt from its requests' long texts
        dict(name="counts: 64 long texts", kind="counts", seqs=64, tokens=20676, vocab=248320),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["verify", "verify", "tables", "cache", "adjust", "counts"])
    if kind == "verify":
        hq, hkv, hd = rng.choice([(24, 4, 256), (32, 8, 128), (12, 1, 256), (8, 2, 128), (16, 16, 128)])
        ctx, rows = _log(rng, 1, 32768), _log(rng, 1, 64)
        # no more cache bytes and no more products than the largest listed cases have
        most = min(7.0e8 / ((ctx + rows) * hkv * hd * 2.125), 1.2e11 / (4.0 * (ctx + rows) * rows * hq * hd))
        return dict(kind=kind, seqs=_log(rng, 1, max(1, min(96, int(most)))), rows=rows, tree=rng.random() < 0.5, ctx=ctx,
                    hq=hq, hkv=hkv, hd=hd, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["f16", "bf16"]))
    if kind == "tables":
        seqs = _log(rng, 1, 1024)
        return dict(kind=kind, seqs=seqs, rows=_log(rng, 1, 16), ctx=_log(rng, 64, 8192), page=rng.choice([16, 32, 64]),
                    prompts=rng.randint(0, min(5, seqs // 2)), gone=rng.randint(0, min(31, seqs // 3)))
    if kind == "cache":
        hkv, hd = rng.choice([(4, 256), (8, 128), (1, 256), (2, 128)])
        return dict(kind=kind, tokens=_log(rng, 1, 16000), hkv=hkv, hd=hd, page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["f32", "f16", "bf16"]))
    if kind == "adjust":
        vocab, rows = rng.choice([248320, 106299, 32000 + rng.randint(0, 999), 1000 + rng.randint(0, 99)]), _log(rng, 1, 64)
        seqs = _log(rng, 1, max(1, min(64, 380 // rows)))
        return dict(kind=kind, seqs=seqs, rows=rows, tree=rng.random() < 0.5, vocab=vocab,
                    dtype=rng.choice(["f32", "f16", "bf16"]), bias=rng.choice([0, 1, 37, 300]))
    return dict(kind=kind, seqs=_log(rng, 1, 60), tokens=_log(rng, 1, 20000), vocab=rng.choice([248320, 106299, 32001]))


def _frac(b):
    return (0.37 + 0.6180339887498949 * b) % 1.0


def _windows(case):
    """(n_new, lens) of every request: the same for every seed, lengths spread over a fourfold range."""
    n, rows, ctx = case["seqs"], case["rows"], case.get("ctx", 0)
    n_new = [rows if b == 0 else max(1, rows - (5 * b) % (rows // 2 + 1)) for b in range(n)]
    lens = [n_new[b] + (ctx if n == 1 else ctx // 4 + int((ctx - ctx // 4) * _frac(b))) for b in range(n)]
    return n_new, lens


def _table_lens(case):
    """(n_new, lens, held): most requests take their window, some end, some bring a prompt."""
    n_new, lens = _windows(case)
    page = case["page"]
    held = [-(-(lens[b] - n_new[b]) // page) + (1 if b % 11 == 3 else 0) for b in range(case["seqs"])]
    for i in range(case["gone"]):  # ended requests give all their pages back
        lens[3 * i + 2] = n_new[3 * i + 2] = 0
    for i in range(case["prompts"]):  # a prompt enters: nothing held yet, all of its tokens new
        b = 2 * i if 2 * i < case["seqs"] else i
        if lens[b]:
            n_new[b], held[b] = lens[b], 0
    return n_new, lens, held


def _text_lens(case):
    n, t = case["seqs"], case["tokens"]
    return [t if b == 0 else max(1, t // 8 + int((t - t // 8) * _frac(b))) for b in range(n)]


def work(case):
    kind = case["kind"]
    if kind == "verify":
        n_new, lens = _windows(case)
        token = case["hkv"] * 2 * (case["hd"] + case["hd"] // 16)
        row = case["hq"] * case["hd"] * 2
        seen = sum((n - t) * t + t * (t + 1) // 2 for t, n in zip(n_new, lens))
        return {"bytes": sum(lens) * token + 2 * sum(n_new) * row, "flops": 4 * case["hd"] * case["hq"] * seen}
    if kind == "tables":
        n_new, lens, held = _table_lens(case)
        page = case["page"]
        moved = sum(abs(-(-n // page) - h) for n, h in zip(lens, held))
        return {"bytes": 20 * case["seqs"] + 12 * sum(n_new) + 8 * moved, "flops": 0}
    if kind == "cache":
        n = case["tokens"] * case["hkv"] * case["hd"]
        slots = _slots(case) * case["hkv"] * case["hd"]
        return {"bytes": 2 * n * (4 if case["dtype"] == "f32" else 2) + 2 * n * 17 // 16 + 2 * slots * 2, "flops": 8 * n}
    if kind == "adjust":
        n_new, _ = _windows(case)
        rows, v = sum(n_new), case["vocab"]
        return {"bytes": rows * v * ((4 if case["dtype"] == "f32" else 2) + 4) + case["seqs"] * v * 4 + rows // 2 * v // 8,
                "flops": 4 * rows * v}
    return {"bytes": 4 * sum(_text_lens(case)) + 4 * case["seqs"] * case["vocab"], "flops": 0}


# ---------------------------------------------------------------- inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(n):
    return _i32([0] + np.cumsum(n).tolist())


def _masks(case, n_new, rng):
    """One 64-bit word a row: itself and its ancestors in the window, node 0 the root."""
    words = []
    for n in n_new:
        seen = []
        for i in range(n):
            up = 0 if i == 0 else seen[int(rng.integers(max(0, i - 8), i))]
            seen.append(up | (1 << i))
        words += seen
    return torch.from_numpy(np.array(words, dtype=np.uint64).view(np.int64)).cuda()


def _planes(pages, hkv, page, hd, gen):
    """Codes and scales of one plane as Q8_0 quantises values of about unit spread."""
    codes = torch.empty((pages, hkv, page, hd), dtype=torch.int8, device="cuda")
    for part in codes.split(max(1, (1 << 27) // (hkv * page * hd))):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(48.0).round_().clamp_(-127, 127))
    scales = torch.randn((pages, hkv, page, hd // 32), generator=gen, device="cuda").mul_(0.25).exp_().mul_(0.021)
    return codes, scales.half()


def _slots(case):
    """Slots of the pool that a cache case writes into: whole pages, and one more."""
    return (-(-case["tokens"] // case["page"]) + 1) * case["page"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": case}
    kind = case["kind"]
    if kind == "verify":
        n_new, lens = _windows(case)
        page, hkv, hd = case["page"], case["hkv"], case["hd"]
        held = [-(-n // page) for n in lens]
        pages = sum(held) + 3
        order = rng.permutation(pages)
        table = np.zeros((case["seqs"], max(held)), dtype=np.int32)
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = order[at:at + n]
            at += n
        s["k_codes"], s["k_scales"] = _planes(pages, hkv, page, hd, gen)
        s["v_codes"], s["v_scales"] = _planes(pages, hkv, page, hd, gen)
        s["table"], s["lens"], s["starts"] = torch.from_numpy(table).cuda(), _i32(lens), _starts(n_new)
        s["n_rows"], s["max_rows"], s["scale"] = sum(n_new), max(n_new), 1.0 / math.sqrt(hd)
        s["q"] = torch.randn((s["n_rows"], case["hq"], hd), generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        s["mask"] = _masks(case, n_new, rng) if case["tree"] else None
    elif kind == "tables":
        n_new, lens, held = _table_lens(case)
        page = case["page"]
        need = [-(-n // page) for n in lens]
        width = max(max(need), max(held))
        spare = sum(max(0, n - h) for n, h in zip(need, held)) + 7
        pages = sum(held) + spare
        order = rng.permutation(pages).astype(np.int32)
        table = np.zeros((case["seqs"], width), dtype=np.int32)
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = order[at:at + n]
            at += n
        head = int(rng.integers(pages))
        ring = np.zeros(pages, dtype=np.int32)
        ring[(head + np.arange(spare)) % pages] = order[at:]
        s["lens"], s["n_new"], s["held"], s["table"] = _i32(lens), _i32(n_new), _i32(held), torch.from_numpy(table).cuda()
        s["ring"], s["ring_state"], s["n_rows"] = torch.from_numpy(ring).cuda(), _i32([head, spare]), sum(n_new) + 3
    elif kind == "cache":
        n, slots = case["tokens"], _slots(case)
        shape = (n, case["hkv"], case["hd"])
        s["k"] = torch.randn(shape, generator=gen, device="cuda")
        s["k"][:, :, 5] *= 8.0  # an outlier channel, as keys have
        s["k"] = s["k"].to(DTYPES[case["dtype"]])
        s["v"] = torch.randn(shape, generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        pages = slots // case["page"]
        order = torch.from_numpy(rng.permutation(pages))
        at = torch.arange(n)
        s["slots"] = (order[at // case["page"]] * case["page"] + at % case["page"]).cuda()
        s["every"] = torch.arange(slots, device="cuda")
        s["k_codes"], s["k_scales"] = _planes(pages, case["hkv"], case["page"], case["hd"], gen)
        s["v_codes"], s["v_scales"] = _planes(pages, case["hkv"], case["page"], case["hd"], gen)
    elif kind == "adjust":
        n_new, _ = _windows(case)
        n, v, rows = case["seqs"], case["vocab"], sum(n_new)
        s["logits"] = torch.randn((rows, v), generator=gen, device="cuda").mul_(3.0).to(DTYPES[case["dtype"]])
        s["starts"] = _starts(n_new)
        # a text of up to some thousand tokens has few of the vocabulary, low ids more often
        s["counts"] = torch.zeros((n + 2, v), dtype=torch.int32, device="cuda")
        text = (torch.rand((n + 2, 4096), generator=gen, device="cuda").pow_(3.0) * v).long().clamp_(max=v - 1)
        s["counts"].scatter_(1, text[:, :2048], PROMPT_BIT)
        s["counts"].scatter_add_(1, text[:, 2048:], torch.ones_like(text[:, 2048:], dtype=torch.int32))
        s["state_of"] = _i32(rng.permutation(n + 2)[:n].tolist())
        p = torch.rand((n, 3), generator=gen, device="cuda")
        s["penalties"] = p * torch.tensor([0.4, 0.8, 0.8], device="cuda") + torch.tensor([1.0, 0.0, 0.0], device="cuda")
        s["tokens"] = (torch.rand(rows, generator=gen, device="cuda").pow_(3.0) * v).int().clamp_(max=v - 1)
        s["mask"] = _masks(case, n_new, rng) if case["tree"] else None
        s["bias_starts"] = _starts([case["bias"]] * n)
        s["bias_tokens"] = torch.randint(0, v, (n * case["bias"],), generator=gen, device="cuda", dtype=torch.int32)
        s["bias_values"] = torch.randn(n * case["bias"], generator=gen, device="cuda").mul_(5.0)
        words = -(-v // 32)
        s["grammar"] = torch.randint(-(1 << 31), 1 << 31, (max(1, rows // 2), words), generator=gen, device="cuda",
                                     dtype=torch.int32)
        of = torch.full((rows,), -1, dtype=torch.int32)
        of[1::2] = torch.arange(rows // 2, dtype=torch.int32)
        s["grammar_of"] = of.cuda()
    else:
        n, v = _text_lens(case), case["vocab"]
        total = sum(n)
        s["tokens"] = (torch.rand(total, generator=gen, device="cuda").pow_(3.0) * v).int().clamp_(max=v - 1)
        s["starts"], s["prompts"] = _starts(n), _i32([x * 3 // 4 for x in n])
        s["state_of"] = _i32(rng.permutation(case["seqs"]).tolist())
        s["counts"] = torch.zeros((case["seqs"], v), dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_calls if own else _plain)[s["case"]["kind"]](s)


def _cache(s):
    """The cache's handle, as a program keeps it beside the planes."""
    import speculative_verify_attention_gb300 as kv
    if "cache" not in s:
        s["cache"] = kv.KVPagedCacheQ8.from_planes(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    return kv, s["cache"]


def _call_verify(s):
    kv, cache = _cache(s)
    if "out" not in s:  # the program's buffers
        s["out"] = torch.empty_like(s["q"])
        n = kv.attn_verify_paged_q8_workspace_bytes(s["case"]["hq"], cache.n_kv_heads, cache.head_dim, s["max_rows"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return kv.attn_verify_paged_q8(s["q"], cache, s["table"], s["lens"], s["starts"], s["max_rows"], s["scale"],
                                   window_mask=s["mask"], out=s["out"], workspace=s["workspace"])


def _call_tables(s):
    import speculative_verify_attention_gb300 as kv
    if "out" not in s:
        n = s["n_rows"]
        s["out"] = dict(held_out=torch.empty_like(s["held"]), ring_out=torch.empty_like(s["ring_state"]),
                        row_starts=torch.empty(len(s["lens"]) + 1, dtype=torch.int32, device="cuda"),
                        slots=torch.empty(n, dtype=torch.int64, device="cuda"),
                        positions=torch.empty(n, dtype=torch.int32, device="cuda"),
                        status=torch.empty(1, dtype=torch.int32, device="cuda"))
    kv.kvq8_paged_tables(s["lens"], s["n_new"], s["held"], s["table"], s["ring"], s["ring_state"], s["case"]["page"],
                         **s["out"])
    return {"table": s["table"], "ring": s["ring"], **s["out"]}


def _call_cache(s):
    kv, cache = _cache(s)
    if "out" not in s:
        shape = (len(s["every"]), cache.n_kv_heads, cache.head_dim)
        s["out"] = [torch.empty(shape, dtype=torch.float16, device="cuda") for _ in range(2)]
    kv.kvq8_paged_append(s["k"], s["v"], cache, s["slots"])
    kv.kvq8_paged_read(cache, s["every"], *s["out"])
    return s["out"]


def _call_adjust(s):
    import speculative_verify_attention_gb300 as kv
    if "out" not in s:
        s["out"] = torch.empty(s["logits"].shape, dtype=torch.float32, device="cuda")
    return kv.logits_adjust(s["logits"], s["starts"], penalties=s["penalties"], counts=s["counts"], state_of=s["state_of"],
                            window_tokens=s["tokens"], window_mask=s["mask"], bias_starts=s["bias_starts"],
                            bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], grammar=s["grammar"],
                            grammar_of=s["grammar_of"], out=s["out"])


def _call_counts(s):
    import speculative_verify_attention_gb300 as kv
    kv.token_counts(s["tokens"], s["starts"], s["counts"], prompt_lens=s["prompts"], state_of=s["state_of"], clear=True)
    return s["counts"]


_calls = {"verify": _call_verify, "tables": _call_tables, "cache": _call_cache, "adjust": _call_adjust, "counts": _call_counts}


# ---------------------------------------------------------------- plain forms

def _values(codes, scales):
    return codes.float().unflatten(-1, (-1, 32)).mul_(scales.float().unsqueeze(-1)).flatten(-2)


def _gathered(codes, scales, table):
    """[pages][heads][page][dim] by a table [seqs][n] -> fp32 [seqs][heads][n * page][dim]."""
    return _values(codes[table], scales[table]).transpose(1, 2).flatten(2, 3)


def _rows(starts, n_rows):
    """Request and place in its window of every row; the rows behind the last belong to the request past the end."""
    r = torch.arange(n_rows, device="cuda")
    seq = torch.searchsorted(starts[1:].contiguous(), r.int(), right=True)
    return seq, r - starts.long()[seq]


def _bits(mask, seq, place, starts, most):
    """[rows][most] truth values: whether a row sees window token j."""
    j = torch.arange(most, device="cuda")
    inside = j < (starts[1:] - starts[:-1]).long()[seq].unsqueeze(1)
    if mask is None:
        return inside & (j <= place.unsqueeze(1))
    return inside & ((mask.unsqueeze(1) >> j) & 1).bool()


def _plain_verify(s):
    table, lens, starts, q = s["table"].long(), s["lens"].long(), s["starts"], s["q"]
    k = _gathered(s["k_codes"], s["k_scales"], table)
    v = _gathered(s["v_codes"], s["v_scales"], table)
    n, heads, keys, dim = k.shape
    group, most = q.shape[1] // heads, s["max_rows"]
    seq, place = _rows(starts, s["n_rows"])
    padded = torch.zeros((n, most) + q.shape[1:], device="cuda")
    padded[seq, place] = q.float()
    x = padded.unflatten(2, (heads, group)).permute(0, 2, 1, 3, 4).flatten(2, 3) @ k.transpose(2, 3) * s["scale"]
    ctx = lens - (starts[1:] - starts[:-1]).long()
    window = torch.zeros((n, most, most), dtype=torch.bool, device="cuda")
    window[seq, place] = _bits(s["mask"], seq, place, starts, most)
    at = torch.arange(keys, device="cuda") - ctx.unsqueeze(1)
    seen = window.gather(2, at.clamp(0, most - 1).unsqueeze(1).expand(-1, most, -1))
    at = at.unsqueeze(1)
    seen = ((at < 0) | (seen & (at < most))).repeat_interleave(group, 1).unsqueeze(1)
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x @ v) / torch.where(total == 0, 1.0, total)
    return o.unflatten(2, (most, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, place].to(q.dtype)


def _plain_tables(s):
    lens, new, held, ring, page = s["lens"].long(), s["n_new"].long(), s["held"].long(), s["ring"], s["case"]["page"]
    head, count = s["ring_state"].long()
    pages, width = len(ring), s["table"].shape[1]
    need = (lens + page - 1) // page
    take, give = (need - held).clamp(min=0), (held - need).clamp(min=0)
    p = torch.arange(width, device="cuda")
    first_take, first_give = (take.cumsum(0) - take).unsqueeze(1), (give.cumsum(0) - give).unsqueeze(1)
    h, m = held.unsqueeze(1), need.unsqueeze(1)
    taken, given = (p >= h) & (p < m), (p >= m) & (p < h)
    table = torch.where(taken, ring[(head + first_take + p - h) % pages], s["table"])
    place = torch.where(given, (head + count + first_give + p - m) % pages, pages)
    ring = torch.cat([ring, ring[:1]]).scatter(0, place.flatten(), s["table"].flatten())[:pages]
    state = torch.stack([(head + take.sum()) % pages, count - take.sum() + give.sum()]).int()
    starts = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), new.cumsum(0)])
    seq, at = _rows(starts.int(), s["n_rows"])
    live, seq = seq < len(lens), seq.clamp(max=len(lens) - 1)
    pos = torch.where(live, lens[seq] - new[seq] + at, 0)
    slots = torch.where(live, table[seq, pos // page].long() * page + pos % page, -1)
    return {"table": table, "ring": ring, "held_out": need.int(), "ring_out": state, "row_starts": starts.int(),
            "slots": slots, "positions": torch.where(live, pos, -1).int(),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _quantised(x):
    x = x.float().unflatten(-1, (-1, 32))
    d = x.abs().amax(-1, keepdim=True) / 127.0
    y = torch.where(d == 0, 0.0, x / d)
    a = y.abs()
    whole = a.floor()
    code = ((whole + (a - whole >= 0.5)).clamp(max=127.0) * y.sign()).flatten(-2)  # ties away from zero
    return code.to(torch.int8), d.squeeze(-1).half()


def _plain_cache(s):
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    outs = []
    for x, codes, scales in ((s["k"], s["k_codes"], s["k_scales"]), (s["v"], s["v_codes"], s["v_scales"])):
        codes[at, :, off], scales[at, :, off] = _quantised(x)
        outs.append(_values(codes, scales).transpose(1, 2).flatten(0, 1)[s["every"]].half())
    return outs


def _plain_adjust(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    starts, most = s["starts"], s["case"]["rows"]
    seq, place = _rows(starts, rows)
    word = s["counts"][s["state_of"].long()[seq]]
    count = word & 0x7fffffff
    token = s["tokens"].long()[(starts.long()[seq].unsqueeze(1) + torch.arange(most, device="cuda")).clamp(max=rows - 1)]
    count.scatter_add_(1, token, _bits(s["mask"], seq, place, starts, most).int())
    repeat, often, once = s["penalties"][seq].unsqueeze(2).unbind(1)
    x = torch.where((count > 0) | (word < 0), torch.where(x > 0, x / repeat, x * repeat), x)
    x = x - (often * count + once * (count > 0))
    listed_at = torch.arange(len(s["bias_tokens"]), device="cuda")
    if len(listed_at):
        of = torch.searchsorted(s["bias_starts"][1:].contiguous(), listed_at.int(), right=True)
        last = torch.full((len(starts) - 1, vocab), -1, dtype=torch.long, device="cuda")  # a token's last entry holds
        last = last.flatten().scatter_reduce_(0, of * vocab + s["bias_tokens"].long(), listed_at, "amax").view(-1, vocab)
        x = x + torch.where(last >= 0, s["bias_values"][last.clamp(min=0)], 0.0)[seq]
    bits = (s["grammar"].unsqueeze(2) >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    allowed = bits.bool().flatten(1)[:, :vocab]
    of = s["grammar_of"].long()
    return torch.where(allowed[of.clamp(min=0)] | (of < 0).unsqueeze(1), x, -math.inf)


def _plain_counts(s):
    total, vocab = len(s["tokens"]), s["case"]["vocab"]
    seq, place = _rows(s["starts"], total)
    prompt = place < s["prompts"].long()[seq]
    at = s["state_of"].long()[seq] * vocab + s["tokens"].long()
    s["counts"].zero_()
    flat = s["counts"].view(-1)
    flat.scatter_add_(0, at, (~prompt).int())
    said = torch.zeros_like(flat).scatter_reduce_(0, at, prompt.int(), "amax")
    flat |= said << 31
    return s["counts"]


_plain = {"verify": _plain_verify, "tables": _plain_tables, "cache": _plain_cache, "adjust": _plain_adjust,
          "counts": _plain_counts}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"verify": _exact_verify, "cache": _exact_cache, "adjust": _exact_adjust}.get(case["kind"], lambda s: None)(s)


def _exact_verify(s):
    """Request by request and head by head, row by row of the window only for what a row sees."""
    q, page = s["q"].double(), s["case"]["page"]
    out = torch.empty_like(q)
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    heads = s["case"]["hkv"]
    group = q.shape[1] // heads
    words = None if s["mask"] is None else [w & (2 ** 64 - 1) for w in s["mask"].tolist()]
    for b, n in enumerate(lens):
        r0, r1 = starts[b], starts[b + 1]
        at = torch.arange(n, device="cuda")
        pg, off = s["table"][b].long()[at // page], at % page
        seen = torch.ones((r1 - r0, n), dtype=torch.bool)
        for t in range(r1 - r0):
            for j in range(r1 - r0):
                seen[t, n - (r1 - r0) + j] = (j <= t) if words is None else bool(words[r0 + t] >> j & 1)
        hidden = torch.where(seen, 0.0, -math.inf).double().cuda()
        for h in range(heads):
            k = s["k_codes"][pg, h, off].double() * s["k_scales"][pg, h, off].double().repeat_interleave(32, 1)
            v = s["v_codes"][pg, h, off].double() * s["v_scales"][pg, h, off].double().repeat_interleave(32, 1)
            for g in range(h * group, (h + 1) * group):
                x = q[r0:r1, g] @ k.T * s["scale"] + hidden
                out[r0:r1, g] = torch.softmax(x, 1) @ v
    return out


def _exact_cache(s):
    page, outs = s["case"]["page"], []
    for x, codes, scales in ((s["k"], s["k_codes"], s["k_scales"]), (s["v"], s["v_codes"], s["v_scales"])):
        pool = codes.double() * scales.double().repeat_interleave(32, 3)
        blocks = x.double().reshape(*x.shape[:2], -1, 32)
        step = (blocks.abs().amax(3).float() / 127.0).double()  # the format's step is a 32-bit quotient
        ratio = (blocks / step.unsqueeze(3)).float().double()  # and so is the number that is rounded
        code = torch.where(step.unsqueeze(3) > 0, torch.trunc(ratio + 0.5 * ratio.sign()), 0.0).clamp(-127, 127)
        pool[s["slots"] // page, :, s["slots"] % page] = (code * step.half().double().unsqueeze(3)).reshape(x.shape)
        outs.append(pool.permute(0, 2, 1, 3).reshape(-1, *x.shape[1:])[s["every"]])
    return outs


def _exact_adjust(s):
    """Row by row: what the row's request holds, then its own path through the window."""
    x = s["logits"].double()
    starts, state = s["starts"].tolist(), s["state_of"].tolist()
    tokens, of = s["tokens"].tolist(), s["grammar_of"].tolist()
    bias_at, bias_tokens, bias = s["bias_starts"].tolist(), s["bias_tokens"].tolist(), s["bias_values"].tolist()
    words = None if s["mask"] is None else [w & (2 ** 64 - 1) for w in s["mask"].tolist()]
    place = torch.arange(x.shape[1], device="cuda")
    for b in range(len(starts) - 1):
        repeat, often, once = s["penalties"][b].double().tolist()
        entries = dict(zip(bias_tokens[bias_at[b]:bias_at[b + 1]], bias[bias_at[b]:bias_at[b + 1]]))
        add = torch.zeros(x.shape[1], dtype=torch.float64)
        add[list(entries.keys())] = torch.tensor(list(entries.values()), dtype=torch.float64)
        add = add.cuda()
        word = s["counts"][state[b]].long()
        for r in range(starts[b], starts[b + 1]):
            path = [tokens[starts[b] + j] for j in range(starts[b + 1] - starts[b])
                    if (j <= r - starts[b] if words is None else words[r] >> j & 1)]
            count = word % (1 << 31) + torch.bincount(torch.tensor(path, device="cuda"), minlength=x.shape[1])
            hit = (count > 0) | (word < 0)
            y = torch.where(hit, torch.where(x[r] > 0, x[r] / repeat, x[r] * repeat), x[r])
            x[r] = y - often * count - once * (count > 0) + add
            if of[r] >= 0:
                x[r][(s["grammar"][of[r]].long()[place // 32] >> (place % 32)) & 1 == 0] = -math.inf
    return x
