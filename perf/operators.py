"""The attention side of a decoder layer, measured: attention of new tokens over a paged cache, the rotary positions of
what is appended to that cache, and the upkeep of its pages.

`run` computes each operator either with the library's kernels (`own` true) or in its plain form: elementary torch
operations in 32 bits, rounded once at the end. Sizes: 32 query heads of 128 values are the rows of 4096 of the
library's own decode product; the rest are generic."""
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases ---------------------------------------------------------------------------------------------------

def listed():
    return [
        # one chat, one token, at its start: nothing but latency
        dict(name="attn-1-token", op="attn", seqs=1, empty=0, q_lo=1, q_hi=1, kv_lo=37, kv_hi=37, heads=32, kv_heads=8,
             dim=128, page=16, window=0, dtype="bf16", mix=1),
        # a serving step: 61 chats of very different lengths, padded to 64 slots with sequences that hold nothing
        dict(name="attn-decode-64", op="attn", seqs=64, empty=3, q_lo=1, q_hi=1, kv_lo=33, kv_hi=8192, heads=32,
             kv_heads=8, dim=128, page=16, window=0, dtype="bf16", mix=2),
        # two long documents, one token each: few rows, a long axis
        dict(name="attn-decode-long", op="attn", seqs=2, empty=0, q_lo=1, q_hi=1, kv_lo=100003, kv_hi=131071, heads=32,
             kv_heads=8, dim=128, page=64, window=0, dtype="f16", mix=3),
        # a prompt from its first token to its last: the matrix product at its largest
        dict(name="attn-prompt-8192", op="attn", seqs=1, empty=0, q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, heads=32,
             kv_heads=8, dim=128, page=32, window=0, dtype="bf16", mix=4),
        # chunks of prompts among single tokens, seven heads to a group, pages that divide nothing, a sliding window
        dict(name="attn-chunks-mixed", op="attn", seqs=17, empty=0, q_lo=1, q_hi=700, kv_lo=701, kv_hi=6000, heads=28,
             kv_heads=4, dim=64, page=24, window=1024, dtype="f16", mix=5),
        # the decode step's keys and values, as the products leave them (32 bits), into the cache
        dict(name="append-decode-33", op="append", seqs=33, empty=0, q_lo=1, q_hi=1, kv_lo=5, kv_hi=8000, heads=32,
             kv_heads=8, dim=128, rot=128, interleaved=False, page=16, source="f32", dtype="bf16", mix=6),
        # a prompt's, with neighbouring pairs and half of each head turned
        dict(name="append-prompts", op="append", seqs=3, empty=0, q_lo=1900, q_hi=4100, kv_lo=4100, kv_hi=9000, heads=32,
             kv_heads=8, dim=128, rot=64, interleaved=True, page=32, source="bf16", dtype="bf16", mix=7),
        # the gradient's way back through the rotation, odd length, heads of 96
        dict(name="rope-gradient", op="rope", tokens=4099, heads=32, dim=96, rot=96, interleaved=False, inverse=True,
             dtype="f16", mix=8),
        # a few samples branch off one chat
        dict(name="fork-4", op="fork", seqs=8, forks=4, kv_lo=40, kv_hi=900, kv_heads=8, dim=128, layers=2, page=16,
             new=3, dtype="bf16", mix=9),
        # many beams at once, over all layers of a stage
        dict(name="fork-200", op="fork", seqs=480, forks=200, kv_lo=17, kv_hi=3000, kv_heads=8, dim=128, layers=8,
             page=64, new=1, dtype="bf16", mix=10),
        # one of three chats ends
        dict(name="compact-small", op="compact", seqs=3, gone=1, kv_lo=100, kv_hi=700, kv_heads=4, dim=64, layers=2,
             page=16, dtype="f16", mix=11),
        # a third of a full cache ends and the rest moves together
        dict(name="compact-large", op="compact", seqs=96, gone=31, kv_lo=900, kv_hi=6000, kv_heads=8, dim=128, layers=4,
             page=32, dtype="bf16", mix=12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "rope", "fork", "compact"])
    mix = rng.randrange(1 << 30)
    kv_heads = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 64, 80, 96, 128, 128, 128])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([16, 16, 24, 32, 64])
    heads = kv_heads * rng.choice([1, 2, 4, 7])
    if op == "attn":
        seqs = _log(rng, 1, 64)
        q_hi = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
        room = 6.0e8 / (seqs * q_hi * heads)  # (query, key) pairs of one query row, so that no case passes the largest
        room = min(room, 2.4e8 / (seqs * kv_heads * dim), 131071)  # and the cache's size
        kv_hi = _log(rng, 16, max(17, int(room)))
        kv_hi = max(kv_hi, 2)
        q_hi = min(q_hi, kv_hi)
        q_lo = rng.choice([1, q_hi])
        return dict(op="attn", seqs=seqs, empty=rng.choice([0, 0, 1]) if seqs > 1 else 0, q_lo=q_lo, q_hi=q_hi, kv_lo=max(q_hi, kv_hi // rng.choice([1, 4, 30])),
                    kv_hi=kv_hi, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    window=rng.choice([0, 0, _log(rng, 16, 4096)]), dtype=dtype, mix=mix)
    if op == "append":
        seqs = _log(rng, 1, 64)
        q_hi = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 12000 // seqs))
        return dict(op="append", seqs=seqs, empty=0, q_lo=rng.choice([1, q_hi]), q_hi=q_hi, kv_lo=q_hi, kv_hi=_log(rng, q_hi + 5, 9000 + q_hi),
                    heads=heads, kv_heads=kv_heads, dim=dim, rot=rng.choice([dim, dim // 2]), interleaved=rng.random() < 0.5,
                    page=page, source=rng.choice(["f32", dtype]), dtype=dtype, mix=mix)
    if op == "rope":
        return dict(op="rope", tokens=_log(rng, 1, 8192), heads=heads, dim=dim, rot=rng.choice([dim, dim // 2]),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, dtype=rng.choice(["f32", "f16", "bf16"]), mix=mix)
    seqs = _log(rng, 3, 300)
    kv_hi = _log(rng, 40, min(6000, 300000 // seqs))
    if op == "fork":
        return dict(op="fork", seqs=seqs, forks=rng.randrange(1, seqs // 2 + 1), kv_lo=max(1, kv_hi // 20), kv_hi=kv_hi, kv_heads=kv_heads,
                    dim=dim, layers=rng.choice([1, 2, 4]), page=page, new=_log(rng, 1, 40), dtype=dtype, mix=mix)
    return dict(op="compact", seqs=seqs, gone=rng.randrange(1, seqs), kv_lo=max(1, kv_hi // 20), kv_hi=kv_hi, kv_heads=kv_heads,
                dim=dim, layers=rng.choice([1, 2, 4]), page=page, dtype=dtype, mix=mix)


def _lengths(case):
    """The sequences' lengths: (new tokens, tokens in the cache with them), a list of pairs, the empty ones last."""
    rng = random.Random(case["mix"])
    got = []
    for _ in range(case["seqs"] - case.get("empty", 0)):
        q = _log(rng, case["q_lo"], case["q_hi"]) if "q_lo" in case else 0
        got.append((q, max(q, _log(rng, case["kv_lo"], case["kv_hi"]))))
    return got + [(1, 0)] * case.get("empty", 0)


def _shape(case):
    """The sequences' lengths of a pages case; a fork's children, the last ones, hold nothing yet."""
    lens = [kv for _, kv in _lengths(case)]
    if case["op"] == "fork":
        lens[case["seqs"] - case["forks"]:] = [0] * case["forks"]
    return lens


# ---- inputs --------------------------------------------------------------------------------------------------------

def _table(case, lens, spare, gen):
    """A page table over shuffled pages: ([sequences, widest] of int32 with -1 behind each row's end, pages in all)."""
    ps = case["page"]
    pages = [-(-n // ps) for n in lens]
    used, width = sum(pages), max(1, max(pages)) + 3
    total = used + spare
    order = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    count = torch.tensor(pages, device="cuda").unsqueeze(1)
    first = torch.cumsum(count, 0) - count
    at = torch.arange(width, device="cuda").unsqueeze(0)
    table = torch.where(at < count, order[(first + at).clamp(max=max(0, total - 1))], -1)
    return table.to(torch.int32).contiguous(), total


def _normal(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _angles(n_pos, rot):
    """cos and sin of position times frequency, [positions, rot / 2, 2], formed in 64 bits and kept in 32."""
    freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2.0 / rot)
    a = torch.arange(n_pos, device="cuda", dtype=torch.float64).unsqueeze(1) * freq
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    d, op = DTYPES[case["dtype"]], case["op"]
    if op == "rope":
        s["x"] = _normal(gen, case["tokens"], case["heads"], case["dim"], dtype=d)
        s["angles"] = _angles(2 * case["tokens"] + 64, case["rot"])
        s["positions"] = torch.randint(0, 2 * case["tokens"] + 64, (case["tokens"],), generator=gen, device="cuda", dtype=torch.int32)
        return s
    if op in ("attn", "append"):
        pairs = _lengths(case)
        lens = [kv for _, kv in pairs]
        s["table"], n = _table(case, lens, 5, gen)
        starts = [0]
        for q, _ in pairs:
            starts.append(starts[-1] + q)
        s["q_starts"] = torch.tensor(starts, device="cuda", dtype=torch.int32)
        s["kv_lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        s["max_q"], s["max_kv"] = max(q for q, _ in pairs), max(lens)
        shape = (n, case["page"], case["kv_heads"], case["dim"])
        s["k"], s["v"] = _normal(gen, *shape, dtype=d), _normal(gen, *shape, dtype=d)
        if op == "attn":
            s["q"] = _normal(gen, starts[-1], case["heads"], case["dim"], dtype=d)
        else:
            src = DTYPES[case["source"]]
            # one product makes all three: q, k and v are slices of its rows
            h, g = case["heads"], case["kv_heads"]
            row = _normal(gen, starts[-1], h + 2 * g, case["dim"], dtype=src)
            s["q"], s["k_new"], s["v_new"] = row[:, :h], row[:, h:h + g], row[:, h + g:]
            s["angles"] = _angles(max(lens) + 1, case["rot"])
        return s
    lens = _shape(case)
    s["table"], n = _table(case, lens, case.get("forks", 2) * (2 + case.get("new", 0) // case["page"]) + 7, gen)
    s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["refs"] = torch.zeros(n, device="cuda", dtype=torch.int32)
    s["refs"][s["table"][s["table"] >= 0].long()] = 1
    shape = (case["layers"], n, case["page"], case["kv_heads"], case["dim"])
    s["k"], s["v"] = _normal(gen, *shape, dtype=d), _normal(gen, *shape, dtype=d)
    if op == "fork":
        live = case["seqs"] - case["forks"]
        s["parents"] = torch.randint(0, live, (case["forks"],), generator=gen, device="cuda", dtype=torch.int32)
        s["children"] = torch.arange(live, case["seqs"], device="cuda", dtype=torch.int32)
        s["n_new"] = torch.zeros(case["seqs"], device="cuda", dtype=torch.int32)
        s["n_new"][live:] = case["new"]
    else:
        s["gone"] = torch.randperm(case["seqs"], generator=gen, device="cuda")[:case["gone"]].to(torch.int32)
    return s


# ---- the plain forms -------------------------------------------------------------------------------------------------

def _plain_attention(s):
    case, q, table = s["case"], s["q"], s["table"].long()
    h, g, d, ps = case["heads"], case["kv_heads"], case["dim"], case["page"]
    starts, kv_len = s["q_starts"].long(), s["kv_lens"].long()
    n, mq, mk = len(kv_len), s["max_q"], s["max_kv"]
    q_len = starts[1:] - starts[:-1]
    # queries padded to [sequence, kv head, (head of the group, row), value]; rows past a sequence's own repeat its last
    row = torch.arange(mq, device=q.device)
    token = (starts[:-1, None] + torch.minimum(row, q_len[:, None] - 1)).clamp(0, len(q) - 1)
    qs = q[token].float().view(n, mq, g, h // g, d).permute(0, 2, 3, 1, 4).reshape(n, g, h // g * mq, d)
    # keys and values of each sequence in order, padded to the longest
    col = torch.arange(mk, device=q.device)
    slot = table[:, col // ps].clamp(min=0) * ps + col % ps
    k = s["k"].reshape(-1, g, d)[slot].float().permute(0, 2, 3, 1).contiguous()
    v = s["v"].reshape(-1, g, d)[slot].float().permute(0, 2, 1, 3).contiguous()
    score = torch.matmul(qs, k) * (d ** -0.5)
    pos = (kv_len - q_len)[:, None] + row
    seen = (col <= pos[:, :, None]) & (col < kv_len[:, None, None])
    if case["window"]:
        seen &= col > pos[:, :, None] - case["window"]
    score = score.view(n, g, h // g, mq, mk).masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == float("-inf"), 0.0, top))
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e.view(n, g, h // g * mq, mk), v).view(n, g, h // g, mq, d) / torch.where(total == 0, 1.0, total)
    out = out.permute(0, 3, 1, 2, 4).reshape(n, mq, h, d)
    t = torch.arange(len(q), device=q.device)
    b = torch.searchsorted(starts, t, right=True) - 1
    return out[b, t - starts[b]].to(q.dtype)


def _plain_rope(x, rows, interleaved, inverse):
    """x [tokens, heads, values] turned by rows [tokens, pairs, 2] of cos and sin; the values behind the pairs stay."""
    f = rows.shape[1]
    c, sn = rows[:, None, :, 0], rows[:, None, :, 1] * (-1.0 if inverse else 1.0)
    x = x.float()
    a, b = (x[..., 0:2 * f:2], x[..., 1:2 * f:2]) if interleaved else (x[..., :f], x[..., f:2 * f])
    u, w = a * c - b * sn, b * c + a * sn
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., 2 * f:]), -1)


def _plain_append(s):
    case, ps, d = s["case"], s["case"]["page"], DTYPES[s["case"]["dtype"]]
    starts, t = s["q_starts"].long(), torch.arange(len(s["q"]), device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    pos = s["kv_lens"].long()[b] - starts[b + 1] + t
    rows = s["angles"][pos]
    slot = s["table"].long()[b, pos // ps] * ps + pos % ps
    q = _plain_rope(s["q"], rows, case["interleaved"], False).to(d)
    s["k"].view(-1, case["kv_heads"], case["dim"])[slot] = _plain_rope(s["k_new"], rows, case["interleaved"], False).to(d)
    s["v"].view(-1, case["kv_heads"], case["dim"])[slot] = s["v_new"].float().to(d)
    return q, s["k"], s["v"]


def _plain_fork(s):
    """Children take their parents' full pages and a copy of the last part of one; then every child gets room for new tokens."""
    case, ps = s["case"], s["case"]["page"]
    table, lens, refs = s["table"].long(), s["lens"].long(), s["refs"].long()
    parent, child = s["parents"].long(), s["children"].long()
    m, at = table.shape[1], torch.arange(table.shape[1], device="cuda")
    n = lens[parent]
    full, tail = n // ps, (n % ps != 0)
    free = torch.argsort((refs > 0).to(torch.int32), stable=True)  # the free pages first, lowest first
    new = free[(torch.cumsum(tail.long(), 0) - tail.long())]
    old = table[parent, full.clamp(max=m - 1)]
    rows = torch.where(at < full[:, None], table[parent], torch.where((at == full[:, None]) & tail[:, None], new[:, None], -1))
    refs = refs.clone()
    refs.index_add_(0, rows.clamp(min=0).flatten(), (rows >= 0).long().flatten())
    table, lens = table.clone(), lens.clone()
    table[child], lens[child] = rows, n
    # the tails' tokens; a fork without one writes a page on itself
    part = (torch.arange(ps, device="cuda") < (n % ps)[:, None])[None, :, :, None, None]
    src, dst = torch.where(tail, old, rows[:, 0]), torch.where(tail, new, rows[:, 0])
    for c in (s["k"], s["v"]):
        c[:, dst] = torch.where(part, c[:, src], c[:, dst])
    # room: the pages that the grown lengths need beyond those there, lowest first, in the order of the sequences
    have, grown = (lens + ps - 1) // ps, lens + s["n_new"].long()
    need = (grown + ps - 1) // ps - have
    free = torch.argsort((refs > 0).to(torch.int32), stable=True)
    first = (torch.cumsum(need, 0) - need)[:, None]
    k = at - have[:, None]
    given = (k >= 0) & (k < need[:, None])
    got = torch.where(given, free[(first + k).clamp(0, len(free) - 1)], -1)
    refs.index_add_(0, got.clamp(min=0).flatten(), given.long().flatten())
    table = torch.where(given, got, table)
    return table.to(torch.int32), grown.to(torch.int32), refs.to(torch.int32), s["k"], s["v"]


def _plain_compact(s):
    """The listed sequences give their pages back; then used pages from the end move into the holes before them."""
    table, lens, refs, gone = s["table"].long(), s["lens"].clone(), s["refs"].long(), s["gone"].long()
    rows = table[gone]
    refs = refs.clone()
    refs.index_add_(0, rows.clamp(min=0).flatten(), -(rows >= 0).long().flatten())
    table = table.clone()
    table[gone], lens[gone] = -1, 0
    used, at = refs > 0, torch.arange(len(refs), device="cuda")
    n = used.sum()
    src, dst = at[used & (at >= n)], at[~used & (at < n)]
    to = at.clone()
    to[src] = dst
    table = torch.where(table >= 0, to[table.clamp(min=0)], -1)
    moved = refs.clone()
    moved[dst], moved[src] = refs[src], 0
    for c in (s["k"], s["v"]):
        c[:, dst] = c[:, src]
    return table.to(torch.int32), lens, moved.to(torch.int32), s["k"], s["v"]


# ---- one pass ----------------------------------------------------------------------------------------------------------

def _own(s):
    import bit_quantized_mat_amd as bqm
    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        return bqm.rope(s["x"], s["angles"], s["positions"], interleaved=case["interleaved"], inverse=case["inverse"])
    cache = bqm.KvCache(s["k"], s["v"])
    if op in ("attn", "append"):
        batch = bqm.KvBatch(s["table"], s["kv_lens"], s["q_starts"], max_q=s["max_q"], max_kv=s["max_kv"])
        if op == "attn":
            return bqm.paged_attention(s["q"], cache, batch, window=case["window"])
        q = bqm.rope_kv_append(s["q"], s["k_new"], s["v_new"], cache, batch, s["angles"], interleaved=case["interleaved"])
        return q, s["k"], s["v"]
    pages = bqm.KvPages(s["table"], s["lens"], s["refs"])
    if op == "fork":
        pages, moves, _ = bqm.kv_fork(pages, s["parents"], s["children"], case["page"])
        bqm.kv_copy_pages(cache, moves)
        pages, _ = bqm.kv_extend(pages, s["n_new"], case["page"])
    else:
        pages = bqm.kv_free(pages, s["gone"])
        pages, moves, _ = bqm.kv_compact(pages, case["page"])
        bqm.kv_copy_pages(cache, moves)
    return pages.table, pages.lens, pages.refs, s["k"], s["v"]


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "attn":
        return _plain_attention(state)
    if case["op"] == "append":
        return _plain_append(state)
    if case["op"] == "rope":
        rows = state["angles"][state["positions"].long()]
        return _plain_rope(state["x"], rows, case["interleaved"], case["inverse"]).to(state["x"].dtype)
    return _plain_fork(state) if case["op"] == "fork" else _plain_compact(state)


# ---- what a pass cannot do without ---------------------------------------------------------------------------------------

def work(case):
    op, size = case["op"], 4 if case["dtype"] == "f32" else 2
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        # the angles of each token are read once (distinct rows: at most the tokens)
        return {"bytes": 2 * n * size + case["tokens"] * (4 * case["rot"] + 4), "flops": 3 * n * case["rot"] // case["dim"]}
    lengths = _lengths(case)
    if op == "append":
        t, row = sum(q for q, _ in lengths), (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        src = 4 if case["source"] == "f32" else 2
        turned = t * (case["heads"] + case["kv_heads"]) * case["rot"]
        return {"bytes": t * row * (src + size) + t * 4 * case["rot"], "flops": 3 * turned}
    token = 2 * case["kv_heads"] * case["dim"] * size
    if op == "attn":
        read = pairs = 0
        for q, kv in lengths:
            w = case["window"] or kv
            # keys that some query of the sequence sees, and the (query, key) pairs
            read += kv - max(0, kv - q + 1 - w) if kv else 0
            first = kv - q + 1  # keys before and with the first query
            cut = min(max(w - first + 1, 0), q)  # queries that see all keys before them
            pairs += cut * first + cut * (cut - 1) // 2 + (q - cut) * w if kv else 0
        t = sum(q for q, _ in lengths)
        return {"bytes": 2 * t * case["heads"] * case["dim"] * size + read * token + 4 * sum(-(-kv // case["page"]) for _, kv in lengths),
                "flops": 4 * case["dim"] * case["heads"] * pairs}
    lens, ps, layers = _shape(case), case["page"], case["layers"]
    n = sum(-(-x // ps) for x in lens)
    meta = 8 * (case["seqs"] * (3 + max(1, max(-(-x // ps) for x in lens))) + n)  # table, lengths and counts, read and written
    if op == "fork":
        live = lens[:case["seqs"] - case["forks"]]
        tails = case["forks"] * sum(x % ps for x in live) / len(live)  # parents are drawn evenly
        return {"bytes": meta + 2 * layers * token * tails, "flops": 0}
    left = n * (1 - case["gone"] / case["seqs"])
    moved = left * (n - left) / n  # used pages behind the first `left` ones, were they spread evenly
    return {"bytes": meta + 2 * layers * token * ps * moved, "flops": 0}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------------------

def _exact_turn(x, pos, table, interleaved, sign):
    """Each pair as a complex number times cos + i sin of its table row."""
    f, y = table.shape[1], x.double().clone()
    turn = torch.complex(table[pos, :, 0].double(), sign * table[pos, :, 1].double())[:, None]
    lo, hi = (slice(0, 2 * f, 2), slice(1, 2 * f, 2)) if interleaved else (slice(0, f), slice(f, 2 * f))
    z = torch.complex(x[..., lo].double(), x[..., hi].double()) * turn
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_moves(s):
    """(from page, to page, tokens) of what a fork or a compaction copies, by the definition, one page at a time."""
    ps, table, lens, refs = s["case"]["page"], s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    if s["case"]["op"] == "fork":
        free = [p for p, r in enumerate(refs) if r == 0]
        return [(table[a][lens[a] // ps], free.pop(0), lens[a] % ps) for a in s["parents"].tolist() if lens[a] % ps]
    for b in s["gone"].tolist():
        for p in table[b]:
            if p >= 0:
                refs[p] -= 1
    n = sum(r > 0 for r in refs)
    return [(a, b, ps) for a, b in zip([p for p in range(n, len(refs)) if refs[p] > 0], [p for p in range(n) if refs[p] == 0])]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rope":
        return _exact_turn(s["x"], s["positions"].long(), s["angles"], case["interleaved"], -1.0 if case["inverse"] else 1.0)
    ps = case["page"]
    if op in ("fork", "compact"):
        k, v = s["k"].double(), s["v"].double()
        for src, dst, n in _exact_moves(s):
            k[:, dst, :n], v[:, dst, :n] = k[:, src, :n], v[:, src, :n]
        return None, None, None, k, v
    g = case["kv_heads"]
    starts, lens, table = s["q_starts"].tolist(), s["kv_lens"].tolist(), s["table"].tolist()
    if op == "append":
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        for b, n in enumerate(lens):
            lo, hi = starts[b], starts[b + 1]
            pos = torch.arange(n - (hi - lo), n, device="cuda")
            page = torch.tensor(table[b], device="cuda")[pos // ps]
            q[lo:hi] = _exact_turn(s["q"][lo:hi], pos, s["angles"], case["interleaved"], 1.0)
            k[page, pos % ps] = _exact_turn(s["k_new"][lo:hi], pos, s["angles"], case["interleaved"], 1.0)
            v[page, pos % ps] = s["v_new"][lo:hi].double()
        return q, k, v
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        pages = [p for p in table[b] if p >= 0]
        keys, vals = (c[pages].reshape(-1, g, case["dim"])[:n].double() if n else None for c in (s["k"], s["v"]))
        for h in range(case["heads"] if n else 0):
            kk, vv = keys[:, h // (case["heads"] // g)], vals[:, h // (case["heads"] // g)]
            for at in range(lo, hi, 2048):  # rows, some at a time
                to = min(hi, at + 2048)
                x = s["q"][at:to, h].double() @ kk.T.contiguous() / case["dim"] ** 0.5
                ahead = torch.arange(n, device="cuda")[None] - (torch.arange(at, to, device="cuda")[:, None] - lo + n - (hi - lo))
                hide = ahead > 0
                if case["window"]:
                    hide |= ahead <= -case["window"]
                out[at:to, h] = torch.softmax(x.masked_fill(hide, float("-inf")), -1) @ vv
    return out
