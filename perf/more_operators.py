"""The token side of a decoder, measured: from a token's row of a 4-bit table, through the norm in front of each product,
to the logits of a 4-bit output matrix and the next token drawn from them.

`run` computes each operator either with the library's kernels (`own` true) or in its plain form: elementary torch
operations in 32 bits, in 64 where values next to a border would fall on either side of it. 4096 values a token and the
14336 x 4096 product are the library's own; the vocabularies and the rest are generic."""
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases ---------------------------------------------------------------------------------------------------

def listed():
    return [
        # one chat's token in front of a product: nothing but latency
        dict(name="norm-1-token", op="norm", tokens=1, dim=4096, stream="f32", add="f32", gain=True, out="q8"),
        # a serving step's tokens, the stream in 16 bits, what the product before it left in 32
        dict(name="norm-decode-61", op="norm", tokens=61, dim=5120, stream="bf16", add="f32", gain=True, out="q8"),
        # a prompt's
        dict(name="norm-prompt", op="norm", tokens=8191, dim=4096, stream="bf16", add="f32", gain=True, out="q8"),
        # one token against a layer's matrix, small groups with offsets
        dict(name="q4-layer-1", op="mm", tokens=1, rows=4096, dim=4096, group=32, zeros=True),
        # one token against the output matrix: the weights' stream
        dict(name="q4-head-1", op="mm", tokens=1, rows=100003, dim=4096, group=64, zeros=False),
        # a serving step's tokens against it
        dict(name="q4-head-17", op="mm", tokens=17, rows=100003, dim=4096, group=128, zeros=False),
        # a prompt against a feed-forward matrix, of a length that no tile divides
        dict(name="q4-prompt", op="mm", tokens=2047, rows=14336, dim=4096, group=128, zeros=True),
        # the last step's tokens looked up
        dict(name="rows-decode-61", op="rows", tokens=61, rows=100003, dim=4096, group=64, zeros=False, dtype="f32"),
        # a prompt's
        dict(name="rows-prompt", op="rows", tokens=8191, rows=100003, dim=4096, group=32, zeros=True, dtype="bf16"),
        # one chat, a small vocabulary, temperature alone
        dict(name="sample-1", op="sample", tokens=1, vocab=32001, dtype="f32", mode="plain", masked=0.0, empty=0),
        # a serving step: every chat with its own settings, greedy ones among them, slots that hold nothing
        dict(name="sample-64", op="sample", tokens=64, vocab=100003, dtype="f32", mode="all", masked=0.0, empty=3),
        # many samples, a nucleus each, 16-bit logits with their ties, a third of the tokens ruled out by a grammar
        dict(name="sample-256", op="sample", tokens=256, vocab=100003, dtype="bf16", mode="p", masked=0.3, empty=0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm", "mm", "mm", "mm", "rows", "sample", "sample"])
    if op == "norm":
        dim = 32 * _log(rng, 1, 512)
        stream = rng.choice(["f32", "f16", "bf16"])
        return dict(op="norm", tokens=_log(rng, 1, min(8191, 8191 * 4096 // dim)), dim=dim, stream=stream,
                    add=rng.choice(["", "f32", "f32", stream]), gain=rng.random() < 0.8, out=rng.choice(["q8", "q8", "values"]))
    if op == "sample":
        vocab = _log(rng, 2, 131071)
        return dict(op="sample", tokens=_log(rng, 1, max(1, min(256, 256 * 100003 // vocab))), vocab=vocab,
                    dtype=rng.choice(["f32", "f32", "f16", "bf16"]), mode=rng.choice(["plain", "k", "p", "min", "all"]),
                    masked=rng.choice([0.0, 0.0, 0.3, 0.9]), empty=rng.choice([0, 0, 1]))
    group = rng.choice([32, 64, 128])
    dim = group * _log(rng, 1, 16384 // group)
    zeros = rng.random() < 0.5
    if op == "rows":
        rows = _log(rng, 64, min(100003, 100003 * 4096 // dim))
        return dict(op="rows", tokens=_log(rng, 1, min(8191, 8191 * 4096 // dim)), rows=rows, dim=dim, group=group, zeros=zeros,
                    dtype=rng.choice(["f32", "f16", "bf16"]))
    tokens = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 16), _log(rng, 17, 100), _log(rng, 17, 4096)])
    rows = _log(rng, 33, min(100003, 100003 * 4096 // dim, 2047 * 14336 * 4096 // (tokens * dim)))
    return dict(op="mm", tokens=tokens, rows=rows, dim=dim, group=group, zeros=zeros)


# ---- inputs --------------------------------------------------------------------------------------------------------

def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _blocks(x):
    """x fp32 [tokens, dim] as Q8_1 blocks: bytes [tokens, dim / 32 * 36], int8 q[32], fp16 d, fp16 d * sum of q each."""
    b = x.view(x.shape[0], -1, 32)
    d = b.abs().amax(-1, keepdim=True) / 127.0
    q = torch.round(b / torch.where(d > 0, d, 1.0)).clamp(-127, 127)
    field = torch.cat((d, d * q.sum(-1, keepdim=True)), -1).half()
    return torch.cat((q.to(torch.int8).view(torch.uint8), field.view(torch.uint8)), -1).flatten(1).contiguous()


def _table(case, gen, s):
    """A matrix in 4 bits: codes uint8 [rows, dim / 2], in each run of 16 bytes those of 32 values, byte i of value i in its
    low half and of value i + 16 in its high half, as two's complement; scales fp16 and, where there are offsets, zeros
    int8 [rows, dim / group]: value = scale * (code - zero)."""
    rows, dim, groups = case["rows"], case["dim"], case["dim"] // case["group"]
    s["codes"] = torch.randint(0, 256, (rows, dim // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s["scales"] = ((0.5 + torch.rand(rows, groups, generator=gen, device="cuda")) / (4.6 * dim ** 0.5)).half()
    s["zeros"] = None
    if case["zeros"]:
        s["zeros"] = torch.randint(-4, 5, (rows, groups), generator=gen, device="cuda", dtype=torch.int8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    op, t = case["op"], case["tokens"]
    if op == "norm":
        s["x"] = _normal(gen, t, case["dim"]).mul_(3.0).to(DTYPES[case["stream"]])
        s["add"] = _normal(gen, t, case["dim"]).to(DTYPES[case["add"]]) if case["add"] else None
        s["gain"] = 1.0 + 0.2 * _normal(gen, case["dim"]) if case["gain"] else None
        return s
    if op == "mm":
        _table(case, gen, s)
        s["a"] = _blocks(_normal(gen, t, case["dim"]))
        return s
    if op == "rows":
        _table(case, gen, s)
        s["ids"] = torch.randint(0, case["rows"], (t,), generator=gen, device="cuda", dtype=torch.int32)
        return s
    # logits: a broad floor and a few likely tokens
    v = case["vocab"]
    x = _normal(gen, t, v).mul_(2.0)
    peaks = torch.randint(0, v, (t, 24), generator=gen, device="cuda")
    x.scatter_add_(1, peaks, 5.0 + 2.0 * _normal(gen, t, 24).abs())
    if case["masked"]:
        x.masked_fill_(torch.rand(t, v, generator=gen, device="cuda") < case["masked"], float("-inf"))
    if case["empty"]:
        x[max(0, t - case["empty"]):] = float("-inf")
    s["logits"] = x.to(DTYPES[case["dtype"]])
    s["u"] = torch.rand(t, generator=gen, device="cuda")

    def one_of(*values, dtype=torch.float32):
        return torch.tensor(values, device="cuda", dtype=dtype)[torch.randint(0, len(values), (t,), generator=gen, device="cuda")]

    mode = case["mode"]
    s["temperature"] = one_of(0.0, 0.6, 0.8, 1.0, 1.3) if mode == "all" else one_of(0.7, 1.0)
    s["top_k"] = one_of(0, 1, 20, 50, 1000, dtype=torch.int32) if mode == "all" else one_of(40, 64, dtype=torch.int32) if mode == "k" else None
    s["top_p"] = one_of(1.0, 0.9, 0.95) if mode == "all" else one_of(0.9, 0.95) if mode == "p" else None
    s["min_p"] = one_of(0.0, 0.02, 0.1) if mode == "all" else one_of(0.05, 0.1) if mode == "min" else None
    return s


# ---- the plain forms -------------------------------------------------------------------------------------------------

def _plain_norm(s):
    case, x = s["case"], s["x"]
    stream = x if s["add"] is None else (x.float() + s["add"].float()).to(x.dtype)
    # the mean of squares in 64 bits: an 8-bit step is a border that 32 bits would fall on either side of
    r = (1.0 / torch.sqrt(stream.double().square().mean(-1, keepdim=True) + 1e-6)).float()
    y = stream.float() * r
    if s["gain"] is not None:
        y = y * s["gain"]
    if case["out"] == "values":
        return y.to(x.dtype), stream
    b = y.view(case["tokens"], -1, 32)
    d = b.abs().amax(-1, keepdim=True) / 127.0
    z = b * torch.where(d > 0, 1.0 / d, 0.0)
    low = torch.floor(z.abs())
    q = torch.copysign(low + (z.abs() - low >= 0.5), z).clamp(-127, 127)  # halves away from zero
    return (q * d.half().float()).half(), stream


def _values(codes, scales, zeros):
    """What rows of 4-bit codes stand for, fp32 [rows, dim]."""
    b = codes.view(codes.shape[0], -1, 16)
    v = torch.cat((b & 15, b >> 4), -1).float()
    v = torch.where(v > 7, v - 16, v).view(codes.shape[0], scales.shape[1], -1)
    if zeros is not None:
        v = v - zeros.float().unsqueeze(-1)
    return (v * scales.float().unsqueeze(-1)).flatten(1)


def _plain_mm(s):
    case = s["case"]
    b = s["a"].view(case["tokens"], -1, 36)
    a = b[..., :32].contiguous().view(torch.int8).float() * b[..., 32:34].contiguous().view(torch.float16).float()
    return torch.matmul(a.view(case["tokens"], -1), _values(s["codes"], s["scales"], s["zeros"]).t())


def _plain_rows(s):
    ids = s["ids"].long()
    v = _values(s["codes"][ids], s["scales"][ids], None if s["zeros"] is None else s["zeros"][ids])
    return (v * _scale(s["case"])).to(DTYPES[s["case"]["dtype"]])


def _plain_sample(s):
    # weights and sums in 64 bits: a token is chosen by which side of a border a sum falls on
    x = s["logits"].double()
    t, v = x.shape
    top = x.amax(-1, keepdim=True)
    heat = s["temperature"].double().unsqueeze(1)
    w = torch.exp((x - torch.where(top == float("-inf"), 0.0, top)) / torch.where(heat > 0, heat, 1.0))
    order = torch.sort(s["logits"], dim=-1, descending=True, stable=True).indices  # equal ones by their place
    ws = w.gather(1, order)
    place = torch.arange(v, device=x.device).unsqueeze(0)
    keep = torch.ones_like(ws, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"].unsqueeze(1)
        keep &= (place < k) | (k <= 0)
    if s["top_p"] is not None:
        p = s["top_p"].double().unsqueeze(1)
        c = torch.cumsum(ws * keep, -1)
        keep &= (c - ws * keep < p * c[:, -1:]) | (p >= 1.0) | (place == 0)
    if s["min_p"] is not None:
        keep &= (ws >= s["min_p"].double().unsqueeze(1)) | (place == 0)
    keep &= (heat > 0) | (place == 0)
    ws = ws * keep
    c = torch.cumsum(ws, -1)
    total = c[:, -1:]
    hit = (c > s["u"].double().unsqueeze(1) * total) & (ws > 0)
    at = hit.to(torch.int8).argmax(-1, keepdim=True)  # the first of the sorted ones
    token = order.gather(1, at)
    none = total == 0
    logprob = torch.log(ws.gather(1, at)) - torch.log(total)
    return torch.where(none, -1, token).squeeze(1).to(torch.int32), torch.where(none, float("-inf"), logprob).squeeze(1).float()


def _scale(case):
    return case["dim"] ** 0.5


# ---- one pass ----------------------------------------------------------------------------------------------------------

def _own(s):
    import bit_quantized_mat_amd as bqm
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        if case["out"] == "values":
            return bqm.rms_norm(s["x"], s["gain"], add=s["add"])
        a, stream = bqm.rms_norm_q8_1(s["x"], s["gain"], add=s["add"])
        b = a.view(case["tokens"], -1, 36)
        return b[..., :32].view(torch.int8) * b[..., 32:34].view(torch.float16), stream
    if op == "sample":
        return bqm.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    m = bqm.Q4Matrix(s["codes"], s["scales"], s["zeros"])
    if op == "mm":
        return bqm.mm_q4(m, s["a"])
    return bqm.q4_dequantize(m, s["ids"], scale=_scale(case), dtype=DTYPES[case["dtype"]])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_norm(state) if op == "norm" else _plain_mm(state) if op == "mm" else _plain_rows(state) if op == "rows" else _plain_sample(state)


# ---- what a pass cannot do without ---------------------------------------------------------------------------------------

def work(case):
    op, t = case["op"], case["tokens"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if op == "norm":
        n, stream = t * case["dim"], size[case["stream"]]
        out = stream if case["out"] == "values" else 36 / 32
        add = size[case["add"]] + stream if case["add"] else 0  # the addend read, the sum written
        return {"bytes": n * (stream + add + out) + 4 * case["dim"] * case["gain"], "flops": 6 * n}
    if op == "sample":
        return {"bytes": t * (case["vocab"] * size[case["dtype"]] + 28), "flops": 4 * t * case["vocab"]}
    row = case["dim"] // 2 + case["dim"] // case["group"] * (3 if case["zeros"] else 2)
    if op == "mm":
        return {"bytes": case["rows"] * row + t * (case["dim"] // 32 * 36 + 4 * case["rows"]), "flops": 2 * t * case["rows"] * case["dim"]}
    distinct = case["rows"] * (1.0 - (1.0 - 1.0 / case["rows"]) ** t)  # rows drawn at least once
    return {"bytes": distinct * row + t * (4 + case["dim"] * size[case["dtype"]]), "flops": 2 * t * case["dim"]}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------------------

def _exact_matrix(s, rows):
    """Rows of the matrix, one nibble place at a time."""
    codes = s["codes"][rows].to(torch.int64)
    n, group = len(codes), s["case"]["group"]
    out = torch.empty(n, codes.shape[1] * 2, dtype=torch.float64, device="cuda")
    for i in range(16):
        for half in range(2):
            c = (codes[:, i::16] >> (4 * half)) & 15
            out[:, i + 16 * half::32] = (c - 16 * (c >= 8)).double()
    col = torch.arange(out.shape[1], device="cuda") // group
    if s["zeros"] is not None:
        out -= s["zeros"][rows].double()[:, col]
    return out * s["scales"][rows].double()[:, col]


def _exact_logprob(x, u, heat, k, p, floor):
    """Of one row of logits: log of the drawn token's share, by going down the sorted tokens."""
    x = x.double()
    x = x[torch.isfinite(x)]
    if not len(x):
        return float("-inf")
    if not heat > 0:
        return 0.0
    val = torch.sort(x, descending=True).values
    if k > 0:
        val = val[:k]
    w = torch.softmax(val / heat, 0)
    if p < 1.0:
        w = w[:int((torch.cumsum(w, 0) < p).sum()) + 1]
    w = w[w >= floor * w[0]]
    w = w / w.sum()
    i = int((torch.cumsum(w, 0) <= u).sum())
    return float(torch.log(w[min(i, len(w) - 1)]))


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        stream = s["x"].double() if s["add"] is None else s["x"].double() + s["add"].double()
        x = stream.to(s["x"].dtype).double()  # the norm is that of the stream as it is kept
        y = x / (x.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6) ** 0.5 * (1.0 if s["gain"] is None else s["gain"].double())
        if case["out"] == "q8":  # whole steps of a block's scale, which is kept in 16 bits
            y = y.unflatten(-1, (-1, 32))
            step = y.abs().amax(-1, keepdim=True) / 127.0
            y = torch.sign(y) * torch.floor(y.abs() / step.clamp(min=1e-300) + 0.5) * step.half().double()
        return y, stream
    if op == "rows":
        return _exact_matrix(s, s["ids"].long()) * _scale(case)
    if op == "mm":
        b = s["a"].cpu().numpy().reshape(case["tokens"], -1, 36)
        q = torch.from_numpy(b[:, :, :32].copy().view("int8")).double()
        d = torch.from_numpy(b[:, :, 32:34].copy().view("float16")).double()
        a = (q * d).flatten(1).cuda()
        out = torch.empty(case["tokens"], case["rows"], dtype=torch.float64, device="cuda")
        for at in range(0, case["rows"], 8192):
            w = _exact_matrix(s, torch.arange(at, min(at + 8192, case["rows"]), device="cuda"))
            out[:, at:at + 8192] = a @ w.t().contiguous()
        return out
    n = case["tokens"]
    heat, u = s["temperature"].tolist(), s["u"].tolist()
    k = [0] * n if s["top_k"] is None else s["top_k"].tolist()
    p = [1.0] * n if s["top_p"] is None else s["top_p"].tolist()
    m = [0.0] * n if s["min_p"] is None else s["min_p"].tolist()
    got = [_exact_logprob(s["logits"][i], u[i], heat[i], k[i], p[i], m[i]) for i in range(n)]
    return None, torch.tensor(got, dtype=torch.float64, device="cuda")
