"""The paged-cache operators at the sizes they serve: appending rotated keys
and values to a page pool, attention over it with a sliding window and first
tokens that stay visible, and attention of a batch that shares a long prefix.

Each case runs one operator once. With `own` false the operator is computed in
its plain form (elementary torch operations in 32 bits, rounded once); with
`own` true by the calls of block_diffusion_drafter_pass_gb300.

The pool of a case is [n_pages, 2, n_kv, 64 * d]: per page of 64 tokens the
keys [n_kv][64][d], then the values transposed [n_kv][d][64].
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# (query heads, kv heads, head dim): the 8B drafter and target, the tiny
# drafter, and generic groups of 1, 2, 5, 7 and 8 heads.
HEADS = ((32, 8, 128), (4, 4, 64), (28, 4, 128), (28, 4, 64), (16, 2, 64), (8, 8, 128), (10, 2, 128), (16, 8, 64))


def listed():
    big = dict(dtype="bf16", heads=32, kv=8, dim=128)
    return [
        # A decoding step of a full serving batch: every sequence appends one token.
        dict(big, name="append decode 32", op="append", seqs=32, q_lo=1, q_hi=1, ctx_lo=64, ctx_hi=512),
        # One drafted block of 16 of the tiny model: pure call latency.
        dict(name="append block small", op="append", dtype="fp16", heads=4, kv=4, dim=64, seqs=1, q_lo=16, q_hi=16,
             ctx_lo=100, ctx_hi=100),
        # Prefill of eight prompts of uneven length, some behind cached tokens.
        dict(big, name="append prefill 8", op="append", seqs=8, q_lo=500, q_hi=2048, ctx_lo=700, ctx_hi=2300),
        # One user's decoding step in a model with windowed layers.
        dict(big, name="window decode 1", op="window", seqs=1, q_lo=1, q_hi=1, ctx_lo=8192, ctx_hi=8192, window=4096,
             sinks=4),
        # The verify pass of the serving batch (contexts 1024 to 8192, block 16), a layer that sees everything.
        dict(big, name="window verify 32", op="window", seqs=32, q_lo=16, q_hi=16, ctx_lo=1024, ctx_hi=8192, window=0,
             sinks=0),
        # The longest context of the benchmark, one block of 16.
        dict(big, name="window long 1", op="window", seqs=1, q_lo=16, q_hi=16, ctx_lo=262144, ctx_hi=262144, window=0,
             sinks=0),
        # Prefill through a windowed layer, uneven prompts.
        dict(big, name="window prefill 3", op="window", seqs=3, q_lo=1200, q_hi=4096, ctx_lo=2000, ctx_hi=6000,
             window=2048, sinks=64),
        # A mixed step: short blocks of uneven length over uneven contexts, groups of 7 heads, half precision.
        dict(name="window mixed 48", op="window", dtype="fp16", heads=28, kv=4, dim=64, seqs=48, q_lo=1, q_hi=7,
             ctx_lo=1, ctx_hi=2500, window=512, sinks=16),
        # A handful of requests on a short common prompt, tiny model.
        dict(name="shared decode small", op="shared", dtype="bf16", heads=4, kv=4, dim=64, seqs=6, q_lo=1, q_hi=1,
             ctx_lo=1, ctx_hi=100, prefix=300),
        # Decoding of 64 users behind one long document.
        dict(big, name="shared decode 64", op="shared", seqs=64, q_lo=1, q_hi=1, ctx_lo=1, ctx_hi=1024, prefix=32768),
        # The verify pass of 32 users behind one long document, block 16.
        dict(big, name="shared verify 32", op="shared", seqs=32, q_lo=16, q_hi=16, ctx_lo=16, ctx_hi=512,
             prefix=32768),
        # Uneven blocks behind a prompt of odd length, groups of 7 heads, half precision.
        dict(name="shared mixed 24", op="shared", dtype="fp16", heads=28, kv=4, dim=128, seqs=24, q_lo=1, q_hi=33,
             ctx_lo=20, ctx_hi=1900, prefix=5003),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = [max(work(c)["bytes"], work(c)["flops"] / 250) for c in listed()]
    while True:
        heads, kv, dim = rng.choice(HEADS)
        case = dict(op=rng.choice(("append", "window", "window", "shared", "shared")), dtype=rng.choice(("bf16", "bf16", "fp16")),
                    heads=heads, kv=kv, dim=dim, seqs=log(1, 64))
        block = rng.random() < 0.7
        if case["op"] == "append":
            case["q_hi"] = log(1, 32) if block else log(32, 4096)
            case["ctx_hi"] = case["q_hi"] + log(1, 2000)
        elif case["op"] == "window":
            case["q_hi"] = log(1, 32) if block else log(32, 4096)
            case["ctx_hi"] = case["q_hi"] + log(1, 131072 if block else 8192)
            case["window"] = 0 if rng.random() < 0.3 else log(16, 8192)
            case["sinks"] = 0 if case["window"] == 0 or rng.random() < 0.3 else log(1, 256)
        else:
            case["q_hi"] = log(1, 32) if block else log(32, 512)
            case["ctx_hi"] = case["q_hi"] + log(1, 4096)
            case["prefix"] = log(64, 65536)
        case["q_lo"] = rng.choice((1, case["q_hi"], (case["q_hi"] + 1) // 2))
        case["ctx_lo"] = rng.choice((case["q_lo"], case["ctx_hi"], (case["ctx_hi"] + 1) // 2))
        w = work(case)
        # the padded scores of the plain form and the pool, in values
        scores = case["seqs"] * case["q_hi"] * case["heads"] * (case["ctx_hi"] + case.get("prefix", 0))
        pool = (case["seqs"] * case["ctx_hi"] + case.get("prefix", 0)) * case["kv"] * case["dim"]
        if max(w["bytes"], w["flops"] / 250) <= max(most) and scores <= 3e9 and pool <= 4e8:
            return case


def _spread(lo, hi, n, k):
    """n lengths spread over [lo, hi], uneven and without a pattern of a power of two."""
    if n == 1:
        return np.array([hi], dtype=np.int64)
    f = np.modf((np.arange(n) + 1) * 0.6180339887498949 + 0.37 * k)[0]
    return lo + np.floor(f * (hi - lo + 1)).astype(np.int64)


def _lengths(case):
    """Per sequence: new tokens, and cached tokens with the new ones among them."""
    q = _spread(case["q_lo"], case["q_hi"], case["seqs"], 0)
    kv = np.maximum(_spread(case["ctx_lo"], case["ctx_hi"], case["seqs"], 1), q)
    return q, kv


def _seen(case, q, kv):
    """Of one sequence: (row, key) pairs that count, and keys that some row sees, in its own cache."""
    pos = kv - q + np.arange(q, dtype=np.int64)
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    lo = np.maximum(0, pos - window + 1) if window else np.zeros_like(pos)
    pairs = int((pos + 1 - lo + np.minimum(lo, sinks)).sum())
    return pairs, int(kv - lo[0] + min(lo[0], sinks))


def work(case):
    q, kv = _lengths(case)
    T, h, n, d, es = int(q.sum()), case["heads"], case["kv"], case["dim"], 2
    ints = 4 * (2 * len(q) + 1)
    if case["op"] == "append":
        # q, k and v read, q and the cache written; a rotation is 3 operations a value
        return {"bytes": 2 * T * (h + 2 * n) * d * es + ints, "flops": 3 * T * (h + n) * d}
    prefix = case.get("prefix", 0)
    seen = [_seen(case, int(a), int(b)) for a, b in zip(q, kv)]
    pairs = sum(p for p, _ in seen) + T * prefix
    keys = sum(k for _, k in seen) + prefix
    return {"bytes": 2 * T * h * d * es + 2 * keys * n * d * es + ints, "flops": 4 * pairs * h * d}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, dev = TYPES[case["dtype"]], "cuda"
    q, kv = _lengths(case)
    T, h, n, d, prefix = int(q.sum()), case["heads"], case["kv"], case["dim"], case.get("prefix", 0)

    def normal(*size):
        return torch.randn(size, generator=g, device=dev, dtype=torch.float32).to(dt)

    pages = (kv + PAGE - 1) // PAGE
    stride, p_pages = int(pages.max()), (prefix + PAGE - 1) // PAGE
    total = int(pages.sum()) + p_pages
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(q), stride, dtype=torch.int32, device=dev)
    ends = np.concatenate([[0], np.cumsum(pages)])
    rows, cols = np.nonzero(np.arange(stride)[None, :] < pages[:, None])
    table[torch.from_numpy(rows).to(dev), torch.from_numpy(cols).to(dev)] = order[torch.from_numpy(ends[rows] + cols).to(dev)]
    s = dict(case, T=T, q_max=int(q.max()), table=table,
             q_start=torch.from_numpy(np.concatenate([[0], np.cumsum(q)]).astype(np.int32)).to(dev),
             kv_len=torch.from_numpy(kv.astype(np.int32)).to(dev),
             pool=torch.empty(total, 2, n, PAGE * d, dtype=dt, device=dev))
    for i in range(0, total, 4096):   # the pages hold a model's normed keys and values; slots past a length hold older tokens
        s["pool"][i:i + 4096] = normal(*s["pool"][i:i + 4096].shape)
    if case["op"] == "append":
        # the new rows are the column ranges of one projection's output
        qkv = normal(T, (h + 2 * n) * d)
        s["q"] = qkv[:, :h * d].view(T, h, d)
        s["k"] = qkv[:, h * d:(h + n) * d].view(T, n, d)
        s["v"] = qkv[:, (h + n) * d:].view(T, n, d)
        s["base"] = 1.0e6 if d == 128 else 1.0e4
    else:
        s["q"] = normal(T, h, d) * 1.5   # scores of standard deviation 1.5
    if prefix:
        s["prefix_table"] = order[total - p_pages:].contiguous()
    return s


def run(s):
    if own:
        import block_diffusion_drafter_pass_gb300 as dfl
        if s["op"] == "append":
            q = dfl.dflash_kv_append(s["pool"], s["k"], s["v"], s["q_start"], s["kv_len"], s["table"], q=s["q"],
                                     rope_base=s["base"])
            return q, s["pool"]
        if s["op"] == "window":
            return dfl.dflash_paged_attn(s["q"], s["pool"], s["q_start"], s["kv_len"], s["table"], window=s["window"],
                                         sinks=s["sinks"])
        return dfl.dflash_shared_prefix_attn(s["q"], s["pool"], s["q_start"], s["kv_len"], s["table"],
                                             s["prefix_table"], s["prefix"])
    return {"append": _append, "window": _window, "shared": _shared}[s["op"]](s)


def _tokens(s):
    """Of every token: its sequence and its place among the sequence's new tokens."""
    t = torch.arange(s["T"], device="cuda")
    seq = torch.searchsorted(s["q_start"].long(), t, right=True) - 1
    return seq, t - s["q_start"].long()[seq]


def _append(s):
    d, half = s["dim"], s["dim"] // 2
    seq, j = _tokens(s)
    start = s["q_start"].long()
    pos = s["kv_len"].long()[seq] - (start[1:] - start[:-1])[seq] + j
    # angles in 64 bits: at far positions 32 bits lose the fraction of a turn
    theta = torch.pow(torch.tensor(s["base"], dtype=torch.float64, device="cuda"),
                      -torch.arange(half, dtype=torch.float64, device="cuda") * 2 / d)
    angle = pos.double()[:, None] * theta
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotated(x):
        a, b = x.float()[..., :half], x.float()[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1).to(x.dtype)

    page, slot = s["table"].long()[seq, pos // PAGE], pos % PAGE
    pool = s["pool"]
    keys = pool[:, 0].view(-1, s["kv"], PAGE, d)
    values = pool[:, 1].view(-1, s["kv"], d, PAGE)
    keys[page, :, slot] = rotated(s["k"])
    values[page, :, :, slot] = s["v"]
    return rotated(s["q"]), pool


def _pages(s, table):
    """Keys [..., n_kv, tokens, d] and values, in 32 bits, of the pages of `table` [..., pages]."""
    pool, n, d = s["pool"], s["kv"], s["dim"]
    t = table.long()
    k = pool[:, 0].view(-1, n, PAGE, d)[t].float().movedim(-4, -3).flatten(-3, -2)
    v = pool[:, 1].view(-1, n, d, PAGE)[t].float().movedim(-4, -3).transpose(-1, -2).flatten(-3, -2)
    return k, v


def _padded(s):
    """Queries [seqs, n_kv, group * q_max, d] in 32 bits, padded to the longest block, and their positions."""
    n, g, d = s["kv"], s["heads"] // s["kv"], s["dim"]
    start, j = s["q_start"].long(), torch.arange(s["q_max"], device="cuda")
    at = (start[:-1, None] + j).clamp(max=s["T"] - 1)
    q = s["q"].float()[at].view(len(at), s["q_max"], n, g, d).permute(0, 2, 3, 1, 4).reshape(len(at), n, -1, d)
    return q, (s["kv_len"].long() - (start[1:] - start[:-1]))[:, None] + j


def _rows(s, out):
    """[seqs, n_kv, group * q_max, d] -> [T, heads, d] in the queries' type."""
    seq, j = _tokens(s)
    g = s["heads"] // s["kv"]
    out = out.view(out.shape[0], s["kv"] * g, s["q_max"], s["dim"])
    return out[seq, :, j].to(s["q"].dtype)


def _visible(s, pos, keys):
    """[seqs, q_max, keys]: which keys of its own cache a row sees."""
    key = torch.arange(keys, device="cuda")
    see = (key <= pos[..., None]) & (key < s["kv_len"].long()[:, None, None])
    if s.get("window"):
        see &= (key > pos[..., None] - s["window"]) | (key < s["sinks"])
    return see


def _masked(s, q, k, see):
    """Scores in 32 bits, -inf where a row does not see the key."""
    g = s["heads"] // s["kv"]
    scores = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(s["dim"]))
    scores = scores.view(*scores.shape[:-2], g, s["q_max"], scores.shape[-1])
    return scores.masked_fill_(~see[:, None, None], float("-inf")).flatten(-3, -2)


def _softmax(scores):
    top = scores.amax(dim=-1, keepdim=True)
    p = scores.sub_(torch.where(top == float("-inf"), torch.zeros_like(top), top)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    return p, torch.where(total > 0, total, torch.ones_like(total))


def _window(s):
    k, v = _pages(s, s["table"])
    q, pos = _padded(s)
    p, total = _softmax(_masked(s, q, k, _visible(s, pos, k.shape[-2])))
    return _rows(s, torch.matmul(p, v) / total)


def _shared(s):
    kp, vp = _pages(s, s["prefix_table"])
    kp, vp = kp[:, :s["prefix"]], vp[:, :s["prefix"]]
    k, v = _pages(s, s["table"])
    q, pos = _padded(s)
    seqs, n, rows, d = q.shape
    flat = q.transpose(0, 1).reshape(n, seqs * rows, d)   # every row of the batch against the one prefix
    first = torch.matmul(flat, kp.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(n, seqs, rows, -1).transpose(0, 1)
    scores = torch.cat([first, _masked(s, q, k, _visible(s, pos, k.shape[-2]))], dim=-1)
    del first
    p, total = _softmax(scores)
    behind = torch.matmul(p[..., :s["prefix"]].transpose(0, 1).reshape(n, seqs * rows, -1), vp)
    out = torch.matmul(p[..., s["prefix"]:], v) + behind.view(n, seqs, rows, d).transpose(0, 1)
    return _rows(s, out / total)


def exact(case, seed):
    """The definition in 64 bits, one sequence at a time."""
    s = prepare(case, seed)
    n, g, d = case["kv"], case["heads"] // case["kv"], case["dim"]
    start, lens, pool = s["q_start"].tolist(), s["kv_len"].tolist(), s["pool"]
    if case["op"] == "append":
        out, q = pool.double(), s["q"].double()
        turn = torch.tensor([s["base"] ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device="cuda")
        for i, total in enumerate(lens):
            a, b = start[i], start[i + 1]
            where = torch.arange(total - (b - a), total, device="cuda")
            z = torch.polar(torch.ones(b - a, d // 2, dtype=torch.float64, device="cuda"), where.double()[:, None] * turn)

            def spin(x):
                w = torch.complex(x[..., :d // 2].double(), x[..., d // 2:].double()) * z[:, None]
                return torch.cat([w.real, w.imag], dim=-1)

            q[a:b] = spin(s["q"][a:b])
            page = s["table"][i].long()[where // PAGE]
            kv = out.view(-1, 2, n, PAGE * d)
            lane = torch.arange(d, device="cuda")
            head = torch.arange(n, device="cuda")[None, :, None]
            slot = (where % PAGE)[:, None, None]
            kv[page[:, None, None], 0, head, slot * d + lane] = spin(s["k"][a:b])
            kv[page[:, None, None], 1, head, lane * PAGE + slot] = s["v"][a:b].double()
        return q, out
    result = torch.zeros(s["T"], n * g, d, dtype=torch.float64, device="cuda")

    def cached(table, count):
        need = table[:(count + PAGE - 1) // PAGE].long()
        k = pool[need, 0].view(-1, n, PAGE, d).permute(1, 0, 2, 3).reshape(n, -1, d)[:, :count]
        v = pool[need, 1].view(-1, n, d, PAGE).permute(1, 0, 3, 2).reshape(n, -1, d)[:, :count]
        return k, v

    prefix = case.get("prefix", 0)
    if prefix:
        kp, vp = cached(s["prefix_table"], prefix)
    for i, total in enumerate(lens):
        a, b = start[i], start[i + 1]
        k, v = cached(s["table"][i], total)
        if prefix:
            k, v = torch.cat([kp, k], dim=1), torch.cat([vp, v], dim=1)
        at = torch.arange(prefix + total - (b - a), prefix + total, device="cuda")[:, None]
        key = torch.arange(prefix + total, device="cuda")[None]
        hidden = key > at
        if case.get("window"):
            hidden = hidden | ((at - key >= case["window"]) & (key >= case["sinks"]))
        for h in range(n * g):
            x = s["q"][a:b, h].double() @ k[h // g].double().T / math.sqrt(d)
            x = torch.softmax(x.masked_fill(hidden, float("-inf")), dim=-1)
            result[a:b, h] = x @ v[h // g].double()
    return result
