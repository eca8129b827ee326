"""Timing cases of the operators that serve many requests from one model at once.

Four kinds of case, named by `op`:

  prefix    attention of one new token per sequence, where groups of sequences share the pages of a long prefix
  adapter   low-rank adapters of many requests at once, added to a shared projection's output
  logprobs  log probabilities of given tokens, entropy and top alternatives of rows of logits
  read      rows of the paged cache back as contiguous keys and values

`run` computes a case in plain torch operations in 32 bits, or through this package where `own` is set.
`exact` restates each definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a handful of requests behind a short system prompt: latency only
        {"name": "prefix 4 behind 512", "op": "prefix", "batch": 4, "prefixes": 1, "plen": 512, "lo": 1, "hi": 64, "hq": 16,
         "hkv": 4, "d": 64, "page": 16, "dtype": "fp16", "cache": "16"},
        # a serving batch behind one system prompt with its documents
        {"name": "prefix 64 behind 8192", "op": "prefix", "batch": 64, "prefixes": 1, "plen": 8192, "lo": 1, "hi": 512,
         "hq": 32, "hkv": 8, "d": 128, "page": 16, "dtype": "bf16", "cache": "16"},
        # three applications' prompts of uneven lengths in one batch, int8 rows, some requests without tokens of their own
        {"name": "prefix int8 96 behind 3", "op": "prefix", "batch": 96, "prefixes": 3, "plen": 6001, "lo": 0, "hi": 384,
         "hq": 32, "hkv": 8, "d": 128, "page": 32, "dtype": "bf16", "cache": "int8"},
        # many samples drawn from one long document: arithmetic, not bytes
        {"name": "prefix 256 behind 32768", "op": "prefix", "batch": 256, "prefixes": 1, "plen": 32768, "lo": 1, "hi": 256,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "dtype": "bf16", "cache": "16"},
        # one token of one request with an adapter: latency only
        {"name": "adapter 1x4096x4096", "op": "adapter", "rows": 1, "n": 4096, "k": 4096, "rank": 16, "adapters": 8,
         "order": "mixed", "dtype": "bf16", "out": "bf16"},
        # a serving batch over two dozen adapters, beside the widest projection of the linear layer's own workloads
        {"name": "adapter 48x28672x5376", "op": "adapter", "rows": 48, "n": 28672, "k": 5376, "rank": 32, "adapters": 24,
         "order": "mixed", "dtype": "bf16", "out": "bf16"},
        # prompts of several requests one after the other, each with its own adapter or none
        {"name": "adapter 8000x4096x4096", "op": "adapter", "rows": 8000, "n": 4096, "k": 4096, "rank": 64, "adapters": 6,
         "order": "runs", "dtype": "bf16", "out": "bf16"},
        # one sampled token, reported with its alternatives
        {"name": "logprobs 1x32000", "op": "logprobs", "rows": 1, "vocab": 32000, "top": 5, "masked": 0.0, "scale": 1.0,
         "dtype": "bf16"},
        # a serving batch of 32-bit logits over a large vocabulary, most of it forbidden by a grammar, at a temperature
        {"name": "logprobs 48x131071", "op": "logprobs", "rows": 48, "vocab": 131071, "top": 20, "masked": 0.6, "scale": 1.25,
         "dtype": "fp32"},
        # a prompt's tokens scored, one alternative each
        {"name": "logprobs 4096x64000", "op": "logprobs", "rows": 4096, "vocab": 64000, "top": 1, "masked": 0.0, "scale": 1.0,
         "dtype": "bf16"},
        # the cached tokens of one short conversation, before its next prompt
        {"name": "read 1x300", "op": "read", "batch": 1, "lo": 300, "hi": 300, "hkv": 8, "d": 128, "page": 16,
         "dtype": "bf16", "cache": "int8"},
        # a batch of cached conversations of every age, int8 rows
        {"name": "read int8 16x..8192", "op": "read", "batch": 16, "lo": 0, "hi": 8192, "hkv": 8, "d": 128, "page": 32,
         "dtype": "bf16", "cache": "int8"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "adapter", "adapter", "logprobs", "logprobs", "read"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "adapter":
        rows = _log_int(rng, 1, 8000)
        n, k = _log_int(rng, 8, 3584) * 8, _log_int(rng, 4, 336) * 16
        rank = rng.choice([8, 16, 24, 32, 64, 128])
        most = 8000 * (4096 + 4096) // (n + k)
        return {"op": op, "rows": max(1, min(rows, most)), "n": n, "k": k, "rank": min(rank, 64) if rows > 1000 else rank,
                "adapters": _log_int(rng, 1, 32), "order": "runs" if rows > 256 else rng.choice(["runs", "mixed"]),
                "dtype": dtype, "out": rng.choice([dtype, dtype, "fp32"])}
    if op == "logprobs":
        vocab = _log_int(rng, 1000, 262143)
        return {"op": op, "rows": min(_log_int(rng, 1, 4096), 4096 * 64000 // (2 * vocab)), "vocab": vocab,
                "top": rng.choice([0, 1, 5, 8, 20, 32]), "masked": rng.choice([0.0, 0.0, 0.6, 0.97]),
                "scale": rng.choice([1.0, 1.25, 0.7]), "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
    hq = hq if hq <= 64 else 32
    d = rng.choice([64, 128])
    page = rng.choice([16, 24, 32, 64])
    cache = rng.choice(["16", "int8"])
    if op == "read":
        batch = _log_int(rng, 1, 64)
        hi = min(_log_int(rng, 8, 8192), 16 * 8192 // batch)
        return {"op": op, "batch": batch, "lo": rng.choice([0, hi // 2, hi]), "hi": hi, "hkv": hkv,
                "d": rng.choice([64, 96, 128]), "page": page, "dtype": dtype, "cache": cache}
    batch = _log_int(rng, 1, 256)
    plen = min(_log_int(rng, 100, 32768), 256 * 32 * 32768 // (batch * hq))
    hi = min(_log_int(rng, 1, 2048), 65536 // batch)
    return {"op": op, "batch": batch, "prefixes": min(batch, rng.choice([1, 1, 2, 3, 5])), "plen": plen,
            "lo": rng.choice([0, 1, hi]), "hi": max(hi, 1), "hq": hq, "hkv": hkv, "d": d, "page": page, "dtype": dtype,
            "cache": cache}


def lengths(case):
    """The case's sequence lengths: lo..hi spread evenly and then mixed, the largest among them."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    even = [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]
    return [even[(i * 37 + 11) % b] if math.gcd(37, b) == 1 else even[i] for i in range(b)]


def groups(case):
    """(length, first sequence, end) of each prefix: the longest first, uneven groups, the last sequence of
    a batch with several prefixes behind none of them."""
    n, batch = case["prefixes"], case["batch"]
    last = batch - 1 if n > 1 and batch > n else batch
    cuts = [last * i * (i + 1) // (n * (n + 1)) for i in range(n + 1)]
    return [(max(1, case["plen"] * (n - i) // n), cuts[i], cuts[i + 1]) for i in range(n)]


def work(case):
    op = case["op"]
    if op == "adapter":
        m, n, k, r = case["rows"], case["n"], case["k"], case["rank"]
        index = _adapter_index(case)
        used, served = len(set(index) - {-1}), sum(i >= 0 for i in index)
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": used * 2 * r * (n + k) + 2 * served * k + 2 * out * m * n + 4 * m, "flops": 2 * served * r * (n + k)}
    if op == "logprobs":
        m, v = case["rows"], case["vocab"]
        return {"bytes": m * (v * (4 if case["dtype"] == "fp32" else 2) + 16 + 8 * case["top"]), "flops": 5 * m * v}
    hkv, d = case["hkv"], case["d"]
    row = (d + 4) if case["cache"] == "int8" else 2 * d
    lens = lengths(case)
    tables = 4 * sum(-(-n // case["page"]) for n in lens)
    if op == "read":
        return {"bytes": sum(lens) * 2 * hkv * (row + 2 * d) + tables, "flops": sum(lens) * 2 * hkv * d}
    shared = groups(case)
    keys = sum(lens) + sum(p for p, a, b in shared if b > a)
    pairs = sum(lens) + sum(p * (b - a) for p, a, b in shared)
    return {"bytes": keys * 2 * hkv * row + case["batch"] * case["hq"] * (4 * d + 4) + tables,
            "flops": 4 * pairs * case["hq"] * d}


# ------------------------------------------------------------------------------------ inputs
def _normal(gen, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def _adapter_index(case):
    """The adapter of each row, -1 for the rows without one (about one in eight)."""
    m, a = case["rows"], case["adapters"]
    if m == 1:
        return [a // 2]
    if case["order"] == "mixed":
        return [-1 if i % 8 == 5 else (i * 7 + i // 8) % a for i in range(m)]
    pieces = 8
    return [-1 if i * pieces // m == 5 else (i * pieces // m * 5 + 1) % a for i in range(m)]


def _tables(need, gen):
    """A block table [len(need), most] over a shuffled pool of pages, with a few pages nobody uses."""
    pool = torch.randperm(sum(need) + 7, generator=gen, device=DEV, dtype=torch.int32).cpu()
    table = torch.zeros((len(need), max(1, max(need))), dtype=torch.int32)
    for i, r in enumerate(torch.split(pool[:sum(need)], need)):
        table[i, :len(r)] = r
    return table, sum(need) + 7


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "adapter":
        m, n, k, r, a = case["rows"], case["n"], case["k"], case["rank"], case["adapters"]
        s["x"] = _normal(gen, m, k, dtype=dtype)
        s["a"] = _normal(gen, a, r, k, dtype=dtype, std=k ** -0.5)
        s["b"] = _normal(gen, a, n, r, dtype=dtype, std=0.5 * r ** -0.5)
        s["index"] = torch.tensor(_adapter_index(case), device=DEV, dtype=torch.int32)
        s["scaling"] = torch.rand(a, generator=gen, device=DEV) + 0.5
        s["base"] = _normal(gen, m, n, dtype=DTYPES[case["out"]])  # the shared projection's output
        return s
    if op == "logprobs":
        m, v = case["rows"], case["vocab"]
        x = _normal(gen, m, v, std=2.5)
        likely = torch.randint(0, v, (m, 4), generator=gen, device=DEV)
        x.scatter_add_(1, likely, torch.rand((m, 4), generator=gen, device=DEV) * 8 + 6)
        if case["masked"]:
            x.masked_fill_(torch.rand((m, v), generator=gen, device=DEV) < case["masked"], -math.inf)
            x.scatter_(1, likely[:, :1], 12.0)
        s["logits"] = x.to(dtype)
        token = likely[:, 0].clone()  # mostly what the model expects, now and then something else it allows
        if not case["masked"]:
            token[::3] = torch.randint(0, v, token[::3].shape, generator=gen, device=DEV)
        s["tokens"] = token.to(torch.int32)
        return s
    lens = lengths(case)
    hkv, d, page = case["hkv"], case["d"], case["page"]
    need = [-(-n // page) for n in lens]
    shared = groups(case) if op == "prefix" else []
    table, pages = _tables([-(-p // page) for p, _, _ in shared] + need, gen)
    n = len(shared)
    if op == "prefix":
        s["prefix_table"] = table[:n, :max(1, -(-case["plen"] // page))].contiguous().to(DEV)
        s["prefix_lens"] = torch.tensor([p for p, _, _ in shared], device=DEV, dtype=torch.int32)
        s["cu_prefix"] = torch.tensor([0] + [b for _, _, b in shared], device=DEV, dtype=torch.int32)
        s["q"] = _normal(gen, len(lens), case["hq"], d, dtype=dtype, std=1.5)
    else:
        s["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        s["total"] = sum(lens)
    s["block_table"] = table[n:, :max(1, max(need))].contiguous().to(DEV)
    s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    shape = (pages, hkv, page, d)
    for name in ("k", "v"):
        if case["cache"] == "int8":
            s[name] = torch.randint(-127, 128, shape, generator=gen, device=DEV, dtype=torch.int8)
            s[name + "_scale"] = torch.rand(shape[:3], generator=gen, device=DEV) * 0.02 + 0.005
        else:
            s[name] = _normal(gen, *shape, dtype=dtype)
    return s


# ------------------------------------------------------------------------------- plain forms
def _gathered(s, name, table):
    """fp32 [tables, kv_heads, pages * page, d]: the rows that a block table names."""
    x = s[name][table.long()].float()
    if s[name].dtype == torch.int8:
        x = x * s[name + "_scale"][table.long()][..., None]
    t, p, h, r, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(t, h, p * r, d)


def _plain_prefix(s):
    case = s["case"]
    hq, hkv, d, batch = case["hq"], case["hkv"], case["d"], case["batch"]
    q = s["q"].float().view(batch, hkv, hq // hkv, d)
    k, v = _gathered(s, "k", s["block_table"]), _gathered(s, "v", s["block_table"])
    mine = (q @ k.transpose(-1, -2)).mul_(d ** -0.5)
    seen = torch.arange(k.shape[2], device=DEV)[None] < s["lens"][:, None]
    mine.masked_fill_(~seen[:, None, None], -math.inf)
    out, lse = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, device=DEV)
    for i, (length, lo, hi) in enumerate(groups(case) + [(0, groups(case)[-1][2], batch)]):
        if hi == lo:
            continue
        both = mine[lo:hi]
        if length:
            pk, pv = (_gathered(s, name, s["prefix_table"][i:i + 1])[0, :, :length] for name in ("k", "v"))
            theirs = torch.einsum("bhgd,hnd->bhgn", q[lo:hi], pk).mul_(d ** -0.5)
            both = torch.cat([theirs, both], -1)
        top = both.amax(-1, keepdim=True).clamp_min(-3.0e38)
        e = both.sub_(top).exp_()
        total = e.sum(-1, keepdim=True)
        acc = e[..., length:] @ v[lo:hi]
        if length:
            acc += torch.einsum("bhgn,hnd->bhgd", e[..., :length], pv)
        out[lo:hi] = acc / total.clamp_min(1e-30)
        lse[lo:hi] = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
    return out.reshape(batch, hq, d).to(s["q"].dtype), lse.reshape(batch, hq)


def _plain_adapter(s):
    y = s["base"].float()
    for i in range(s["case"]["adapters"]):
        rows = (s["index"] == i).nonzero()[:, 0]
        if rows.numel():
            h = s["x"][rows].float() @ s["a"][i].float().t()
            y[rows] += (h @ s["b"][i].float().t()) * s["scaling"][i]
    return y.to(s["base"].dtype)


def _plain_logprobs(s):
    case = s["case"]
    x = s["logits"].float()
    top, first = x.max(-1, keepdim=True)
    t = (x - top) * case["scale"]  # relative to the largest, whose own 1 would swallow the rest of a sharp row's sum
    e = torch.exp(t)
    rest = e.scatter(1, first, 0.0).sum(-1)
    log_total = torch.log1p(rest)
    entropy = log_total - torch.where(e > 0, e * t, 0.0).sum(-1) / (1 + rest)
    logprob = t.gather(1, s["tokens"].long()[:, None])[:, 0] - log_total
    lse = top[:, 0] * case["scale"] + log_total
    if not case["top"]:
        return [logprob, entropy, lse]
    best, index = torch.sort(x, dim=-1, descending=True, stable=True)
    n = case["top"]
    return [logprob, entropy, lse, (best[:, :n] - top) * case["scale"] - log_total[:, None], index[:, :n].to(torch.int32)]


def _plain_read(s):
    page = s["case"]["page"]
    token = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(s["cu"][1:].long(), token, right=True)
    at = token - s["cu"][seq].long()
    pages, off = s["block_table"][seq, at // page].long(), at % page
    out = []
    for name in ("k", "v"):
        x = s[name][pages, :, off].float()
        if s[name].dtype == torch.int8:
            x = x * s[name + "_scale"][pages, :, off][..., None]
        out.append(x.to(DTYPES[s["case"]["dtype"]]))
    return out


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import int8_weight_quantized_gb300 as ck
        if op == "adapter":
            return ck.ck_adapter_linear(s["x"], s["a"], s["b"], s["index"], scaling=s["scaling"], residual=s["base"])
        if op == "logprobs":
            r = ck.ck_token_logprobs(s["logits"], s["tokens"], top=case["top"], scale=case["scale"])
            return [r.logprob, r.entropy, r.lse] + ([r.top, r.index] if case["top"] else [])
        cache = ck.KVCache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
        if op == "read":
            return ck.ck_cache_read(cache, s["block_table"], s["cu"], s["total"], dtype=DTYPES[case["dtype"]])
        return ck.ck_prefix_attention(s["q"], cache, s["prefix_table"], s["prefix_lens"], s["cu_prefix"], s["block_table"],
                                      s["lens"], return_lse=True)
    return {"prefix": _plain_prefix, "adapter": _plain_adapter, "logprobs": _plain_logprobs, "read": _plain_read}[op](s)


# ---------------------------------------------------------------------- definitions in 64 bits
def _exact_rows(s, name, head, table, n):
    """The first n cached rows of one head along one row of a block table, [n, d] in 64 bits."""
    at = torch.arange(n, device=DEV)
    page = s["case"]["page"]
    p, r = table[at // page].long(), at % page
    rows = s[name][p, head, r].double()
    return rows * s[name + "_scale"][p, head, r].double().unsqueeze(1) if name + "_scale" in s else rows


def _exact_prefix(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full((case["batch"], hq), -math.inf, dtype=torch.float64, device=DEV)
    lens = lengths(case)
    behind = {b: (i, p) for i, (p, lo, hi) in enumerate(groups(case)) for b in range(lo, hi)}
    for h in range(hkv):
        shared = {i: [_exact_rows(s, name, h, s["prefix_table"][i], p) for name in ("k", "v")]
                  for i, p in set(behind.values())}
        for b, n in enumerate(lens):
            k, v = (_exact_rows(s, name, h, s["block_table"][b], n) for name in ("k", "v"))
            heads = slice(h * g, (h + 1) * g)
            q = s["q"][b, heads].double() / math.sqrt(d)
            parts = [(q @ k.t(), v)]
            if b in behind:
                pk, pv = shared[behind[b][0]]
                parts.insert(0, (q @ pk.t(), pv))
            score = torch.cat([x for x, _ in parts], -1)
            if score.shape[-1] == 0:
                continue
            lse[b, heads] = torch.logsumexp(score, -1)
            weight = torch.softmax(score, -1)
            split = weight.split([x.shape[-1] for x, _ in parts], -1)
            out[b, heads] = sum(w @ y for w, (_, y) in zip(split, parts))
    return out, lse


def _exact_logprobs(s):
    case = s["case"]
    result = []
    for logits, token in zip(s["logits"].split(256), s["tokens"].split(256)):
        x = logits.double() * case["scale"]
        log_p = x - torch.logsumexp(x, -1, keepdim=True)
        p = log_p.exp()
        row = [log_p[torch.arange(len(token), device=DEV), token.long()], -torch.special.xlogy(p, p).sum(-1),
               torch.logsumexp(x, -1)]
        if case["top"]:
            place = torch.arange(x.shape[1], device=DEV)
            left, best, index = logits.double(), [], []
            for _ in range(case["top"]):
                high = left.max(-1, keepdim=True).values
                first = torch.where(left == high, place, x.shape[1]).min(-1).values
                index.append(first)
                best.append(log_p.gather(1, first[:, None])[:, 0])
                left = left.scatter(1, first[:, None], math.nan).nan_to_num(nan=-1e300, neginf=-1e299)
            row += [torch.stack(best, 1), torch.stack(index, 1).to(torch.int32)]
        result.append(row)
    return [torch.cat(parts) for parts in zip(*result)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefix":
        return _exact_prefix(s)
    if op == "logprobs":
        return _exact_logprobs(s)
    if op == "adapter":
        y = s["base"].double()
        which = s["index"].tolist()
        for i in sorted(set(which) - {-1}):
            at = torch.tensor([m for m, w in enumerate(which) if w == i], device=DEV)
            low = s["x"][at].double() @ s["a"][i].double().transpose(0, 1)
            y[at] = y[at] + s["scaling"][i].double() * (low @ s["b"][i].double().transpose(0, 1))
        return y
    out = [torch.zeros((s["total"], case["hkv"], case["d"]), dtype=torch.float64, device=DEV) for _ in range(2)]
    start = 0
    for b, n in enumerate(lengths(case)):
        for o, name in zip(out, ("k", "v")):
            for h in range(case["hkv"]):
                o[start:start + n, h] = _exact_rows(s, name, h, s["block_table"][b], n)
        start += n
    return out
