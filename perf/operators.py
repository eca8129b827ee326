"""Timing cases of the transformer operators that stand between the quantized linear layers.

Five kinds of case, named by `op`:

  norm_rope    per-head RMS norm of queries and keys, rotary position, keys and values into the paged cache
  decode       attention of one new token per sequence over the paged cache
  decode_step  the two together, on a cache of int8 codes
  int4         a linear layer with 4-bit weights and group scales, for few rows
  prompt       attention over whole prompts, causal or not, with a sliding window and first tokens that stay visible

`run` computes a case in plain torch operations in 32 bits, or through this package where `own` is set.
`exact` restates each definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest call of a decode loop: one sequence's new token
        {"name": "rope 1 token", "op": "norm_rope", "tokens": 1, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "dtype": "bf16", "page": 16, "keep_k": False},
        # a prompt on its way into the cache, its keys also kept contiguous for the prompt's attention
        {"name": "rope 8192 tokens", "op": "norm_rope", "tokens": 8192, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "dtype": "bf16", "page": 16, "keep_k": True},
        # one user early in a conversation: latency only
        {"name": "decode 1x274", "op": "decode", "batch": 1, "lo": 274, "hi": 274, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "window": 0, "sinks": 0, "dtype": "bf16", "cache": "16"},
        # a serving batch of conversations of every age, one of them empty
        {"name": "decode 64x0..8192", "op": "decode", "batch": 64, "lo": 0, "hi": 8192, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "window": 0, "sinks": 0, "dtype": "bf16", "cache": "16"},
        # one long document: the length has to be split to fill the GPU
        {"name": "decode 1x131071", "op": "decode", "batch": 1, "lo": 131071, "hi": 131071, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16", "cache": "16"},
        # a batch's whole attention step on an int8 cache: rotate, quantize, append, attend
        {"name": "step int8 32x..16384", "op": "decode_step", "batch": 32, "lo": 1025, "hi": 16384, "hq": 32, "hkv": 8,
         "d": 128, "rot": 128, "interleaved": False, "page": 32, "window": 0, "sinks": 0, "dtype": "bf16"},
        # one token through a square projection
        {"name": "int4 1x4096x4096", "op": "int4", "rows": 1, "n": 4096, "k": 4096, "group": 128, "bias": False,
         "dtype": "bf16"},
        # one token through the widest projection of the linear layer's own workloads
        {"name": "int4 1x28672x5376", "op": "int4", "rows": 1, "n": 28672, "k": 5376, "group": 128, "bias": False,
         "dtype": "bf16"},
        # a small serving batch through a feed-forward projection, finer groups, with bias
        {"name": "int4 16x16384x4096", "op": "int4", "rows": 16, "n": 16384, "k": 4096, "group": 64, "bias": True,
         "dtype": "fp16"},
        # short prompts of ragged lengths batched together
        {"name": "prompt ragged 6x..700", "op": "prompt", "batch": 6, "lo": 1, "hi": 700, "hq": 16, "hkv": 4, "d": 64,
         "causal": True, "window": 128, "sinks": 4, "dtype": "fp16"},
        # a long prompt, every key up to the query
        {"name": "prompt 1x16384", "op": "prompt", "batch": 1, "lo": 16384, "hi": 16384, "hq": 16, "hkv": 4, "d": 128,
         "causal": True, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a long prompt through a layer with a window and four first tokens that stay visible
        {"name": "prompt 1x16000 window", "op": "prompt", "batch": 1, "lo": 16000, "hi": 16000, "hq": 16, "hkv": 2,
         "d": 128, "causal": True, "window": 1024, "sinks": 4, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "decode", "decode", "decode_step", "int4", "int4", "prompt", "prompt"])
    dtype = rng.choice(["bf16", "fp16"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
    hq = hq if hq <= 64 else 32
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64])
    if op == "norm_rope":
        d = rng.choice([64, 96, 128, 256])
        return {"op": op, "tokens": min(_log_int(rng, 1, 8192), (8192 * 48 * 128) // ((hq + 2 * hkv) * d)), "hq": hq,
                "hkv": hkv, "d": d, "rot": rng.choice([d, d // 2]), "interleaved": rng.random() < 0.5,
                "dtype": dtype, "page": page, "keep_k": rng.random() < 0.5}
    if op == "int4":
        group = rng.choice([32, 64, 128])
        n, k = _log_int(rng, 64, 3584) * 8, _log_int(rng, 2, 42) * 128
        return {"op": op, "rows": _log_int(rng, 1, 32), "n": n, "k": k, "group": group, "bias": rng.random() < 0.5,
                "dtype": dtype}
    windowed = rng.random() < 0.4
    window, sinks = (_log_int(rng, 16, 2048), rng.choice([0, 1, 4, 5])) if windowed else (0, 0)
    if op == "prompt":
        causal = windowed or rng.random() < 0.6
        hi = _log_int(rng, 16, 6000)
        batch = min(_log_int(rng, 1, 8), max(1, 8000 // hi))
        return {"op": op, "batch": batch, "lo": 1 if batch > 1 else hi, "hi": hi, "hq": min(hq, 16),
                "hkv": hkv if min(hq, 16) % hkv == 0 else 1, "d": d, "causal": causal, "window": window,
                "sinks": sinks, "dtype": dtype}
    batch = _log_int(rng, 1, 96)
    hi = min(_log_int(rng, 16, 65536), 260000 // (batch * hkv) * 8 // (d // 64))
    lo = rng.choice([1, max(1, hi // 2), hi])
    case = {"op": op, "batch": batch, "lo": lo, "hi": max(lo, hi), "hq": hq, "hkv": hkv, "d": d, "page": page,
            "window": window, "sinks": sinks, "dtype": dtype}
    if op == "decode":
        case["cache"] = rng.choice(["16", "int8"])
    else:
        case.update(rot=d, interleaved=rng.random() < 0.5)
    return case


def lengths(case):
    """The case's sequence lengths: lo..hi spread evenly and then mixed, the largest among them."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    even = [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]
    return [even[(i * 37 + 11) % b] if math.gcd(37, b) == 1 else even[i] for i in range(b)]


def visible_keys(length, case):
    """Keys that the last of `length` tokens sees."""
    if not case["window"] or length <= case["window"]:
        return length
    return case["window"] + min(case["sinks"], length - case["window"])


def work(case):
    op = case["op"]
    if op == "int4":
        m, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": n * k / 2 + 2 * n * k / case["group"] + 2 * m * (n + k) + (2 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "norm_rope":
        t = case["tokens"]
        copies = (hq + 2 * hkv) * 2 + (hkv if case["keep_k"] else 0)
        return {"bytes": t * (2 * d * copies + 4 * case["rot"] + 12) + 4 * d, "flops": t * (hq + hkv) * (4 * d + 3 * case["rot"])}
    lens = lengths(case)
    if op == "prompt":
        pairs = sum(sum(visible_keys(i + 1, case) for i in range(n)) if case["causal"] else n * n for n in lens)
        return {"bytes": 2 * sum(lens) * d * (2 * hq + 2 * hkv) + 4 * sum(lens) * hq, "flops": 4 * pairs * hq * d}
    keys = sum(visible_keys(n, case) for n in lens)
    per_key = 2 * hkv * ((d + 4) if op == "decode_step" or case["cache"] == "int8" else 2 * d)
    small = 2 * 2 * case["batch"] * hq * d + 4 * sum(-(-n // case["page"]) for n in lens)
    if op == "decode_step":
        small += case["batch"] * (2 * d * (hq + 2 * hkv) + 4 * case["rot"])
    return {"bytes": keys * per_key + small, "flops": 4 * keys * hq * d}


# ------------------------------------------------------------------------------------ inputs
def _normal(gen, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def _rope_table(positions, rot):
    """fp32 [positions, rot]: the cosines of a position's rot/2 angles, then their sines."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    angle = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _pages(case, gen, lens):
    """A block table over a shuffled pool of pages, with a few pages nobody uses."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    pool = torch.randperm(sum(need) + 7, generator=gen, device=DEV, dtype=torch.int32)
    width = max(1, max(need))
    table = torch.zeros((len(lens), width), dtype=torch.int32)
    rows = torch.split(pool[:sum(need)].cpu(), need)
    for i, r in enumerate(rows):
        table[i, :len(r)] = r
    return table.to(DEV), sum(need) + 7


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "int4":
        m, n, k, group = case["rows"], case["n"], case["k"], case["group"]
        s["x"] = _normal(gen, m, k, dtype=dtype)
        codes = _normal(gen, n, k, std=2.5).round_().clamp_(-7, 7).to(torch.int32).add_(8).view(n, k // 8, 4, 2)
        shift = torch.arange(0, 16, 4, device=DEV, dtype=torch.int32)[:, None] + torch.tensor([0, 16], device=DEV, dtype=torch.int32)
        s["w4"] = (codes << shift).sum((2, 3)).to(torch.int32)  # 8 codes a word: even k in the low half, odd k in the high
        s["w_scale"] = (torch.rand((n, k // group), generator=gen, device=DEV) * 0.01 + 0.002).to(torch.bfloat16)
        s["bias"] = _normal(gen, n, dtype=dtype, std=0.02) if case["bias"] else None
        return s
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "prompt":
        lens = lengths(case)
        t = sum(lens)
        s["q"], s["k"] = _normal(gen, t, hq, d, dtype=dtype, std=1.5), _normal(gen, t, hkv, d, dtype=dtype)
        s["v"] = _normal(gen, t, hkv, d, dtype=dtype)
        s["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        return s
    if op == "norm_rope":
        t, page = case["tokens"], case["page"]
        pages = -(-t // page) + 3
        s["positions"] = torch.arange(t, device=DEV, dtype=torch.int32) + 5
        table = torch.randperm(pages, generator=gen, device=DEV)
        i = torch.arange(t, device=DEV)
        s["slots"] = table[i // page] * page + i % page
        s["table"] = _rope_table(t + 5, case["rot"])
    else:
        lens = lengths(case)
        t, page = len(lens), case["page"]
        s["block_table"], pages = _pages(case, gen, lens)
        s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    int8 = op == "decode_step" or case.get("cache") == "int8"
    shape = (pages, hkv, page, d)
    if int8:
        for name in ("k", "v"):
            s[name] = torch.randint(-127, 128, shape, generator=gen, device=DEV, dtype=torch.int8)
            s[name + "_scale"] = torch.rand(shape[:3], generator=gen, device=DEV) * 0.02 + 0.005
    else:
        s["k"], s["v"] = _normal(gen, *shape, dtype=dtype), _normal(gen, *shape, dtype=dtype)
    if op == "decode":
        s["q"] = _normal(gen, t, hq, d, dtype=dtype, std=1.5)
    else:
        s["qkv"] = _normal(gen, t, (hq + 2 * hkv) * d, dtype=dtype)
        s["q_weight"] = (1 + _normal(gen, d, std=0.1)).to(dtype)
        s["k_weight"] = (1 + _normal(gen, d, std=0.1)).to(dtype)
    if op == "decode_step":
        last = s["lens"].long() - 1
        s["positions"] = last.to(torch.int32)
        s["slots"] = s["block_table"].long().gather(1, (last // page)[:, None])[:, 0] * page + last % page
        s["table"] = _rope_table(max(lens), case["rot"])
    return s


# ------------------------------------------------------------------------------- plain forms
EPS = 1e-6


def _plain_rotate(x, weight, s):
    """Norm and rotation of x [T, H, D], in 32 bits."""
    case = s["case"]
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    rot = case["rot"]
    cos, sin = s["table"][s["positions"].long()][:, None].split(rot // 2, -1)
    head, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, rest], -1)


def _plain_qkv(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    x = s["qkv"].view(-1, hq + 2 * hkv, d)
    q = _plain_rotate(x[:, :hq], s["q_weight"], s)
    k = _plain_rotate(x[:, hq:hq + hkv], s["k_weight"], s)
    return q, k, x[:, hq + hkv:].float()


def _plain_quantize(x):
    scale = x.abs().amax(-1) / 127
    codes = (x / scale.clamp_min(1e-38)[..., None]).round().clamp(-127, 127)
    return codes.to(torch.int8), scale


def _written(s):
    page = s["case"]["page"]
    return s["slots"] // page, s["slots"] % page


def _stored(s):
    """The values that the written rows of an int8 cache stand for, in the queries' type."""
    at, off = _written(s)
    dtype = s["qkv"].dtype
    return [(s[n][at, :, off].float() * s[n + "_scale"][at, :, off][..., None]).to(dtype) for n in ("k", "v")]


def _plain_decode(q, s):
    """q [B, Hq, D] fp32 against the paged cache."""
    case = s["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    table = s["block_table"].long()
    b, n = table.shape[0], table.shape[1] * page

    def gathered(name):
        x = s[name][table].float()
        if s[name].dtype == torch.int8:
            x = x * s[name + "_scale"][table][..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(b, hkv, n, d)

    lens = s["lens"].long()[:, None]
    j = torch.arange(n, device=DEV)[None]
    seen = j < lens
    if case["window"]:
        seen = seen & ((j >= lens - case["window"]) | (j < case["sinks"]))
    seen = seen[:, None, None]
    score = q.view(b, hkv, hq // hkv, d) @ gathered("k").transpose(-1, -2) * d ** -0.5
    score = score.masked_fill(~seen, -3.0e38)
    e = torch.exp(score - score.amax(-1, keepdim=True)) * seen
    total = e.sum(-1, keepdim=True)
    out = (e @ gathered("v")) / total.clamp_min(1e-30)
    return out.reshape(b, hq, d)


def _plain_int4(s):
    case, x, w4 = s["case"], s["x"], s["w4"]
    shift = torch.arange(0, 16, 4, device=DEV, dtype=torch.int32)[:, None] + torch.tensor([0, 16], device=DEV, dtype=torch.int32)
    codes = ((w4[:, :, None, None] >> shift) & 15) - 8
    w = codes.reshape(case["n"], -1, case["group"]).float() * s["w_scale"].float()[..., None]
    y = x.float() @ w.reshape(case["n"], case["k"]).t()
    return (y if s["bias"] is None else y + s["bias"].float()).to(x.dtype)


def _plain_prompt(s):
    case, cu = s["case"], s["cu"].long()
    hq, hkv = case["hq"], case["hkv"]
    t = s["q"].shape[0]
    i = torch.arange(t, device=DEV)
    seq = torch.searchsorted(cu[1:], i, right=True)
    seen = seq[:, None] == seq[None]
    if case["causal"]:
        at = i - cu[seq]
        seen &= i[None] <= i[:, None]
        if case["window"]:
            seen &= (i[:, None] - i[None] < case["window"]) | (at[None] < case["sinks"])
    q = s["q"].float().transpose(0, 1).reshape(hkv, hq // hkv, t, -1)
    k, v = s["k"].float().transpose(0, 1)[:, None], s["v"].float().transpose(0, 1)[:, None]
    score = (q @ k.transpose(-1, -2)).mul_(case["d"] ** -0.5)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    out = (e @ v) / total
    lse = (top + total.log()).reshape(hq, t)
    return out.reshape(hq, t, -1).transpose(0, 1).to(s["q"].dtype).contiguous(), lse


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import int8_weight_quantized_gb300 as ck
        if op == "int4":
            return ck.ck_int4_linear(s["x"], s["w4"], s["w_scale"], bias=s["bias"])
        if op == "prompt":
            return ck.ck_attention(s["q"], s["k"], s["v"], s["cu"], causal=case["causal"], window=case["window"],
                                   sinks=case["sinks"], return_lse=True)
        cache = ck.KVCache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
        if op == "decode":
            return ck.ck_paged_attention(s["q"], cache, s["block_table"], s["lens"], window=case["window"],
                                         sinks=case["sinks"])
        q, k = ck.ck_qk_norm_rope(s["qkv"], s["positions"], s["table"], case["hq"], case["hkv"],
                                  q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                  interleaved=case["interleaved"], cache=cache, slots=s["slots"],
                                  return_k=case.get("keep_k", False))
        if op == "norm_rope":
            return [q, s["k"], s["v"]] + ([k] if case["keep_k"] else [])
        out = ck.ck_paged_attention(q, cache, s["block_table"], s["lens"], window=case["window"],
                                    sinks=case["sinks"])
        return [out, q] + _stored(s)
    if op == "int4":
        return _plain_int4(s)
    if op == "prompt":
        return _plain_prompt(s)
    if op == "decode":
        return _plain_decode(s["q"].float(), s).to(s["q"].dtype)
    dtype = s["qkv"].dtype
    q, k, v = _plain_qkv(s)
    q = q.to(dtype)
    at, off = _written(s)
    if op == "norm_rope":
        k = k.to(dtype)
        s["k"][at, :, off] = k
        s["v"][at, :, off] = v.to(dtype)
        return [q, s["k"], s["v"]] + ([k] if case["keep_k"] else [])
    for name, x in (("k", k), ("v", v)):
        codes, scale = _plain_quantize(x)
        s[name][at, :, off] = codes
        s[name + "_scale"][at, :, off] = scale
    out = _plain_decode(q.float(), s).to(dtype)
    return [out, q] + _stored(s)


# ---------------------------------------------------------------------- definitions in 64 bits
def _exact_rotate(x, weight, positions, case):
    """x [T, H, D] in 64 bits; the table's 32-bit cosines and sines are part of the input."""
    x = x.double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    half = case["rot"] // 2
    t = _rope_table(int(positions.max()) + 1, case["rot"])[positions.long()].double()
    y = x.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        c, d = t[:, i, None], t[:, i + half, None]
        y[..., a] = x[..., a] * c - x[..., b] * d
        y[..., b] = x[..., a] * d + x[..., b] * c
    return y


def _exact_attend(q, k, v, scale):
    """softmax(q k^T scale) v for q [G, D], k and v [n, D] whose keys are all visible; zeros where n is 0."""
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    p = torch.softmax(q @ k.t() * scale, -1)
    return p @ v


def _exact_decode(q, s):
    case, page = s["case"], s["case"]["page"]
    g, out = case["hq"] // case["hkv"], torch.zeros_like(q)
    for b, n in enumerate(lengths(case)):
        keep = [j for j in range(n) if not case["window"] or j >= n - case["window"] or j < case["sinks"]]
        at = torch.tensor(keep, device=DEV, dtype=torch.long)
        pages, off = s["block_table"][b].long()[at // page], at % page
        for h in range(case["hkv"]):
            rows = []
            for name in ("k", "v"):
                x = s[name][pages, h, off].double()
                rows.append(x * s[name + "_scale"][pages, h, off].double()[:, None] if name + "_scale" in s else x)
            out[b, h * g:(h + 1) * g] = _exact_attend(q[b, h * g:(h + 1) * g], rows[0], rows[1], case["d"] ** -0.5)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "int4":
        w = torch.empty((case["n"], case["k"]), dtype=torch.float64, device=DEV)
        for e in range(8):
            w[:, e::8] = ((s["w4"] >> (4 * (e // 2) + 16 * (e % 2))) & 15).double() - 8
        w *= s["w_scale"].double().repeat_interleave(case["group"], 1)
        y = (w @ s["x"].double().t()).t()
        return y if s["bias"] is None else y + s["bias"].double()
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    if op == "prompt":
        cu = s["cu"].tolist()
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros((hq, cu[-1]), dtype=torch.float64, device=DEV)
        for lo, hi in zip(cu, cu[1:]):
            n = hi - lo
            if n == 0:
                continue
            hidden = torch.zeros((n, n), dtype=torch.bool, device=DEV)
            if case["causal"]:
                hidden = torch.ones((n, n), dtype=torch.bool, device=DEV).triu(1)
                if case["window"]:
                    old = torch.ones((n, n), dtype=torch.bool, device=DEV).tril(-case["window"])
                    old[:, :case["sinks"]] = False
                    hidden |= old
            for h in range(hq):
                score = s["q"][lo:hi, h].double() @ s["k"][lo:hi, h // g].double().t() / math.sqrt(d)
                score[hidden] = -math.inf
                lse[h, lo:hi] = torch.logsumexp(score, -1)
                out[lo:hi, h] = torch.softmax(score, -1) @ s["v"][lo:hi, h // g].double()
        return out, lse
    if op == "decode":
        return _exact_decode(s["q"].double(), s)
    x = s["qkv"].view(-1, hq + 2 * hkv, d)
    q = _exact_rotate(x[:, :hq], s["q_weight"], s["positions"], case)
    k = _exact_rotate(x[:, hq:hq + hkv], s["k_weight"], s["positions"], case)
    v = x[:, hq + hkv:].double()
    page = case["page"]
    if op == "norm_rope":
        caches = []
        for name, rows in (("k", k), ("v", v)):
            c = s[name].double()
            for h in range(hkv):
                c[s["slots"] // page, h, s["slots"] % page] = rows[:, h]
            caches.append(c)
        return [q] + caches + ([k] if case["keep_k"] else [])
    stored = []
    for name, rows in (("k", k), ("v", v)):
        scale = rows.abs().max(-1).values / 127
        codes = torch.where(scale[..., None] > 0, rows / scale[..., None], 0.0).round().clamp(-127, 127)
        for h in range(hkv):
            s[name][s["slots"] // page, h, s["slots"] % page] = codes[:, h].to(torch.int8)
            s[name + "_scale"][s["slots"] // page, h, s["slots"] % page] = scale[:, h].float()
        stored.append(codes * scale[..., None])
    # the queries meet the cache in their own 16-bit type
    out = _exact_decode(q.to(s["qkv"].dtype).double(), s)
    return [out, q] + stored
