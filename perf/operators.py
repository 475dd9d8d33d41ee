"""Cases of the attention operators around the block-quantized products: keys
and values appended to a paged cache held in 4 bits (the position rotation
applied on the way), attention of a few new tokens over that cache, and causal
attention over whole packed prompts.

The cache is one uint8 tensor, [page][kv head][page_size / 16 groups]. A group
holds 16 tokens of one head in 18 D bytes: 16 rows of D/2 key-code bytes, 16
rows of D/2 value-code bytes, 16 x D/32 f16 key scales, 16 x D/32 f16 value
scales. Codes and scales are Q4_0's (per 32 elements: d = signed max / -8,
value (code - 8) d); only the order of the code bytes is the cache's own, see
byte_maps(). Token `slot` of the cache lies in page slot // page_size, row
slot % page_size.
"""
import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one generated token of one request: only latency counts
        dict(name="append, 1 token", op="append", n_tok=1, n_seq=1, heads=32, kv_heads=8, head_dim=128, rot=128,
             pairs=False, dtype="f32", page=64, prompt=False),
        # a decode step of 64 requests, all 32 heads with keys and values of their own
        dict(name="append, 64 requests", op="append", n_tok=64, n_seq=64, heads=32, kv_heads=32, head_dim=128, rot=128,
             pairs=True, dtype="f32", page=16, prompt=False),
        # small heads, half of each rotated, a few short prompts packed together
        dict(name="append, short prompts", op="append", n_tok=1037, n_seq=7, heads=24, kv_heads=8, head_dim=64, rot=32,
             pairs=False, dtype="f32", page=32, prompt=True),
        # a long prompt's projections in f16, cut out of one fused product
        dict(name="append, 8191-token prompt", op="append", n_tok=8191, n_seq=1, heads=32, kv_heads=8, head_dim=128,
             rot=128, pairs=False, dtype="f16", page=64, prompt=True),
        # one request's decode step after a short prompt: latency
        dict(name="cache, 1 short", op="cache", n_seq=1, lo=777, hi=777, lens=1, q_len=1, heads=32, kv_heads=8,
             head_dim=128, page=64, dtype="f32"),
        # a decode step of a ragged batch, every head with its own keys
        dict(name="cache, 24 ragged", op="cache", n_seq=24, lo=200, hi=4096, lens=2, q_len=1, heads=32, kv_heads=32,
             head_dim=128, page=16, dtype="f16"),
        # a decode step over one very long context, eight query heads to a key head
        dict(name="cache, 1 long", op="cache", n_seq=1, lo=131071, hi=131071, lens=3, q_len=1, heads=64, kv_heads=8,
             head_dim=128, page=128, dtype="f32"),
        # five drafted tokens of each request checked at once, small heads
        dict(name="cache, drafts", op="cache", n_seq=16, lo=5, hi=6000, lens=4, q_len=5, heads=24, kv_heads=8,
             head_dim=64, page=32, dtype="f16"),
        # a chat line: latency, most of a tile empty
        dict(name="prompt, 61 tokens", op="prompt", n_seq=1, lo=61, hi=61, lens=5, heads=32, kv_heads=8, head_dim=128),
        # a batch of chat turns, packed
        dict(name="prompt, 16 packed", op="prompt", n_seq=16, lo=1, hi=700, lens=6, heads=32, kv_heads=8,
             head_dim=128),
        # small heads, as many key heads as query heads, odd lengths
        dict(name="prompt, 5 packed, D 64", op="prompt", n_seq=5, lo=300, hi=1501, lens=7, heads=24, kv_heads=24,
             head_dim=64),
        # a long document
        dict(name="prompt, 8192 tokens", op="prompt", n_seq=1, lo=8192, hi=8192, lens=8, heads=32, kv_heads=8,
             head_dim=128),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["append", "cache", "cache", "prompt", "prompt"])
    head_dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * kv_heads <= 64])
    c = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim)
    if op == "append":
        prompt = rng.random() < 0.6
        n_tok = _log(rng, 1, 8191 if prompt else 256)
        while n_tok > 1 and n_tok * (c["heads"] + 2 * kv_heads) * head_dim > 8191 * 48 * 128:
            n_tok = n_tok // 2 + 1
        c.update(n_tok=n_tok, n_seq=min(n_tok, _log(rng, 1, 16)) if prompt else n_tok,
                 rot=rng.choice([head_dim, head_dim, head_dim // 2]), pairs=rng.random() < 0.4,
                 dtype=rng.choice(["f32", "f16"]), page=rng.choice([16, 32, 64, 128]), prompt=prompt)
    elif op == "cache":
        n_seq = _log(rng, 1, 64)
        most = max(64, int(131071 * 8 / kv_heads / n_seq))  # about the longest listed case's cache in all
        hi = _log(rng, 16, min(131071, most))
        c.update(n_seq=n_seq, lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, lens=rng.randrange(1 << 20),
                 q_len=rng.choice([1, 1, 1, 2, 3, 5, 8]), page=rng.choice([16, 32, 64, 128]),
                 dtype=rng.choice(["f32", "f16"]))
        c["lo"], c["hi"] = max(c["lo"], c["q_len"]), max(c["hi"], c["q_len"])
    else:
        n_seq = _log(rng, 1, 32)
        hi = _log(rng, 16, int(8192 / n_seq * (1 if c["heads"] <= 32 else 0.6)))
        c.update(n_seq=n_seq, lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, lens=rng.randrange(1 << 20))
    return c


def lengths(case):
    """The case's sequence lengths: the longest one, the shortest one and what lies between."""
    r = random.Random(case["lens"])
    n = [int(r.uniform(case["lo"], case["hi"] + 0.999)) for _ in range(case["n_seq"])]
    n[0] = case["hi"]
    n[-1] = case["lo"] if case["n_seq"] > 1 else n[-1]
    return n


def work(case):
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        n, b = case["n_tok"], 4 if case["dtype"] == "f32" else 2
        o = 2 if case["prompt"] else b
        # projections in, rotated queries out (and for a prompt keys and values), 4-bit rows out, and the
        # rows' values, read from the cache (they were just written: counted once) and written in f32
        out = n * h * d * o + (2 * n * hk * d * o if case["prompt"] else 0)
        table = 4 * case["rot"] * min(n, 8192)
        return {"bytes": n * (h + 2 * hk) * d * b + out + 2 * n * hk * (d // 2 + d // 16) + 8 * n * hk * d + table,
                "flops": n * ((h + hk) * 3 * case["rot"] + 2 * hk * 4 * d)}
    lens = lengths(case)
    if case["op"] == "cache":
        t, b = case["q_len"], 4 if case["dtype"] == "f32" else 2
        seen = sum(sum(max(0, n - t + i + 1) for i in range(t)) for n in lens)
        return {"bytes": sum(lens) * hk * 2 * (d // 2 + d // 16) + 2 * len(lens) * t * h * d * b,
                "flops": 4 * d * h * seen}
    n = sum(lens)
    return {"bytes": 2 * n * (2 * h + 2 * hk) * d, "flops": 4 * d * h * sum(m * (m + 1) // 2 for m in lens)}


# ---------------------------------------------------------------- the inputs
DTYPE = {"f32": torch.float32, "f16": torch.float16}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _channels(g, heads, d):
    """Per-channel sizes: keys of trained models have a few channels much larger than the rest."""
    return torch.exp(0.6 * _normal(g, 1, heads, d)) * (1 + 4 * (torch.rand(1, heads, d, generator=g, device="cuda") > 0.97))


def byte_maps(d):
    """Where the code bytes of a 16-token group lie: [16, D/2] offsets of the bytes of token row i in Q4_0 order
    (block b's byte j at 16 b + j), for keys and for values. Keys: the 4-byte words of a row, word t of every
    block together. Values: the rows in the order 0 2 4 6 1 3 5 7 (and the same of the upper eight), the 2-byte
    units of a row, unit u of every block together, the halves of the row swapped in rows 2, 3, 6, 7 of that order."""
    nb = d // 32
    i, byte = torch.arange(16)[:, None], torch.arange(d // 2)[None, :]
    b, j = byte // 16, byte % 16
    keys = i * (d // 2) + ((j // 4) * nb + b) * 4 + j % 4
    row = (i & 8) | ((i & 1) << 2) | ((i >> 1) & 3)
    unit = (j // 2) ^ torch.where((row & 2) > 0, 4, 0)
    values = 8 * d + row * (d // 2) + (unit * nb + b) * 2 + j % 2
    return keys, values


def quantise(x):
    """Q4_0 of f32 [..., D]: codes uint8 [..., D] (0..15) and scales f16 [..., D/32], each step rounded in f32."""
    y = x.unflatten(-1, (-1, 32))
    at = y.abs().argmax(-1, keepdim=True)
    d = y.gather(-1, at) / -8.0
    inv = torch.where(d != 0, torch.reciprocal(d), torch.zeros_like(d))
    code = (y * inv + 8.5).floor().clamp(0, 15).to(torch.uint8)
    return code.flatten(-2), d.squeeze(-1).half()


def packed(codes):
    """[..., D] codes to [..., D/2] bytes: element j of a block in the low nibble of byte j, j + 16 in the high."""
    y = codes.unflatten(-1, (-1, 2, 16))
    return (y[..., 0, :] | (y[..., 1, :] << 4)).flatten(-2)


def cache_offsets(case, slots):
    """Byte offsets in the cache of the rows of `slots`: key codes, value codes, key scales, value scales."""
    d, hk, page = case["head_dim"], case["kv_heads"], case["page"]
    heads = torch.arange(hk, device=slots.device)
    p, r = slots // page, slots % page
    group = (((p[:, None] * hk + heads) * (page // 16)) + (r // 16)[:, None]) * (18 * d)
    keys, values = (m.to(slots.device)[r % 16][:, None, :] for m in byte_maps(d))
    scale = 16 * d + ((r % 16)[:, None] * (d // 16) + torch.arange(d // 16, device=slots.device))[:, None, :]
    g = group[:, :, None]
    return g + keys, g + values, g + scale, g + scale + d


def write_rows(case, data, slots, k, v):
    kc, ks = quantise(k)
    vc, vs = quantise(v)
    at = cache_offsets(case, slots.long())
    data[at[0]], data[at[1]] = packed(kc), packed(vc)
    data[at[2]], data[at[3]] = ks.view(torch.uint8), vs.view(torch.uint8)


def read_rows(case, data, slots):
    """The f32 values of the rows of `slots`: keys and values [n, kv heads, D]."""
    at = cache_offsets(case, slots.long())
    return tuple(_values(data[c], data[s]) for c, s in ((at[0], at[2]), (at[1], at[3])))


def _values(code_bytes, scale_bytes):
    c = code_bytes.unflatten(-1, (-1, 16))
    c = torch.stack([c & 15, c >> 4], -2).flatten(-2).float() - 8.0
    return (c * scale_bytes.contiguous().view(torch.float16).float()[..., None]).flatten(-2)


def _append_inputs(case, seed):
    g = _generator(seed)
    n, h, hk, d, page = case["n_tok"], case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    x = _normal(g, n, h + 2 * hk, d)
    x[:, h:h + hk] *= _channels(g, hk, d)[0]
    x = x.to(DTYPE[case["dtype"]])
    r = random.Random(seed)
    if case["prompt"]:  # packed prompts from position 0 on, cut out of one fused projection
        cuts = sorted(r.sample(range(1, n), case["n_seq"] - 1)) if case["n_seq"] > 1 else []
        lens = [b - a for a, b in zip([0] + cuts, cuts + [n])]
        pos = [i for m in lens for i in range(m)]
        q, k, v = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
        n_pages = sum(-(-m // page) for m in lens) + 3
        pages = list(range(n_pages))
        r.shuffle(pages)
        slots, used = [], 0
        for m in lens:
            slots += [pages[used + i // page] * page + i % page for i in range(m)]
            used += -(-m // page)
    else:  # the next token of each request, somewhere in a page of its own
        pos = [r.randrange(0, 8192) for _ in range(n)]
        n_pages = 2 * n
        pages = r.sample(range(n_pages), n)
        slots = [pages[i] * page + pos[i] % page for i in range(n)]
        q, k, v = (t.contiguous() for t in (x[:, :h], x[:, h:h + hk], x[:, h + hk:]))
    half = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    angle = torch.arange(8192, dtype=torch.float64)[:, None] * freq
    rope = torch.stack([angle.cos(), angle.sin()], -1).float().cuda()  # [position][pair][cos, sin]
    data = torch.zeros(n_pages * hk * (page // 16) * 18 * d, dtype=torch.uint8, device="cuda")
    return dict(q=q, k=k, v=v, rope=rope, data=data, pos=torch.tensor(pos, dtype=torch.int32, device="cuda"),
                slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))


def _cache_inputs(case, seed):
    g = _generator(seed)
    n_seq, hk, d, page, t = case["n_seq"], case["kv_heads"], case["head_dim"], case["page"], case["q_len"]
    lens = lengths(case)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 2
    pages = list(range(n_pages))
    random.Random(seed).shuffle(pages)
    table, slots, used = torch.full((n_seq, max(need)), -1, dtype=torch.int32), [], 0
    for s, n in enumerate(lens):
        mine = torch.tensor(pages[used:used + need[s]], dtype=torch.int32)
        table[s, :need[s]] = mine
        slots.append((mine.long()[:, None] * page + torch.arange(page)).flatten()[:n])
        used += need[s]
    # what was never written is arbitrary, NaN scales among it
    data = torch.randint(0, 256, (n_pages * hk * (page // 16) * 18 * d,), dtype=torch.uint8, generator=g, device="cuda")
    slots = torch.cat(slots).cuda()
    size = _channels(g, hk, d)
    for part in slots.split(1 << 16):
        write_rows(case, data, part, _normal(g, part.numel(), hk, d) * size, _normal(g, part.numel(), hk, d) + 0.2)
    q = (_normal(g, n_seq * t, case["heads"], d) * 1.3).to(DTYPE[case["dtype"]])
    offsets = torch.arange(0, n_seq * t + 1, t, dtype=torch.int32, device="cuda") if t > 1 else None
    return dict(data=data, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q=q,
                offsets=offsets)


def _prompt_inputs(case, seed):
    g = _generator(seed)
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    lens = lengths(case)
    x = _normal(g, sum(lens), h + 2 * hk, d)
    x[:, h:h + hk] *= _channels(g, hk, d)[0]
    x[:, h + hk:] += 0.2
    x = x.half()
    ends = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    return dict(q=x[:, :h], k=x[:, h:h + hk], v=x[:, h + hk:], offsets=ends)


INPUTS = {"append": _append_inputs, "cache": _cache_inputs, "prompt": _prompt_inputs}


def prepare(case, seed):
    s = INPUTS[case["op"]](case, seed)
    s["case"] = case
    if case["op"] == "append":
        t = torch.float16 if case["prompt"] else DTYPE[case["dtype"]]
        make = lambda x, dtype: torch.empty(x.shape, dtype=dtype, device="cuda")  # noqa: E731
        s["q_out"] = make(s["q"], t)
        s["k_out"], s["v_out"] = (make(s["k"], t), make(s["v"], t)) if case["prompt"] else (None, None)
        s["k_rows"], s["v_rows"] = make(s["k"], torch.float32), make(s["v"], torch.float32)
    else:
        s["out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    return OPS[state["case"]["op"]](state)


def run_append(s):
    c = s["case"]
    if own:
        import ggml_block_quantized_gb300 as qg
        cache = qg.KVCache(c["kv_heads"], c["head_dim"], c["page"], s["data"])
        qg.kv_append(cache, s["k"], s["v"], s["slots"], positions=s["pos"], rope=s["rope"], rope_pairs=c["pairs"],
                     q=s["q"], q_out=s["q_out"], k_out=s["k_out"], v_out=s["v_out"])
        qg.kv_read(cache, s["slots"], k_out=s["k_rows"], v_out=s["v_rows"])
        return {n: s[n] for n in ("q_out", "k_out", "v_out", "k_rows", "v_rows")}
    cos, sin = s["rope"][s["pos"].long()].unbind(-1)
    q, k, v = (rotate(s["q"].float(), cos, sin, c["pairs"]), rotate(s["k"].float(), cos, sin, c["pairs"]),
               s["v"].float())
    write_rows(c, s["data"], s["slots"], k, v)
    k_rows, v_rows = read_rows(c, s["data"], s["slots"])
    t = s["q_out"].dtype
    return dict(q_out=q.to(t), k_out=k.to(t) if c["prompt"] else None, v_out=v.to(t) if c["prompt"] else None,
                k_rows=k_rows, v_rows=v_rows)


def rotate(x, cos, sin, pairs):
    """The first 2 * cos.shape[-1] channels of [n, heads, D] turned by each token's angles: channels i and i + rot/2
    make pair i, or 2 i and 2 i + 1 where `pairs` is true."""
    half = cos.shape[-1]
    y, c, s = x.clone(), cos[:, None], sin[:, None]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def softmax_product(scores, seen, v):
    """softmax over the keys that are seen, times v; zeros where none is."""
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1.0)


def run_cache(s):
    c = s["case"]
    if own:
        import ggml_block_quantized_gb300 as qg
        cache = qg.KVCache(c["kv_heads"], c["head_dim"], c["page"], s["data"])
        return qg.kv_attend(cache, s["q"], s["table"], s["lens"], q_offsets=s["offsets"], max_q_len=c["q_len"],
                            out=s["out"])
    n_seq, hk, d, t = c["n_seq"], c["kv_heads"], c["head_dim"], c["q_len"]
    g = c["heads"] // hk
    # the sequences' pages, key and value rows as values: [n_seq, kv heads, tokens, D]
    x = s["data"].view(-1, hk, c["page"] // 16, 18 * d)[s["table"].clamp(min=0).long()]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
    keys, values = (m.flatten().cuda() for m in byte_maps(d))
    k = _values(x[..., keys].unflatten(-1, (16, -1)), x[..., 16 * d:17 * d].unflatten(-1, (16, -1))).flatten(2, 3)
    v = _values(x[..., values].unflatten(-1, (16, -1)), x[..., 17 * d:].unflatten(-1, (16, -1))).flatten(2, 3)
    at = torch.arange(k.shape[2], device="cuda")
    lens = s["lens"].long()
    v = torch.where((at < lens[:, None])[:, None, :, None], v, 0.0)
    q = s["q"].float().view(n_seq, t, hk, g, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # rows: head of the group, token
    last = (lens - t)[:, None] + torch.arange(t, device="cuda")
    seen = (at <= last[..., None])[:, None, None].expand(-1, 1, g, -1, -1).flatten(2, 3)
    o = softmax_product(torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5, seen, v)
    return o.view(n_seq, hk, g, t, d).permute(0, 3, 1, 2, 4).reshape(n_seq * t, c["heads"], d).to(s["q"].dtype)


def run_prompt(s):
    c = s["case"]
    if own:
        import ggml_block_quantized_gb300 as qg
        return qg.prompt_attend(s["q"], s["k"], s["v"], s["offsets"], out=s["out"])
    n, hk, d = s["q"].shape[0], c["kv_heads"], c["head_dim"]
    q = s["q"].float().unflatten(1, (hk, -1)).permute(1, 2, 0, 3)
    k, v = (s[x].float().transpose(0, 1)[:, None] for x in ("k", "v"))
    at = torch.arange(n, device="cuda")
    seq = torch.bucketize(at, s["offsets"][1:].long(), right=True)
    seen = (seq[:, None] == seq) & (at[:, None] >= at)
    o = softmax_product(torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5, seen, v)
    return o.permute(2, 0, 1, 3).reshape(n, c["heads"], d).half()


OPS = {"append": run_append, "cache": run_cache, "prompt": run_prompt}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    return {"append": exact_append, "cache": exact_cache, "prompt": exact_prompt}[case["op"]](case, seed)


def _q4_0_numpy(x):
    """The values that Q4_0 stores for f32 rows [n, D]. The rule is stated in f32 steps (a code is the result of a
    rounding, so it has no meaning in more bits): the first element of largest magnitude over -8, its inverse, and
    the product and the sum with 8.5 rounded one after the other."""
    b = x.reshape(-1, 32)
    big = b[np.arange(len(b)), np.abs(b).argmax(1)]
    d = (big / np.float32(-8)).astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(d != 0, np.float32(1) / d, np.float32(0)).astype(np.float32)
    code = np.minimum(15, np.trunc((b * inv[:, None]).astype(np.float32) + np.float32(8.5)))
    return ((code - 8).astype(np.float64) * d.astype(np.float16).astype(np.float64)[:, None]).reshape(x.shape)


def exact_append(case, seed):
    s = _append_inputs(case, seed)
    table = s["rope"].cpu().numpy()[s["pos"].cpu().numpy()]
    half = case["rot"] // 2

    def turned(x, kind):
        """The rotated rows; in f32 (`kind`) each product and their sum are rounded, as the cache's rule has it."""
        x = x.float().cpu().numpy().astype(kind)
        c, sn = table[:, None, :, 0].astype(kind), table[:, None, :, 1].astype(kind)
        y = x.copy()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["pairs"] else (i, half + i)
            y[:, :, a] = x[:, :, a] * c[:, :, i] - x[:, :, b] * sn[:, :, i]
            y[:, :, b] = x[:, :, a] * sn[:, :, i] + x[:, :, b] * c[:, :, i]
        return y

    v = s["v"].float().cpu().numpy()
    got = dict(q_out=turned(s["q"], np.float64), k_rows=_q4_0_numpy(turned(s["k"], np.float32)), v_rows=_q4_0_numpy(v))
    got["k_out"] = turned(s["k"], np.float64) if case["prompt"] else None
    got["v_out"] = v.astype(np.float64) if case["prompt"] else None
    return {n: torch.from_numpy(np.ascontiguousarray(x)) if x is not None else None for n, x in got.items()}


def exact_cache(case, seed):
    s = _cache_inputs(case, seed)
    hk, d, page, t = case["kv_heads"], case["head_dim"], case["page"], case["q_len"]
    g, nb = case["heads"] // hk, d // 32
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    pages = s["data"].view(-1, hk, page // 16, 18 * d)
    order = [i // 2 + 4 * (i % 2) for i in range(8)]  # the row of a half group in which value row i lies
    for n, length in enumerate(lengths(case)):
        x = pages[s["table"][n, :-(-length // page)].long()].transpose(0, 1).reshape(hk, -1, 18 * d)
        kc = x[..., :8 * d].reshape(hk, -1, 4, nb, 4).transpose(2, 3).reshape(hk, -1, nb, 16)
        u = x[..., 8 * d:16 * d].reshape(hk, -1, 2, 8, 2, 4, nb, 2)
        u = torch.stack([u[:, :, :, r].flip(3) if r & 2 else u[:, :, :, r] for r in order], 3)
        vc = u.flatten(4, 5).transpose(4, 5).reshape(hk, -1, nb, 16)
        ks, vs = (x[..., i * d:(i + 1) * d].contiguous().view(torch.float16).double().reshape(hk, -1, nb, 1)
                  for i in (16, 17))
        k, v = ((torch.cat([(c & 15), (c >> 4)], -1).double().sub(8) * sc).reshape(hk, -1, d)[:, :length]
                for c, sc in ((kc, ks), (vc, vs)))
        for i in range(t):
            m = length - t + i + 1
            if m <= 0:
                continue
            q = s["q"][n * t + i].double().view(hk, g, d)
            p = torch.softmax(torch.einsum("hgd,hmd->hgm", q, k[:, :m]) / math.sqrt(d), -1)
            out[n * t + i] = torch.einsum("hgm,hmd->hgd", p, v[:, :m]).reshape(-1, d)
    return out


def exact_prompt(case, seed):
    s = _prompt_inputs(case, seed)
    g, d = case["heads"] // case["kv_heads"], case["head_dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for n in lengths(case):
        at = slice(start, start + n)
        start += n
        hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for h in range(case["heads"]):
            a = s["q"][at, h].double() @ s["k"][at, h // g].double().T / math.sqrt(d)
            out[at, h] = torch.softmax(a.masked_fill(hidden, -math.inf), -1) @ s["v"][at, h // g].double()
    return out
