"""Cases of the operators that stand around the block-quantized products and the
attention in a generation step of a batch: the norms before and after a block
fused with its gate and residual, attention of a batch that shares a long prefix
over the paged 4-bit cache, and the choice of the next tokens from the logits.

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
        # one generated token between two blocks: only latency counts
        dict(name="norm 1 token", op="norm", n=1, d=4096, h="f32", y="f32", x="f32", post=False, gate="none",
             layer=False),
        # a decode step of 48 requests, a norm on both sides of the block and a gate for each channel
        dict(name="norm 48 tokens both sides", op="norm", n=48, d=5120, h="f32", y="f32", x="f32", post=True,
             gate="channel", layer=False),
        # odd rows, layer norms, a gate for each token and channel
        dict(name="norm 1037 odd rows", op="norm", n=1037, d=1283, h="f32", y="f32", x="f32", post=True,
             gate="token", layer=True),
        # a long prompt, the stream held in f16, the products' f32 results added
        dict(name="norm 8191-token prompt", op="norm", n=8191, d=4096, h="f16", y="f32", x="f16", post=False,
             gate="none", layer=False),
        # two requests on a short common instruction: latency
        dict(name="shared 2 on 300", op="shared", n_seq=2, prefix=300, lo=1, hi=40, lens=1, q_len=1, heads=32,
             kv_heads=8, head_dim=128, page=16, dtype="f32"),
        # a decode step of a batch on one long instruction
        dict(name="shared 32 on 8200", op="shared", n_seq=32, prefix=8200, lo=1, hi=600, lens=2, q_len=1, heads=32,
             kv_heads=8, head_dim=128, page=64, dtype="f32"),
        # three drafted tokens of each request checked at once, small heads
        dict(name="shared drafts", op="shared", n_seq=40, prefix=4099, lo=3, hi=300, lens=3, q_len=3, heads=24,
             kv_heads=8, head_dim=64, page=32, dtype="f16"),
        # questions on one very long document
        dict(name="shared 16 on 65521", op="shared", n_seq=16, prefix=65521, lo=1, hi=2000, lens=4, q_len=1, heads=64,
             kv_heads=8, head_dim=128, page=128, dtype="f16"),
        # one request's next token, every filter on: latency
        dict(name="sample 1 row", op="sample", n=1, vocab=32000, dtype="f32", filters="all", spread=2.5, cut=0.0),
        # a batch of requests with settings of their own, a grammar's mask on some
        dict(name="sample 64 rows", op="sample", n=64, vocab=32000, dtype="f32", filters="mixed", spread=2.5, cut=0.3),
        # plain sampling at a temperature from a large vocabulary
        dict(name="sample 8 rows no filter", op="sample", n=8, vocab=130001, dtype="f32", filters="none", spread=3.0,
             cut=0.0),
        # a large batch over a large vocabulary
        dict(name="sample 256 rows of 130001", op="sample", n=256, vocab=130001, dtype="f16", filters="mixed",
             spread=2.5, cut=0.05),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["norm", "shared", "shared", "sample", "sample"])
    if op == "norm":
        d = _log(rng, 32, 16384)
        if rng.random() < 0.6:
            d = max(32, d // 32 * 32)
        n = _log(rng, 1, min(8191, 8191 * 4096 // d))
        return dict(op=op, n=n, d=d, h=rng.choice(["f32", "f16"]), y=rng.choice(["f32", "f16"]),
                    x=rng.choice(["f32", "f16"]), post=rng.random() < 0.4, gate=rng.choice(["none", "channel", "token"]),
                    layer=rng.random() < 0.3)
    if op == "sample":
        vocab = _log(rng, 50, 262144)
        return dict(op=op, n=_log(rng, 1, min(256, 256 * 130001 // vocab)), vocab=vocab, dtype=rng.choice(["f32", "f16"]),
                    filters=rng.choice(["none", "mixed", "mixed", "all"]), spread=rng.choice([0.5, 2.5, 2.5, 4.0]),
                    cut=rng.choice([0.0, 0.0, 0.3, 0.95]))
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * kv_heads <= 64])
    q_len = rng.choice([1, 1, 1, 2, 3, 5])
    n_seq = _log(rng, 1, 64)
    # no more products and no longer cache than the longest listed case
    most = min(65521, 65521 * 8 // kv_heads, 65521 * 64 * 16 // (kv_heads * group * n_seq * q_len))
    hi = _log(rng, q_len, min(2000, max(16, 32000 * 8 // kv_heads // n_seq)))
    return dict(op=op, n_seq=n_seq, prefix=_log(rng, 16, max(16, most)), lo=max(q_len, hi // rng.choice([1, 4, 64])), hi=max(hi, q_len),
                lens=rng.randrange(1 << 20), q_len=q_len, heads=kv_heads * group, kv_heads=kv_heads,
                head_dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["f32", "f16"]))


def lengths(case):
    """The sequences' own lengths: the longest one, the shortest one and what lies between."""
    r = random.Random(case["lens"])
    n = [int(r.uniform(case["lo"], case["hi"] + 0.999)) for _ in range(case["n_seq"])]
    n[0] = case["hi"]
    n[-1] = case["lo"] if case["n_seq"] > 1 else n[-1]
    return n


SIZE = {"f32": 4, "f16": 2}


def work(case):
    if case["op"] == "norm":
        n, d = case["n"], case["d"]
        row = 2 * SIZE[case["h"]] + SIZE[case["y"]] + SIZE[case["x"]] + (4 if case["gate"] == "token" else 0)
        vectors = 1 + case["post"] + (1 + case["post"]) * case["layer"] + (case["gate"] == "channel")
        return {"bytes": n * d * row + 4 * d * vectors, "flops": n * d * (6 + 4 * case["post"] + (case["gate"] != "none"))}
    if case["op"] == "sample":
        n, v = case["n"], case["vocab"]
        # a logit's difference, exponential and sums; the settings and what is chosen
        return {"bytes": n * v * SIZE[case["dtype"]] + 28 * n, "flops": 6 * n * v}
    h, hk, d, t, b = case["heads"], case["kv_heads"], case["head_dim"], case["q_len"], SIZE[case["dtype"]]
    lens = lengths(case)
    seen = sum(sum(max(0, n - t + i + 1) for i in range(t)) for n in lens) + case["prefix"] * t * len(lens)
    return {"bytes": (sum(lens) + case["prefix"]) * hk * 2 * (d // 2 + d // 16) + 2 * len(lens) * t * h * d * b,
            "flops": 4 * d * h * seen}


# ---------------------------------------------------------------- the inputs
DTYPE = {"f32": torch.float32, "f16": torch.float16}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _norm_inputs(case, seed):
    g = _generator(seed)
    n, d = case["n"], case["d"]
    # the stream of a trained model has a few channels far larger than the rest
    size = torch.exp(0.5 * _normal(g, d)) * (1 + 12 * (_uniform(g, d) > 0.995))
    s = dict(h=(_normal(g, n, d) * size + 0.1).to(DTYPE[case["h"]]), y=(_normal(g, n, d) * 0.7).to(DTYPE[case["y"]]),
             weight=1 + 0.2 * _normal(g, d), bias=0.1 * _normal(g, d) if case["layer"] else None, post_weight=None,
             post_bias=None, gate=None, scale=0.75, eps=1e-5)
    if case["post"]:
        s["post_weight"] = 0.6 + 0.2 * _normal(g, d)
        s["post_bias"] = 0.1 * _normal(g, d) if case["layer"] else None
    if case["gate"] != "none":
        s["gate"] = torch.tanh(_normal(g, *((n, d) if case["gate"] == "token" else (d,))))
    return s


def _sample_inputs(case, seed):
    g = _generator(seed)
    n, v = case["n"], case["vocab"]
    x = _normal(g, n, v) * case["spread"]
    # a few likely tokens in each row, fewer in some rows than in others
    lift = _uniform(g, n, v) < torch.exp(-6 - 4 * _uniform(g, n, 1))
    x += lift * 8 * _uniform(g, n, v)
    if case["cut"]:  # tokens that a grammar forbids, in half of the rows
        x.masked_fill_((_uniform(g, n, v) < case["cut"]) & (_uniform(g, n, 1) < 0.5), -math.inf)
    s = dict(logits=x.to(DTYPE[case["dtype"]]), uniform=_uniform(g, n), temperature=0.5 + _uniform(g, n))
    s["top_k"] = s["top_p"] = s["min_p"] = None
    if case["filters"] == "all":
        s["top_k"] = torch.full((n,), 40, dtype=torch.int32, device="cuda")
        s["top_p"], s["min_p"] = torch.full((n,), 0.95, device="cuda"), torch.full((n,), 0.02, device="cuda")
    elif case["filters"] == "mixed":  # each setting in some rows; now and then a temperature of 0
        at = torch.randint(0, 4, (3, n), generator=g, device="cuda")
        k = torch.exp(_uniform(g, n) * math.log(2000)).to(torch.int32)
        s["top_k"] = torch.where(at[0] < 2, k, 0).to(torch.int32)
        s["top_p"] = torch.where(at[1] < 3, 0.3 + 0.69 * _uniform(g, n), 1.0)
        s["min_p"] = torch.where(at[2] < 1, 0.1 * _uniform(g, n), 0.0)
        s["temperature"] *= _uniform(g, n) > 0.1
    return s


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


def write_rows(case, data, slots, k, v):
    """The rows of `slots` of the cache, from f32 keys and values [n, kv heads, D]."""
    d, hk, page = case["head_dim"], case["kv_heads"], case["page"]
    p, r = slots // page, slots % page
    group = (((p[:, None] * hk + torch.arange(hk, device="cuda")) * (page // 16)) + (r // 16)[:, None]) * (18 * d)
    scale = (16 * d + ((r % 16)[:, None] * (d // 16) + torch.arange(d // 16, device="cuda")))[:, None, :]
    for x, m, s in zip((k, v), byte_maps(d), (scale, scale + d)):
        codes, scales = quantise(x)
        data[group[..., None] + m.cuda()[r % 16][:, None, :]] = packed(codes)
        data[group[..., None] + s] = scales.view(torch.uint8)


def _shared_inputs(case, seed):
    g = _generator(seed)
    n_seq, hk, d, page, t = case["n_seq"], case["kv_heads"], case["head_dim"], case["page"], case["q_len"]
    lens = [case["prefix"]] + lengths(case)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 2
    pages = list(range(n_pages))
    random.Random(seed).shuffle(pages)
    pages, ends = torch.tensor(pages, dtype=torch.int32), np.cumsum([0] + need)
    table, slots = torch.full((n_seq + 1, max(need)), -1, dtype=torch.int32), []
    for s, n in enumerate(lens):
        mine = pages[ends[s]:ends[s + 1]]
        table[s, :need[s]] = mine
        slots.append((mine.long()[:, None] * page + torch.arange(page)).flatten()[:n])
    # what was never written is arbitrary, NaN scales among it
    data = torch.randint(0, 256, (n_pages * hk * (page // 16) * 18 * d,), dtype=torch.uint8, generator=g, device="cuda")
    # per-channel sizes: keys of trained models have a few channels much larger than the rest
    size = torch.exp(0.6 * _normal(g, 1, hk, d)) * (1 + 4 * (_uniform(g, 1, hk, d) > 0.97))
    for part in torch.cat(slots).cuda().split(1 << 16):
        write_rows(case, data, part, _normal(g, part.numel(), hk, d) * size, _normal(g, part.numel(), hk, d) + 0.2)
    q = (_normal(g, n_seq * t, case["heads"], d) * 1.3).to(DTYPE[case["dtype"]])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(data=data, q=q, prefix_table=table[0, :need[0]].contiguous().cuda(), prefix_len=i32([lens[0]]),
                table=table[1:, :max(need[1:])].contiguous().cuda(), lens=i32(lens[1:]),
                offsets=i32(range(0, n_seq * t + 1, t)) if t > 1 else None)


INPUTS = {"norm": _norm_inputs, "shared": _shared_inputs, "sample": _sample_inputs}


def prepare(case, seed):
    s = INPUTS[case["op"]](case, seed)
    s["case"] = case
    empty = lambda like, dtype: torch.empty(like.shape, dtype=dtype, device="cuda")  # noqa: E731
    if case["op"] == "norm":
        s["h_out"], s["x_out"] = empty(s["h"], s["h"].dtype), empty(s["h"], DTYPE[case["x"]])
    elif case["op"] == "shared":
        s["out"] = empty(s["q"], s["q"].dtype)
        s["maps"] = [m.flatten().cuda() for m in byte_maps(case["head_dim"])]
    else:
        s["token"], s["prob"] = empty(s["uniform"], torch.int32), empty(s["uniform"], torch.float32)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    return OPS[state["case"]["op"]](state)


def normed(x, weight, bias, layer, eps):
    """x / rms(x) * weight, or with its mean taken off first, and the bias added."""
    if layer:
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    return y if bias is None else y + bias


def run_norm(s):
    layer, eps = s["case"]["layer"], s["eps"]
    if own:
        import ggml_block_quantized_gb300 as qg
        h, x = qg.norm_residual(s["h"], s["y"], s["weight"], bias=s["bias"], post_weight=s["post_weight"],
                                post_bias=s["post_bias"], gate=s["gate"], scale=s["scale"], eps=eps, layer=layer,
                                h_out=s["h_out"], x_out=s["x_out"])
        return dict(h=h, x=x)
    u = s["y"].float()
    if s["post_weight"] is not None:
        u = normed(u, s["post_weight"], s["post_bias"], layer, eps)
    if s["gate"] is not None:
        u = u * s["gate"]
    h = s["h"].float() + s["scale"] * u
    return dict(h=h.to(s["h"].dtype), x=normed(h, s["weight"], s["bias"], layer, eps).to(s["x_out"].dtype))


def run_sample(s):
    if own:
        import ggml_block_quantized_gb300 as qg
        token, prob = qg.sample_tokens(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"],
                                       top_p=s["top_p"], min_p=s["min_p"], out=s["token"], prob_out=s["prob"])
        return dict(token=token, prob=prob)
    # in 64 bits throughout: what is chosen goes by sums of many weights against a border
    x, at = s["logits"].double().sort(dim=-1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    place, some = torch.arange(x.shape[1], device="cuda"), x[:, :1] > -math.inf
    w = torch.exp((x - torch.where(some, x[:, :1], 0.0)) / torch.where(t > 0, t, 1.0))
    w = torch.where(t > 0, w, (place == 0).double())
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        w = torch.where((place < k) | (k <= 0), w, 0.0)
    keep = place == 0
    if s["top_p"] is not None:
        before = w.cumsum(-1) - w
        keep = keep | (before < s["top_p"].double()[:, None] * w.sum(-1, keepdim=True)) | (s["top_p"][:, None] >= 1)
    else:
        keep = keep | (place >= 0)
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"].double()[:, None]) | (place == 0)
    kept = torch.zeros_like(w).scatter_(-1, at, torch.where(keep, w, 0.0))
    total = kept.cumsum(-1)
    token = (total <= s["uniform"].double()[:, None] * total[:, -1:]).sum(-1, keepdim=True).clamp(max=x.shape[1] - 1)
    prob = kept.gather(-1, token) / total[:, -1:]
    # a row whose tokens are all forbidden has none
    return dict(token=torch.where(some, token, -1)[:, 0].int(), prob=torch.where(some, prob, 0.0)[:, 0].float())


def _values(code_bytes, scale_bytes):
    c = code_bytes.unflatten(-1, (-1, 16))
    c = torch.stack([c & 15, c >> 4], -2).flatten(-2).float() - 8.0
    return (c * scale_bytes.contiguous().view(torch.float16).float()[..., None]).flatten(-2)


def rows_of(case, data, pages, maps):
    """Key and value rows of pages [..., n] as values, [..., kv heads, tokens, D]."""
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    x = data.view(-1, hk, page // 16, 18 * d)[pages.clamp(min=0).long()]
    x = x.transpose(-4, -3).flatten(-3, -2)
    keys, values = maps
    k = _values(x[..., keys].unflatten(-1, (16, -1)), x[..., 16 * d:17 * d].unflatten(-1, (16, -1))).flatten(-3, -2)
    v = _values(x[..., values].unflatten(-1, (16, -1)), x[..., 17 * d:].unflatten(-1, (16, -1))).flatten(-3, -2)
    return k, v


def run_shared(s):
    c = s["case"]
    if own:
        import ggml_block_quantized_gb300 as qg
        cache = qg.KVCache(c["kv_heads"], c["head_dim"], c["page"], s["data"])
        return qg.kv_attend_shared(cache, s["q"], s["prefix_table"], s["prefix_len"], s["table"], s["lens"],
                                   q_offsets=s["offsets"], max_q_len=c["q_len"], out=s["out"])
    n_seq, hk, d, t = c["n_seq"], c["kv_heads"], c["head_dim"], c["q_len"]
    g = c["heads"] // hk
    q = s["q"].float().view(n_seq, t, hk, g, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # rows: head of the group, token
    pk, pv = rows_of(c, s["data"], s["prefix_table"], s["maps"])
    at = torch.arange(pk.shape[1], device="cuda")
    seen_p = at < s["prefix_len"]
    sp = torch.matmul(q.transpose(0, 1).flatten(1, 2), pk.transpose(-1, -2)) * d ** -0.5
    sp = torch.where(seen_p, sp, -math.inf).unflatten(1, (n_seq, -1)).transpose(0, 1)
    k, v = rows_of(c, s["data"], s["table"], s["maps"])
    at = torch.arange(k.shape[2], device="cuda")
    lens = s["lens"].long()
    last = (lens - t)[:, None] + torch.arange(t, device="cuda")
    seen = (at <= last[..., None])[:, None, None].expand(-1, 1, g, -1, -1).flatten(2, 3)
    so = torch.where(seen, torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5, -math.inf)
    top = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    top = torch.where(torch.isfinite(top), top, 0.0)
    wp, wo = torch.exp(sp - top), torch.exp(so - top)
    total = wp.sum(-1, keepdim=True) + wo.sum(-1, keepdim=True)
    pv = torch.where(seen_p[:, None], pv, 0.0)
    v = torch.where((at < lens[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(wp.transpose(0, 1).flatten(1, 2), pv).unflatten(1, (n_seq, -1)).transpose(0, 1) + torch.matmul(wo, v)
    o = o / torch.where(total > 0, total, 1.0)
    return o.view(n_seq, hk, g, t, d).permute(0, 3, 1, 2, 4).reshape(n_seq * t, c["heads"], d).to(s["q"].dtype)


OPS = {"norm": run_norm, "shared": run_shared, "sample": run_sample}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    return {"norm": exact_norm, "shared": exact_shared, "sample": exact_sample}[case["op"]](case, seed)


def exact_norm(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in _norm_inputs(case, seed).items()}

    def apply(x, weight, bias):
        moment = torch.einsum("nd,nd->n", x, x) / x.shape[1]
        if case["layer"]:
            mean = x.sum(1) / x.shape[1]
            x, moment = x - mean[:, None], torch.einsum("nd,nd->n", x - mean[:, None], x - mean[:, None]) / x.shape[1]
        y = torch.einsum("nd,n,d->nd", x, (moment + s["eps"]) ** -0.5, weight)
        return y + bias if bias is not None else y

    u = s["y"] if s["post_weight"] is None else apply(s["y"], s["post_weight"], s["post_bias"])
    h = s["h"] + (s["scale"] * u if s["gate"] is None else s["scale"] * s["gate"] * u)
    return dict(h=h, x=apply(h, s["weight"], s["bias"]))


def exact_sample(case, seed):
    s = {k: v.cpu().numpy() if isinstance(v, torch.Tensor) else v for k, v in _sample_inputs(case, seed).items()}
    token, prob = np.zeros(case["n"], np.int32), np.zeros(case["n"])
    for r in range(case["n"]):
        x, t = s["logits"][r].astype(np.float64), float(s["temperature"][r])
        if x.max() == -np.inf:
            token[r] = -1
            continue
        if t <= 0:
            token[r], prob[r] = x.argmax(), 1.0
            continue
        w = np.exp((x - x.max()) / t)
        order = np.argsort(-x, kind="stable")
        if s["top_k"] is not None and s["top_k"][r] > 0:
            order = order[:s["top_k"][r]]
        if s["top_p"] is not None and s["top_p"][r] < 1:
            sums = np.concatenate([[0.0], np.cumsum(w[order])])
            order = order[:max(1, int((sums[:-1] < float(s["top_p"][r]) * sums[-1]).sum()))]
        if s["min_p"] is not None:
            order = order[w[order] >= float(s["min_p"][r])]
        order = np.sort(order)
        sums = np.cumsum(w[order])
        token[r] = order[np.searchsorted(sums, float(s["uniform"][r]) * sums[-1], side="right")]
        prob[r] = w[token[r]] / sums[-1]
    return dict(token=torch.from_numpy(token), prob=torch.from_numpy(prob))


def exact_shared(case, seed):
    s = _shared_inputs(case, seed)
    hk, d, page, t = case["kv_heads"], case["head_dim"], case["page"], case["q_len"]
    g, nb = case["heads"] // hk, d // 32
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    pages = s["data"].view(-1, hk, page // 16, 18 * d)
    order = [i // 2 + 4 * (i % 2) for i in range(8)]  # the row of a half group in which value row i lies

    def rows(mine, length):
        x = pages[mine[:-(-length // page)].long()].transpose(0, 1).reshape(hk, -1, 18 * d)
        kc = x[..., :8 * d].reshape(hk, -1, 4, nb, 4).transpose(2, 3).reshape(hk, -1, nb, 16)
        u = x[..., 8 * d:16 * d].reshape(hk, -1, 2, 8, 2, 4, nb, 2)
        u = torch.stack([u[:, :, :, r].flip(3) if r & 2 else u[:, :, :, r] for r in order], 3)
        vc = u.flatten(4, 5).transpose(4, 5).reshape(hk, -1, nb, 16)
        ks, vs = (x[..., i * d:(i + 1) * d].contiguous().view(torch.float16).double().reshape(hk, -1, nb, 1) for i in (16, 17))
        return tuple((torch.cat([(c & 15), (c >> 4)], -1).double().sub(8) * sc).reshape(hk, -1, d)[:, :length]
                     for c, sc in ((kc, ks), (vc, vs)))

    pk, pv = rows(s["prefix_table"], case["prefix"])
    for n, length in enumerate(lengths(case)):
        k, v = rows(s["table"][n], length)
        for i in range(t):
            m = max(0, length - t + i + 1)
            q = s["q"][n * t + i].double().view(hk, g, d) / math.sqrt(d)
            a = torch.cat([torch.einsum("hgd,hmd->hgm", q, x) for x in (pk, k[:, :m])], -1)
            p = torch.softmax(a, -1)
            o = torch.einsum("hgm,hmd->hgd", p[..., :case["prefix"]], pv) + torch.einsum("hgm,hmd->hgd", p[..., case["prefix"]:], v[:, :m])
            out[n * t + i] = o.reshape(-1, d)
    return out
