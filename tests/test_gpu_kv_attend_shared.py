"""qkv_attend_shared against the formula in 64 bits (attn_ref.attend) on the cache's
own values: every row over the prefix and the sequence's own tokens together. The
tolerance is attn_ref.bound's, as for qkv_attend; the prefix's sums of D products
are formed in three parts (or two), which the bound's D 2^-23 of a score covers."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attn_ref  # noqa: E402
import ggml_block_quantized_gb300 as qg  # noqa: E402
from test_gpu_kv_attend import filled, i32  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert qg.device_error() == 0


def call(cache, q, table, lens, prefix, **kw):
    """Row 0 of `table` is the prefix's, the others are the sequences'."""
    page = cache.page_size
    return qg.kv_attend_shared(cache, q, i32(table[0][:max(1, -(-prefix // page))]), i32([prefix]), i32(table[1:]), i32(lens), **kw)


def check(got, q, ks, vs, prefix, lens, q_lens, group, scale, f16, rows=None):
    got, q = got.detach().cpu().numpy().astype(np.float64), q.cpu().numpy().astype(np.float64)
    d, at = q.shape[2], 0
    for s, m in enumerate(q_lens):
        if rows is None or s in rows:
            seen = [prefix + max(0, lens[s] - m + i + 1) for i in range(m)]
            for h in range(q.shape[1]):
                k, v = (np.concatenate([x[0][:prefix, h // group], x[s + 1][:, h // group]]) for x in (ks, vs))
                out, pv, mag, big = attn_ref.attend(q[at:at + m, h], k, v, seen, scale)
                tol = attn_ref.bound(out, pv, mag, big, d, len(k), 24 if f16 else 20, 10 if f16 else 20, f16)
                err = np.abs(got[at:at + m, h] - out)
                assert np.isfinite(got[at:at + m, h]).all(), (s, h)
                assert (err <= tol).all(), (s, h, float((err / tol).max()))
        at += m


CASES = [  # D, type, kv heads, group, page, prefix, own lengths, queries of each sequence (None: one)
    (128, "f32", 8, 4, 64, 300, [20, 1], None), (128, "f16", 8, 4, 64, 777, [33, 5, 0], None),
    (128, "f32", 2, 1, 16, 1, [0, 1, 17], None), (64, "f16", 3, 1, 16, 0, [3, 0, 20], None),
    (64, "f32", 1, 8, 32, 127, [300, 5, 1000], None), (64, "f16", 2, 3, 48, 128, [2, 1], [2, 3]),
    (128, "f16", 1, 7, 128, 129, [90, 7, 260], [5, 3, 2]), (128, "f32", 1, 16, 16, 2049, [41, 3, 9, 500], [4, 8, 2, 7]),
    (64, "f32", 4, 2, 64, 5000, [4, 3], [2, 0]), (128, "f32", 1, 64, 64, 1000, [70, 9], [2, 3]),
    (128, "f16", 32, 1, 16, 511, [9] * 20, None), (128, "f32", 1, 1, 128, 20000, [10], None),
    (64, "f16", 1, 5, 16, 15, [1] * 70, None), (128, "f32", 2, 3, 32, 260, [8] * 50, [1] * 50),
    (64, "f32", 8, 8, 256, 700, [5] * 40, None), (128, "f16", 2, 16, 16, 384, [6] * 33, [3] * 33),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", "")[:60])
def test_attend(case):
    d, t, hk, group, page, prefix, lens, q_lens = case
    rng = np.random.default_rng(sum(map(ord, str(case))))
    cache, table, ks, vs = filled(rng, [prefix] + lens, hk, d, page)
    per = q_lens or [1] * len(lens)
    q = torch.from_numpy(rng.standard_normal((sum(per), hk * group, d)).astype(np.float32) * 1.5).cuda().to(TYPES[t])
    kw = dict(q_offsets=i32(np.cumsum([0] + per)) if q_lens else None, max_q_len=max(per))
    got = call(cache, q, table, lens, prefix, **kw)
    assert got.dtype == q.dtype
    check(got, q, ks, vs, prefix, lens, per, group, d ** -0.5, t == "f16")
    assert torch.equal(got, call(cache, q, table, lens, prefix, **kw))


@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("k_size,v_size,q_size,scale", [
    (1, 1, 1, -0.2), (1, 1, 1, 0.0), (30, 1, 8, 1.0), (1, 3e3, 1, 0.09), (1, 1e-4, 1, 0.09), (1e-4, 1, 300, 0.09),
    (2e3, 1, 1e-4, 0.09), (6e4, 1e4, 1e-5, 0.09)])
def test_sizes_of_values(t, k_size, v_size, q_size, scale):
    """Steep, flat and reversed softmaxes; keys, values and queries far from 1."""
    rng = np.random.default_rng(17)
    cache, table, ks, vs = filled(rng, [700, 33, 4], 2, 128, 64, k_size, v_size)
    q = torch.from_numpy(rng.standard_normal((2, 6, 128)).astype(np.float32) * q_size).cuda().to(TYPES[t])
    if t == "f16" and v_size > 5e3:
        pytest.skip("results past f16's range")
    got = call(cache, q, table, [33, 4], 700, scale=scale)
    check(got, q, ks, vs, 700, [33, 4], [1, 1], 3, scale, t == "f16")


@pytest.mark.parametrize("e", [-125, -100, 90, 120])
def test_queries_near_the_ends_of_f32(e):
    rng = np.random.default_rng(42)
    cache, table, ks, vs = filled(rng, [300, 40, 7], 2, 128, 64)
    q = np.ldexp(rng.standard_normal((2, 6, 128)).astype(np.float32).astype(np.float64), e).astype(np.float32)
    q, scale = torch.from_numpy(q).cuda(), float(np.ldexp(128 ** -0.5, -e))
    check(call(cache, q, table, [40, 7], 300, scale=scale), q, ks, vs, 300, [40, 7], [1, 1], 3, scale, False)


@pytest.mark.parametrize("t", ["f32", "f16"])
def test_values_of_mixed_size(t):
    """Tokens and blocks whose keys and values differ by many orders of magnitude."""
    rng = np.random.default_rng(18)
    n, d, page = 700, 128, 16
    cache, table, ks, vs = filled(rng, [n, 5], 1, d, page)
    flat = (i32(table[0])[:, None] * page + torch.arange(page, device="cuda", dtype=torch.int32)).reshape(-1)[:n].contiguous()
    for order in (1, -1):
        size = torch.logspace(-4, 3, n, device="cuda")
        size = (size if order > 0 else size.flip(0))[:, None, None] * torch.tensor([1.0, 1e-3, 1e-1, 1e-2], device="cuda").repeat_interleave(32)
        qg.kv_append(cache, torch.randn(n, 1, d, device="cuda") * size.clamp(max=1), torch.randn(n, 1, d, device="cuda") * size, flat)
        k, v = (x.cpu().numpy().astype(np.float64) for x in qg.kv_read(cache, flat))
        q = torch.randn(1, 4, d, device="cuda").to(TYPES[t])
        check(call(cache, q, table, [5], n), q, [k, ks[1]], [v, vs[1]], n, [5], [1], 4, d ** -0.5, t == "f16")


@pytest.mark.parametrize("t", ["f32", "f16"])
def test_where_the_weight_lies(t):
    """All of it on one prefix token, on one own token, in the first and the last of many tiles."""
    rng = np.random.default_rng(3)
    n, d = 3000, 128
    cache, table, ks, vs = filled(rng, [n, 20, 20], 1, d, 64)
    q = torch.zeros(2, 8, d)
    for h, (s, tok) in enumerate([(0, 0), (0, 127), (0, 128), (0, n - 1), (0, 1500), (1, 0), (1, 19), (2, 19)]):
        for i in range(2):
            k = ks[s if s == 0 or s == i + 1 else i + 1][tok, 0]
            q[i, h] = torch.from_numpy(k / np.abs(k).max() * 20)
    q = q.cuda().to(TYPES[t])
    check(call(cache, q, table, [20, 20], n), q, ks, vs, n, [20, 20], [1, 1], 8, d ** -0.5, t == "f16")


# Powers of 2 by which the first token outweighs each of the others. Beside a largest weight of 2^14 the weights' f16 parts
# end at 2^-24: one lies between that and the next step, one below the half of it, others far above.
@pytest.mark.parametrize("less", [38.415, 39.32, 31.415, 32.32, 20.7])
@pytest.mark.parametrize("d", [64, 128])
def test_many_small_equal_weights(d, less):
    """Tokens that are all alike beside one that outweighs them, in parts of the whole prefix: all roundings have one sign.
    A weight is off by 2^-39 of the largest at most (half a step of 2^-24 beside 2^14) and in two parts by 2^-22 of
    itself. The sums over the units, n / 128 additions, round by 2^-24 of them each; where all values are 1 by the same
    above and below the line. A unit's sum is off by 64 additions (2^-24 each) and 32 steps of the products (2^-23)."""
    n, page, seqs, group = (1 << 18) - 16, 128, 320, 64
    pages = -(-n // page)
    cache = qg.KVCache.empty(pages, 1, d, page)
    k, v = torch.zeros(n, 1, d, device="cuda"), torch.ones(n, 1, d, device="cuda")
    k[0, 0, 0] = -8.0  # (a block's scale is 1, its first code 0)
    v[1:, 0, d // 2:] = -3.0
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    qg.kv_append(cache, k, v, slots)
    kept = qg.kv_read(cache, slots)
    assert torch.equal(kept[0], k) and torch.equal(kept[1], v)
    q = torch.zeros(seqs, group, d, device="cuda")
    q[..., 0] = -less * float(np.log(2.0)) / 8.0
    got = qg.kv_attend_shared(cache, q, slots[:pages], i32([n]), i32([[0]] * seqs), i32([0] * seqs), scale=1.0).double().cpu().numpy()
    share = (n - 1) * 2.0 ** (8.0 * float(q[0, 0, 0]) / np.log(2.0))
    of_weights = (n - 1) * 2.0 ** -39 + 2.0 ** -22 * share
    of_units = 64 * 2.0 ** -24 + 32 * 2.0 ** -23
    assert np.abs(got[..., :d // 2] - 1.0).max() <= of_weights + of_units
    want = (1.0 - 3.0 * share) / (1.0 + share)
    assert np.abs(got[..., d // 2:] - want).max() <= of_weights * (want + 3.0) + (of_units + n / 128 * 2.0 ** -24) * (1.0 + 3.0 * share + abs(want))


def test_the_same_as_one_cache():
    """What qkv_attend gives on sequences whose tables begin with the prefix's pages."""
    rng = np.random.default_rng(5)
    d, page, prefix, lens = 128, 64, 64 * 9, [70, 3, 129]
    cache, table, ks, vs = filled(rng, [prefix] + lens, 2, d, page)
    whole = np.concatenate([np.repeat(table[:1, :9], 3, 0), table[1:]], 1)
    q = torch.from_numpy(rng.standard_normal((3, 8, d)).astype(np.float32)).cuda()
    a = call(cache, q, table, lens, prefix)
    b = qg.kv_attend(cache, q, i32(whole), i32([prefix + n for n in lens]))
    assert (a - b).abs().max() < 2e-6 * b.abs().max()


@pytest.mark.parametrize("t,d", [("f32", 64), ("f16", 64), ("f32", 128), ("f16", 128)])
@pytest.mark.parametrize("seqs,group,hk", [(9, 16, 97), (60, 16, 13), (20, 64, 16), (16, 64, 1)])
@pytest.mark.parametrize("pages", [1, 12, 45])
def test_parts_of_many_items(t, d, seqs, group, hk, pages):
    """Thread blocks that go from one head's or rows' tiles to the next ones', and items of one block each: what
    qkv_attend gives on whole tables, within both calls' bounds (each is held to 64 bits elsewhere; a score's error and
    a weight's are those of attn_ref.bound, 2^-17 of the largest value here, and two roundings to f16)."""
    rng = np.random.default_rng(pages * seqs)
    page = 128
    table = torch.arange((pages + seqs), dtype=torch.int32, device="cuda")
    cache = qg.KVCache.empty(pages + seqs, hk, d, page)
    n = (pages + seqs) * page
    for s in range(0, n, 2048):
        m = min(2048, n - s)
        kv = torch.from_numpy(rng.standard_normal((2, m, hk, d)).astype(np.float32)).cuda()
        qg.kv_append(cache, kv[0], kv[1], torch.arange(s, s + m, dtype=torch.int32, device="cuda"))
    lens = i32(rng.integers(1, page, seqs))
    q = torch.from_numpy(rng.standard_normal((seqs, hk * group, d)).astype(np.float32)).cuda().to(TYPES[t])
    own = table[pages:, None].contiguous()
    got = qg.kv_attend_shared(cache, q, table[:pages], i32([pages * page]), own, lens)
    want = qg.kv_attend(cache, q, torch.cat([table[None, :pages].expand(seqs, -1), own], 1).contiguous(), lens + pages * page)
    off = (got.double() - want.double()).abs().max()
    assert off < 4 * 2.0 ** -17 + (2 * 2.0 ** -11 * want.double().abs().max() if t == "f16" else 0), off


def test_strided_queries_out_and_stream():
    rng = np.random.default_rng(19)
    lens = [130, 64, 9]
    cache, table, ks, vs = filled(rng, [400] + lens, 2, 128, 32)
    x = torch.from_numpy(rng.standard_normal((3, 8 + 4, 128)).astype(np.float32)).cuda()
    q = x[:, :8]
    out = torch.full((3, 8, 128), np.nan, device="cuda")
    need = qg.kv_attend_shared_workspace_bytes(cache, 8, 3)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    args = (cache, q, i32(table[0][:13]), i32([400]), i32(table[1:]), i32(lens))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    assert qg.kv_attend_shared(*args, out=out, workspace=ws, stream=side) is out
    side.synchronize()
    check(out, q, ks, vs, 400, lens, [1, 1, 1], 4, 128 ** -0.5, False)
    other = qg.kv_attend_shared(*args, stream=side)
    side.synchronize()
    assert torch.equal(other, out)


def test_captured_with_lengths_that_change():
    """A graph's prefix length, own lengths and queries are read when it runs; two graphs on one workspace take turns."""
    rng = np.random.default_rng(6)
    d, lens = 64, [30, 40]
    cache, table, ks, vs = filled(rng, [1000] + lens, 2, d, 16)
    q = torch.from_numpy(rng.standard_normal((2, 4, d)).astype(np.float32)).cuda()
    pt, pl, tab, ln = i32(table[0][:63]), i32([1000]), i32(table[1:]), i32(lens)
    ws = torch.empty(qg.kv_attend_shared_workspace_bytes(cache, 4, 2), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            qg.kv_attend_shared(cache, q, pt, pl, tab, ln, out=o, workspace=ws)
    for prefix, own in ((1000, [30, 40]), (130, [1, 40]), (0, [30, 0]), (999, [0, 0])):
        pl.copy_(i32([prefix]))
        ln.copy_(i32(own))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        check(outs[0], q, [ks[0][:prefix], ks[1][:own[0]], ks[2][:own[1]]], [vs[0][:prefix], vs[1][:own[0]], vs[2][:own[1]]],
              prefix, own, [1, 1], 2, d ** -0.5, False)


@pytest.mark.parametrize("t", ["f32", "f16"])
def test_nothing_seen(t):
    cache, table, ks, vs = filled(np.random.default_rng(1), [0, 0, 3], 2, 64, 16)
    q = torch.randn(2, 4, 64, device="cuda").to(TYPES[t])
    got = call(cache, q, table, [0, 3], 0)
    assert not got[0].any()
    check(got, q, ks, vs, 0, [0, 3], [1, 1], 2, 64 ** -0.5, t == "f16")


def test_rows_in_no_sequence_are_left():
    rng = np.random.default_rng(2)
    lens = [10, 20, 30]
    cache, table, ks, vs = filled(rng, [200] + lens, 1, 128, 16)
    q = torch.from_numpy(rng.standard_normal((9, 2, 128)).astype(np.float32)).cuda()
    out = torch.full((9, 2, 128), 3.0, device="cuda")
    call(cache, q, table, lens, 200, q_offsets=i32([1, 3, 3, 6]), max_q_len=3, out=out)
    assert (out[:1] == 3).all() and (out[6:] == 3).all()
    check(out[1:6], q[1:6], ks, vs, 200, lens, [2, 0, 3], 2, 128 ** -0.5, False)
    out.fill_(3.0)
    call(cache, q, table, lens, 200, q_offsets=i32([0, 2, 6, 9]), max_q_len=3, out=out)  # the second has four
    assert qg.device_error() == 4
    assert (out[2:6] == 3).all() and not (out[:2] == 3).any() and not (out[6:] == 3).any()


@pytest.mark.parametrize("d,heads,n_seq,max_q_len", [(64, 8, (1 << 20) + 77, 2), (128, 256, 100003, 64), (64, 8, 5000, 300)])
def test_many_sequences_most_of_them_empty(d, heads, n_seq, max_q_len):
    """The bits of a call that names the others alone."""
    rng = np.random.default_rng(23)
    held = sorted({0, 5, 31, 32, 33, n_seq - 1, *range(47, n_seq, 50021)})
    per = rng.integers(1, max_q_len + 1, len(held)) % 7 + 1 if max_q_len > 6 else rng.integers(1, max_q_len + 1, len(held))
    n = int(per.sum())
    own = rng.integers(0, 16, len(held))
    cache = qg.KVCache.empty(20, 1, d, 16)
    kv = torch.from_numpy(rng.standard_normal((2, 320, 1, d)).astype(np.float32)).cuda()
    qg.kv_append(cache, kv[0], kv[1], torch.arange(320, dtype=torch.int32, device="cuda"))
    q = torch.from_numpy(rng.standard_normal((n, heads, d)).astype(np.float32)).cuda()
    table = torch.from_numpy(rng.integers(0, 20, (len(held), 1)).astype(np.int32)).cuda()
    offsets = np.concatenate([[0], np.cumsum(per)]).astype(np.int32)
    args = (cache, q, torch.arange(18, dtype=torch.int32, device="cuda"), i32([283]))
    want = qg.kv_attend_shared(*args, table, i32(own), q_offsets=i32(offsets), max_q_len=max_q_len)
    at = torch.tensor(held, device="cuda")
    all_table, all_own, all_per = torch.zeros(n_seq, 1, dtype=torch.int32, device="cuda"), torch.zeros(n_seq, dtype=torch.int32, device="cuda"), np.zeros(n_seq + 1, np.int64)
    all_table[at], all_own[at], all_per[np.array(held) + 1] = table, i32(own), per
    got = qg.kv_attend_shared(*args, all_table, all_own, q_offsets=i32(np.cumsum(all_per)), max_q_len=max_q_len)
    assert torch.equal(got, want)
    assert qg.device_error() == 0


def test_indexes_out_of_range():
    """A bad page counts as unseen, a length past the table as the table's end."""
    rng = np.random.default_rng(21)
    d, prefix = 64, 250
    cache, table, ks, vs = filled(rng, [prefix, 60], 1, d, 16)
    q = torch.randn(1, 2, d, device="cuda")
    broken = table.copy()
    broken[0, 1], broken[0, 9] = 1 << 20, -7
    got = call(cache, q, broken, [60], prefix)
    assert qg.device_error() == 4
    keep = [t for t in range(prefix) if not 16 <= t < 32 and not 144 <= t < 160]
    check(got, q, [ks[0][keep], ks[1]], [vs[0][keep], vs[1]], len(keep), [60], [1], 2, d ** -0.5, False)
    cache, table, ks, vs = filled(rng, [256, 60], 1, d, 16)
    want = call(cache, q, table, [60], 256)
    for bad in (257, 2 ** 31 - 1):
        got = qg.kv_attend_shared(cache, q, i32(table[0]), i32([bad]), i32(table[1:]), i32([60]))
        assert qg.device_error() == 4 and torch.equal(got, want)
    got = qg.kv_attend_shared(cache, q, i32(table[0]), i32([-1]), i32(table[1:]), i32([60]))
    assert qg.device_error() == 4
    check(got, q, ks, vs, 0, [60], [1], 2, d ** -0.5, False)


@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("bits", [0x7C00, 0xFC00, 0x7E00], ids=["inf", "-inf", "nan"])
@pytest.mark.parametrize("tok", [0, 127, 130, 299])
def test_scales_that_are_not_finite(t, bits, tok):
    """A value block's: NaN in its 32 channels of every row, and nothing else; past the prefix's end: nothing."""
    rng = np.random.default_rng(40)
    n, d = 300, 128
    cache, table, ks, vs = filled(rng, [n, 20], 1, d, 16)
    at = attn_ref.slot_bytes(16, 1, d, int(table[0, tok // 16]) * 16 + tok % 16, 0)[3][2]
    cache.data[torch.from_numpy(at).cuda()] = torch.tensor([bits & 255, bits >> 8], dtype=torch.uint8, device="cuda")
    q = torch.from_numpy(rng.standard_normal((1, 4, d)).astype(np.float32)).cuda().to(TYPES[t])
    got = call(cache, q, table, [20], n)
    block = torch.arange(d, device="cuda") // 32 == 2
    assert torch.equal(torch.isnan(got), block.expand_as(got))
    other = [np.where(np.arange(d) // 32 == 2, 0, v) for v in vs]
    check(torch.where(block, torch.zeros_like(got), got), q, ks, other, n, [20], [1], 4, d ** -0.5, t == "f16")
    check(call(cache, q, table, [20], tok), q, [ks[0][:tok], ks[1]], [vs[0][:tok], vs[1]], tok, [20], [1], 4, d ** -0.5, t == "f16")


@pytest.mark.parametrize("t", ["f32", "f16"])
def test_odd_queries_keep_to_their_row(t):
    rng = np.random.default_rng(31)
    cache, table, ks, vs = filled(rng, [900, 4, 40], 2, 128, 32)
    q = torch.from_numpy(rng.standard_normal((2, 8, 128)).astype(np.float32)).cuda().to(TYPES[t])
    clean = call(cache, q, table, [4, 40], 900)
    q[0, 1, 77] = float("nan")
    q[1, 6, ::9] = float("inf")
    got = call(cache, q, table, [4, 40], 900)
    assert torch.isnan(got[0, 1]).all() and torch.isnan(got[1, 6]).all()
    rest = torch.ones(2, 8, dtype=torch.bool, device="cuda")
    rest[0, 1] = rest[1, 6] = False
    assert torch.equal(got[rest], clean[rest])


def test_a_prefix_past_32_bits():
    """Pages at the far end of a 5 GB cache."""
    hk, d, page, n = 32, 128, 64, 300
    n_pages = 5 * (1 << 30) // (page * hk * 144)
    cache = qg.KVCache.empty(n_pages, hk, d, page)
    rng = np.random.default_rng(22)
    table = np.arange(n_pages - 6, n_pages, dtype=np.int32)
    slots = i32(np.arange((n_pages - 6) * page, (n_pages - 6) * page + n + 64))
    k, v = (torch.randn(n + 64, hk, d, device="cuda") for _ in range(2))
    qg.kv_append(cache, k, v, slots)
    k, v = (x.cpu().numpy().astype(np.float64) for x in qg.kv_read(cache, slots))
    q = torch.from_numpy(rng.standard_normal((1, hk, d)).astype(np.float32)).cuda()
    got = qg.kv_attend_shared(cache, q, i32(table[:5]), i32([n]), i32(table[None, 5:]), i32([40]))
    check(got, q, [k[:n], k[320:360]], [v[:n], v[320:360]], n, [40], [1], 1, d ** -0.5, False)


def batch(seed, t, d=128, hk=2, group=5, prefix=1500, seqs=7, page=32):
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(1, 90, seqs)]
    cache, table, ks, vs = filled(rng, [prefix] + lens, hk, d, page)
    q = torch.from_numpy(rng.standard_normal((seqs, hk * group, d)).astype(np.float32)).cuda().to(TYPES[t])
    return cache, q, i32(table[0][:-(-prefix // page)]), i32([prefix]), i32(table[1:]), i32(lens)


@pytest.mark.parametrize("t", ["f32", "f16"])
def test_an_empty_prefix_table(t):
    a = list(batch(7, t))
    a[2], a[3] = a[2][:0], i32([0])
    assert torch.equal(qg.kv_attend_shared(*a), qg.kv_attend_shared(*a[:2], i32([0]), *a[3:]))
    want = qg.kv_attend(a[0], a[1], a[4], a[5])
    assert (qg.kv_attend_shared(*a).double() - want.double()).abs().max() <= (2.0 ** -17 if t == "f32" else 2.0 ** -9) * want.abs().max()


def test_what_lies_in_the_workspace_does_not_matter():
    """Nor whose it was: two graphs of other shapes and a call on its own share one, each after the other."""
    a, b = batch(8, "f32"), batch(9, "f16", 64, 3, 4, 700, 11, 16)
    want = [qg.kv_attend_shared(*x) for x in (a, b)]
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(x[1]) for x in (a, b)], []
    side = torch.cuda.Stream()
    for x, out in zip((a, b), outs):
        with torch.cuda.stream(side):
            qg.kv_attend_shared(*x, out=out, workspace=ws)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qg.kv_attend_shared(*x, out=out, workspace=ws)
        graphs.append(g)
    for k in (0, 1, 1, 0, 1, 0):
        outs[k].fill_(float("nan"))
        graphs[k].replay()
        assert torch.equal(outs[k], want[k])
        assert torch.equal(qg.kv_attend_shared(*(a, b)[1 - k], workspace=ws), want[1 - k])


@pytest.mark.parametrize("t,d", [("f32", 64), ("f16", 64), ("f32", 128), ("f16", 128)])
@pytest.mark.parametrize("first", [16, 48, 112, 240])
def test_a_workspace_on_a_16_byte_boundary(t, d, first):
    """As many bytes as are asked for, 16 into an allocation; what lies before and behind stays."""
    a = batch(10, t, d, prefix=700)
    want = qg.kv_attend_shared(*a)
    need = qg.kv_attend_shared_workspace_bytes(a[0], a[1].shape[1], a[1].shape[0])
    arena = torch.full((first + need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    assert arena.data_ptr() % 32 == 0
    assert torch.equal(qg.kv_attend_shared(*a, workspace=arena[first:first + need]), want)
    assert (arena[:first] == 0x5A).all() and (arena[first + need:] == 0x5A).all()


@pytest.mark.parametrize("t,d", [("f32", 64), ("f16", 64), ("f32", 128), ("f16", 128)])
@pytest.mark.parametrize("hk,prefix,seqs", [(1, 20000, 30), (7, 3000, 60), (40, 1000, 60)])
def test_the_same_bits_beside_other_work(t, d, hk, prefix, seqs):
    """Many calls, two at a time on two streams and beside products that keep the multiprocessors busy now and then: the
    roles of a block then run at other paces towards each other."""
    a, b = batch(11, t, d, hk, 16, prefix, seqs, 64), batch(12, t, d, 2, 16, 900, 40, 16)
    want = [qg.kv_attend_shared(*x) for x in (a, b)]
    m = torch.randn(1024, 1024, device="cuda").half()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(12):
        got = []
        for x, s in zip((a, b), streams):
            got.append([qg.kv_attend_shared(*x, stream=s) for _ in range(3)])
        with torch.cuda.stream(streams[2]):
            for _ in range(i % 4):
                m @ m
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, w) for x in g)


def test_refusals():
    cache = qg.KVCache.empty(4, 2, 128, 16)
    q, pt, pl, tab, ln = torch.zeros(2, 4, 128, device="cuda"), i32([0]), i32([9]), i32([[1], [2]]), i32([3, 4])
    f = qg.kv_attend_shared
    bad = [(TypeError, lambda: f(cache, q.double(), pt, pl, tab, ln)),
           (TypeError, lambda: f(cache, q, pt.long(), pl, tab, ln)),
           (TypeError, lambda: f(cache, q, pt, pl.float(), tab, ln)),
           (TypeError, lambda: f(cache, q, pt, 9, tab, ln)),
           (ValueError, lambda: f(cache, q, pt[None], pl, tab, ln)),
           (ValueError, lambda: f(cache, q, pt, ln, tab, ln)),
           (ValueError, lambda: f(cache, q[:1], pt, pl, tab, ln)),
           (ValueError, lambda: f(cache, q, pt, pl, tab[:1], ln)),
           (ValueError, lambda: f(cache, q, pt, pl, tab, ln, out=q[:1])),
           (qg.QGError, lambda: f(cache, q, pt, pl, tab, ln, max_q_len=0)),
           (qg.QGError, lambda: f(cache, q, pt, pl, tab, ln, scale=float("inf"))),
           (qg.QGError, lambda: f(cache, q, pt, pl, tab, ln, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")))]
    for error, go in bad:
        with pytest.raises(error):
            go()
    assert f(cache, q[:0], pt, pl, tab[:0], ln[:0]).shape == (0, 4, 128)
    assert qg.device_error() == 0
