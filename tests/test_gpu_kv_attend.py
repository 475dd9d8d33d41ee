"""qkv_attend against the formula in 64 bits (attn_ref.attend) on the cache's own
values. The tolerance is attn_ref.bound: f32 queries and weights carry 20 bits
or more, f16 queries are exact and their weights carry 11 (2^-10 of a weight
at most, with the value's scale folded in)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attn_ref  # noqa: E402
import ggml_block_quantized_gb300 as qg  # noqa: E402

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


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def filled(rng, lens, hk, d, page, k_size=1.0, v_size=1.0, garbage=True, extra=2):
    """A cache of sequences of the given lengths in shuffled pages; what is not
    written is random bytes (NaN and infinite scales among them). Returns the
    cache, the table (-1 past the used pages), and each sequence's k and v in f64."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + extra
    data = torch.from_numpy(rng.integers(0, 256, n_pages * hk * page * d // 8 * 9).astype(np.uint8)).cuda()
    if garbage:  # half of the scales of what is not written are NaN or infinite
        data.view(torch.float16)[torch.rand(data.numel() // 2, device="cuda") < 0.5] = float("nan")
        data.view(torch.float16)[torch.rand(data.numel() // 2, device="cuda") < 0.2] = float("inf")
    cache = qg.KVCache(hk, d, page, data)
    pages = rng.permutation(n_pages)
    table = np.full((len(lens), max(need + [1])), -1, np.int32)
    slots, used = [], 0
    for s, n in enumerate(lens):
        mine = pages[used:used + need[s]]
        used += need[s]
        table[s, :need[s]] = mine
        slots.append((mine[:, None].astype(np.int64) * page + np.arange(page)).reshape(-1)[:n])
    flat = np.concatenate(slots) if slots else np.zeros(0)
    k = rng.standard_normal((len(flat), hk, d)).astype(np.float32) * np.float32(k_size)
    v = (rng.standard_normal((len(flat), hk, d)).astype(np.float32) + np.float32(0.3)) * np.float32(v_size)
    kd, vd = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    qg.kv_append(cache, kd, vd, i32(flat))
    kr, vr = (t.cpu().numpy().astype(np.float64) for t in qg.kv_read(cache, i32(flat)))
    cut = np.cumsum([0] + list(lens))
    return cache, table, [kr[a:b] for a, b in zip(cut, cut[1:])], [vr[a:b] for a, b in zip(cut, cut[1:])]


def check(got, q, ks, vs, lens, q_lens, group, scale, f16):
    """Every row of got [n_tok, heads, D] against the formula, within the bound."""
    got, q = got.detach().cpu().numpy().astype(np.float64), q.cpu().numpy().astype(np.float64)
    d, at = q.shape[2], 0
    for s, m in enumerate(q_lens):
        seen = [lens[s] - m + i + 1 for i in range(m)]
        for h in range(q.shape[1]):
            out, pv, mag, big = attn_ref.attend(q[at:at + m, h], ks[s][:, h // group], vs[s][:, h // group], seen, scale)
            tol = attn_ref.bound(out, pv, mag, big, d, lens[s], 24 if f16 else 20, 10 if f16 else 20, f16)
            err = np.abs(got[at:at + m, h] - out)
            assert np.isfinite(got[at:at + m, h]).all(), (s, h)
            assert (err <= tol).all(), (s, h, float((err / tol).max()))
            for i in range(m):
                if seen[i] <= 0:
                    assert not got[at + i, h].any()
        at += m


CASES = [  # D, type, kv heads, group, page, lengths, queries of each sequence (None: one)
    (128, "f32", 8, 4, 64, [777], None), (128, "f16", 8, 4, 64, [777], None),
    (128, "f32", 2, 1, 16, [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129], None),
    (64, "f16", 3, 1, 16, [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129], None),
    (64, "f32", 1, 8, 32, [300, 5, 1000], None), (128, "f16", 1, 7, 48, [511, 513, 2049], None),
    (128, "f32", 2, 3, 32, [90, 7, 260], [5, 3, 2]), (64, "f16", 4, 4, 16, [41, 3, 0, 500], [4, 8, 2, 7]),
    (128, "f16", 1, 16, 64, [200, 70], [2, 0]), (64, "f32", 2, 5, 128, [129, 1], [1, 4]),
    (128, "f32", 1, 8, 16, [333], [37]), (64, "f32", 1, 64, 64, [150, 40], [2, 3]),
    (128, "f16", 1, 40, 64, [150, 40], None), (128, "f32", 32, 1, 16, [257, 100, 31], None),
    (128, "f32", 1, 1, 128, [40000], None), (64, "f16", 2, 8, 64, [30011, 5], None),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", "")[:60])
def test_attend(case):
    d, t, hk, group, page, lens, q_lens = case
    rng = np.random.default_rng(sum(map(ord, str(case))))
    cache, table, ks, vs = filled(rng, lens, hk, d, page)
    per = q_lens or [1] * len(lens)
    q = torch.from_numpy(rng.standard_normal((sum(per), hk * group, d)).astype(np.float32) * 1.5).cuda().to(TYPES[t])
    offsets = i32(np.cumsum([0] + per)) if q_lens else None
    got = qg.kv_attend(cache, q, i32(table), i32(lens), q_offsets=offsets, max_q_len=max(per))
    assert got.dtype == q.dtype
    check(got, q, ks, vs, lens, per, group, d ** -0.5, t == "f16")
    again = qg.kv_attend(cache, q, i32(table), i32(lens), q_offsets=offsets, max_q_len=max(per) + 3)
    check(again, q, ks, vs, lens, per, group, d ** -0.5, t == "f16")
    assert torch.equal(got, qg.kv_attend(cache, q, i32(table), i32(lens), q_offsets=offsets, max_q_len=max(per)))


@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("k_size,v_size,q_size,scale", [
    (1, 1, 1, -0.2), (1, 1, 1, 0.0), (30, 1, 8, 1.0), (1, 3e3, 1, 0.09), (1, 1e-4, 1, 0.09), (1e-4, 1, 300, 0.09),
    (2e3, 1, 1e-4, 0.09)])
def test_sizes_of_values(t, k_size, v_size, q_size, scale):
    """Steep, flat and reversed softmaxes; keys, values and queries far from 1."""
    rng = np.random.default_rng(17)
    lens = [700, 33]
    cache, table, ks, vs = filled(rng, lens, 2, 128, 64, k_size, v_size)
    q = torch.from_numpy(rng.standard_normal((2, 6, 128)).astype(np.float32) * q_size).cuda().to(TYPES[t])
    got = qg.kv_attend(cache, q, i32(table), i32(lens), scale=scale)
    check(got, q, ks, vs, lens, [1, 1], 3, scale, t == "f16")


@pytest.mark.parametrize("e", [-125, -118, -100, 90, 110, 120])
def test_queries_near_the_ends_of_f32(e):
    """Queries of 2^e with a scale of 2^-e: the scores are ordinary ones."""
    rng = np.random.default_rng(42)
    lens = [300, 40]
    cache, table, ks, vs = filled(rng, lens, 2, 128, 64)
    q = np.ldexp(rng.standard_normal((2, 6, 128)).astype(np.float32).astype(np.float64), e).astype(np.float32)
    q, scale = torch.from_numpy(q).cuda(), float(np.ldexp(128 ** -0.5, -e))
    check(qg.kv_attend(cache, q, i32(table), i32(lens), scale=scale), q, ks, vs, lens, [1, 1], 3, scale, False)


def test_values_of_mixed_size():
    """Tokens whose values differ by ten orders of magnitude, large ones late and early."""
    rng = np.random.default_rng(18)
    n, d = 600, 64
    for order in (1, -1):
        cache, table, ks, vs = filled(rng, [n], 1, d, 16)
        flat = (i32(table[0])[:, None] * 16 + torch.arange(16, device="cuda", dtype=torch.int32)).reshape(-1)[:n]
        size = torch.logspace(-5, 3, n, device="cuda")[::1]
        v = torch.randn(n, 1, d, device="cuda") * (size if order > 0 else size.flip(0))[:, None, None]
        qg.kv_append(cache, torch.randn(n, 1, d, device="cuda"), v, flat.contiguous())
        k, v = (x.cpu().numpy().astype(np.float64) for x in qg.kv_read(cache, flat.contiguous()))
        for t in ("f32", "f16"):
            q = torch.randn(1, 4, d, device="cuda").to(TYPES[t])
            check(qg.kv_attend(cache, q, i32(table), i32([n])), q, [k], [v], [n], [1], 4, d ** -0.5, t == "f16")


@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("by", ["token", "block", "both"])
@pytest.mark.parametrize("d,n", [(128, 512), (64, 97)])
def test_strong_scores_beside_large_values(d, n, by, t):
    """Tokens with nearly all of the weight and values 10^7 times smaller than the others', and blocks of a head 10^4
    times smaller than its largest: the loss is of the largest weighted value's size, not of the largest value's
    (attn_ref.tight_bound)."""
    rng = np.random.default_rng(43)
    cache, table, _, _ = filled(rng, [n], 1, d, 16)
    flat = (i32(table[0])[:, None] * 16 + torch.arange(16, device="cuda", dtype=torch.int32)).reshape(-1)[:n].contiguous()
    q = rng.standard_normal((1, 4, d)).astype(np.float32)
    k, v = (rng.standard_normal((n, 1, d)).astype(np.float32) for _ in range(2))
    if by != "block":
        v *= 1e4
        for h in range(4):
            k[n // 5 + n // 7 * h, 0] = q[0, h] * 8
            v[n // 5 + n // 7 * h, 0] *= 1e-7
    if by != "token":
        v *= np.resize(np.repeat(np.float32([1, 1e-2, 1e-4, 1e-1]), 32), d)
    qg.kv_append(cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), flat)
    kr, vr = (x.cpu().numpy().astype(np.float64)[:, 0] for x in qg.kv_read(cache, flat))
    q = torch.from_numpy(q).cuda().to(TYPES[t])
    got = qg.kv_attend(cache, q, i32(table), i32([n]))[0].cpu().numpy().astype(np.float64)
    out, tol = attn_ref.tight_bound(q[0].cpu().numpy().astype(np.float64), kr, vr, d ** -0.5, t == "f16")
    assert (np.abs(got - out) <= tol).all(), float((np.abs(got - out) / tol).max())


def test_strided_queries_out_and_stream():
    rng = np.random.default_rng(19)
    lens = [130, 64, 9]
    cache, table, ks, vs = filled(rng, lens, 2, 128, 32)
    x = torch.from_numpy(rng.standard_normal((3, 8 + 4, 128)).astype(np.float32)).cuda()
    q = x[:, :8]
    assert not q.is_contiguous()
    out = torch.full((3, 8, 128), np.nan, device="cuda")
    need = qg.kv_attend_workspace_bytes(cache, 8)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    tab, ln = i32(table), i32(lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    assert qg.kv_attend(cache, q, tab, ln, out=out, workspace=ws, stream=side) is out
    side.synchronize()
    check(out, q, ks, vs, lens, [1, 1, 1], 4, 128 ** -0.5, False)
    other = qg.kv_attend(cache, q, tab, ln, stream=side)
    side.synchronize()
    assert torch.equal(other, out)


def test_infinite_and_nan_tokens_reach_only_those_who_see_them():
    rng = np.random.default_rng(20)
    n, d = 100, 128
    cache, table, ks, vs = filled(rng, [n], 1, d, 16)
    slot = lambda t: int(table[0, t // 16]) * 16 + t % 16  # noqa: E731
    bad = torch.full((1, 1, d), float("inf"), device="cuda")
    good = torch.ones(1, 1, d, device="cuda")
    qg.kv_append(cache, good, bad, i32([slot(97)]))  # its values are infinite: d = -inf, f16
    q = torch.randn(6, 4, d, device="cuda")
    got = qg.kv_attend(cache, q, i32(table), i32([n]), q_offsets=i32([0, 6]), max_q_len=6)
    assert torch.isfinite(got[:3]).all()  # tokens 94, 95, 96
    assert not torch.isfinite(got[3:]).all(-1).any()
    check(got[:3], q[:3], [ks[0][:97]], [vs[0][:97]], [97], [3], 4, d ** -0.5, False)


@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("d,group,per", [(64, 2, 4), (128, 3, 4), (128, 1, 8), (64, 3, 5)], ids=lambda x: str(x))
def test_segments_one_after_another_in_a_thread_block(d, group, per, t):
    """More segments than thread blocks, each of a few tiles, so that a block goes from one to the next; in every other
    sequence the values of a token that only the later queries see are not finite. Each row has its own result in its
    own place, NaN in the affected block's channels where it sees the token, and the same bits each time."""
    rng = np.random.default_rng(41)
    n_seq, hk = 150, 8
    lens = rng.integers(per, 120, n_seq).tolist()
    cache, table, ks, vs = filled(rng, lens, hk, d, 16)
    marked = list(range(0, n_seq, 2))
    for s in marked:  # the third token from the end: its second value block's scale becomes NaN
        tok = lens[s] - 3
        slot = int(table[s, tok // 16]) * 16 + tok % 16
        for h in range(hk):
            at = attn_ref.slot_bytes(16, hk, d, slot, h)[3][1]
            cache.data[torch.from_numpy(at).cuda()] = torch.tensor([0, 0x7E], dtype=torch.uint8, device="cuda")
    q = torch.from_numpy(rng.standard_normal((n_seq * per, hk * group, d)).astype(np.float32)).cuda().to(TYPES[t])
    off = i32(np.arange(n_seq + 1) * per)
    got = qg.kv_attend(cache, q, i32(table), i32(lens), q_offsets=off, max_q_len=per)
    for _ in range(10):
        again = qg.kv_attend(cache, q, i32(table), i32(lens), q_offsets=off, max_q_len=per)
        assert torch.equal(got.nan_to_num(7.0), again.nan_to_num(7.0))
    sees = torch.zeros(n_seq, per, dtype=torch.bool, device="cuda")
    sees[::2, per - 3:] = True
    nan = torch.isnan(got)
    want = sees.view(-1, 1, 1) & ((torch.arange(d, device="cuda") // 32) == 1)
    assert torch.equal(nan, want.expand_as(nan))
    filled_in = torch.where(nan, torch.zeros_like(got), got)
    some = [s for s in range(n_seq) if s % 2 or s % 10 == 0]
    for s in some:
        rows = slice(s * per, (s + 1) * per)
        keep = torch.ones(per, dtype=torch.bool) if s % 2 else ~sees[s].cpu()
        m = int(keep.sum())
        check(filled_in[rows][:m], q[rows][:m], [ks[s][:lens[s] - per + m]], [vs[s][:lens[s] - per + m]],
              [lens[s] - per + m], [m], group, d ** -0.5, t == "f16")


@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("bits", [0x7C00, 0xFC00, 0x7E00], ids=["inf", "-inf", "nan"])
@pytest.mark.parametrize("tok", [3, 40, 94, 95, 96, 98, 99])
def test_a_value_scale_that_is_not_finite(t, bits, tok):
    """All 32 channels of its block are NaN in the rows that see its token, and nothing else is, wherever among the
    tiles and the rows' limits the token lies."""
    rng = np.random.default_rng(40)
    n, d, m = 100, 128, 6
    for group in (4, 2):
        cache, table, ks, vs = filled(rng, [n], 1, d, 16)
        slot = int(table[0, tok // 16]) * 16 + tok % 16
        at = attn_ref.slot_bytes(16, 1, d, slot, 0)[3][2]
        cache.data[torch.from_numpy(at).cuda()] = torch.tensor([bits & 255, bits >> 8], dtype=torch.uint8, device="cuda")
        q = torch.from_numpy(rng.standard_normal((m, group, d)).astype(np.float32)).cuda().to(TYPES[t])
        got = qg.kv_attend(cache, q, i32(table), i32([n]), q_offsets=i32([0, m]), max_q_len=m)
        sees = torch.arange(m, device="cuda") + n - m >= tok
        want = sees.view(-1, 1, 1) & (torch.arange(d, device="cuda") // 32 == 2)
        assert torch.equal(torch.isnan(got), want.expand_as(got))
        # the other channels as if the block were of zeros
        ref = [attn_ref.attend(q[:, h].cpu().numpy().astype(np.float64), ks[0][:, 0], np.where(np.arange(d) // 32 == 2, 0, vs[0][:, 0]),
                               n - m + 1 + np.arange(m), d ** -0.5) for h in range(group)]
        for h, (out, pv, mag, big) in enumerate(ref):
            tol = attn_ref.bound(out, pv, mag, big, d, n, 24 if t == "f16" else 20, 10 if t == "f16" else 20, t == "f16")
            other = np.arange(d) // 32 != 2
            assert (np.abs(got[:, h].cpu().numpy().astype(np.float64) - out) <= tol)[:, other].all()


@pytest.mark.parametrize("t", [torch.float32, torch.float16], ids=["f32", "f16"])
@pytest.mark.parametrize("lens", [[5, 40], [777, 3, 40000]], ids=["short", "split"])
def test_nan_queries_give_nan(t, lens):
    """A query that is not a number makes its own row NaN, split over thread blocks or not, and no other one."""
    rng = np.random.default_rng(31)
    cache, table, ks, vs = filled(rng, lens, 2, 128, 32)
    q = torch.from_numpy(rng.standard_normal((len(lens), 8, 128)).astype(np.float32)).cuda().to(t)
    clean = qg.kv_attend(cache, q, i32(table), i32(lens))
    check(clean, q, ks, vs, lens, [1] * len(lens), 4, 128 ** -0.5, t == torch.float16)
    q[0, 1, 77] = float("nan")
    q[-1, 6] = float("nan")
    got = qg.kv_attend(cache, q, i32(table), i32(lens))
    assert torch.isnan(got[0, 1]).all() and torch.isnan(got[-1, 6]).all()
    rest = torch.ones(len(lens), 8, dtype=torch.bool, device="cuda")
    rest[0, 1] = rest[-1, 6] = False
    assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("t", [torch.float32, torch.float16], ids=["f32", "f16"])
def test_infinite_queries_give_nan(t):
    """Infinities in a query have scores of both signs of it, or NaN: its row is NaN, and no other one."""
    rng, lens = np.random.default_rng(36), [300, 9000]
    cache, table, ks, vs = filled(rng, lens, 2, 64, 16)
    q = torch.from_numpy(rng.standard_normal((2, 6, 64)).astype(np.float32)).cuda().to(t)
    clean = qg.kv_attend(cache, q, i32(table), i32(lens))
    q[0, 4, ::9], q[1, 0, ::5] = float("inf"), -float("inf")
    got = qg.kv_attend(cache, q, i32(table), i32(lens))
    assert torch.isnan(got[0, 4]).all() and torch.isnan(got[1, 0]).all()
    rest = torch.ones(2, 6, dtype=torch.bool, device="cuda")
    rest[0, 4] = rest[1, 0] = False
    assert torch.equal(got[rest], clean[rest])


def test_indexes_out_of_range():
    """A bad page counts as unseen, a length past the table as the table's end, a bad sequence is left out."""
    rng = np.random.default_rng(21)
    d, lens = 64, [60, 60, 60, 60]
    cache, table, ks, vs = filled(rng, lens, 1, d, 16)
    q = torch.randn(4, 2, d, device="cuda")
    ref = qg.kv_attend(cache, q, i32(table), i32([60, 60, 64, 0]))
    broken = table.copy()
    broken[0, 1], broken[1, 3] = 1 << 20, -7
    got = qg.kv_attend(cache, q, i32(broken), i32([60, 60, 1000, -3]))
    assert qg.device_error() == 4
    keep0 = [t for t in range(60) if not 16 <= t < 32]
    check(got[:1], q[:1], [ks[0][keep0]], [vs[0][keep0]], [44], [1], 2, d ** -0.5, False)
    check(got[1:2], q[1:2], [ks[1][:48]], [vs[1][:48]], [48], [1], 2, d ** -0.5, False)
    assert not got[3].any()
    assert bool(torch.isfinite(got[2]).all()) == bool(torch.isfinite(ref[2]).all())
    out = torch.full((4, 2, d), 3.0, device="cuda")
    qg.kv_attend(cache, q, i32(table), i32(lens), q_offsets=i32([0, 1, 0, 4, 9]), max_q_len=2, out=out)
    assert qg.device_error() == 4
    assert bool((out[1:] == 3).all()) and not bool((out[0] == 3).any())


def test_a_length_past_the_table_is_the_tables_end():
    """And one below zero no tokens, whatever its place among the sequences."""
    rng = np.random.default_rng(48)
    lens = [48, 20, 48, 5]
    cache, table, ks, vs = filled(rng, lens, 2, 128, 16)
    q = torch.from_numpy(rng.standard_normal((4, 4, 128)).astype(np.float32)).cuda()
    want = qg.kv_attend(cache, q, i32(table), i32([48, 0, 48, 5]))
    check(want, q, ks, vs, [48, 0, 48, 5], [1] * 4, 2, 128 ** -0.5, False)
    assert qg.device_error() == 0
    for bad in ([49, -1, 2 ** 31 - 1, 5], [1 << 20, -2 ** 31, 48, 5]):
        assert torch.equal(qg.kv_attend(cache, q, i32(table), i32(bad)), want)
        assert qg.device_error() == 4


@pytest.mark.parametrize("t", ["f32", "f16"])
def test_very_large_scores(t):
    """Scores up to 2^23: all of the weight is on the token with the largest one, whose values are the result."""
    rng = np.random.default_rng(49)
    n, d = 700, 128
    cache, table, ks, vs = filled(rng, [n], 1, d, 32)
    q = torch.from_numpy(rng.standard_normal((1, 4, d)).astype(np.float32)).cuda().to(TYPES[t])
    s = q[0].cpu().numpy().astype(np.float64) @ ks[0][:, 0].T
    scale = 0.9 * 2.0 ** 23 / np.abs(s).max()
    two = np.sort(s * scale, -1)[:, -2:]
    assert (two[:, 1] - two[:, 0] > 2.0 ** 12).all()  # far above the scores' error, 2^-20 of 2^23 times D terms' size
    got = qg.kv_attend(cache, q, i32(table), i32([n]), scale=scale)[0].cpu().numpy().astype(np.float64)
    v = vs[0][s.argmax(-1), 0]
    assert (np.abs(got - v) <= (2.0 ** -20 + (2.0 ** -10 if t == "f16" else 0)) * np.abs(v)).all()


def test_a_long_cache_past_32_bits():
    """A sequence at the far end of a 5 GB cache."""
    hk, d, page, n = 32, 128, 64, 300
    n_pages = 5 * (1 << 30) // (page * hk * 144)
    cache = qg.KVCache.empty(n_pages, hk, d, page)
    rng = np.random.default_rng(22)
    table = np.arange(n_pages - 5, n_pages, dtype=np.int32)[None]
    slots = i32(np.arange((n_pages - 5) * page, (n_pages - 5) * page + n))
    k, v = (torch.randn(n, hk, d, device="cuda") for _ in range(2))
    qg.kv_append(cache, k, v, slots)
    k, v = (x.cpu().numpy().astype(np.float64) for x in qg.kv_read(cache, slots))
    q = torch.from_numpy(rng.standard_normal((1, hk, d)).astype(np.float32)).cuda()
    check(qg.kv_attend(cache, q, i32(table), i32([n])), q, [k], [v], [n], [1], 1, d ** -0.5, False)


def test_refusals():
    cache = qg.KVCache.empty(4, 2, 128, 16)
    q, tab, ln = torch.zeros(2, 4, 128, device="cuda"), i32([[0, 1], [2, 3]]), i32([3, 4])
    bad = [(TypeError, lambda: qg.kv_attend(cache, q.double(), tab, ln)),
           (TypeError, lambda: qg.kv_attend(cache, q, tab.long(), ln)),
           (ValueError, lambda: qg.kv_attend(cache, q[:, :3], tab, ln)),
           (ValueError, lambda: qg.kv_attend(cache, q[..., :64], tab, ln)),
           (ValueError, lambda: qg.kv_attend(cache, q[:1], tab, ln)),
           (ValueError, lambda: qg.kv_attend(cache, q, tab[:1], ln)),
           (ValueError, lambda: qg.kv_attend(cache, q, tab, ln, q_offsets=i32([0, 1]))),
           (TypeError, lambda: qg.kv_attend(cache, q, tab, ln, out=q.half())),
           (ValueError, lambda: qg.kv_attend(cache, q, tab, ln, out=q[:1])),
           (qg.QGError, lambda: qg.kv_attend(cache, q, tab, ln, max_q_len=0)),
           (qg.QGError, lambda: qg.kv_attend(cache, q, tab, ln, scale=float("nan"))),
           (qg.QGError, lambda: qg.kv_attend(cache, q, tab, ln, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")))]
    for error, call in bad:
        with pytest.raises(error):
            call()
    assert qg.kv_attend(cache, q[:0], tab[:0], ln[:0]).shape == (0, 4, 128)
    assert qg.device_error() == 0
