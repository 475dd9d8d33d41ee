"""qkv_append and qkv_read against the rule they are defined by: the rotation's
f32 steps (numpy rounds each, as the formula does), the oracle's Q4_0 on the
rotated rows, and the cache layout written out byte by byte. Everything but
the f16 outputs of f32 rows is one rounding after another, so all of it is
compared bit for bit."""
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


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def i32(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


def same_bits(a, b):
    u = {4: np.uint32, 2: np.uint16, 1: np.uint8}
    return np.array_equal(np.ascontiguousarray(a).view(u[a.itemsize]), np.ascontiguousarray(b).view(u[b.itemsize]))


CASES = [  # n_tok, heads, kv_heads, D, rot, pairs, in, out, page, fused (q, k and v cut out of one product)
    (1, 8, 8, 128, 128, False, "f32", "f32", 16, False), (1, 5, 1, 64, 64, True, "f16", "f16", 16, False),
    (7, 12, 4, 128, 64, False, "f16", "f32", 32, True), (33, 6, 3, 64, 32, False, "f32", "f16", 48, True),
    (50, 4, 2, 128, 8, True, "f32", "f16", 64, True), (19, 7, 7, 64, 56, False, "f16", "f16", 16, False),
    (130, 16, 2, 128, 128, True, "f32", "f32", 128, True), (257, 3, 1, 64, 40, False, "f32", "f32", 16, True),
    (64, 32, 8, 128, 128, False, "f16", "f16", 64, True), (5, 2, 1, 128, 0, False, "f32", "f32", 16, False),
    # rows enough for two a warp, and for eight; heads that do not divide by them
    (301, 14, 7, 128, 96, False, "f16", "f32", 32, True), (1201, 6, 3, 64, 64, True, "f32", "f32", 16, False),
    (1201, 54, 9, 128, 128, False, "f16", "f16", 64, True), (3101, 48, 2, 64, 0, False, "f32", "f16", 16, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_append_bytes(case):
    n, heads, hk, d, rot, pairs, tin, tout, page, fused = case
    rng = np.random.default_rng(sum(map(ord, str(case))))
    x = (rng.standard_normal((n, heads + 2 * hk, d)) * np.exp(rng.standard_normal((1, heads + 2 * hk, 1)) * 3))
    x = x.astype(np.float16 if tin == "f16" else np.float32)
    x[0, heads:, :32] = 0  # a block of zeros
    x[-1, heads + hk:, 32:64] = x[-1, heads + hk:, 32:33]  # magnitudes that tie
    x[-1, heads + hk:, 33:64:2] *= -1
    xd = dev(x)
    q, k, v = xd[:, :heads], xd[:, heads:heads + hk], xd[:, heads + hk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    n_pages = -(-n // page) + 2
    slots = rng.permutation(n_pages * page)[:n].astype(np.int32)
    slots[n // 2] = slots[n // 2] if n < 3 else -1
    table = rng.standard_normal((77, rot // 2, 2)).astype(np.float32) if rot else None
    pos = rng.integers(0, 77, n).astype(np.int32)
    filler = rng.integers(0, 256, n_pages * page * hk * d // 8 * 9).astype(np.uint8)
    cache = qg.KVCache(hk, d, page, dev(filler))
    k_out, v_out = (torch.empty(n, hk, d, dtype=TYPES[tout], device="cuda") for _ in range(2))
    q_out = torch.empty(n, heads, d, dtype=TYPES[tout], device="cuda")
    got = qg.kv_append(cache, k, v, dev(slots), positions=dev(pos) if rot else None, rope=dev(table) if rot else None,
                       rope_pairs=pairs, q=q, q_out=q_out, k_out=k_out, v_out=v_out)
    assert got is q_out
    xf = x.astype(np.float32)
    qr, kr, vr = xf[:, :heads], xf[:, heads:heads + hk], xf[:, heads + hk:]
    if rot:
        qr, kr = (attn_ref.rotate(t, table[pos], pairs, np.float32) for t in (qr, kr))
    want = filler.copy()
    rows = {}
    for i, s in enumerate(slots):
        if s < 0:
            continue
        for h in range(hk):
            at = attn_ref.slot_bytes(page, hk, d, int(s), h)
            rows[i, h] = []
            for c, (r, codes, scales) in enumerate(((kr, at[0], at[2]), (vr, at[1], at[3]))):
                sc, co = attn_ref.q4_0(r[i, h][None])
                want[codes], want[scales] = co[0], np.ascontiguousarray(sc[0]).view(np.uint8).reshape(-1, 2)
                rows[i, h].append(attn_ref.q4_0_values(sc, co)[0])
    assert np.array_equal(cache.data.cpu().numpy(), want)
    npt = np.float16 if tout == "f16" else np.float32
    for t, r in ((q_out, qr), (k_out, kr), (v_out, vr)):
        assert same_bits(t.cpu().numpy(), r.astype(npt))
    # the values of the rows, from both and from either
    k_rows, v_rows = qg.kv_read(cache, dev(slots))
    for i in range(n):
        for h in range(hk):
            a, b = rows.get((i, h), (np.zeros(d), np.zeros(d)))
            assert np.array_equal(k_rows[i, h].cpu().numpy().astype(np.float64), a)
            assert np.array_equal(v_rows[i, h].cpu().numpy().astype(np.float64), b)
    alone = torch.full_like(v_rows, np.nan)
    assert qg.kv_read(cache, dev(slots), v_out=alone)[0] is None and torch.equal(alone, v_rows)
    alone.fill_(np.nan)
    qg.kv_read(cache, dev(slots), k_out=alone)
    assert torch.equal(alone, k_rows)


@pytest.mark.parametrize("n,heads,hk", [(3, 2, 1), (40, 8, 2), (1500, 4, 4), (1500, 6, 2), (9000, 16, 1), (9000, 18, 3)])
def test_batches_that_end_with_the_heads(n, heads, hk):
    """Heads of 64, two side by side in a warp, one, two and eight pairs at a time: query heads that fill a token's
    last batch, and ones that end a head or a pair before its end, each rotated by halves."""
    d, page = 64, 16
    rng = np.random.default_rng(n + heads)
    x = rng.standard_normal((n, heads + 2 * hk, d)).astype(np.float32)
    table, pos = rng.standard_normal((31, d // 2, 2)).astype(np.float32), rng.integers(0, 31, n).astype(np.int32)
    cache = qg.KVCache.empty(-(-n // page), hk, d, page)
    xd = dev(x)
    q, k, v = xd[:, :heads], xd[:, heads:heads + hk], xd[:, heads + hk:]
    k_out = torch.empty(n, hk, d, device="cuda")
    got = qg.kv_append(cache, k, v, dev(np.arange(n, dtype=np.int32)), positions=dev(pos), rope=dev(table), q=q, k_out=k_out)
    assert same_bits(got.cpu().numpy(), attn_ref.rotate(x[:, :heads], table[pos], False, np.float32))
    assert same_bits(k_out.cpu().numpy(), attn_ref.rotate(x[:, heads:heads + hk], table[pos], False, np.float32))


def test_special_values_keep_the_quantizer_rule():
    """NaN, infinite and subnormal rows get the bytes that Q4_0's rule gives them."""
    d, page = 128, 16
    rng = np.random.default_rng(5)
    x = rng.standard_normal((6, 1, d)).astype(np.float32)
    x[0, 0, 3] = np.nan
    x[1, 0, 40:50] = np.inf
    x[2, 0, 64:96] = np.nan
    x[3, 0, :32] *= np.float32(1e-41)
    x[3, 0, 32:64] *= np.float32(1e30)
    x[4, 0, 5] = -np.inf
    x[5] = -0.0
    cache = qg.KVCache(1, d, page, torch.zeros(16 * 144, dtype=torch.uint8, device="cuda"))
    qg.kv_append(cache, dev(x), dev(x), i32(range(6)))
    got = cache.data.cpu().numpy()
    for i in range(6):
        at = attn_ref.slot_bytes(page, 1, d, i, 0)
        sc, co = attn_ref.q4_0(x[i])
        for c, s in ((at[0], at[2]), (at[1], at[3])):
            assert np.array_equal(got[c], co[0])
            assert np.array_equal(got[s], np.ascontiguousarray(sc[0]).view(np.uint8).reshape(-1, 2))


def test_in_place_no_query_and_empty():
    rng = np.random.default_rng(6)
    n, d, table = 9, 128, qg.rope_table(32, 128)
    x = dev(rng.standard_normal((n, 2, d)).astype(np.float32))
    pos = i32(range(n))
    make = lambda: qg.KVCache(2, d, 16, torch.zeros(16 * 2 * 144, dtype=torch.uint8, device="cuda"))  # noqa: E731
    a, b = make(), make()
    q = x.clone()
    qg.kv_append(a, x, x, pos, positions=pos, rope=table, q=q, q_out=q)
    assert qg.kv_append(b, x, x, pos, positions=pos, rope=table) is None
    assert torch.equal(a.data, b.data)
    fresh = qg.kv_append(a, x, x, pos, positions=pos, rope=table, q=x)
    assert torch.equal(fresh, q) and fresh.dtype == torch.float32
    y = x.clone()
    qg.kv_append(a, y, x, pos, positions=pos, rope=table, k_out=y)
    assert torch.equal(y, q) and torch.equal(a.data, b.data)
    empty = x[:0]
    qg.kv_append(a, empty, empty, pos[:0], q=empty)
    assert qg.kv_read(a, pos[:0])[0].shape == (0, 2, d)
    assert torch.equal(a.data, b.data)


def test_indexes_out_of_range_are_left_out():
    rng = np.random.default_rng(7)
    d, table = 64, qg.rope_table(8, 64)
    x = dev(rng.standard_normal((3, 1, d)).astype(np.float32))
    data = torch.full((32 * 72,), 7, dtype=torch.uint8, device="cuda")
    cache = qg.KVCache(1, d, 16, data)
    out = torch.full((3, 1, d), 5.0, device="cuda")
    qg.kv_append(cache, x, x, i32([32, 1, 2]), positions=i32([1, 8, -1]), rope=table, q=x, q_out=out)
    assert qg.device_error() == 4
    assert bool((data == 7).all()) and bool((out[1:] == 5).all()) and not bool((out[0] == 5).any())
    k, v = qg.kv_read(cache, i32([1 << 30, -5, 3]))
    assert qg.device_error() == 4
    assert not k[:2].any() and not v[:2].any() and bool((k[2] != 0).any())


def test_a_cache_past_32_bits():
    """Offsets of more than 2^32 bytes: rows at both ends of a 5 GB cache."""
    hk, d, page = 32, 128, 64
    n_pages = 5 * (1 << 30) // (page * hk * 144)
    cache = qg.KVCache.empty(n_pages, hk, d, page)
    assert cache.data.numel() > 1 << 32
    rng = np.random.default_rng(8)
    x = dev(rng.standard_normal((4, hk, d)).astype(np.float32))
    slots = i32([0, n_pages * page - 1, n_pages * page - 17, n_pages * page // 2])
    qg.kv_append(cache, x, -x, slots)
    k, v = qg.kv_read(cache, slots)
    sc, co = attn_ref.q4_0(x.cpu().numpy().reshape(-1, d))
    assert np.array_equal(k.cpu().numpy().reshape(-1, d).astype(np.float64), attn_ref.q4_0_values(sc, co))
    sc, co = attn_ref.q4_0(-x.cpu().numpy().reshape(-1, d))
    assert np.array_equal(v.cpu().numpy().reshape(-1, d).astype(np.float64), attn_ref.q4_0_values(sc, co))
    at = attn_ref.slot_bytes(page, hk, d, n_pages * page - 1, hk - 1)
    assert at[0].min() > 1 << 32


def test_an_empty_rope_is_refused():
    """It is no rotation that any position could have; without tokens there is nothing to rotate."""
    cache = qg.KVCache(2, 128, 16, torch.full((16 * 2 * 144,), 7, dtype=torch.uint8, device="cuda"))
    x, s, empty = torch.ones(3, 2, 128, device="cuda"), i32(range(3)), qg.rope_table(0, 128)
    with pytest.raises(ValueError):
        qg.kv_append(cache, x, x, s, positions=s, rope=empty)
    qg.kv_append(cache, x[:0], x[:0], s[:0], positions=s[:0], rope=empty)
    assert bool((cache.data == 7).all())


def test_refusals():
    d = 128
    cache = qg.KVCache.empty(2, 2, d, 16)
    x = torch.zeros(3, 2, d, device="cuda")
    s, table = i32(range(3)), qg.rope_table(4, 128)
    bad = [(TypeError, lambda: qg.kv_append(cache, x.double(), x.double(), s)),
           (TypeError, lambda: qg.kv_append(cache, x, x.half(), s)),
           (TypeError, lambda: qg.kv_append(cache, x, x, s.long())),
           (TypeError, lambda: qg.kv_append(cache, x, x, s.cpu())),
           (ValueError, lambda: qg.kv_append(cache, x[:, :1], x[:, :1], s)),
           (ValueError, lambda: qg.kv_append(cache, x, x, s[:2])),
           (ValueError, lambda: qg.kv_append(cache, x, x, s, rope=table)),
           (ValueError, lambda: qg.kv_append(cache, x, x, s, positions=s, rope=table[:, :3])),
           (ValueError, lambda: qg.kv_append(cache, x, x, s, q=x[:2])),
           (ValueError, lambda: qg.kv_append(cache, x, x, s, q_out=x)),
           (TypeError, lambda: qg.kv_append(cache, x, x, s, q=x, k_out=x.half(), q_out=x)),
           (ValueError, lambda: qg.kv_append(cache, x, x, s, k_out=x[:2])),
           (ValueError, lambda: qg.kv_append(cache, x.transpose(0, 1), x.transpose(0, 1), s)),
           (qg.QGError, lambda: qg.kv_append(cache, x[:1].expand(3, 2, d), x, s)),
           (qg.QGError, lambda: qg.kv_append(cache, torch.zeros(3, 2 * d + 2, device="cuda")[:, :2 * d].unflatten(1, (2, d)), x, s)),
           (qg.QGError, lambda: qg.kv_append(cache, torch.zeros(3 * 2 * d + 1, device="cuda")[1:].view(3, 2, d), x, s)),
           (ValueError, lambda: qg.kv_read(cache, s, k_out=x[:2])),
           (TypeError, lambda: qg.kv_read(cache, s, k_out=x.half())),
           (ValueError, lambda: qg.KVCache(2, d, 16, cache.data[:-1]))]
    for error, call in bad:
        with pytest.raises(error):
            call()
    assert qg.device_error() == 0
