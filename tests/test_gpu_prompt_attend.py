"""qattn_prompt against the formula in 64 bits (attn_ref.attend). The inputs are
f16, exact in the products; the softmax weights are rounded to f16, half an
ulp, 2^-11 of a weight: attn_ref.bound with 10 bits for it (weights and their
sum) is the tolerance."""
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attn_ref  # noqa: E402
import ggml_block_quantized_gb300 as qg  # noqa: E402

pytestmark = pytest.mark.gpu


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


def inputs(rng, n, heads, hk, d, fused=True, q_size=1.5, v_size=1.0):
    x = rng.standard_normal((n, heads + 2 * hk, d)).astype(np.float32)
    x[:, :heads] *= q_size
    x[:, heads + hk:] = (x[:, heads + hk:] + 0.3) * v_size
    x = torch.from_numpy(x).cuda().half()
    q, k, v = x[:, :heads], x[:, heads:heads + hk], x[:, heads + hk:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def check(got, q, k, v, lens, scale, f16=True, rows=None, heads=None):
    got, q, k, v = (t.detach().cpu().numpy().astype(np.float64) for t in (got, q, k, v))
    d, group, at = q.shape[2], q.shape[1] // k.shape[1], 0
    for n in lens:
        mine = np.arange(n) if rows is None else np.array(sorted({r for r in rows if 0 <= r < n}))
        for h in range(q.shape[1]) if heads is None else heads:
            if not len(mine):
                continue
            out, pv, mag, big = attn_ref.attend(q[at + mine, h], k[at:at + n, h // group], v[at:at + n, h // group],
                                                mine + 1, scale)
            tol = attn_ref.bound(out, pv, mag, big, d, n, 24, 10, f16)
            err = np.abs(got[at + mine, h] - out)
            assert np.isfinite(got[at + mine, h]).all(), (n, h)
            assert (err <= tol).all(), (n, h, float((err / tol).max()))
        at += n


CASES = [  # D, kv heads, group, lengths, fused
    (128, 2, 4, [1], True), (64, 1, 1, [2], False), (128, 8, 4, [61], True), (64, 3, 1, [127, 128, 129], True),
    (128, 1, 8, [0, 1, 0, 2, 3, 15, 16, 17, 31, 33, 0], True), (128, 2, 2, [255, 1, 257], True),
    (64, 2, 8, [300, 5, 700], True), (128, 2, 5, [37, 1, 260], True), (64, 1, 12, [9, 130], False), (128, 1, 6, [300, 43], True),
    (64, 1, 48, [70, 3], True), (128, 1, 19, [14], False), (128, 1, 3, [190, 64], True), (64, 1, 7, [100, 333], False),
    (128, 1, 16, [130, 40], True), (128, 4, 1, [513], True), (64, 1, 5, [385, 1, 1, 1], True),
    (128, 1, 128, [3, 2], True), (64, 1, 200, [5], True), (128, 1, 6, [260], False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", "")[:60])
def test_prompt(case):
    d, hk, group, lens, fused = case
    rng = np.random.default_rng(sum(map(ord, str(case))))
    q, k, v = inputs(rng, sum(lens), hk * group, hk, d, fused)
    off = i32(np.cumsum([0] + lens))
    got = qg.prompt_attend(q, k, v, off)
    assert got.dtype == torch.float16
    check(got, q, k, v, lens, d ** -0.5)
    assert torch.equal(got, qg.prompt_attend(q, k, v, off))
    wide = torch.full(got.shape, np.nan, device="cuda")
    assert qg.prompt_attend(q, k, v, off, out=wide) is wide
    check(wide, q, k, v, lens, d ** -0.5, f16=False)


def test_long_prompt():
    """Many key tiles; sampled rows, among them the tiles' borders."""
    rng = np.random.default_rng(30)
    lens = [2500, 3, 1797]
    q, k, v = inputs(rng, sum(lens), 6, 2, 128)
    got = qg.prompt_attend(q, k, v, i32(np.cumsum([0] + lens)))
    rows = [0, 1, 2, 63, 64, 127, 128, 129, 255, 256, 1000, 1023, 1024, 1796, 2047, 2048, 2303, 2304, 2498, 2499]
    check(got, q, k, v, lens, 128 ** -0.5, rows=rows)


@pytest.mark.parametrize("d,heads,hk,n_seq,most", [(128, 8, 2, 700, 3), (64, 4, 4, 900, 2), (128, 16, 1, 300, 40)])
def test_many_short_prompts(d, heads, hk, n_seq, most):
    """More work items than multiprocessors, most of a single tile or less."""
    rng = np.random.default_rng(36)
    lens = rng.integers(0, most + 1, n_seq).tolist()
    q, k, v = inputs(rng, sum(lens), heads, hk, d)
    off = i32(np.cumsum([0] + lens))
    got = qg.prompt_attend(q, k, v, off)
    for _ in range(20):
        assert torch.equal(got, qg.prompt_attend(q, k, v, off))
    check(got, q, k, v, lens, d ** -0.5, heads=[0, heads - 1])


@pytest.mark.parametrize("lens", [[1] * 20 + [700, 2, 0, 129, 300] + [0] * 9 + [260] * 3 + [64, 1], [513] + [5] * 40 + [257, 128],
                                  [0] * 70 + [3] + [0] * 100 + [1000]], ids=["mixed", "long-first", "gaps"])
def test_more_sequences_than_a_warp(lens):
    """More than 32 sequences, of one tile and of several, with empty ones among them: the bits of calls that take
    them one by one."""
    rng = np.random.default_rng(44)
    q, k, v = inputs(rng, sum(lens), 8, 2, 64)
    got, at = qg.prompt_attend(q, k, v, i32(np.cumsum([0] + lens))), 0
    for n in lens:
        if n:
            rows = slice(at, at + n)
            assert torch.equal(got[rows], qg.prompt_attend(q[rows], k[rows], v[rows], i32([0, n])))
        at += n


def test_very_many_sequences():
    """300000 sequences of 0 .. 2 rows and a few long ones: the time is that of the work, not of looking through all
    sequences for each item."""
    rng = np.random.default_rng(45)
    lens = rng.integers(0, 3, 300000)
    lens[[7, 150000, 299990]] = 700, 300, 129
    ends = np.cumsum(np.concatenate([[0], lens]))
    q, k, v = inputs(rng, int(ends[-1]), 1, 1, 64)
    off = i32(ends)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    got = qg.prompt_attend(q, k, v, off)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 2.0
    one = torch.from_numpy(ends[:-1][lens == 1]).cuda()
    assert torch.equal(got[one], v[one])  # (one key: its value)
    for s in (0, 140000, 149990, 299980):
        a, b = int(ends[s]), int(ends[s + 20])
        assert torch.equal(got[a:b], qg.prompt_attend(q[a:b], k[a:b], v[a:b], i32(ends[s:s + 21] - a)))


@pytest.mark.parametrize("q_size,v_size,scale", [(1, 1, -0.3), (1, 1, 0.0), (20, 1, 1.0), (1, 5000.0, 0.09),
                                                 (1, 1e-4, 0.09), (3000, 1, 0.01)])
def test_sizes_of_values(q_size, v_size, scale):
    rng = np.random.default_rng(31)
    lens = [200, 70]
    q, k, v = inputs(rng, sum(lens), 4, 2, 128, q_size=q_size, v_size=v_size)
    check(qg.prompt_attend(q, k, v, i32([0, 200, 270]), scale=scale), q, k, v, lens, scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_unseen_nan_and_infinity(d, bad):
    """Row 150 of the first prompt and row 5 of the second hold what is not
    finite: no row before them, and no row of another prompt, sees it."""
    rng = np.random.default_rng(32)
    lens = [300, 40, 90]
    q, k, v = (t.clone() for t in inputs(rng, sum(lens), 4, 2, d, fused=False))
    k[150], v[150], k[305], v[305] = bad, bad, bad, bad
    got = qg.prompt_attend(q, k, v, i32(np.cumsum([0] + lens)))
    check(got[:150], q[:150], k[:150], v[:150], [150], d ** -0.5)
    check(got[300:305], q[300:305], k[300:305], v[300:305], [5], d ** -0.5)
    check(got[340:], q[340:], k[340:], v[340:], [90], d ** -0.5)
    assert not torch.isfinite(got[150:300]).all(-1).all() and not torch.isfinite(got[305:340]).all(-1).all()


@pytest.mark.parametrize("n_hidden", [1, 127, 128, 129, 256, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_minus_infinity(d, n_hidden):
    """The first keys hold -inf in a channel where the queries are 1: their scores are -inf and their weights 0, for
    whole key tiles and parts of one. The rows after them see only the other keys."""
    rng = np.random.default_rng(39)
    q, k, v = (t.clone() for t in inputs(rng, 430, 4, 2, d, fused=False))
    q[..., 0] = 1.0
    k[:n_hidden, :, 0] = -float("inf")
    got = qg.prompt_attend(q, k, v, i32([0, 430]))
    check(got[n_hidden:], q[n_hidden:], k[n_hidden:], v[n_hidden:], [430 - n_hidden], d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [3, 5, 7, 12, 4])
def test_same_bits_whatever_ran_before(d, group):
    """Groups whose tiles have rows without a query: what an earlier launch left there, zeros or large numbers, has no
    say in the other rows. The same for rows past a sequence's end, which hold the next sequence."""
    rng = np.random.default_rng(47)
    n_seq, n = 6, 700
    q, k, v = inputs(rng, n_seq * n, 2 * group, 2, d, q_size=4.0)
    off = i32(np.arange(n_seq + 1) * n)
    x = torch.randn(40 * 256, 12, d, device="cuda").half()
    ends = i32(np.arange(0, 40 * 256 + 1, 256))

    def after(size):
        qg.prompt_attend(x[:, :8] * size, x[:, 8:10] * min(size, 1), x[:, 10:], ends)
        return qg.prompt_attend(q, k, v, off)

    got = after(0.0)
    for size in (100.0, 0.0, 3000.0):
        assert torch.equal(after(size), got)
    qn = q.clone()  # the last sequence alone, with and without queries after it
    qn[n:2 * n] *= 50
    assert torch.equal(qg.prompt_attend(qn[:2 * n], k[:2 * n], v[:2 * n], i32([0, n, 2 * n]))[:n], got[:n])


def test_infinite_value_that_is_seen():
    """An infinite value with a weight above zero gives that infinity."""
    rng = np.random.default_rng(33)
    q, k, v = (t.clone() for t in inputs(rng, 140, 2, 1, 128, fused=False))
    v[3, 0, 7] = float("inf")
    v[130, 0, 9] = -float("inf")
    got = qg.prompt_attend(q, k, v, i32([0, 140]))
    assert bool((got[3:, :, 7] == float("inf")).all()) and bool((got[130:, :, 9] == -float("inf")).all())
    clean = torch.isfinite(got)
    clean[3:, :, 7] = True
    clean[130:, :, 9] = True
    assert bool(clean.all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d,group", [(64, 1), (128, 3), (128, 4)])
def test_a_query_that_is_not_finite(d, group, bad):
    """It gives NaN in its own row and head and changes no other one (a query with an infinity has scores of both
    signs of it, or NaN)."""
    rng = np.random.default_rng(35)
    lens = [290, 33]
    q, k, v = (t.clone() for t in inputs(rng, sum(lens), 2 * group, 2, d, fused=False))
    clean = qg.prompt_attend(q, k, v, i32([0, 290, 323]))
    rows, heads = [7, 200, 289, 291, 322], [0, 2 * group - 1, group, group - 1, 1]
    for r, h in zip(rows, heads):
        q[r, h, ::9] = bad
    got = qg.prompt_attend(q, k, v, i32([0, 290, 323]))
    rest = torch.ones(323, 2 * group, dtype=torch.bool, device="cuda")
    for r, h in zip(rows, heads):
        assert torch.isnan(got[r, h]).all()
        rest[r, h] = False
    assert torch.equal(got[rest], clean[rest])


def test_very_large_scores():
    """Scores up to 2^23: a row is the values of the key with its largest one."""
    rng = np.random.default_rng(49)
    n, d = 400, 64
    q, k, v = inputs(rng, n, 2, 1, d)
    s = np.einsum("mhd,nd->hmn", q.cpu().numpy().astype(np.float64), k[:, 0].cpu().numpy().astype(np.float64))
    s[:, np.arange(n)[:, None] < np.arange(n)] = -np.inf
    scale = 0.9 * 2.0 ** 23 / np.abs(s[np.isfinite(s)]).max()
    two = np.sort(s, -1)[..., -2:] * scale
    clear = (two[..., 1] - two[..., 0] > 2.0 ** 9).T  # (a score may be off by D 2^-23 of its terms' size)
    assert clear.mean() > 0.98
    got = qg.prompt_attend(q, k, v, i32([0, n]), scale=scale).cpu().numpy()
    want = v[:, 0].cpu().numpy()[s.argmax(-1)].transpose(1, 0, 2)
    off = np.abs(got.astype(np.float64) - want)  # weight and result rounded to f16 once each
    assert (off <= 2.0 ** -10 * 1.01 * np.abs(want) + 2.0 ** -24)[clear].all()


def test_strides_rows_in_no_sequence_and_stream():
    rng = np.random.default_rng(34)
    q, k, v = inputs(rng, 100, 4, 2, 64)
    out = torch.full((100, 4, 64), 9.0, device="cuda", dtype=torch.float16)
    off = i32([10, 40, 40, 90])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    qg.prompt_attend(q, k, v, off, out=out, stream=side)
    side.synchronize()
    assert bool((out[:10] == 9).all()) and bool((out[90:] == 9).all())
    check(out[10:90], q[10:90], k[10:90], v[10:90], [30, 50], 64 ** -0.5)


@pytest.mark.parametrize("t", [torch.float16, torch.float32], ids=["f16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_an_output_on_a_16_byte_boundary(d, t):
    """`out` begins 16 bytes into a buffer: the same bits, and nothing beside it."""
    rng = np.random.default_rng(37)
    lens = [140, 3]
    q, k, v = inputs(rng, sum(lens), 6, 2, d)
    off = i32([0, 140, 143])
    want = qg.prompt_attend(q, k, v, off, out=torch.empty(143, 6, d, dtype=t, device="cuda"))
    check(want, q, k, v, lens, d ** -0.5, f16=t == torch.float16)
    pad = 16 // want.element_size()
    buffer = torch.full((pad + want.numel() + pad,), 9.0, dtype=t, device="cuda")
    out = buffer[pad:-pad].view(143, 6, d)
    assert out.data_ptr() % 32 == 16
    qg.prompt_attend(q, k, v, off, out=out)
    assert torch.equal(out, want)
    assert bool((buffer[:pad] == 9).all()) and bool((buffer[-pad:] == 9).all())


def test_offsets_out_of_range():
    rng = np.random.default_rng(35)
    q, k, v = inputs(rng, 50, 2, 1, 64)
    out = torch.full((50, 2, 64), 9.0, device="cuda", dtype=torch.float16)
    qg.prompt_attend(q, k, v, i32([0, 20, 10, 60]), out=out)  # the second falls, the third ends past the rows
    assert qg.device_error() == 4
    check(out[:20], q[:20], k[:20], v[:20], [20], 64 ** -0.5)
    assert bool((out[20:] == 9).all())
    qg.prompt_attend(q, k, v, i32([-3, 20, 50]), out=out)
    assert qg.device_error() == 4
    check(out[20:], q[20:], k[20:], v[20:], [30], 64 ** -0.5)


@pytest.mark.parametrize("offsets,kept", [
    ([0, 2048, 0, 2048], [(0, 2048)]),  # the third begins again where the first has been
    ([0, 900, 300, 900, 2048], [(0, 900), (900, 2048)]),
    ([0, 1100, 4000, 1100, 1100, -1, 1200, 2000, 1999, 2000, 2048], [(0, 1100), (1200, 2000), (2000, 2048)]),
    ([700, 100, 200, 2048], [(100, 200), (200, 2048)]),  # the falling first one holds no other back
    ([0, 2048] + [0, 2048] * 40, [(0, 2048)]),  # more than 32 sequences
    ([0] + [5, 3] * 40 + [2048], [(0, 5)]), ([900, 100] + [100] * 40 + [1800, 1700, 2048], [(100, 1800)])],
    ids=["again", "inside", "several", "first", "many", "many-short", "many-first"])
def test_falling_offsets_lose_no_other_rows(offsets, kept):
    """Sequences of many tiles around offsets that fall: each row of a sequence that is not left out has its result,
    the others are not written, every time."""
    rng = np.random.default_rng(38)
    q, k, v = inputs(rng, 2048, 1, 1, 64)
    want = torch.full((2048, 1, 64), 9.0, device="cuda", dtype=torch.float16)
    for a, b in kept:
        want[a:b] = qg.prompt_attend(q[a:b], k[a:b], v[a:b], i32([0, b - a]))
    for _ in range(3):
        out = torch.full((2048, 1, 64), 9.0, device="cuda", dtype=torch.float16)
        qg.prompt_attend(q, k, v, i32(offsets), out=out)
        assert qg.device_error() == 4
        assert torch.equal(out, want)


def test_refusals():
    q, k = torch.zeros(5, 4, 128, device="cuda", dtype=torch.float16), torch.zeros(5, 2, 128, device="cuda", dtype=torch.float16)
    off = i32([0, 5])
    bad = [(TypeError, lambda: qg.prompt_attend(q.float(), k, k, off)),
           (TypeError, lambda: qg.prompt_attend(q, k, k, off.long())),
           (ValueError, lambda: qg.prompt_attend(q, k[:4], k[:4], off)),
           (ValueError, lambda: qg.prompt_attend(q[:, :3], k, k, off)),
           (qg.QGError, lambda: qg.prompt_attend(q[..., :96].contiguous(), k[..., :96].contiguous(), k[..., :96].contiguous(), off)),
           (ValueError, lambda: qg.prompt_attend(q, k, k, off, out=q[:2])),
           (TypeError, lambda: qg.prompt_attend(q, k, k, off, out=q.double())),
           (qg.QGError, lambda: qg.prompt_attend(q, k, k, off, scale=float("inf"))),
           (qg.QGError, lambda: qg.prompt_attend(q[:1].expand(5, 4, 128), k, k, off))]
    for error, call in bad:
        with pytest.raises(error):
            call()
    assert qg.prompt_attend(q[:0], k[:0], k[:0], i32([0])).shape == (0, 4, 128)
    assert qg.device_error() == 0
