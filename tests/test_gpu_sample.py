"""sample_tokens (include/qstep.h) on the GPU against its definition in 64 bits:
the tokens are the same, the probabilities off by their rounding to f32 (two
conversions and a division, each 2^-24) and by their weights' unit (weights are
whole multiples of 2^-44 of a power of 2 within a 90th of the largest, so off by
2^-44.9 of it, and the sum is no less than the largest)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ggml_block_quantized_gb300 as qg  # noqa: E402
import step_ref  # noqa: E402

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def cuda(x, dtype):
    return None if x is None else torch.as_tensor(np.asarray(x), dtype=dtype, device="cuda")


def both(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None):
    """The GPU's tokens and the definition's; asserts that they agree."""
    f = torch.float32
    n = logits.shape[0]
    u = cuda(uniform, f)
    token, prob = qg.sample_tokens(logits, u, temperature=cuda(temperature, f), top_k=cuda(top_k, torch.int32),
                                   top_p=cuda(top_p, f), min_p=cuda(min_p, f), prob_out=torch.full((n,), 7.0, device="cuda"))
    f32 = lambda x: None if x is None else np.asarray(x, np.float32)  # noqa: E731
    want, want_p = step_ref.sample(logits.float().cpu().numpy(), f32(uniform), f32(temperature), top_k, f32(top_p), f32(min_p))
    got = token.cpu().numpy()
    assert token.dtype == torch.int32 and np.array_equal(got, want), (np.nonzero(got != want)[0][:5], got[got != want][:5], want[got != want][:5])
    assert np.all(np.abs(prob.double().cpu().numpy() - want_p) <= 2.0 ** -22 * want_p + 2.0 ** -44.9)
    return want


def rows(n, vocab, seed, spread=2.5, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, vocab, generator=g, device="cuda") * spread
    x += (torch.rand(n, vocab, generator=g, device="cuda") < 0.003) * 8 * torch.rand(n, vocab, generator=g, device="cuda")
    return x.to(dtype), np.random.default_rng(seed)


def u01(rng, n):
    return rng.integers(0, 1 << 24, n) / float(1 << 24)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("n,vocab", [(1, 1), (4, 2), (3, 31), (5, 33), (7, 1000), (2, 1025), (40, 4099), (1, 32000), (6, 32768),
                                     (3, 50257), (2, 130001), (1, 262144), (2, 524288), (200, 777)])
def test_sizes_without_filters(n, vocab, dtype):
    x, rng = rows(n, vocab, n + vocab, dtype=dtype)
    both(x, u01(rng, n))
    both(x, u01(rng, n), temperature=rng.uniform(0.3, 3.0, n))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("n,vocab", [(3, 5), (9, 700), (64, 3000), (5, 32000), (2, 130001), (1, 524288)])
@pytest.mark.parametrize("spread", [0.0, 0.3, 2.5, 12.0])
def test_filters(n, vocab, spread, dtype):
    x, rng = rows(n, vocab, n * 3 + vocab, spread, dtype)
    t = rng.uniform(0.4, 2.0, n)
    k = np.minimum(rng.choice([0, 1, 2, 5, 40, 129, 1000, 20000, 1 << 20], n), 1 << 20)
    p = rng.choice([1.0, 0.999, 0.95, 0.7, 0.2, 0.01], n)
    q = rng.choice([0.0, 0.02, 0.3, 1.0], n)
    both(x, u01(rng, n), t, k)
    both(x, u01(rng, n), t, None, p)
    both(x, u01(rng, n), t, None, None, q)
    both(x, u01(rng, n), t, k, p, q)


@pytest.mark.parametrize("vocab", [100, 5000, 40000])
def test_equal_logits_go_by_index(vocab):
    """Ties at the border: the lowest indexes stay."""
    x = torch.full((8, vocab), 1.5, device="cuda")
    x[4:, ::3] = 2.0
    x[6:, 5] = 9.0
    k = [7, vocab // 2, 0, 0, 7, vocab // 2, 2, 0]
    p = [1.0, 1.0, 0.5, 0.37, 1.0, 0.9, 1.0, 0.8]
    for u in (0.0, 0.25, 0.999999):
        got = both(x, [u] * 8, [1.0] * 8, k, p)
    assert got[0] == 6 and got[1] == vocab // 2 - 1
    both(x.half(), [0.5] * 8, [0.7] * 8, k, p)


def test_few_values():
    """Logits of few distinct values, as after a coarse rounding: every border lies among equal ones."""
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randint(-6, 7, (24, 30011), generator=g, device="cuda").float()
    rng = np.random.default_rng(1)
    both(x, u01(rng, 24), rng.uniform(0.5, 2, 24), rng.integers(1, 30000, 24), rng.uniform(0.05, 1, 24), rng.choice([0, 0.1], 24))
    both(x * 1e-30, u01(rng, 24), rng.uniform(0.5, 2, 24), rng.integers(1, 30000, 24), rng.uniform(0.05, 1, 24))


@pytest.mark.parametrize("vocab", [4001, 130001, 524288])
@pytest.mark.parametrize("tail", [-28.0, -30.8, -31.15, -31.26])  # 6.2, 0.7, 0.52 and 0.47 of a weight's unit
@pytest.mark.parametrize("at", [0, -1])
def test_a_flat_tail(tail, vocab, at):
    """One likely token and very many equally unlikely ones, whose weights' roundings have one sign: a sum is off by 2^-35
    of itself and by 2^-45 of the largest weight for each token, times 2^(1/128), by which the unit may be larger. The
    token chosen is one whose borders are no further off than that (top_p's border beside it: as far, and by one token)."""
    x = torch.full((1, vocab), tail, device="cuda")
    x[0, at] = 0.0
    w = np.exp(x[0].double().cpu().numpy())
    sums = np.cumsum(w)
    whole = sums[-1]
    off = 2.0 ** -35 * whole + vocab * 2.0 ** -45 * 2.0 ** (1 / 128)
    u = np.array([0.0, 2.0 ** -40, 2.0 ** -30, 2.0 ** -28, 2.0 ** -27, 2.0 ** -26, 2.0 ** -25, 0.25, 0.5, 1 - 2.0 ** -10, 1 - 2.0 ** -23, 1 - 2.0 ** -24])
    for p in (None, 0.99999994):
        token, prob = qg.sample_tokens(x.expand(len(u), vocab), cuda(u, torch.float32), top_p=None if p is None else torch.full((len(u),), p, device="cuda"),
                                       prob_out=torch.empty(len(u), device="cuda"))
        kept = sums
        if p is not None:
            order = np.argsort(-w, kind="stable")
            stay = order[np.concatenate([[0.0], np.cumsum(w[order])[:-1]]) < float(np.float32(p)) * whole]
            kept = np.cumsum(np.where(np.isin(np.arange(vocab), stay), w, 0.0))
        slack = (0.0 if p is None else 2 * off + np.exp(tail)) + 2 * off
        for t, q, v in zip(token.tolist(), prob.tolist(), np.float32(u).astype(np.float64)):
            before, past = (kept[t - 1] if t > 0 else 0.0), kept[t]
            assert before - slack <= v * kept[-1] <= past + slack, (t, v)
            assert abs(q - w[t] / kept[-1]) <= 2.0 ** -22 * w[t] + 2.0 ** -44 + slack * w[t], (t, q)


def test_masks_and_odd_values():
    x, rng = rows(12, 4001, 5)
    x[0] = -INF
    x[1] = NAN
    x[2, :-1] = -INF                      # one token left
    x[3, 100:] = torch.finfo(torch.float32).min  # masked by the type's lowest value
    x[4, ::2] = NAN
    x[5, 7] = INF
    x[6, [9, 4000]] = INF
    x[7] = -1e30
    x[7, 3000] = 1e30
    x[8] = torch.finfo(torch.float32).min
    x[9, 50:] = -1e9
    x[10] = -0.0
    x[10, 1::2] = 0.0
    for k, p, q in ((None, None, None), ([40] * 12, [0.9] * 12, [0.01] * 12), (None, [0.9] * 12, None), ([3000] * 12, None, None),
                    (None, [0.999999] * 12, None)):
        got = both(x, u01(rng, 12), [1.1] * 12, k, p, q)
        assert got[0] == got[1] == -1 and got[2] == 4000 and got[5] == 7 and got[6] in (9, 4000) and got[7] == 3000


def test_settings_at_their_ends():
    n = 16
    x, rng = rows(n, 2500, 8)
    t = np.array([0.0, -1.0, NAN, 1e-30, 2.0 ** -60, 1e-3, 1e6, INF, 1e-38, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0], np.float32)
    k = [0, 0, 0, 0, 0, 0, 0, 0, 0, -5, 1, 2500, 2501, 1 << 30, 0, 0]
    p = np.array([1.0] * 9 + [0.0, -1.0, 2.0, NAN, 0.5, 1e-20, 0.99999994], np.float32)
    q = np.array([0.0] * 12 + [NAN, 2.0, -1.0, 1e-30], np.float32)
    with np.errstate(invalid="ignore"):
        both(x, u01(rng, n), t)
        both(x, u01(rng, n), None, k)
        both(x, u01(rng, n), None, None, p)
        both(x, u01(rng, n), None, None, None, q)
        both(x, u01(rng, n), np.where(t > 0, t, 1), k, p, q)
        for u in (0.0, 1.0 - 2.0 ** -24, 1.0, 5.0, -1.0, NAN, 2.0 ** -149, INF):
            both(x, [u] * n, [1.0] * n, k, p)


@pytest.mark.parametrize("vocab,finite", [(4000, 2500), (9000, 3), (50001, 4100), (50001, 2100), (130001, 0)])
@pytest.mark.parametrize("k", [2600, 4099, 30000])
def test_more_asked_for_than_there_are(vocab, finite, k):
    """top_k beyond the tokens that are not -inf, alone and with the other filters."""
    x, rng = rows(3, vocab, vocab + finite + k)
    for r in range(3):
        x[r, torch.from_numpy(rng.permutation(vocab)[finite:]).cuda()] = -INF
    x[0, :7] = 0.25
    u, ks = u01(rng, 3), np.full(3, k)
    both(x, u, None, ks)
    both(x, u, np.full(3, 1.3), ks, np.full(3, 0.8))
    both(x, u, np.full(3, 0.8), ks, np.full(3, 0.95), np.full(3, 0.001))


@pytest.mark.parametrize("n", [305, 400, 512, 513, 1100])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_more_rows_than_run_at_once(n, dtype):
    """Settings of every kind, in any order among the rows."""
    x, rng = rows(n, 1700, n, dtype=dtype)
    x[rng.integers(0, n, 9)] = -INF
    k = rng.choice([0, 0, 1, 3, 40, 700, 1699, 5000, -2], n)
    p = rng.choice([1.0, 1.0, 0.9, 0.3, 0.0, NAN], n)
    m = rng.choice([0.0, 0.0, 0.05, 2.0, NAN], n)
    t = rng.choice([1.0, 0.0, 0.7, 1.9], n)
    both(x, u01(rng, n), t, np.maximum(k, 0), np.where(np.isnan(p), 1.0, p), np.where(np.isnan(m), 0.0, m))
    f = lambda a, d=torch.float32: cuda(a, d)  # noqa: E731
    u = f(u01(rng, n))
    whole = qg.sample_tokens(x, u, f(t), f(k, torch.int32), f(p), f(m), prob_out=torch.empty(n, device="cuda"))
    for r0 in range(0, n, 100):
        part = slice(r0, min(n, r0 + 100))
        some = qg.sample_tokens(x[part], u[part], f(t[part]), f(k[part], torch.int32), f(p[part]), f(m[part]),
                                prob_out=torch.empty(part.stop - r0, device="cuda"))
        assert torch.equal(whole[0][part], some[0]) and torch.equal(whole[1][part], some[1])


def test_every_token_has_its_share():
    """The unit interval in 4096 steps: as many of them choose a token as its probability says, in the indexes' order."""
    x, _ = rows(1, 300, 3, 1.0)
    n = 4096
    u = (np.arange(n) + 0.5) / n
    got = both(x.expand(n, 300), u, np.full(n, 0.8), np.full(n, 50), np.full(n, 0.9))
    assert np.all(np.diff(got) >= 0) and len(set(got.tolist())) > 20


def test_strides_places_and_a_vocabulary_that_is_padded():
    x, rng = rows(9, 3000, 4)
    u = u01(rng, 9)
    want = both(x[:, :2717].contiguous(), u, [0.9] * 9, [50] * 9, [0.8] * 9)
    assert np.array_equal(both(x[:, :2717], u, [0.9] * 9, [50] * 9, [0.8] * 9), want)  # what lies behind has no say
    for first in (1, 2, 3, 5):
        both(x[::2, first:first + 2700], u[:5], [0.9] * 5, [50] * 5, [0.8] * 5)
        both(x.half()[:, first:2001 + first], u, [0.9] * 9, None, [0.8] * 9)
    both(x[:1].expand(9, 3000), u)


def test_a_row_does_not_depend_on_the_others():
    """One row alone (many blocks a row) and among many (one block a row), same bits each time."""
    x, rng = rows(300, 20011, 6)
    u, t, k, p = u01(rng, 300), rng.uniform(0.5, 1.5, 300), rng.integers(0, 100, 300), rng.uniform(0.5, 1, 300)
    f, i = torch.float32, torch.int32
    args = lambda s: dict(temperature=cuda(t[s], f), top_k=cuda(k[s], i), top_p=cuda(p[s], f), prob_out=torch.empty(len(u[s]), device="cuda"))  # noqa: E731
    a, pa = qg.sample_tokens(x, cuda(u, f), **args(slice(None)))
    b, pb = qg.sample_tokens(x, cuda(u, f), **args(slice(None)))
    assert torch.equal(a, b) and torch.equal(pa, pb)
    for r in (0, 17, 299):
        s = slice(r, r + 1)
        c, pc = qg.sample_tokens(x[s], cuda(u[s], f), **args(s))
        assert torch.equal(c, a[s]) and torch.equal(pc, pa[s])


def test_streams_and_graphs():
    x, rng = rows(5, 32000, 2)
    u, p = cuda(u01(rng, 5), torch.float32), cuda([0.9] * 5, torch.float32)
    want, _ = qg.sample_tokens(x, u, top_p=p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = qg.sample_tokens(x, u, top_p=p, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.sample_tokens(x, u, top_p=p, out=out)
    for _ in range(3):
        u.copy_(torch.rand(5, device="cuda"))
        graph.replay()
        want, _ = qg.sample_tokens(x, u, top_p=p)
        assert torch.equal(out, want)


def test_no_rows():
    token, prob = qg.sample_tokens(torch.empty(0, 50, device="cuda"), torch.empty(0, device="cuda"))
    assert token.shape == (0,) and prob is None


def test_rows_past_32_bits():
    """Rows 2^28 elements apart: the last begins behind 2^31."""
    apart, n, vocab = 1 << 28, 9, 1001
    logits = torch.empty(apart * (n - 1) + vocab, dtype=torch.float16, device="cuda").as_strided((n, vocab), (apart, 1))
    x, rng = rows(n, vocab, 77, dtype=torch.float16)
    logits.copy_(x)
    u, k = cuda(u01(rng, n), torch.float32), cuda([40] * n, torch.int32)
    for kw in (dict(), dict(top_k=k), dict(top_p=torch.full((n,), 0.9, device="cuda"))):
        assert torch.equal(qg.sample_tokens(logits, u, **kw)[0], qg.sample_tokens(x, u, **kw)[0])
