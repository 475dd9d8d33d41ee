"""norm_residual (include/qstep.h) on the GPU against its formula in 64 bits;
the bounds are step_ref's, from the arithmetic."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ggml_block_quantized_gb300 as qg  # noqa: E402
import step_ref  # noqa: E402
from ggml_block_quantized_gb300 import step  # noqa: E402

pytestmark = pytest.mark.gpu
F32, F16 = torch.float32, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def make(n, d, seed=0, h=F32, y=F32, post=True, gate=None, bias=True, mean=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    size = torch.exp(0.7 * r(d))
    return dict(h=(r(n, d) * size + mean).to(h), y=(r(n, d) + mean).to(y), weight=1 + 0.3 * r(d),
                bias=0.2 * r(d) if bias else None, post_weight=0.5 + 0.3 * r(d) if post else None,
                post_bias=0.2 * r(d) if post and bias else None,
                gate=None if gate is None else r(n, d) if gate == "rows" else r(d))


def wanted(a, **kw):
    npy = {k: None if v is None else v.float().cpu().numpy() for k, v in a.items()}
    return step_ref.norm_residual(npy["h"], npy["y"], npy["weight"], npy["bias"], npy["post_weight"], npy["post_bias"],
                                  npy["gate"], **kw)


def check(got, want, off):
    f = got.double().cpu().numpy()
    if got.dtype == F16:
        off = step_ref.half(off, want)
    worst = np.max(np.abs(f - want) - off)
    assert worst <= 0, worst


def run(a, **kw):
    return qg.norm_residual(a["h"], a["y"], a["weight"], a["bias"], a["post_weight"], a["post_bias"], a["gate"], **kw)


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 7), (1, 4096), (2, 8200), (5, 16384), (1, 16383), (9, 1283), (70, 64),
                                 (33, 256), (300, 40), (1, 8192), (2, 8193), (4, 31), (13, 513)])
def test_sizes(n, d, layer):
    a = make(n, d, seed=n + d)
    h, x = run(a, layer=layer, scale=0.75)
    hw, ho, xw, xo = wanted(a, layer=layer, scale=0.75)
    check(h, hw, ho)
    check(x, xw, xo)


@pytest.mark.parametrize("h", [F32, F16])
@pytest.mark.parametrize("y", [F32, F16, None])
@pytest.mark.parametrize("x", [F32, F16])
@pytest.mark.parametrize("post,gate,bias,d", [(False, None, False, 96), (True, "channel", False, 1024), (True, "rows", True, 515),
                                              (False, "rows", False, 4104)])
def test_forms(h, y, x, post, gate, bias, d):
    a = make(6, d, seed=d, h=h, y=y or F32, post=post and y is not None, gate=gate if y is not None else None, bias=bias)
    if y is None:
        a["y"] = None
    out = torch.empty(6, d, dtype=x, device="cuda")
    ho, xo = run(a, x_out=out, scale=-1.5, eps=1e-6)
    hw, hb, xw, xb = wanted(a, scale=-1.5, eps=1e-6)
    assert xo is out
    check(out, xw, xb)
    if y is None:
        assert ho is None
    else:
        assert ho.dtype == h
        check(ho, hw, hb)


@pytest.mark.parametrize("d", [1024, 1021])
def test_strides_and_places(d):
    """Rows that lie apart, off a 16-byte boundary, shared by all (stride 0); h_out over h; what lies between rows stays."""
    g = torch.Generator(device="cuda").manual_seed(3)
    big = torch.randn(9, 2 * d + 37, generator=g, device="cuda")
    h, y = big[:, 1:1 + d], big[:, d + 8:2 * d + 8]
    w = torch.randn(d + 1, generator=g, device="cuda")[1:]
    gate = torch.randn(1, d, generator=g, device="cuda").expand(9, d)
    a = dict(h=h, y=y, weight=w, bias=None, post_weight=None, post_bias=None, gate=gate)
    hw, hb, xw, xb = wanted(a)
    before = big.clone()
    ho, x = qg.norm_residual(h, y, w, gate=gate, h_out=h)
    assert ho.data_ptr() == h.data_ptr()
    check(h, hw, hb)
    check(x, xw, xb)
    big[:, 1:1 + d] = before[:, 1:1 + d]
    assert torch.equal(big, before)
    # every row the same one
    one = torch.randn(1, d, generator=g, device="cuda").expand(5, d)
    ho, x = qg.norm_residual(one, y[:5], w)
    hw, hb, xw, xb = step_ref.norm_residual(one.cpu().numpy(), y[:5].cpu().numpy(), w.cpu().numpy())
    check(ho, hw, hb)
    check(x, xw, xb)


def test_a_large_mean_costs_no_bits():
    """layer: deviations of 1 beside a mean of 4096 (the squares' sum before the mean is known would lose them)."""
    a = make(4, 2000, seed=5, mean=4096.0, post=False, bias=False)
    h, x = run(a, layer=True)
    hw, hb, xw, xb = wanted(a, layer=True)
    check(x, xw, xb)


@pytest.mark.parametrize("d", [256, 2048, 8448])
@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("act", ["Q8_0", "Q8_1", "Q8_K"])
def test_blocks_are_quantize_act(act, n, d):
    t = getattr(qg, act)
    a = make(n, d, seed=d + n, gate="channel")
    a["h"][0, :40] = 0
    xq = torch.zeros(n * qg.qtype_nbytes(t, d) + 16, dtype=torch.uint8, device="cuda")
    h, x = run(a, x_out=torch.empty(n, d, device="cuda"), xq=xq, act_type=t)
    assert torch.equal(xq[:-16], qg.quantize_act(t, x, n)) and not xq[-16:].any()
    # without x_out
    xq2 = torch.zeros_like(xq)
    h2, none = run(a, xq=xq2, act_type=t)
    assert none is None and torch.equal(xq2, xq) and torch.equal(h, h2)


@pytest.mark.parametrize("x_out", [True, False])
@pytest.mark.parametrize("act", ["Q8_0", "Q8_1", "Q8_K"])
def test_strides_of_what_is_not_there_do_not_count(act, x_out):
    """Through the C interface: without y, gate and h_out their strides may be anything."""
    t, n, d = getattr(qg, act), 3, 512
    a = make(n, d, seed=7)
    want = torch.empty(n, d, device="cuda")
    qg.norm_residual(a["h"], weight=a["weight"], bias=a["bias"], x_out=want)
    x = torch.empty_like(want)
    xq = torch.full((n * qg.qtype_nbytes(t, d),), 0x5A, dtype=torch.uint8, device="cuda")
    args = step._NormArgs(a["h"].data_ptr(), None, d, 1, None, None, None, 3, a["weight"].data_ptr(), a["bias"].data_ptr(), None,
                          d + 5, x.data_ptr() if x_out else None, xq.data_ptr(), n, d, qg.F32, qg.F16, qg.F32, t, 0, 1.0, 1e-5)
    assert step._lib().qnorm_residual(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(xq, qg.quantize_act(t, want, n).flatten())
    if x_out:
        assert torch.equal(x, want)


def test_blocks_of_zeros_and_odd_values():
    d = 512
    h = torch.zeros(3, d, device="cuda")
    h[1, 3], h[2, 300] = float("inf"), float("nan")
    for t in (qg.Q8_0, qg.Q8_1, qg.Q8_K):
        xq = torch.empty(3 * qg.qtype_nbytes(t, d), dtype=torch.uint8, device="cuda")
        x = torch.empty(3, d, device="cuda")
        qg.norm_residual(h, x_out=x, xq=xq, act_type=t)
        assert torch.equal(xq, qg.quantize_act(t, x, 3))
    assert not x[0].any() and x[1].isnan().any() and x[2].isnan().all()


def test_only_the_sum():
    a = make(5, 700, seed=1, gate="channel")
    h, x = run(a, x_out=False)
    hw, hb, _, _ = wanted(a)
    check(h, hw, hb)
    assert x is None


def test_rows_do_not_meet():
    """A row's NaN stays in it, a row's result does not depend on the others, same bits each time."""
    a = make(40, 200, seed=9)
    h, x = run(a)
    b = {k: None if v is None else v.clone() for k, v in a.items()}
    b["y"][7, 3] = float("nan")
    h2, x2 = run(b)
    keep = [i for i in range(40) if i != 7]
    assert torch.equal(h2[keep], h[keep]) and torch.equal(x2[keep], x[keep]) and x2[7].isnan().all()
    c = {k: v[11:12] if v is not None and v.dim() == 2 else v for k, v in a.items()}
    h3, x3 = run(c)
    assert torch.equal(h3, h[11:12]) and torch.equal(x3, x[11:12])


def test_no_rows():
    a = make(0, 64)
    h, x = run(a)
    assert h.shape == x.shape == (0, 64)


def test_streams_and_graphs():
    a = make(17, 1536, seed=4, gate="rows")
    h, x = run(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h1, x1 = run(a, stream=s)
    s.synchronize()
    assert torch.equal(h1, h) and torch.equal(x1, x)
    ho, xo = torch.empty_like(h), torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(a, h_out=ho, x_out=xo)
    for k in (1.0, -2.0):
        a["y"].mul_(k)
        graph.replay()
        h, x = run(a)
        assert torch.equal(ho, h) and torch.equal(xo, x)


def test_many_rows():
    """More rows than blocks run at once, the last ones among them."""
    n, d = 70001, 96
    a = make(n, d, seed=2, post=False, bias=False)
    h, x = run(a)
    rows = [0, 1, 35000, n - 2, n - 1]
    b = {k: v[rows] if v is not None and v.dim() == 2 else v for k, v in a.items()}
    hw, hb, xw, xb = wanted(b)
    check(h[rows], hw, hb)
    check(x[rows], xw, xb)


def test_a_chain_into_a_product():
    """norm -> activation blocks -> product equals norm -> product (which quantizes x itself), bit for bit."""
    d, n_out = 1024, 200
    g = torch.Generator(device="cuda").manual_seed(8)
    W = qg.quantize_rows(qg.Q4_0, torch.randn(n_out * d, generator=g, device="cuda"), n_out)
    a = make(2, d, seed=6)
    xq = torch.empty(2 * qg.qtype_nbytes(qg.Q8_0, d), dtype=torch.uint8, device="cuda")
    h, x = run(a, x_out=torch.empty(2, d, device="cuda"), xq=xq, act_type=qg.Q8_0)
    assert torch.equal(qg.qgemv_xq(qg.Q4_0, W, xq, n_out, d, 2), qg.qgemv(qg.Q4_0, W, x, n_out, d, 2))


def test_rows_past_32_bits():
    """Rows of every matrix 2^28 elements apart: the last begins behind 2^31."""
    apart, n, d = 1 << 28, 9, 96
    far = lambda x: torch.empty(apart * (n - 1) + d, dtype=x.dtype, device="cuda").as_strided((n, d), (apart, 1)).copy_(x)  # noqa: E731
    a = make(n, d, h=F16, y=F16, gate=None)
    want = run(a)
    b = dict(a, h=far(a["h"]), y=far(a["y"]))
    got = run(b, h_out=far(torch.zeros_like(a["h"])))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
