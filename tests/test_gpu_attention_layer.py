"""The example's layer: products, append, prompt attention and attention over
the cache, one after the other on one stream, as a user runs them."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attn_ref  # noqa: E402
import ggml_block_quantized_gb300 as qg  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import attention_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu
LENGTHS, STEPS, PAGE = [37, 1, 130], 3, 32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert qg.device_error() == 0


@pytest.mark.parametrize("heads,kv_heads,head_dim", [(6, 2, 64), (4, 4, 128)])
def test_layer(heads, kv_heads, head_dim):
    """Each sequence's prompt rows against 64-bit attention over f16 rows, each step's against 64-bit attention over
    the 4-bit values of all its rows. The bounds are the operators' own (f16 rows and weights for a prompt; f32 rows
    and split weights for a step)."""
    n_in = 256
    layer = ex.random_layer(heads, kv_heads, head_dim, n_in, n_pos=256)
    g = torch.Generator(device="cuda").manual_seed(head_dim)
    x = [torch.randn(n + STEPS, n_in, generator=g, device="cuda") for n in LENGTHS]
    got, _, _ = ex.run(layer, x, LENGTHS, STEPS, PAGE)
    assert [tuple(r.shape) for r in got] == [(sum(LENGTHS), heads, head_dim)] + [(len(LENGTHS), heads, head_dim)] * STEPS
    assert layer.output(got[1]).shape == (len(LENGTHS), n_in)
    packed = torch.cat([r[:n] for r, n in zip(x, LENGTHS)])
    pq, pk, pv = (t.cpu().numpy() for t in layer.project(packed))  # as the prompts' one product gives them
    scale, group, at = head_dim ** -0.5, heads // kv_heads, 0
    for s, n in enumerate(LENGTHS):
        table = layer.rope.cpu().numpy()[:n + STEPS]
        q, k, v = pq[at:at + n], pk[at:at + n], pv[at:at + n]
        q, k = (attn_ref.rotate(t, table[:n], False, np.float32) for t in (q, k))
        mine = got[0][at:at + n].cpu().numpy()
        for h in range(heads):
            a, b, c = (t.astype(np.float16).astype(np.float64) for t in (q[:, h], k[:, h // group], v[:, h // group]))
            out, p_v, mag, big = attn_ref.attend(a, b, c, np.arange(1, n + 1), scale)
            assert np.all(np.abs(mine[:, h] - out) <= attn_ref.bound(out, p_v, mag, big, head_dim, n, 24, 10, False))
        for i in range(STEPS):  # a step's three rows are one product; the next row of k and v joins the sequence's
            new = torch.stack([r[m + i] for r, m in zip(x, LENGTHS)])
            nq, nk, nv = (t.cpu().numpy()[s:s + 1] for t in layer.project(new))
            nq, nk = (attn_ref.rotate(t, table[n + i:n + i + 1], False, np.float32) for t in (nq, nk))
            k, v = np.concatenate([k, nk]), np.concatenate([v, nv])
            mine_s = got[1 + i][s].cpu().numpy()
            for h in range(heads):
                b, c = (attn_ref.q4_0_values(*attn_ref.q4_0(t[:, h // group])) for t in (k, v))
                out, p_v, mag, big = attn_ref.attend(nq[:, h].astype(np.float64), b, c, [len(k)], scale)
                assert np.all(np.abs(mine_s[h:h + 1] - out) <=
                              attn_ref.bound(out, p_v, mag, big, head_dim, len(k), 20, 20, False))
        at += n


def test_outputs_for_another_stream_are_its_own():
    """Work on the current stream that still writes to memory it has given back does not reach what a call on another
    stream allocates for itself (outputs and workspace)."""
    rng = np.random.default_rng(50)
    x = torch.from_numpy(rng.standard_normal((40, 12, 128)).astype(np.float32)).cuda()
    q, k, v = x[:, :8].contiguous(), x[:, 8:10].contiguous(), x[:, 10:].contiguous()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    slots, table, lengths, ends = i32(list(range(40))), i32([[0, 1, 2]]), i32([40]), i32([0, 40])
    cache = qg.KVCache(2, 128, 16, torch.zeros(48 * 2 * 144, dtype=torch.uint8, device="cuda"))
    h = [t.half() for t in (q, k, v)]
    calls = [lambda s: qg.kv_append(cache, k, v, slots, q=q, stream=s),
             lambda s: torch.cat(qg.kv_read(cache, slots, stream=s)) if s is None else qg.kv_read(cache, slots, stream=s),
             lambda s: qg.kv_attend(cache, q, table, lengths, q_offsets=ends, max_q_len=40, stream=s),
             lambda s: qg.prompt_attend(*h, ends, stream=s)]
    want = [c(None) for c in calls]
    sizes = sorted({t.numel() * t.element_size() for t in want} | {x.numel(), qg.kv_attend_workspace_bytes(cache, 8, 40)} |
                   {k.numel() * 4})
    side = torch.cuda.Stream()
    for c, w in zip(calls, want):
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)  # some 50 ms, and then writes to blocks that have been given back by then
        for n in sizes * 3:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        got = c(side)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(torch.cat(got) if isinstance(got, tuple) else got, w)


def test_example_command(capsys):
    ex.main()
    text = capsys.readouterr().out
    assert "prompt rows" in text and "apart" in text
