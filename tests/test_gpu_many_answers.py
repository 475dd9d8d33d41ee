"""The example's steps: norm, product, append, attention over the shared prompt,
product, norm, logits and sample, one after the other on one stream, as a user
runs them; each call's result against its own formula in 64 bits on the inputs
that the calls before it made."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attn_ref  # noqa: E402
import ggml_block_quantized_gb300 as qg  # noqa: E402
import step_ref  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import many_answers as ex  # noqa: E402

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


def model(head_dim=64, heads=6, kv_heads=2):
    return ex.Model(vocab=1003, n_in=256, n_layers=2, heads=heads, kv_heads=kv_heads, head_dim=head_dim, n_pos=512)


def npy(t):
    return t.detach().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("n,prompt_len", [(3, 150), (8, 64), (1, 1)])
def test_graph_and_eager_draw_alike(n, prompt_len):
    m = model()
    prompt = torch.randint(0, m.vocab, (prompt_len,), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda")
    eager = ex.run(m, prompt, n, 40, False, page_size=16)
    graph = ex.run(m, prompt, n, 40, True, page_size=16)
    assert torch.equal(eager[0], graph[0]) and torch.equal(eager[1], graph[1])
    assert ((eager[0] >= 0) & (eager[0] < m.vocab)).all() and ((eager[1] > 0) & (eager[1] <= 1)).all()


@pytest.mark.parametrize("head_dim,heads,kv_heads", [(64, 6, 2), (128, 4, 4)])
def test_every_call_of_a_step(monkeypatch, head_dim, heads, kv_heads):
    """The bounds are the operators' own: step_ref's of a norm, attn_ref's of attention, tokens equal and their
    probabilities off by three roundings and the weights' unit. A norm's blocks are those of quantize_act of its x."""
    m, n, prompt_len, steps = model(head_dim, heads, kv_heads), 5, 140, 4
    seen = {"norm": 0, "attend": 0, "sample": 0}
    real = qg.norm_residual, qg.kv_attend_shared, qg.sample_tokens

    def norm(h, y=None, weight=None, **kw):
        if "xq" not in kw:  # (the prompt's)
            return real[0](h, y, weight, **kw)
        seen["norm"] += 1
        hn, yn = npy(h), None if y is None else npy(y)
        x = real[0](h, y, weight)[1]
        out = real[0](h, y, weight, **kw)
        hw, hb, xw, xb = step_ref.norm_residual(hn, yn, npy(weight))
        if y is not None:
            assert np.all(np.abs(npy(h) - hw) <= step_ref.half(hb, hw))
        assert np.all(np.abs(npy(x) - xw) <= xb)
        assert torch.equal(kw["xq"], qg.quantize_act(m.act, x, n).flatten())
        return out

    def attend(cache, q, prefix, prefix_len, table, lengths):
        seen["attend"] += 1
        out = real[1](cache, q, prefix, prefix_len, table, lengths)
        page, own = cache.page_size, int(lengths[0])
        for s in range(n):
            at = [int(prefix[i // page]) * page + i % page for i in range(prompt_len)]
            at += [int(table[s, i // page]) * page + i % page for i in range(own)]
            k, v = (npy(t) for t in qg.kv_read(cache, torch.tensor(at, dtype=torch.int32, device="cuda")))
            for h in range(heads):
                g = h // (heads // kv_heads)
                want, pv, mag, big = attn_ref.attend(npy(q[s:s + 1, h]), k[:, g], v[:, g], [len(at)], head_dim ** -0.5)
                assert np.all(np.abs(npy(out[s:s + 1, h]) - want) <=
                              attn_ref.bound(want, pv, mag, big, head_dim, len(at), 20, 20, False))
        return out

    def sample(logits, uniform, temperature, top_k, top_p, prob_out):
        seen["sample"] += 1
        out = real[2](logits, uniform, temperature, top_k, top_p, prob_out=prob_out)
        tokens, probs = step_ref.sample(npy(logits), npy(uniform), npy(temperature), top_k.cpu().numpy(), npy(top_p))
        assert np.array_equal(out[0].cpu().numpy(), tokens)
        assert np.all(np.abs(npy(prob_out) - probs) <= 2.0 ** -22 * probs + 2.0 ** -44.9)
        return out

    for name, f in (("norm_residual", norm), ("kv_attend_shared", attend), ("sample_tokens", sample)):
        monkeypatch.setattr(qg, name, f)
    g = torch.Generator(device="cuda").manual_seed(head_dim)
    prompt = torch.randint(0, m.vocab, (prompt_len,), generator=g, device="cuda")
    ex.run(m, prompt, n, steps, False, page_size=16)
    assert seen == {"norm": 3 * steps, "attend": 2 * steps, "sample": steps}


def test_example_command(capsys):
    ex.main()
    text = capsys.readouterr().out
    assert "answers to a prompt" in text and "same tokens" in text
