"""Several answers to one prompt, drawn token by token on this library alone: the
prompt's keys and values lie in the cache once, and every step's attention reads
them once for all answers.

    a layer     norm_residual -> qgemv_xq -> kv_append -> kv_attend_shared -> qgemv
    the end     norm_residual -> qgemv_xq -> sample_tokens

`python examples/many_answers.py` runs a small model of random weights, attention
layers only, eagerly and as one CUDA graph a step, and prints the times and
whether both drew the same tokens.
"""
import os
import sys

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import ggml_block_quantized_gb300 as qg  # noqa: E402
from attention_layer import AttentionLayer, _i32  # noqa: E402


class Model:
    """Layers of attention between a token's row and the logits; every norm is one with the residual's addition."""

    def __init__(self, vocab, n_in, n_layers, heads, kv_heads, head_dim, n_pos, t=qg.Q8_0, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weights(n_out, n):
            return qg.quantize_rows(t, torch.randn(n_out * n, generator=g, device="cuda") * n ** -0.5, n_out)

        self.t, self.act, self.vocab, self.n_in = t, qg.qtype_act_type(t), vocab, n_in
        self.kv_heads, self.head_dim = kv_heads, head_dim
        rope = qg.rope_table(n_pos, head_dim)
        self.layers = [AttentionLayer(t, weights((heads + 2 * kv_heads) * head_dim, n_in),
                                      weights(n_in, heads * head_dim), n_in, heads, kv_heads, head_dim, rope)
                       for _ in range(n_layers)]
        self.rows = torch.randn(vocab, n_in, generator=g, device="cuda").half()
        self.norms = [1 + 0.1 * torch.randn(n_in, generator=g, device="cuda") for _ in range(n_layers + 1)]
        self.w_logits = weights(vocab, n_in)

    def prompt(self, caches, tokens):
        """The prompt's keys and values, into the pages 0, 1, ... of every layer's cache."""
        n = tokens.shape[0]
        h, y, places, ends = self.rows[tokens], None, torch.arange(n, dtype=torch.int32, device="cuda"), _i32([0, n])
        for layer, cache, w in zip(self.layers, caches, self.norms):
            h2, x = qg.norm_residual(h, y, w)
            h = h if h2 is None else h2
            y = layer.output(layer.prompts(cache, x, places, places, ends))


class Answers:
    """n answers to one prompt: the state of a step, all of it on the device, so that a step can be captured."""

    def __init__(self, model, prompt, n, steps, page_size=64, temperature=0.8, top_k=40, top_p=0.95, seed=2):
        assert n <= qg.MAX_NVEC
        self.m, self.n = model, n
        shared, own = -(-prompt.shape[0] // page_size), -(-steps // page_size)
        self.caches = [qg.KVCache.empty(shared + n * own, model.kv_heads, model.head_dim, page_size)
                       for _ in model.layers]
        model.prompt(self.caches, prompt)
        self.prefix, self.prefix_len = _i32(list(range(shared))), _i32([prompt.shape[0]])
        self.table = _i32([[shared + s * own + i for i in range(own)] for s in range(n)])
        places = self.table.long() * page_size
        self.slots = (places[:, :, None] + torch.arange(page_size, device="cuda")).flatten(1).int()  # [n, tokens]
        self.step = torch.zeros(1, dtype=torch.long, device="cuda")
        self.lengths = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.last = prompt[-1:].repeat(n)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.uniform = torch.rand(steps, n, generator=g, device="cuda")
        full = lambda v, t=torch.float32: torch.full((n,), v, dtype=t, device="cuda")  # noqa: E731
        self.temperature, self.top_k, self.top_p = full(temperature), full(top_k, torch.int32), full(top_p)
        self.xq = torch.empty(n * qg.qtype_nbytes(model.act, model.n_in), dtype=torch.uint8, device="cuda")
        self.tokens = torch.full((steps, n), -1, dtype=torch.int32, device="cuda")
        self.probs = torch.zeros(steps, n, device="cuda")

    def product(self, W, n_out):
        return qg.qgemv_xq(self.m.t, W, self.xq, n_out, self.m.n_in, self.n)

    def one_step(self):
        """The next token of every answer."""
        m, n = self.m, self.n
        slots = self.slots.index_select(1, self.step).flatten()
        self.lengths += 1
        positions = self.prefix_len + self.lengths - 1
        h, y = m.rows[self.last], None
        for layer, cache, w in zip(m.layers, self.caches, m.norms):
            qg.norm_residual(h, y, w, h_out=None if y is None else h, x_out=False, xq=self.xq, act_type=m.act)
            heads = layer.heads
            qkv = self.product(layer.w_qkv, (heads + 2 * m.kv_heads) * m.head_dim).view(n, -1, m.head_dim)
            q = qg.kv_append(cache, qkv[:, heads:heads + m.kv_heads], qkv[:, heads + m.kv_heads:], slots,
                             positions=positions, rope=layer.rope, q=qkv[:, :heads])
            y = layer.output(qg.kv_attend_shared(cache, q, self.prefix, self.prefix_len, self.table, self.lengths))
        qg.norm_residual(h, y, m.norms[-1], h_out=h, x_out=False, xq=self.xq, act_type=m.act)
        prob = torch.empty(n, device="cuda")
        token, _ = qg.sample_tokens(self.product(m.w_logits, m.vocab).view(n, -1), self.uniform[self.step].flatten(),
                                    self.temperature, self.top_k, self.top_p, prob_out=prob)
        self.tokens.index_copy_(0, self.step, token[None])
        self.probs.index_copy_(0, self.step, prob[None])
        self.last.copy_(token)
        self.step += 1


def run(model, prompt, n, steps, graph, **kw):
    """The tokens [steps, n], their probabilities and a step's milliseconds."""
    a = Answers(model, prompt, n, steps, **kw)
    once = a.one_step
    if graph:
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # one step on its own first, as a capture wants; the graph goes on from it
            a.one_step()
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(g):
            a.one_step()
        once = g.replay
    marks = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    marks[0].record()
    for _ in range(steps - 1 if graph else steps):
        once()
    marks[1].record()
    torch.cuda.synchronize()
    return a.tokens, a.probs, marks[0].elapsed_time(marks[1]) / max(1, steps - 1 if graph else steps)


def main():
    model = Model(vocab=32000, n_in=2048, n_layers=4, heads=16, kv_heads=4, head_dim=128, n_pos=2048)
    prompt = torch.randint(0, model.vocab, (1500,), device="cuda")
    run(model, prompt, 8, 4, False)
    tokens, _, eager = run(model, prompt, 8, 32, False)
    again, _, captured = run(model, prompt, 8, 32, True)
    if qg.device_error():
        raise SystemExit("a kernel reported an error")
    print(f"8 answers to a prompt of 1500 tokens, a step: {eager:.3f} ms, as a graph {captured:.3f} ms")
    print("the graph drew " + ("the same tokens" if torch.equal(tokens, again) else "other tokens"))


if __name__ == "__main__":
    main()
