"""The attention half of a decoder layer on this library alone: block-quantized
products around a paged 4-bit cache of keys and values.

    prompts        qgemm -> kv_append -> prompt_attend -> qgemm
    a step         qgemv -> kv_append -> kv_attend     -> qgemv

`python examples/attention_layer.py` packs a few prompts of random rows,
generates from them for some steps, and prints the times and how far the last
step is from the same tokens run as whole prompts, whose keys and values never
went through 4 bits.
"""
import os
import sys

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import ggml_block_quantized_gb300 as qg  # noqa: E402


class Pages:
    """Which pages of a cache each sequence holds, on the host."""

    def __init__(self, n_pages, page_size, n_seq):
        self.page_size, self.free, self.of = page_size, list(range(n_pages)), [[] for _ in range(n_seq)]
        self.lengths = [0] * n_seq

    def take(self, counts):
        """Room for counts[s] more tokens of each sequence: their slots and positions, packed."""
        slots, positions = [], []
        for s, n in enumerate(counts):
            first, self.lengths[s] = self.lengths[s], self.lengths[s] + n
            while len(self.of[s]) * self.page_size < self.lengths[s]:
                self.of[s].append(self.free.pop())
            positions += range(first, self.lengths[s])
            slots += [self.of[s][i // self.page_size] * self.page_size + i % self.page_size
                      for i in range(first, self.lengths[s])]
        return _i32(slots), _i32(positions)

    def table(self):
        most = max(map(len, self.of))
        return _i32([p + [-1] * (most - len(p)) for p in self.of]), _i32(self.lengths)


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class AttentionLayer:
    """w_qkv [(heads + 2 kv_heads) * head_dim, n_in] and w_out [n_in, heads * head_dim],
    in blocks of weight type t."""

    def __init__(self, t, w_qkv, w_out, n_in, heads, kv_heads, head_dim, rope):
        self.t, self.w_qkv, self.w_out, self.rope = t, w_qkv, w_out, rope
        self.n_in, self.heads, self.kv_heads, self.head_dim = n_in, heads, kv_heads, head_dim

    def _product(self, W, x, n_out, n_in):
        n = x.shape[0]
        f = qg.qgemv if n <= qg.MAX_NVEC else qg.qgemm  # few rows: W is read once a call; many: a matrix product
        return f(self.t, W, x, n_out, n_in, n)

    def project(self, x):
        """x f32 [n, n_in] -> q, k, v: the columns of one product, none copied."""
        h, hk, d = self.heads, self.kv_heads, self.head_dim
        y = self._product(self.w_qkv, x, (h + 2 * hk) * d, self.n_in).view(x.shape[0], h + 2 * hk, d)
        return y[:, :h], y[:, h:h + hk], y[:, h + hk:]

    def prompts(self, cache, x, slots, positions, offsets):
        """Whole prompts, packed: the attended rows, f32 [n, heads, head_dim]. Their keys and values go to the
        cache; the prompts' own attention reads the f16 rows that kv_append hands out."""
        q, k, v = self.project(x)
        k16, v16 = (torch.empty(k.shape, dtype=torch.float16, device=x.device) for _ in range(2))
        q16 = qg.kv_append(cache, k, v, slots, positions=positions, rope=self.rope, q=q, k_out=k16, v_out=v16)
        out = torch.empty(q.shape, dtype=torch.float32, device=x.device)
        return qg.prompt_attend(q16, k16, v16, offsets, out=out)

    def step(self, cache, x, slots, positions, table, lengths):
        """The next token of every sequence: the attended rows, f32 [n_seq, heads, head_dim]."""
        q, k, v = self.project(x)
        q = qg.kv_append(cache, k, v, slots, positions=positions, rope=self.rope, q=q)
        return qg.kv_attend(cache, q, table, lengths)

    def output(self, rows):
        return self._product(self.w_out, rows.flatten(1), self.n_in, self.heads * self.head_dim)


def random_layer(heads=32, kv_heads=8, head_dim=128, n_in=4096, n_pos=4096, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_qkv = (heads + 2 * kv_heads) * head_dim

    def weights(n_out, n):
        w = torch.randn(n_out * n, generator=g, device="cuda") * n ** -0.5
        return qg.quantize_rows(qg.Q8_0, w, n_out)

    return AttentionLayer(qg.Q8_0, weights(n_qkv, n_in), weights(n_in, heads * head_dim), n_in, heads, kv_heads,
                          head_dim, qg.rope_table(n_pos, head_dim))


def run(layer, x, lengths, steps, page_size=64):
    """x[s]: the rows of sequence s, its prompt of lengths[s] rows and then one a step. Returns the attended rows of
    the prompts and of each step, and the milliseconds of the prompts and of the last step."""
    pages = Pages(sum(-(-(n + steps) // page_size) for n in lengths) + 1, page_size, len(lengths))
    cache = qg.KVCache.empty(len(pages.free), layer.kv_heads, layer.head_dim, page_size)
    slots, positions = pages.take(lengths)
    offsets = torch.tensor([0] + lengths).cumsum(0).int().cuda()
    marks = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    packed = torch.cat([r[:n] for r, n in zip(x, lengths)])
    marks[0].record()
    rows = [layer.prompts(cache, packed, slots, positions, offsets)]
    layer.output(rows[0])
    marks[1].record()
    for i in range(steps):
        slots, positions = pages.take([1] * len(lengths))
        table, held = pages.table()
        new = torch.stack([r[n + i] for r, n in zip(x, lengths)])
        marks[2].record()
        rows.append(layer.step(cache, new, slots, positions, table, held))
        layer.output(rows[-1])
        marks[3].record()
    torch.cuda.synchronize()
    return rows, marks[0].elapsed_time(marks[1]), marks[2].elapsed_time(marks[3]) if steps else 0.0


def main():
    lengths, steps = [700, 61, 1500, 1], 8
    layer = random_layer()
    g = torch.Generator(device="cuda").manual_seed(2)
    x = [torch.randn(n + steps, layer.n_in, generator=g, device="cuda") for n in lengths]
    run(layer, x, lengths, steps)
    rows, t_prompt, t_step = run(layer, x, lengths, steps)
    whole, _, _ = run(layer, x, [n + steps for n in lengths], 0)
    ends = torch.tensor([n + steps for n in lengths]).cumsum(0) - 1
    want = whole[0][ends.cuda()]
    off = ((rows[-1] - want).norm() / want.norm()).item()
    if qg.device_error():
        raise SystemExit("a kernel reported an error")
    print(f"{sum(lengths)} prompt rows: {t_prompt:.3f} ms; a step of {len(lengths)} sequences: {t_step:.3f} ms")
    print(f"step {steps} against the same rows run as prompts: {100 * off:.1f}% apart (keys and values in 4 bits)")


if __name__ == "__main__":
    main()
