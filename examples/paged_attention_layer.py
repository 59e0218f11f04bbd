"""The attention half of one decoder layer, served with a paged NVFP4 cache.

The W4A4 linears of the library on both sides of the cache's three calls:

    qkv linear -> kv_tables (pages and slots of the step) -> kv_append (keys and
    values to 4 bits) -> kv_attention -> o linear

Three requests with prompts of different lengths are admitted in one step (all
their tokens attend in one call) and then decoded a token at a time, their pages
taken from a free list on the GPU as they grow; one decode step is captured in
a CUDA graph and replayed.  Weights and inputs are random.  Run from the
repository's root on a machine with the library built:

    python examples/paged_attention_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_w4a4_decode_gb300 as nv  # noqa: E402


class AttentionLayer:
    """Packed qkv and o weights, and the layer's cache."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, pages, page_size, calibration, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        rows = (q_heads + 2 * kv_heads) * head_dim
        self.w_qkv = torch.randn((rows, hidden), generator=gen, device="cuda") * hidden ** -0.5
        self.w_o = torch.randn((hidden, q_heads * head_dim), generator=gen, device="cuda") * hidden ** -0.5
        self.qkv, self.o = nv.pack_weight(self.w_qkv), nv.pack_weight(self.w_o)
        # tensor scales from calibration rows: the layer's input, keys, values, and the
        # attention's output (averages of values, so the values' scale covers it)
        self.x_g = nv.global_scale(calibration)
        _, k, v = self.split(calibration @ self.w_qkv.T)
        self.cache = nv.KVCache(nv.kv_pool(pages, kv_heads, head_dim, page_size),
                                nv.global_scale(k.contiguous()), nv.global_scale(v.contiguous()),
                                page_size=page_size, head_dim=head_dim)

    def split(self, qkv):
        """[tokens, ...] rows of the qkv linear as q, k, v heads (views)."""
        heads = qkv.unflatten(-1, (-1, self.head_dim))
        return heads.split((self.q_heads, self.kv_heads, self.kv_heads), dim=1)

    def project(self, x, weight, x_g):
        """x . W^T for any number of rows, eight at a time (the linears' limit)."""
        return torch.cat([nv.linear(r, x_g, *weight, out_dtype=torch.bfloat16) for r in x.split(nv.MAX_M)])

    def step(self, x, step, table, max_q):
        """The rows x of a step through the layer: writes the cache, returns the o linear's rows."""
        q, k, v = self.split(self.project(x, self.qkv, self.x_g))
        nv.kv_append(self.cache, k, v, step.slots)
        y = nv.kv_attention(self.cache, q, table, step.seq_len, step.q_start, max_q=max_q)
        return self.project(y.flatten(1), self.o, self.cache.v_g)


def run(prompts=(37, 5, 90), steps=20, hidden=512, q_heads=8, kv_heads=2, head_dim=64, page_size=16, seed=0):
    """Serves the prompts and `steps` tokens each.  Returns the layer, the block
    table, the lengths, and every row's input and output in order, a request each."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    reqs = len(prompts)
    blocks = -(-(max(prompts) + steps) // page_size)
    pages = reqs * blocks
    layer = AttentionLayer(hidden, q_heads, kv_heads, head_dim, pages, page_size,
                           torch.randn((64, hidden), generator=gen, device="cuda") * 1.5, seed)
    free = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((reqs, blocks), -1, dtype=torch.int32, device="cuda")
    inputs, outputs = [[] for _ in prompts], [[] for _ in prompts]

    # all prompts in one step
    x = torch.randn((sum(prompts), hidden), generator=gen, device="cuda")
    t = nv.kv_tables(ints([0] * reqs), ints(prompts), free, ints([0]), table, page_size=page_size,
                     tokens=sum(prompts))
    y = layer.step(x, t, table, max(prompts))
    for r, (a, b) in enumerate(zip(x.split(prompts), y.split(prompts))):
        inputs[r].append(a)
        outputs[r].append(b)

    # one decode step as a graph: lengths, the free list's head and the inputs are its buffers
    lens, head, one = t.seq_len.clone(), t.free_head.clone(), ints([1] * reqs)
    x = torch.randn((reqs, hidden), generator=gen, device="cuda")

    def decode():
        t = nv.kv_tables(lens, one, free, head, table, page_size=page_size, tokens=reqs)
        y = layer.step(x, t, table, 1)
        lens.copy_(t.seq_len)
        head.copy_(t.free_head)
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = [v.clone() for v in (lens, head, table)]
    with torch.cuda.stream(side):
        decode()  # once outside the capture (its tokens are written again below)
        for v, was in zip((lens, head, table), keep):
            v.copy_(was)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = decode()
    for _ in range(steps):
        x.copy_(torch.randn((reqs, hidden), generator=gen, device="cuda"))
        graph.replay()
        for r in range(reqs):
            inputs[r].append(x[r:r + 1].clone())
            outputs[r].append(y[r:r + 1].clone())
    torch.cuda.synchronize()
    return layer, table, lens.tolist(), [torch.cat(v) for v in inputs], [torch.cat(v) for v in outputs]


def dense(layer, x):
    """The same layer without quantisation: float32 weights, keys, values and softmax."""
    q, k, v = (h.transpose(0, 1) for h in layer.split(x @ layer.w_qkv.T))
    group = layer.q_heads // layer.kv_heads
    k, v = (h.repeat_interleave(group, 0) for h in (k, v))
    s = q @ k.transpose(1, 2) * layer.head_dim ** -0.5
    s = s.masked_fill(torch.ones_like(s, dtype=torch.bool).triu(1), float("-inf"))
    return (torch.softmax(s, -1) @ v).transpose(0, 1).flatten(1) @ layer.w_o.T


def main():
    layer, table, lens, inputs, outputs = run()
    assert nv.device_status() == 0
    print(f"lengths {lens}, pages {[(row >= 0).sum().item() for row in table]}")
    for r, (x, y) in enumerate(zip(inputs, outputs)):
        want = dense(layer, x)
        cos = torch.nn.functional.cosine_similarity(y.float().flatten(), want.flatten(), dim=0).item()
        print(f"request {r}: {len(x)} rows, cosine to the unquantised layer {cos:.4f}")


if __name__ == "__main__":
    main()
