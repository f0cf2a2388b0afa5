"""The attention half of a decoder layer, served from a paged int8 cache.

Per step, for every sequence of the batch at once (prompt chunks and decode
steps mixed as they come):

    r  = residual + h;  y = rmsnorm(r) * w     tern_add_rmsnorm_s8 (int8 codes)
    qkv = y W_qkv                              tern_linear_s8
    cache <- k, v                              tern_kv8_append
    o  = attention(q, cache)                   tern_kv8_attention
    h' = o W_o                                 tern_linear

The next block's norm takes (h', r).  A position embedding would go between
the projection and the cache; queries, keys and values are used as they come.

    python examples/attention_block.py
"""
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch  # noqa: E402

import ternary_weight_linear_gb300 as tl  # noqa: E402


class Pages:
    """Pages of one pool for a fixed set of sequences: a free list on the host,
    the table and the lengths on the device."""

    def __init__(self, pages, seqs, width):
        self.free = list(range(pages - 1, -1, -1))
        self.owned = [[] for _ in range(seqs)]
        self.lens = [0] * seqs
        self.host = torch.zeros(seqs, width, dtype=torch.int32).pin_memory()
        self.table = self.host.cuda()

    def grow(self, new):
        """new[b] more tokens for sequence b -> (row starts, lengths) on the device."""
        for b, m in enumerate(new):
            self.lens[b] += m
            while len(self.owned[b]) * tl.KV8_BLOCK < self.lens[b]:
                if not self.free:
                    raise RuntimeError("the pool has no free page")
                self.host[b, len(self.owned[b])] = self.free[-1]
                self.owned[b].append(self.free.pop())
        self.table.copy_(self.host)
        start = [0]
        for m in new:
            start.append(start[-1] + m)
        return (torch.tensor(start, dtype=torch.int32, device="cuda"),
                torch.tensor(self.lens, dtype=torch.int32, device="cuda"))

    def release(self, b):
        """Sequence b has ended: its pages are free."""
        self.free += reversed(self.owned[b])
        self.owned[b], self.lens[b] = [], 0


class AttentionBlock:
    """norm [hidden] bf16; qkv and out: (packed weights, scales) of the
    projections, [(heads + 2 kv_heads) dim, hidden] and [hidden, heads dim]."""

    def __init__(self, norm, qkv, out, heads, kv_heads, dim, pages, window=0, sinks=0, eps=1e-6):
        self.norm, self.qkv, self.out = norm, qkv, out
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.window, self.sinks, self.eps = window, sinks, eps
        self.codes = torch.zeros(pages, 2, kv_heads, tl.KV8_BLOCK, dim, dtype=torch.int8,
                                 device="cuda")
        self.scales = torch.zeros(pages, 2, kv_heads, device="cuda")
        self.workspaces = {}

    def _workspace(self, name, need):
        """Kept across calls; zeroed once, as the library asks."""
        ws = self.workspaces.get(name)
        if need and (ws is None or ws.numel() < need):
            ws = self.workspaces[name] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        return ws

    def __call__(self, h, residual, table, start, lens, max_new):
        """h fp32 and residual bf16 [rows, hidden] -> the next block's pair."""
        rows, hidden = h.shape
        n, d = self.heads, self.dim
        q, x_scale, residual = tl.tern_add_rmsnorm_s8(h, self.norm, residual, self.eps)
        width = (n + 2 * self.kv_heads) * d
        y = tl.tern_linear_s8(*self.qkv, q, x_scale, workspace=self._workspace(
            "linear", tl.tern_linear_workspace_bytes(rows, hidden, width)))
        y = y.view(rows, -1, d)
        tl.tern_kv8_append(y[:, n:n + self.kv_heads], y[:, n + self.kv_heads:], self.codes,
                           self.scales, table, start, lens, max_new=max_new)
        o = tl.tern_kv8_attention(
            y[:, :n].bfloat16(), self.codes, self.scales, table, start, lens, max_new=max_new,
            window=self.window, sinks=self.sinks, workspace=self._workspace(
                "attention", tl.tern_kv8_attention_workspace_bytes(len(lens), rows, n,
                                                                   self.kv_heads, d)))
        h = tl.tern_linear(*self.out, o.view(rows, n * d), workspace=self._workspace(
            "linear", tl.tern_linear_workspace_bytes(rows, n * d, hidden)))
        return h, residual


def random_projection(rows, width, gen):
    """(packed weights, scales) of a random ternary matrix whose outputs have
    about the size of its inputs."""
    w = (torch.rand(rows, width, generator=gen, device="cuda") * 3).floor().to(torch.int8) - 1
    scale = torch.full((rows, width // 128), (1.5 / width) ** 0.5, device="cuda").half()
    return tl.tern_pack(w), scale


def main():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    hidden, heads, kv_heads, dim = 5120, 48, 8, 128
    block = AttentionBlock(
        torch.ones(hidden, device="cuda").bfloat16(),
        random_projection((heads + 2 * kv_heads) * dim, hidden, gen),
        random_projection(hidden, heads * dim, gen), heads, kv_heads, dim, pages=256)
    pages = Pages(256, 3, 64)
    # two prompts in chunks, a third sequence that starts when they decode
    steps = [[500, 300, 0], [500, 200, 0], [1, 1, 400]] + [[1, 1, 1]] * 5
    for new in steps:
        start, lens = pages.grow(new)
        rows = sum(new)
        h = torch.randn(rows, hidden, generator=gen, device="cuda")
        residual = torch.randn(rows, hidden, generator=gen, device="cuda").bfloat16()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        h, residual = block(h, residual, pages.table, start, lens, max(new))
        end.record()
        end.synchronize()
        print(f"{rows:5d} new tokens, {sum(pages.lens):5d} cached: "
              f"{begin.elapsed_time(end) * 1e3:8.1f} us")
    status = tl.tern_device_status()  # (reading it clears it)
    if status:
        raise RuntimeError(tl.tern_status_string(status))


if __name__ == "__main__":
    main()
