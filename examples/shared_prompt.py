"""The attention half of a decoder layer for a batch that shares its prompt, with
rotary positions and a norm on either side of the residual's addition.

Per step, for every sequence of the batch at once:

    qkv = codes W_qkv                              tern_linear_s8
    q, cache <- turned q, k and v                  tern_kv8_append_rope
    o  = attention(q, shared pages and own)        tern_kv8_attention_shared
    h  = o W_o                                     tern_linear
    r  = residual + gate * rmsnorm(h) * w1
    codes of rmsnorm(r) * w2                       tern_norm_add_norm_s8

The prompt's keys and values are computed once; every sequence's row of the page
table then begins with its pages.

    python examples/shared_prompt.py
"""
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch  # noqa: E402

import ternary_weight_linear_gb300 as tl  # noqa: E402


class Block:
    """qkv and out: (packed weights, scales) of the projections; post, norm [hidden]
    and gate [hidden] bf16; freq, magnitude: tern_rope_frequencies."""

    def __init__(self, qkv, out, post, gate, norm, freq, magnitude, heads, kv_heads, dim, pages):
        self.qkv, self.out, self.post, self.gate, self.norm = qkv, out, post, gate, norm
        self.freq, self.magnitude = freq, magnitude
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.codes = torch.zeros(pages, 2, kv_heads, tl.KV8_BLOCK, dim, dtype=torch.int8,
                                 device="cuda")
        self.scales = torch.zeros(pages, 2, kv_heads, device="cuda")
        self.workspaces = {}

    def _workspace(self, name, need):
        """Kept across calls; zeroed once, as the library asks."""
        ws = self.workspaces.get(name)
        if ws is None or ws.numel() < need:
            ws = self.workspaces[name] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        return ws

    def __call__(self, q, x_scale, residual, table, start, lens, max_new, shared):
        """Codes and scales of the block's input, the residual [rows, hidden] -> the
        same for what follows."""
        rows, hidden = q.shape
        n, kv, d = self.heads, self.kv_heads, self.dim
        width = (n + 2 * kv) * d
        y = tl.tern_linear_s8(*self.qkv, q, x_scale, workspace=self._workspace(
            "linear", tl.tern_linear_workspace_bytes(rows, hidden, width))).view(rows, -1, d)
        turned = tl.tern_kv8_append_rope(
            y[:, :n], y[:, n:n + kv], y[:, n + kv:], self.codes, self.scales, table, start, lens,
            self.freq, magnitude=self.magnitude, max_new=max_new)
        need = (tl.tern_kv8_attention_shared_workspace_bytes if shared and len(lens) > 1
                else tl.tern_kv8_attention_workspace_bytes)
        o = tl.tern_kv8_attention_shared(
            turned, self.codes, self.scales, table, start, lens, shared, max_new=max_new,
            workspace=self._workspace("attention", need(len(lens), rows, n, kv, d)))
        h = tl.tern_linear(*self.out, o.view(rows, n * d), workspace=self._workspace(
            "linear", tl.tern_linear_workspace_bytes(rows, n * d, hidden)))
        return tl.tern_norm_add_norm_s8(h, self.post, residual, self.norm, gate=self.gate)


def random_projection(rows, width, gen):
    """(packed weights, scales) of a random ternary matrix whose outputs have
    about the size of its inputs."""
    w = (torch.rand(rows, width, generator=gen, device="cuda") * 3).floor().to(torch.int8) - 1
    scale = torch.full((rows, width // 128), (1.5 / width) ** 0.5, device="cuda").half()
    return tl.tern_pack(w), scale


def serve(block, hidden, prompt, seqs, steps, gen):
    """`prompt` tokens once, then `steps` decode steps of `seqs` sequences behind them.
    -> the last step's (codes, x_scale, residual)."""
    page = tl.KV8_BLOCK
    common = prompt // page  # whole pages are shared, the rest is each sequence's own
    own = -(-(prompt - common * page + steps) // page)
    table = torch.arange(common, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    table = torch.cat((table, common + torch.arange(seqs * own, dtype=torch.int32,
                                                    device="cuda").view(seqs, own)), 1)

    def tokens(rows):
        x = torch.randn(rows, hidden, generator=gen, device="cuda")
        r = torch.randn(rows, hidden, generator=gen, device="cuda").bfloat16()
        return tl.tern_norm_add_norm_s8(x, None, r, block.norm)

    def lengths(*values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    # the shared pages, by the first sequence alone; then what is left of the prompt
    # behind them, in pages of each
    if common:
        block(*tokens(common * page), table[:1], lengths(0, common * page),
              lengths(common * page), common * page, 0)
    rest = prompt - common * page
    if rest:
        q, x_scale, r = tokens(rest)
        block(q.repeat(seqs, 1), x_scale.repeat(seqs), r.repeat(seqs, 1), table,
              lengths(*range(0, seqs * rest + 1, rest)), lengths(*[prompt] * seqs), rest,
              common * page)
    got = None
    for step in range(1, steps + 1):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        inputs = tokens(seqs)
        begin.record()
        got = block(*inputs, table, lengths(*range(seqs + 1)), lengths(*[prompt + step] * seqs), 1,
                    common * page)
        end.record()
        end.synchronize()
        print(f"step {step}: {seqs} sequences behind {common * page} shared tokens: "
              f"{begin.elapsed_time(end) * 1e3:8.1f} us")
    return got


def main():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    hidden, heads, kv_heads, dim = 5120, 48, 8, 128
    freq, magnitude = tl.tern_rope_frequencies(dim, base=1e6, scaling="ramp", factor=4.0,
                                               trained=8192)
    ones = torch.ones(hidden, device="cuda").bfloat16()
    block = Block(random_projection((heads + 2 * kv_heads) * dim, hidden, gen),
                  random_projection(hidden, heads * dim, gen), ones, 0.5 * ones, ones, freq,
                  magnitude, heads, kv_heads, dim, pages=256)
    serve(block, hidden, 8000, 32, 6, gen)
    status = tl.tern_device_status()  # (reading it clears it)
    if status:
        raise RuntimeError(tl.tern_status_string(status))


if __name__ == "__main__":
    main()
