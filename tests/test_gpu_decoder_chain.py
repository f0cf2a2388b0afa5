"""Chains of the library's own kernels on one stream: each starts while the one
before it ends, and has to read what that one wrote.

Each step's result has to be, bit for bit, what the same calls give with the
GPU idle between them.
"""
import pytest

import synth
from helpers import to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tl():
    import torch
    import ternary_weight_linear_gb300 as tl
    tl.build()
    tl.load()
    torch.cuda.init()
    return tl


def _same(step, count):
    """step(i) -> a tensor: `count` of them back to back and one by one."""
    import torch
    chained = [step(i).clone() for i in range(count)]
    torch.cuda.synchronize()
    for i in range(count):
        torch.cuda.synchronize()
        got = step(i)
        torch.cuda.synchronize()
        assert torch.equal(got, chained[i]), i


@pytest.mark.parametrize("m", [1, 9, 70])  # few rows, the split form, prompt rows
def test_attention_reads_what_append_wrote(tl, m):
    """The same slots of the cache, written again at each step."""
    import torch
    seqs, heads, kv, dim, count = 3, 8, 2, 128, 12
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    codes = torch.zeros(12, 2, kv, 64, dim, dtype=torch.int8, device="cuda")
    scales = torch.zeros(12, 2, kv, device="cuda")
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(seqs, 4)
    lens = torch.full((seqs,), 128 + m, dtype=torch.int32, device="cuda")
    first = torch.randn(seqs * 128, kv, dim, generator=g, device="cuda")
    ix = [torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * n for n in (128, m)]
    tl.tern_kv8_append(first, first, codes, scales, table, ix[0],
                       torch.full_like(lens, 128), max_new=128)
    kvs = [torch.randn(2, seqs * m, kv, dim, generator=g, device="cuda") for _ in range(count)]
    q = torch.randn(seqs * m, heads, dim, generator=g, device="cuda").bfloat16()
    ws = torch.zeros(tl.tern_kv8_attention_workspace_bytes(seqs, seqs * m, heads, kv, dim),
                     dtype=torch.uint8, device="cuda")

    def step(i):
        tl.tern_kv8_append(kvs[i][0], kvs[i][1], codes, scales, table, ix[1], lens, max_new=m)
        return tl.tern_kv8_attention(q, codes, scales, table, ix[1], lens, max_new=m, workspace=ws)

    _same(step, count)
    assert tl.tern_device_status() == 0


@pytest.mark.parametrize("T", [1, 5, 16, 40])
def test_layer_reads_the_codes_that_the_norm_wrote(tl, T):
    import torch
    c = synth.case("tiny", T, K=2048, N=700, seed=T)
    W, s, _ = to_device(c)
    Wp = tl.tern_pack(W)
    xs = [torch.randn(T, 2048, device="cuda") for _ in range(12)]
    w = torch.ones(2048, device="cuda")
    q = torch.empty(T, 2048, dtype=torch.int8, device="cuda")
    scale = torch.empty(T, device="cuda")
    ws = torch.zeros(tl.tern_linear_workspace_bytes(T, 2048, 700), dtype=torch.uint8,
                     device="cuda")

    def step(i):
        tl.tern_add_rmsnorm_s8(xs[i], w, q=q, x_scale=scale)
        return tl.tern_linear_s8(Wp, s, q, scale, workspace=ws)

    _same(step, 12)
    assert tl.tern_device_status() == 0


# T of every token tile and rung; the switches that choose another reader of x
@pytest.mark.parametrize("T", [1, 4, 12, 40])
@pytest.mark.parametrize("env", [{}, {"TERN_DECODE_ACT": "int8", "TERN_PREFILL": "bf16"},
                                 {"TERN_ROTATE": "1"},
                                 {"TERN_ROTATE": "1", "TERN_PREFILL": "bf16"}])
def test_layer_reads_the_activations_that_the_norm_wrote(tl, monkeypatch, T, env):
    import torch
    c = synth.case("tiny", T, K=2048, N=700, seed=T)
    W, s, _ = to_device(c)
    Wp = tl.tern_pack(W)
    xs = [torch.randn(T, 2048, device="cuda") for _ in range(12)]
    w = torch.ones(2048, device="cuda")
    y = torch.empty(T, 2048, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(tl.tern_linear_workspace_bytes(T, 2048, 700), dtype=torch.uint8,
                     device="cuda")

    def step(i):
        tl.tern_add_rmsnorm_s8(xs[i], w, y=y, quantise=False)
        return tl.tern_linear(Wp, s, y, workspace=ws)

    for k, v in env.items():
        monkeypatch.setenv(k, v)
    tl.tern_reload_env()
    try:
        _same(step, 12)
    finally:
        for k in env:
            monkeypatch.delenv(k)
        tl.tern_reload_env()
    assert tl.tern_device_status() == 0
