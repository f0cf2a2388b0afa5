"""The attention block's operators together: the example, link by link against the
oracle, and chains of their kernels, each of which starts while the one before it
ends and has to read what that one wrote."""
import importlib.util
import os

import numpy as np
import pytest

import oracle
import synth
from helpers import assert_s8_parity
from oracle import attention_block as ab
from oracle import decoder as od

pytestmark = pytest.mark.gpu

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")


@pytest.fixture(scope="module")
def example():
    import torch
    import ternary_weight_linear_gb300 as tl
    tl.build()
    tl.load()
    torch.cuda.init()
    spec = importlib.util.spec_from_file_location(
        "shared_prompt", os.path.join(ROOT, "examples", "shared_prompt.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _np(t):
    return t.double().cpu().numpy()


class Recorder:
    """The library, with each call checked against the oracle as it is made."""

    def __init__(self, tl, weights):
        self.tl, self.weights, self.seen = tl, weights, []

    def __getattr__(self, name):
        f = getattr(self.tl, name)
        check = getattr(self, "check_" + name[5:], None) if name != "check_" else None
        if check is None:
            return f

        def call(*args, **kw):
            import torch
            torch.cuda.synchronize()
            self.seen.append(name)
            return check(f, *args, **kw)
        return call

    def check_linear_s8(self, f, Wp, scales, q, xs, **kw):
        y = f(Wp, scales, q, xs, **kw)
        c, wp = self.weights
        ref, m, _ = oracle.linear_s8(wp, c.scales, q.cpu().numpy(), xs.cpu().numpy(), len(q), c.K,
                                     c.N)
        assert_s8_parity(_np(y), ref, m, "qkv")
        return y

    def check_kv8_append_rope(self, f, q, k, v, codes, scales, table, start, lens, freq, *,
                              magnitude, max_new):
        before = codes.cpu().numpy(), scales.cpu().numpy()
        out = f(q, k, v, codes, scales, table, start, lens, freq, magnitude=magnitude,
                max_new=max_new)
        ix = [t.cpu().numpy() for t in (table, start, lens)]
        pos = np.concatenate([np.arange(n - m, n) for n, m in zip(ix[2], np.diff(ix[1]))])
        turns = [t % 2 ** 64 for t in freq.cpu().tolist()]
        m = np.float64(np.float32(magnitude))
        want, size = ab.rope(_np(q), pos, turns, False, m)
        bound = 2.0 ** -21 * m * size
        assert np.all(np.abs(_np(out) - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound))
        # the cache of the keys as tern_rope turns them, bit for bit
        import torch
        k32 = self.tl.tern_rope(k, torch.from_numpy(pos.astype(np.int32)).cuda(), freq,
                                magnitude=magnitude)
        ref = od.kv8_append(*before, *ix, k32.cpu().numpy(), v.cpu().numpy())
        assert np.array_equal(codes.cpu().numpy(), ref[0])
        assert np.array_equal(scales.cpu().numpy(), ref[1])
        return out

    def check_kv8_attention_shared(self, f, q, codes, scales, table, start, lens, shared, **kw):
        o = f(q, codes, scales, table, start, lens, shared, **kw)
        ref, _, absum = od.kv8_attention(_np(q), *[t.cpu().numpy() for t in
                                                   (codes, scales, table, start, lens)], 0, 0,
                                         q.shape[2] ** -0.5)
        assert np.all(np.abs(_np(o) - ref)
                      <= 5 * 2.0 ** -11 * absum + 2.0 ** -9 * np.abs(ref) + 2.0 ** -16)
        return o

    def check_norm_add_norm_s8(self, f, x, post, residual, weight, gate=None):
        q, xs, r = f(x, post, residual, weight, gate=gate)
        opt = lambda t: None if t is None else _np(t)  # noqa: E731
        eps = float(np.float32(1e-6))
        want, mag = ab.norm_add_norm(_np(x), opt(post), opt(gate), 1.0, _np(residual), 1.0, eps)
        assert np.all(np.abs(_np(r) - want) <= 2.0 ** -17 * mag + 2.0 ** -8 * np.abs(want))
        _, scale, ratio = ab.norm(_np(r), _np(weight), eps)
        assert np.all(np.abs(_np(xs) - scale) <= 2.0 ** -18 * scale)
        assert np.all(np.abs(_np(q) - ratio) <= 0.5 + 127 * 2.0 ** -17)
        return q, xs, r


# whole pages shared, and a prompt that ends inside one
@pytest.mark.parametrize("prompt", [128, 200])
def test_the_examples_links(example, monkeypatch, prompt):
    import torch
    tl = example.tl
    hidden, heads, kv, dim, seqs = 256, 6, 2, 64, 5
    cq = synth.case("tiny", 1, K=hidden, N=(heads + 2 * kv) * dim, seed=1)
    co = synth.case("tiny", 1, K=heads * dim, N=hidden, seed=2)

    def projection(c):
        return (tl.tern_pack(torch.from_numpy(c.W).cuda()),
                torch.from_numpy(c.scales.view(np.uint16)).view(torch.float16).cuda())

    rec = Recorder(tl, (cq, oracle.pack(cq.W)[0]))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(prompt)
    vec = lambda a, b: (a + b * torch.randn(hidden, generator=gen, device="cuda")).bfloat16()  # noqa: E731
    freq, magnitude = tl.tern_rope_frequencies(dim, scaling="ramp", factor=4.0, trained=256)
    block = example.Block(projection(cq), projection(co), vec(1, 0.2), vec(0.5, 0.2), vec(1, 0.2),
                          freq, magnitude, heads, kv, dim, pages=16)
    monkeypatch.setattr(example, "tl", rec)
    got = example.serve(block, hidden, prompt, seqs, 3, gen)
    assert tl.tern_device_status() == 0
    assert got[0].shape == (seqs, hidden)
    calls = 1 + (prompt % 64 > 0) + 3
    assert rec.seen.count("tern_kv8_attention_shared") == calls


@pytest.mark.parametrize("prompt", [0, 40])
def test_the_example_without_a_whole_page_to_share(example, monkeypatch, prompt):
    import torch
    tl = example.tl
    hidden, heads, kv, dim, seqs = 256, 6, 2, 64, 5
    cq = synth.case("tiny", 1, K=hidden, N=(heads + 2 * kv) * dim, seed=1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    freq, magnitude = tl.tern_rope_frequencies(dim)
    ones = torch.ones(hidden, device="cuda").bfloat16()
    qkv = (tl.tern_pack(torch.from_numpy(cq.W).cuda()),
           torch.from_numpy(cq.scales.view(np.uint16)).view(torch.float16).cuda())
    block = example.Block(qkv, example.random_projection(hidden, heads * dim, gen), ones, ones, ones,
                          freq, magnitude, heads, kv, dim, pages=16)
    rec = Recorder(tl, (cq, oracle.pack(cq.W)[0]))
    monkeypatch.setattr(example, "tl", rec)
    got = example.serve(block, hidden, prompt, seqs, 3, gen)
    assert tl.tern_device_status() == 0
    assert got[0].shape == (seqs, hidden)
    assert rec.seen.count("tern_kv8_attention_shared") == (prompt > 0) + 3


def _same(step, count):
    """step(i) -> tensors: `count` of them back to back and one by one."""
    import torch
    chained = [[t.clone() for t in step(i)] for i in range(count)]
    torch.cuda.synchronize()
    for i in range(count):
        torch.cuda.synchronize()
        got = step(i)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, chained[i])), i


@pytest.mark.parametrize("seqs,m,shared", [(3, 1, 128), (9, 2, 64 * 40), (40, 1, 64 * 90),
                                           (21, 1, 64 * 90)])
def test_attention_reads_what_the_append_wrote(example, seqs, m, shared):
    """The same slots of the cache, written again at each step; queries straight
    from the append."""
    import torch
    tl = example.tl
    heads, kv, dim, count = 12, 2, 128, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(seqs)
    common = shared // 64
    pages = common + 2 * seqs
    codes = torch.randint(-127, 128, (pages, 2, kv, 64, dim), generator=g, device="cuda",
                          dtype=torch.int8)
    scales = torch.rand(pages, 2, kv, generator=g, device="cuda") * 0.02
    table = torch.cat((torch.arange(common, device="cuda").repeat(seqs, 1),
                       common + torch.arange(2 * seqs, device="cuda").view(seqs, 2)), 1).int()
    lens = torch.full((seqs,), shared + 64 + m, dtype=torch.int32, device="cuda")
    start = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * m
    ys = [torch.randn(seqs * m, heads + 2 * kv, dim, generator=g, device="cuda")
          for _ in range(count)]
    freq, _ = tl.tern_rope_frequencies(64)
    ws = torch.zeros(tl.tern_kv8_attention_shared_workspace_bytes(seqs, seqs * m, heads, kv, dim),
                     dtype=torch.uint8, device="cuda")

    def step(i):
        q, k, v = ys[i].split((heads, kv, kv), 1)
        q = tl.tern_kv8_append_rope(q, k, v, codes, scales, table, start, lens, freq, max_new=m)
        return [tl.tern_kv8_attention_shared(q, codes, scales, table, start, lens, shared,
                                             max_new=m, workspace=ws)]

    _same(step, count)
    assert tl.tern_device_status() == 0


# the prefix as spans, beside the spans, under a window, and a chunk among single tokens
@pytest.mark.parametrize("new,shared,window", [([1] * 3, 128, 0), ([1, 2, 1, 0, 3] * 8, 64 * 90, 0),
                                               ([2] * 21, 64 * 90, 64 * 70),
                                               ([20] + [1] * 20, 64 * 90, 0)])
@pytest.mark.parametrize("captured", [False, True])
def test_lengths_and_tables_that_the_device_advances(example, new, shared, window, captured):
    """What a serving loop does between steps, on the stream alone: lengths, rows,
    the table, the cache and the queries are written by kernels before each call, and
    every launch of the call has to see them.  Bit for bit the same call with the GPU
    idle between the calls."""
    import torch
    tl = example.tl
    seqs, heads, kv, dim, count, own = len(new), 12, 2, 128, 8, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(seqs)
    common = shared // 64
    codes0 = torch.randint(-127, 128, (common + own * seqs, 2, kv, 64, dim), generator=g,
                           device="cuda", dtype=torch.int8)
    scales0 = torch.rand(len(codes0), 2, kv, generator=g, device="cuda") * 0.02
    codes, scales = codes0.clone(), scales0.clone()
    rng = np.random.default_rng(seqs)
    tables, lens, starts = [], [], []
    for i in range(count):
        m = rng.permutation(new)
        starts.append(np.concatenate([[0], np.cumsum(m)]))
        lens.append(shared + m + rng.integers(0, 64 * own - 63, seqs))
        order = rng.permutation(len(codes0))
        tables.append(np.concatenate([np.tile(order[:common], (seqs, 1)),
                                      order[common:].reshape(seqs, own)], 1))
    dev = lambda a: torch.from_numpy(np.stack(a).astype(np.int32)).cuda()  # noqa: E731
    tables, lens, starts = dev(tables), dev(lens), dev(starts)
    table, length, start = (torch.zeros_like(t[0]) for t in (tables, lens, starts))
    rows = sum(new)
    ys = [torch.randn(rows, heads + 2 * kv, dim, generator=g, device="cuda") for _ in range(count)]
    freq, _ = tl.tern_rope_frequencies(64)
    ws = torch.zeros(tl.tern_kv8_attention_shared_workspace_bytes(seqs, rows, heads, kv, dim),
                     dtype=torch.uint8, device="cuda")
    turned = torch.empty(rows, heads, dim, device="cuda").bfloat16()

    def step(i, out):
        codes.copy_(codes0)
        scales.copy_(scales0)
        torch.add(tables[i], 0, out=table)
        torch.add(starts[i], 0, out=start)
        torch.add(lens[i], 0, out=length)
        q, k, v = ys[i].split((heads, kv, kv), 1)
        tl.tern_kv8_append_rope(q, k, v, codes, scales, table, start, length, freq,
                                max_new=max(new), q_out=turned)
        return tl.tern_kv8_attention_shared(turned, codes, scales, table, start, length, shared,
                                            max_new=max(new), window=window, sinks=3, out=out,
                                            workspace=ws)

    outs = [torch.zeros_like(turned) for _ in range(count)]
    if captured:
        step(0, outs[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(count):
                step(i, outs[i])
        for _ in range(3):
            graph.replay()
    else:
        for i in range(count):
            step(i, outs[i])
    torch.cuda.synchronize()
    for i in range(count):
        want = torch.zeros_like(turned)
        step(i, want)
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want) and (want != 0).any(2).all(), i
    assert not ws[:tl.SYNC_BYTES].any()
    assert tl.tern_device_status() == 0


@pytest.mark.parametrize("T", [1, 5, 40])
def test_norms_and_rotation_in_a_chain(example, T):
    """rotation -> norms -> layer, in buffers that each step writes again."""
    import torch
    tl = example.tl
    c = synth.case("tiny", T, K=1024, N=512, seed=T)
    Wp = tl.tern_pack(torch.from_numpy(c.W).cuda())
    s = torch.from_numpy(c.scales.view(np.uint16)).view(torch.float16).cuda()
    xs = [torch.randn(T, 16, 64, device="cuda") for _ in range(8)]
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    freq, _ = tl.tern_rope_frequencies(64, base=1e6)
    w = torch.ones(1024, device="cuda")
    turned = torch.empty(T, 16, 64, device="cuda")
    q = torch.empty(T, 1024, dtype=torch.int8, device="cuda")
    scale = torch.empty(T, device="cuda")
    residual = torch.empty(T, 1024, device="cuda").bfloat16()
    res0 = torch.randn(T, 1024, device="cuda").bfloat16()
    ws = torch.zeros(tl.tern_linear_workspace_bytes(T, 1024, 512), dtype=torch.uint8, device="cuda")

    def step(i):
        tl.tern_rope(xs[i], pos, freq, out=turned)
        tl.tern_norm_add_norm_s8(turned.view(T, 1024), w, res0, w, q=q, x_scale=scale,
                                 residual_out=residual)
        return [tl.tern_linear_s8(Wp, s, q, scale, workspace=ws), residual]

    _same(step, 8)
    assert tl.tern_device_status() == 0
