"""The example's attention block, link by link against the oracle: prompt
chunks, decode steps, a sequence that ends and one that takes its pages.

Each call's inputs are what the call before it gave, so each link has its own
bar: exact for the codes of the cache, the other operators' own elsewhere.
"""
import importlib.util
import os

import numpy as np
import pytest

import oracle
import synth
from helpers import assert_s8_parity
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
        "attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _np(t):
    return t.float().cpu().numpy()


class Recorder:
    """The library with a note of each call's arguments and results."""

    def __init__(self, tl):
        self.tl, self.calls = tl, {}

    def __getattr__(self, name):
        f = getattr(self.tl, name)
        if not name.startswith("tern_") or name.endswith("_bytes"):
            return f

        def call(*args, **kw):
            self.calls[name] = (args, kw, f(*args, **kw))
            return self.calls[name][2]
        return call


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_block_steps(example, monkeypatch, window, sinks):
    import torch
    tl = example.tl
    hidden, heads, kv, dim = 256, 4, 2, 64
    rec = Recorder(tl)
    monkeypatch.setattr(example, "tl", rec)
    cq = synth.case("tiny", 1, K=hidden, N=(heads + 2 * kv) * dim, seed=1)
    co = synth.case("tiny", 1, K=heads * dim, N=hidden, seed=2)

    def projection(c):
        return (tl.tern_pack(torch.from_numpy(c.W).cuda()),
                torch.from_numpy(c.scales.view(np.uint16)).view(torch.float16).cuda())

    rng = np.random.default_rng(3)
    norm = torch.from_numpy((1 + 0.2 * rng.standard_normal(hidden)).astype(np.float32))
    block = example.AttentionBlock(norm.cuda().bfloat16(), projection(cq), projection(co), heads,
                                   kv, dim, pages=9, window=window, sinks=sinks)
    pages = example.Pages(9, 3, 6)
    for new in [[70, 30, 0], [75, 1, 20], [1, 1, 1], "end 0", [1, 40, 1], [2, 2, 2]]:
        if new == "end 0":
            pages.release(0)
            continue
        start, lens = pages.grow(new)
        rows = sum(new)
        h = torch.from_numpy(rng.standard_normal((rows, hidden)).astype(np.float32)).cuda()
        res = torch.from_numpy(rng.standard_normal((rows, hidden)).astype(np.float32)).cuda()
        res = res.bfloat16()
        codes, scales = block.codes.cpu().numpy(), block.scales.cpu().numpy()
        rec.calls = {}
        out, r = block(h, res, pages.table, start, lens, max(new))
        torch.cuda.synchronize()
        assert tl.tern_device_status() == 0

        # norm: a code is within half a step of the exact quotient, but for
        # the relative 2^-17 that the norm's tests derive
        q, xs, r_got = rec.calls["tern_add_rmsnorm_s8"][2]
        bf16 = lambda a: torch.from_numpy(np.float32(a)).bfloat16().float().numpy()  # noqa: E731
        r_ref, _, _, ratio = od.add_rmsnorm(_np(h), _np(res), _np(block.norm), block.eps, bf16)
        assert r is r_got and np.array_equal(_np(r).astype(np.float64), r_ref)
        assert np.all(np.abs(_np(q) - ratio) <= 0.5 + 127 * 2.0 ** -17)

        # projection
        y = rec.calls["tern_linear_s8"][2]
        wp, _ = oracle.pack(cq.W)
        y_ref, m, _ = oracle.linear_s8(wp, cq.scales, q.cpu().numpy(), xs.cpu().numpy(), rows,
                                       hidden, cq.N)
        assert_s8_parity(y.cpu().numpy(), y_ref, m, f"{new}")

        # cache
        qkv = _np(y).reshape(rows, heads + 2 * kv, dim)
        table, st, ln = (t.cpu().numpy() for t in (pages.table, start, lens))
        codes, scales = od.kv8_append(codes, scales, table, st, ln, qkv[:, heads:heads + kv],
                                      qkv[:, heads + kv:])
        assert np.array_equal(block.codes.cpu().numpy(), codes)
        assert np.array_equal(block.scales.cpu().numpy(), scales)

        # attention, at its tests' bar
        o = rec.calls["tern_kv8_attention"][2]
        o_ref, _, absum = od.kv8_attention(bf16(qkv[:, :heads]).astype(np.float64), codes, scales,
                                           table, st, ln, window, sinks, dim ** -0.5)
        bound = 5 * 2.0 ** -11 * absum + 2.0 ** -9 * np.abs(o_ref) + 2.0 ** -25
        assert np.all(np.abs(_np(o) - o_ref) <= bound)

        # output projection: the small-T bar, the s8 rung's beyond 16 rows
        x = o.view(rows, heads * dim)
        wp, _ = oracle.pack(co.W)
        bits = x.view(torch.int16).cpu().numpy().view(np.uint16)
        got = out.cpu().numpy().astype(np.float64)
        if rows <= 16:
            ref, m = oracle.linear_f64(wp, co.scales, bits, rows, heads * dim, hidden)
            assert np.all(np.abs(got - ref) <= 1e-3 * m + 1e-6)
        else:
            qo, xo = oracle.quant_s8(bits, rows, heads * dim)
            ref, m, _ = oracle.linear_s8(wp, co.scales, qo, xo, rows, heads * dim, hidden)
            assert_s8_parity(out.cpu().numpy(), ref, m, f"{new}")


def test_pages_run_out(example):
    pages = example.Pages(2, 2, 4)
    pages.grow([64, 1])
    with pytest.raises(RuntimeError):
        pages.grow([1, 0])


def test_example_runs(example, capsys):
    example.main()
    assert len(capsys.readouterr().out.splitlines()) == 8
