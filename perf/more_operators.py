"""What is measured of the operators that an attention block needs around its
projections, its norm and its cache.

Four operators:

  rope     rotary positions of queries or keys: half and interleaved pairs,
           all of the head or its first part, frequencies scaled for contexts
           longer than the trained ones
  append   new keys and values into the paged int8 cache, the keys rotated on
           the way, and the same rows' queries rotated into 16 bits
  norms    the norm after a block, its gate and the residual's scale, the
           residual's addition, and the norm before the next block with its
           int8 codes
  attn     attention of a batch whose sequences begin with the same pages of
           the cache, each with tokens of its own behind them

`run` computes them in plain torch operations (fp32, angles in 64 bits) or,
where `own` is set, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 64  # tokens of a cache page, which is the block that shares a scale


def listed():
    return [
        # the queries of one decode step of a full batch: latency
        dict(name="rope_step", op="rope", tokens=32, heads=48, dim=128, rotary=128,
             interleaved=False, x="float32", out="bfloat16", far=40000, base=1e6, scaling="none",
             factor=1.0, trained=0),
        # a prompt chunk's queries and keys together, a quarter of the head
        # turned, at positions far past the trained context
        dict(name="rope_chunk", op="rope", tokens=2048, heads=56, dim=128, rotary=32,
             interleaved=True, x="bfloat16", out="bfloat16", far=900000, base=5e5,
             scaling="bands", factor=8.0, trained=8192),
        # a decode step of sixteen sequences writes one token each
        dict(name="append_step", op="append", seqs=16, new=1, ragged=False, min_len=70,
             max_len=4000, heads=48, kv_heads=8, dim=128, rotary=128, interleaved=False,
             x="float32", base=1e6, scaling="none", factor=1.0, trained=0),
        # prompt chunks of several sequences at once, ragged, not starting on a page
        dict(name="append_prompts", op="append", seqs=3, new=2048, ragged=True, min_len=2100,
             max_len=5000, heads=48, kv_heads=8, dim=128, rotary=128, interleaved=False,
             x="float32", base=1e4, scaling="ramp", factor=4.0, trained=4096),
        # small heads of which half is turned, 16-bit projections
        dict(name="append_small_heads", op="append", seqs=5, new=700, ragged=True, min_len=701,
             max_len=3001, heads=16, kv_heads=16, dim=64, rotary=32, interleaved=True,
             x="bfloat16", base=1e4, scaling="linear", factor=2.0, trained=0),
        # one token of a decode step through the model's width: latency
        dict(name="norms_token", op="norms", tokens=1, width=5120, x="float32", gate="none",
             y=True),
        # a prompt chunk, with a gate for each channel
        dict(name="norms_prompt", op="norms", tokens=2048, width=5120, x="float32",
             gate="channel", y=False),
        # a short shared prompt and a small batch: latency
        dict(name="attn_small", op="attn", shared=2048, seqs=6, new=1, min_own=3, max_own=300,
             heads=48, kv_heads=8, dim=128, window=0, sinks=0),
        # a decode step of a full batch behind a long common prompt
        dict(name="attn_batch", op="attn", shared=16384, seqs=32, new=1, min_own=40, max_own=1500,
             heads=48, kv_heads=8, dim=128, window=0, sinks=0),
        # verify steps of four tokens behind a common document
        dict(name="attn_verify", op="attn", shared=32768, seqs=40, new=4, min_own=60,
             max_own=900, heads=40, kv_heads=8, dim=128, window=0, sinks=0),
        # small heads under a window that reaches into the prefix, with sink tokens
        dict(name="attn_window", op="attn", shared=6016, seqs=23, new=2, min_own=20, max_own=2500,
             heads=32, kv_heads=8, dim=64, window=3000, sinks=70),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rotation(rng, dim):
    scaling = rng.choice(["none", "linear", "base", "bands", "ramp"])
    return dict(rotary=16 * rng.randrange(1, dim // 16 + 1), interleaved=rng.random() < 0.5,
                base=rng.choice([1e4, 5e5, 1e6]), scaling=scaling,
                factor=1.0 if scaling == "none" else round(rng.uniform(1.5, 16), 2),
                trained=2048 * _log(rng, 1, 16))


def draw(rng):
    op = rng.choice(["rope", "append", "norms", "attn", "attn"])
    if op == "norms":
        return dict(op=op, tokens=_log(rng, 1, 2048), width=16 * _log(rng, 16, 320),
                    x=rng.choice(["float32", "bfloat16"]),
                    gate=rng.choice(["none", "channel", "token"]), y=rng.random() < 0.5)
    if op == "rope":
        dim = rng.choice([64, 96, 128])
        return dict(op=op, tokens=_log(rng, 1, 1024), heads=_log(rng, 1, 56), dim=dim,
                    x=rng.choice(["float32", "bfloat16", "float16"]),
                    out=rng.choice(["float32", "bfloat16", "float16"]), far=_log(rng, 10, 10 ** 6),
                    **_draw_rotation(rng, dim))
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 4, 5, 6])
    if op == "append":
        new = _log(rng, 1, 2048)
        low = new + rng.randrange(0, 200)
        return dict(op=op, seqs=_log(rng, 1, 3 if new > 64 else 40), new=new,
                    ragged=rng.random() < 0.5, min_len=low, max_len=low + _log(rng, 1, 3000),
                    heads=kv * group, kv_heads=kv, dim=dim,
                    x=rng.choice(["float32", "bfloat16", "float16"]), **_draw_rotation(rng, dim))
    window = _log(rng, 100, 8000) if rng.random() < 0.3 else 0
    new = 1 if rng.random() < 0.6 else rng.randrange(2, 5)
    least = new + rng.randrange(0, 30)
    return dict(op=op, shared=64 * _log(rng, 4, 400), seqs=_log(rng, 2, 32), new=new,
                min_own=least, max_own=least + _log(rng, 1, 1500),
                heads=kv * group, kv_heads=kv, dim=dim, window=window,
                sinks=rng.choice([0, 4, 100]) if window else 0)


# ------------------------------------------------------------------ lengths


def _lengths(case):
    """Tokens of each sequence, the new ones among them, and how many are new:
    spread by the fractions of multiples of two irrational numbers."""
    b = np.arange(case["seqs"])
    f = np.mod(b * 0.6180339887498949, 1.0)
    if case["op"] == "attn":
        lens = np.rint(case["max_own"] - (case["max_own"] - case["min_own"]) * f).astype(np.int64)
        new = np.full(case["seqs"], case["new"], dtype=np.int64)
        return case["shared"] + np.maximum(lens, new), new
    lens = np.rint(case["max_len"] - (case["max_len"] - case["min_len"]) * f).astype(np.int64)
    new = np.full(case["seqs"], case["new"], dtype=np.int64)
    if case["ragged"]:
        new = 1 + np.floor((case["new"] - 1) * (1 - np.mod(b * 0.7548776662466927, 1.0))).astype(
            np.int64)
    return lens, np.minimum(new, lens)


def _size(name):
    return 4 if name == "float32" else 2


def work(case):
    op = case["op"]
    if op == "norms":
        n = case["tokens"] * case["width"]
        per = _size(case["x"]) + 2 + 2 + 1 + (2 if case["y"] else 0)
        per += 2 if case["gate"] == "token" else 0
        rows = 2 + (case["gate"] == "channel")
        return {"bytes": n * per + 2 * rows * case["width"] + 4 * case["tokens"], "flops": 12 * n}
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        turned = case["tokens"] * case["heads"] * case["rotary"]
        return {"bytes": n * (_size(case["x"]) + _size(case["out"])) + 4 * case["tokens"]
                + 4 * case["rotary"], "flops": 3 * turned}
    h, d = case["kv_heads"], case["dim"]
    lens, new = _lengths(case)
    n = int(new.sum())
    if op == "append":
        pages = int(np.sum((lens + BLOCK - 1) // BLOCK - (lens - new) // BLOCK))
        return {"bytes": n * 2 * h * d * (_size(case["x"]) + 1) + pages * 2 * h * 8
                + n * case["heads"] * d * (_size(case["x"]) + 2),
                "flops": n * (2 * h * d * 3 + 3 * (h + case["heads"]) * case["rotary"])}
    w, s, shared = case["window"], case["sinks"], case["shared"]
    pairs = tokens = 0
    deep = shared  # the first token of the prefix, past the sinks, that a row sees
    for length, m in zip(lens.tolist(), new.tolist()):
        p = np.arange(length - m, length)
        low = np.maximum(0, p - w + 1) if w else np.zeros_like(p)
        pairs += int(np.sum(p - low + 1 + np.minimum(low, s)))
        tokens += length - max(shared, int(low[0]))
        deep = min(deep, int(low[0]))
    tokens += shared - deep + min(deep, s)
    return {"bytes": tokens * 2 * h * (d + 4 / BLOCK) + n * case["heads"] * d * 4,
            "flops": 4 * pairs * case["heads"] * d}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _table(st, case):
    """What a program that rotates holds: the framework's table of frequencies."""
    if own:
        import ternary_weight_linear_gb300 as tl
        st["freq"], st["magnitude"] = tl.tern_rope_frequencies(
            case["rotary"], base=case["base"], scaling=case["scaling"], factor=case["factor"],
            trained=case["trained"])


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "norms":
        t, k = case["tokens"], case["width"]
        # a projection's output, the residual stream with a few outlier
        # channels, norm weights near one, gates of a trained block
        out = (torch.rand(k, generator=g, device=DEV) < 0.01).float() * 19 + 1
        st["x"] = (_rand(g, t, k) * 3).to(getattr(torch, case["x"]))
        st["residual"] = (_rand(g, t, k) * out).bfloat16()
        st["post"] = (1 + 0.2 * _rand(g, k)).bfloat16()
        st["weight"] = (1 + 0.2 * _rand(g, k)).bfloat16()
        st["gate"] = None
        if case["gate"] != "none":
            shape = (k,) if case["gate"] == "channel" else (t, k)
            st["gate"] = (0.5 + 0.2 * _rand(g, *shape)).bfloat16()
        st["values"] = torch.empty(t, k, dtype=torch.bfloat16, device=DEV)
        return st
    if case["op"] == "rope":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        _table(st, case)
        x = _rand(g, t, h, d).to(getattr(torch, case["x"]))
        st["x"] = x
        # a chunk of consecutive positions, or the steps of several sequences
        if t > 64:
            first = int(torch.randint(0, case["far"], (1,), generator=g, device=DEV))
            st["pos"] = torch.arange(first, first + t, dtype=torch.int32, device=DEV)
        else:
            st["pos"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV,
                                      dtype=torch.int32)
        st["out"] = torch.empty(t, h, d, dtype=getattr(torch, case["out"]), device=DEV)
        return st
    h, d = case["kv_heads"], case["dim"]
    lens, new = _lengths(case)
    seqs, total = case["seqs"], int(new.sum())
    each = (lens + BLOCK - 1) // BLOCK
    width = max(1, int(each.max()))
    common = case["shared"] // BLOCK if case["op"] == "attn" else 0
    # pages handed out in a shuffled order, as after some time of serving
    pages = int((each - common).sum()) + common + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(seqs, width, dtype=torch.int32, device=DEV)
    table[:, :common] = order[:common]
    at = common
    for b, e in enumerate(each.tolist()):
        table[b, common:e] = order[at:at + e - common]
        at += e - common
    codes = torch.empty(pages, 2, h, BLOCK, d, dtype=torch.int8, device=DEV)
    for p in range(0, pages, 256):
        part = codes[p:p + 256]
        part.copy_((_rand(g, *part.shape) * 36).round_().clamp_(-127, 127))
    st["codes"] = codes
    st["scales"] = (0.02 + 0.02 * torch.rand(pages, 2, h, generator=g, device=DEV))
    st["table"] = table
    st["lens"] = torch.from_numpy(lens).to(device=DEV, dtype=torch.int32)
    st["start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).to(
        device=DEV, dtype=torch.int32)
    st["max_new"] = int(new.max())
    # which (sequence, new token) each row is, for the plain forms
    rows = np.repeat(np.arange(seqs), new)
    first = np.concatenate([[0], np.cumsum(new)])[rows]
    st["row_seq"] = torch.from_numpy(rows).to(DEV)
    st["row_pos"] = torch.from_numpy((lens - new)[rows] + np.arange(total) - first).to(DEV)
    if case["op"] == "append":
        _table(st, case)
        # queries, keys and values as one projection writes them
        y = _rand(g, total, case["heads"] + 2 * h, d).to(getattr(torch, case["x"]))
        st["q"], st["k"], st["v"] = y.split((case["heads"], h, h), dim=1)
        st["q_out"] = torch.empty(total, case["heads"], d, dtype=torch.bfloat16, device=DEV)
        # the pages that hold new tokens, and whether they hold older ones
        touched, older = [], []
        for b, (n, m) in enumerate(zip(lens.tolist(), new.tolist())):
            for j in range((n - m) // BLOCK, (n + BLOCK - 1) // BLOCK if m else 0):
                touched.append((b, j))
                older.append(j * BLOCK < n - m)
        at = torch.tensor(touched, device=DEV).long()
        st["touched"] = table[at[:, 0], at[:, 1]].long()
        st["older"] = torch.tensor(older, device=DEV)
        st["values"] = torch.empty(len(at), 2, h, BLOCK, d, dtype=torch.bfloat16, device=DEV)
        place = {p: i for i, p in enumerate(touched)}
        pos = st["row_pos"].tolist()
        slots = [place[(b, p // BLOCK)] for b, p in zip(rows.tolist(), pos)]
        st["row_touched"] = torch.tensor(slots, device=DEV)
        st["row_slot"] = st["row_pos"] % BLOCK
        # older tokens of the touched pages lie before the first new one
        head = [max(0, min(BLOCK, int(lens[b] - new[b]) - j * BLOCK)) for b, j in touched]
        st["old_tokens"] = (torch.arange(BLOCK, device=DEV)[None]
                            < torch.tensor(head, device=DEV)[:, None])
    else:
        st["q"] = (_rand(g, total, case["heads"], d) * 0.8).bfloat16()
        st["workspace"] = {}
    return st


# ------------------------------------------------------------------ plain forms


def _frequencies(case):
    """(radians a token of each pair in 64 bits, the factor of turned elements)."""
    rot, base, factor, trained = case["rotary"], case["base"], case["factor"], case["trained"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    if case["scaling"] == "base":
        base = base * factor ** (rot / (rot - 2))
    theta = base ** (-2 * i / rot)
    if case["scaling"] == "linear":
        return theta / factor, 1.0
    if case["scaling"] == "bands":
        # pairs that turn 4 times and more in the trained context stay, those
        # that turn once or less are slowed by the factor
        keep = ((trained * theta / (2 * math.pi) - 1) / 3).clamp(0, 1)
        return theta * (keep + (1 - keep) / factor), 1.0
    if case["scaling"] == "ramp":
        # the same between the pairs that turn 32 times and once, straight in
        # the pair's number
        def pair(turns):
            return rot * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot - 1)
        slow = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return theta * (1 - slow + slow / factor), 0.1 * math.log(factor) + 1
    return theta, 1.0


def _turned(case, x, pos):
    """fp32 rows x [rows, heads, dim] with the pairs of their first part turned."""
    rot = case["rotary"]
    theta, magnitude = _frequencies(case)
    angle = pos.double()[:, None] * theta
    c = (angle.cos() * magnitude).float()[:, None]
    s = (angle.sin() * magnitude).float()[:, None]
    part = x[..., :rot]
    if case["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rope(st):
    return _turned(st["case"], st["x"].float(), st["pos"]).to(st["out"].dtype)


def _touched_values(st):
    """The pages with new tokens as the values that their codes stand for (in 16
    bits: the codes have eight)."""
    at = st["touched"]
    return torch.mul(st["codes"][at], st["scales"][at][..., None, None], out=st["values"])


def _plain_append(st):
    case = st["case"]
    at, h = st["touched"], case["kv_heads"]
    k = _turned(case, st["k"].float(), st["row_pos"])
    x = torch.stack((k, st["v"].float()), 1)  # [rows, 2, heads, dim]
    big = torch.zeros(len(at), 2, h, device=DEV)
    big.index_reduce_(0, st["row_touched"], x.abs().amax(-1), "amax")
    was = torch.where(st["older"][:, None, None], st["scales"][at], 0)
    # (a tensor: torch multiplies by the rounded reciprocal of a plain number)
    now = torch.maximum(was, big / torch.full((1,), 127.0, device=DEV))
    part = st["codes"][at]
    shrunk = (part.float() * (was / now)[..., None, None]).round().to(torch.int8)
    grew = (now > was)[..., None, None] & st["old_tokens"][:, None, None, :, None]
    part = torch.where(grew, shrunk, part)
    q = (x / now[st["row_touched"]][..., None]).round().clamp(-127, 127).to(torch.int8)
    part[st["row_touched"], :, :, st["row_slot"]] = q
    st["codes"][at] = part
    st["scales"][at] = now
    return {"q": _turned(case, st["q"].float(), st["row_pos"]).bfloat16(),
            "values": _touched_values(st), "scales": st["scales"]}


def _plain_norms(st):
    case = st["case"]
    x = st["x"].float()
    n = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * st["post"].float()
    if st["gate"] is not None:
        n = n * st["gate"].float()
    r = (0.9 * st["residual"].float() + 1.25 * n).bfloat16()
    f = r.float()
    y = f * torch.rsqrt(f.square().mean(1, keepdim=True) + 1e-6) * st["weight"].float()
    scale = y.abs().amax(1) / torch.full((1,), 127.0, device=DEV)
    q = (y / scale[:, None]).round().clamp(-127, 127)
    got = {"residual": r, "x_scale": scale, "values": (q * scale[:, None]).bfloat16()}
    if case["y"]:
        got["y"] = y.bfloat16()
    return got


def _seen(case, pos, key):
    seen = key <= pos[..., None]
    if case["window"]:
        seen &= (key > pos[..., None] - case["window"]) | (key < case["sinks"])
    return seen


def _plain_attn(st):
    """The prefix's scores for all rows in one product, the own tokens' for each
    sequence, and one softmax over both."""
    case = st["case"]
    seqs, h, d, t = case["seqs"], case["kv_heads"], case["dim"], case["new"]
    group, shared = case["heads"] // h, case["shared"]
    common = shared // BLOCK

    first = st["table"][0, :common].long()
    kv = st["codes"][first].float() * st["scales"][first][..., None, None]
    k0, v0 = kv.permute(1, 2, 0, 3, 4).reshape(2, h, shared, d)
    rest = st["table"][:, common:].long()
    n = rest.shape[1] * BLOCK
    kv = st["codes"][rest].float() * st["scales"][rest][..., None, None]
    k1, v1 = kv.permute(2, 3, 0, 1, 4, 5).reshape(2, h, seqs, n, d)
    q = st["q"].float().view(seqs, t, h, group, d).permute(2, 0, 1, 3, 4)  # [h, seqs, t, group, d]
    s0 = (q.reshape(h, seqs * t * group, d) @ k0.transpose(1, 2)).view(h, seqs, t, group, shared)
    s1 = (q.reshape(h, seqs, t * group, d) @ k1.transpose(2, 3)).view(h, seqs, t, group, n)
    s = torch.cat((s0, s1), -1) / math.sqrt(d)
    pos = st["row_pos"].view(seqs, t)
    s = s.masked_fill(~_seen(case, pos, torch.arange(shared + n, device=DEV))[None, :, :, None],
                      -torch.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = (p[..., :shared].reshape(h, seqs * t * group, shared) @ v0).view(h, seqs, t, group, d)
    o = o + (p[..., shared:].reshape(h, seqs, t * group, n) @ v1).view(h, seqs, t, group, d)
    o = o / p.sum(-1, keepdim=True)
    return o.permute(1, 2, 0, 3, 4).reshape(seqs * t, case["heads"], d).bfloat16()


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"norms": _plain_norms, "rope": _plain_rope, "append": _plain_append,
                "attn": _plain_attn}[op](st)
    import ternary_weight_linear_gb300 as tl
    if op == "rope":
        return tl.tern_rope(st["x"], st["pos"], st["freq"], interleaved=case["interleaved"],
                            magnitude=st["magnitude"], out=st["out"])
    if op == "norms":
        t, k = st["x"].shape
        y = torch.empty(t, k, dtype=torch.bfloat16, device=DEV) if case["y"] else None
        q, scale, r = tl.tern_norm_add_norm_s8(
            st["x"], st["post"], st["residual"], st["weight"], gate=st["gate"],
            residual_scale=0.9, branch_scale=1.25, eps=1e-6, y=y)
        # the codes as the values that they stand for
        got = {"residual": r, "x_scale": scale,
               "values": torch.mul(q, scale[:, None], out=st["values"])}
        if case["y"]:
            got["y"] = y
        return got
    if op == "append":
        q = tl.tern_kv8_append_rope(
            st["q"], st["k"], st["v"], st["codes"], st["scales"], st["table"], st["start"],
            st["lens"], st["freq"], interleaved=case["interleaved"], magnitude=st["magnitude"],
            max_new=st["max_new"], q_out=st["q_out"])
        return {"q": q, "values": _touched_values(st), "scales": st["scales"]}
    if not st["workspace"]:
        st["workspace"]["at"] = torch.zeros(
            tl.tern_kv8_attention_shared_workspace_bytes(
                case["seqs"], st["q"].shape[0], case["heads"], case["kv_heads"], case["dim"]),
            dtype=torch.uint8, device=DEV)
    return tl.tern_kv8_attention_shared(
        st["q"], st["codes"], st["scales"], st["table"], st["start"], st["lens"], case["shared"],
        max_new=st["max_new"], window=case["window"], sinks=case["sinks"],
        workspace=st["workspace"]["at"])


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    st = prepare(case, seed)

    def rotate(x, pos):
        # pair by pair
        rot = case["rotary"]
        out = x.double().clone()
        base, factor, trained = case["base"], case["factor"], case["trained"]
        grow = 0.1 * math.log(factor) + 1 if case["scaling"] == "ramp" else 1.0
        for i in range(rot // 2):
            b = base * factor ** (rot / (rot - 2.0)) if case["scaling"] == "base" else base
            f = math.exp(-2.0 * i / rot * math.log(b))
            if case["scaling"] == "linear":
                f /= factor
            elif case["scaling"] == "bands":
                turns = trained * f / (2 * math.pi)
                share = min(1.0, max(0.0, (turns - 1.0) / (4.0 - 1.0)))
                f = share * f + (1 - share) * f / factor
            elif case["scaling"] == "ramp":
                at = [rot * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))
                      for n in (32, 1)]
                lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
                share = min(1.0, max(0.0, (i - lo) / max(0.001, hi - lo)))
                f = (1 - share) * f + share * f / factor
            c = torch.cos(pos.double() * f)[:, None] * grow
            s = torch.sin(pos.double() * f)[:, None] * grow
            m, n = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
            u, v = x[..., m].double(), x[..., n].double()
            out[..., m] = u * c - v * s
            out[..., n] = u * s + v * c
        return out

    def rope():
        return rotate(st["x"], st["pos"])

    def norms():
        x, w = st["x"].double(), st["post"].double()
        n = x * w / (torch.einsum("tk,tk->t", x, x) / x.shape[1] + 1e-6).sqrt()[:, None]
        if st["gate"] is not None:
            n = n * st["gate"].double()
        # (the stored residual is what the second norm takes)
        r = (0.9 * st["residual"].double() + 1.25 * n)
        f = r.bfloat16().double()
        power = torch.einsum("tk,tk->t", f, f) / f.shape[1]
        y = (f * st["weight"].double()) / (power + 1e-6).sqrt()[:, None]
        scale = y.abs().max(dim=1).values / 127
        got = {"residual": r, "x_scale": scale,
               "values": torch.round(y / scale[:, None]) * scale[:, None]}
        if case["y"]:
            got["y"] = y
        return got

    def append():
        # sequence by sequence, page by page
        k_all, q_all = rotate(st["k"], st["row_pos"]), rotate(st["q"], st["row_pos"])
        lens, start = st["lens"].tolist(), st["start"].tolist()
        scales = st["scales"].double().clone()
        values = []
        for b, n in enumerate(lens):
            m = start[b + 1] - start[b]
            done = n - m
            while done < n:
                j, off = divmod(done, BLOCK)
                take = min(BLOCK - off, n - done)
                page = int(st["table"][b, j])
                row = start[b] + done - (n - m)
                x = torch.stack((k_all[row:row + take], st["v"][row:row + take].double()))
                x = x.transpose(1, 2)  # [2, heads, take, dim]
                s = x.abs().amax((2, 3)) / 127
                c = st["codes"][page].double()
                if off:
                    # the stored scales are fp32: the growth is judged on them
                    was = st["scales"][page]
                    s32 = torch.maximum(was, s.float())
                    keep = (s32 == was)[..., None, None]
                    s = torch.where(s32 == was, was.double(), s)
                    old = c[:, :, :off]
                    c[:, :, :off] = torch.where(
                        keep, old, torch.round(old * (was.double() / s)[..., None, None]))
                c[:, :, off:off + take] = torch.round(x / s[..., None, None])
                scales[page] = s
                values.append(c * s[..., None, None])
                done += take
        return {"q": q_all, "values": torch.stack(values), "scales": scales}

    def attn():
        h, d = case["kv_heads"], case["dim"]
        group = case["heads"] // h
        w, sinks = case["window"], case["sinks"]
        lens, start = st["lens"].tolist(), st["start"].tolist()
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(lens):
            m = start[b + 1] - start[b]
            used = st["table"][b, :(n + BLOCK - 1) // BLOCK].long()
            pos = torch.arange(n - m, n, device=DEV)[:, None]
            key = torch.arange(n, device=DEV)[None]
            seen = key <= pos
            if w:
                seen = seen & ((pos - key < w) | (key < sinks))
            for kh in range(h):
                kv = (st["codes"][used, :, kh].double()
                      * st["scales"][used, :, kh].double()[..., None, None])
                k = kv[:, 0].reshape(-1, d)[:n]
                v = kv[:, 1].reshape(-1, d)[:n]
                x = st["q"][start[b]:start[b + 1], kh * group:(kh + 1) * group].double()
                s = torch.einsum("tgd,jd->tgj", x, k) / math.sqrt(d)
                p = torch.softmax(torch.where(seen[:, None], s, -math.inf), dim=2)
                out[start[b]:start[b + 1], kh * group:(kh + 1) * group] = p @ v
        return out

    return {"rope": rope, "append": append, "norms": norms, "attn": attn}[case["op"]]()
