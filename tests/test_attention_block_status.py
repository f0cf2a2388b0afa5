"""The example reports the device's error, and not that of a word it has
cleared: its library and device replaced, no GPU needed."""
import importlib.util
import os

import pytest

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")


class Device:
    """The library's status word: a read clears it."""
    word = -7

    def tern_device_status(self):
        was, self.word = self.word, 0
        return was

    def tern_status_string(self, status):
        return {0: "ok", -7: "index out of range"}[status]


def test_failure_message_is_the_errors(monkeypatch):
    import torch
    spec = importlib.util.spec_from_file_location(
        "attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)

    class Event:
        def __init__(self, **kw):
            pass

        record = synchronize = lambda self: None
        elapsed_time = lambda self, other: 0.0

    class Pages:
        table, lens = None, [1]
        __init__ = grow = lambda self, *a: (None, None)

    def on_cpu(f):
        return lambda *a, generator=None, device=None, **kw: f(*a, **kw)

    monkeypatch.setattr(example, "tl", Device())
    monkeypatch.setattr(Pages, "__init__", lambda self, *a: None)
    monkeypatch.setattr(example, "Pages", Pages)
    monkeypatch.setattr(example, "AttentionBlock", lambda *a, **kw: lambda h, r, *rest: (h, r))
    monkeypatch.setattr(example, "random_projection", lambda *a: None)
    monkeypatch.setattr(torch, "Generator", lambda device: torch.default_generator)
    monkeypatch.setattr(torch.cuda, "Event", Event)
    for name in ("ones", "randn"):
        monkeypatch.setattr(torch, name, on_cpu(getattr(torch, name)))
    with pytest.raises(RuntimeError, match="index out of range"):
        example.main()
