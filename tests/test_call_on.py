"""Calls on a given stream, without a GPU: which stream's memory results come from and what the allocator is told,
on stand-ins for streams and tensors."""
import contextlib

import pytest
import torch

from combine_moe_get_amd import binding as B
from combine_moe_get_amd import experts


class Stream:
    def __init__(self, name):
        self.name, self.device = name, torch.device("cuda:0")


class Tensor(torch.Tensor):
    @staticmethod
    def make(log, name):
        t = torch.zeros(1).as_subclass(Tensor)
        t.record_stream = lambda s: log.append((name, s.name))
        return t


@pytest.fixture
def world(monkeypatch):
    now = [Stream("main")]

    @contextlib.contextmanager
    def use(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", use)
    return now


def _prepare(now, log, made):
    def prepare(x):
        made.append(now[-1].name)
        out = Tensor.make(log, "out")

        def call(stream=None):
            log.append(("ran", (stream or now[-1]).name))
            return (out, None)

        call._keep = ("shape", x, None, (x, 3))
        return call

    return prepare


def test_another_stream(world):
    log, made = [], []
    x = Tensor.make(log, "x")
    B.call_on(Stream("side"), _prepare(world, log, made), x)
    assert made == ["side"]
    assert log == [("ran", "side"), ("x", "side"), ("x", "side"), ("out", "side"), ("out", "main")]


@pytest.mark.parametrize("given", [False, True])
def test_the_current_stream(world, given):
    log, made = [], []
    B.call_on(world[0] if given else None, _prepare(world, log, made), Tensor.make(log, "x"))
    assert made == ["main"] and log == [("ran", "main")]


NAMES = ["experts_matmul", "experts_matmul_dgrad", "experts_matmul_wgrad", "quantize_rows", "combine_grad"]


@pytest.mark.parametrize("name", NAMES)
def test_the_functions_go_this_way(name, monkeypatch):
    seen = []
    monkeypatch.setattr(B, "call_on", lambda stream, prepare, *args: seen.append((stream, prepare)))
    f = getattr(experts, name)
    f(*[None] * (2 if name == "quantize_rows" else 6 if name == "combine_grad" else 4), stream="s")
    assert seen == [("s", getattr(experts, "prepare_" + name))]


@pytest.mark.parametrize("name,required", [("layout", 2), ("layout_noalloc", 2), ("dispatch", 4), ("combine", 5),
                                           ("layout_dispatch", 4)])
def test_the_layers_functions_go_this_way(name, required, monkeypatch):
    seen = []
    monkeypatch.setattr(B, "call_on", lambda stream, prepare, *args: seen.append((stream, prepare)))
    getattr(B, name)(*[None] * required, stream="s")
    assert seen == [("s", getattr(B, "prepare_" + name))]
