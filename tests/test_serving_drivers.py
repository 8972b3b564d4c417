"""Host logic of the serving drivers (no GPU needed): the library calls are replaced by
recorders, the rest runs on CPU tensors."""
import contextlib

import pytest
import torch


@pytest.fixture(scope="module")
def mods():
    from long_context_compressed_compress_b200 import build
    build.build()
    from long_context_compressed_compress_b200 import layer, ops, paged
    return layer, ops, paged


def cache(paged, R=4, N=12, P=4, D=64, max_entries=24):
    return paged.PagedEntries(1, N, P, D, R, max_entries, dtype=torch.float32, device="cpu")


@pytest.mark.parametrize("stream", ["side", None])
def test_host_lists_are_made_on_the_stream_of_their_call(mods, monkeypatch, stream):
    """A list's device copy is released when the call returns: it has to belong to the
    stream whose kernels read it."""
    _, ops, paged = mods
    c = cache(paged)
    now, seen = [], []

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()
    monkeypatch.setattr(torch.cuda, "stream", on)
    for name in ("reserve", "fork", "free"):
        monkeypatch.setattr(ops, "kv_pages_" + name, lambda *a: None)
    make = torch.tensor
    monkeypatch.setattr(torch, "tensor", lambda *a, **k: (seen.append(now[-1] if now else "none"), make(*a, **k))[1])
    c.reserve([0, 1], [3, 4], stream=stream)
    c.fork([0], [2], [3], stream=stream)
    c.free([0, 1], stream=stream)
    assert seen == [stream] * 6
