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


def decode(mods, R=4, **kw):
    layer, _, paged = mods
    from long_context_compressed_compress_b200 import configs
    cfg = configs._hca(B=R, T=64, H=2, D=64, m=4, W=kw.pop("W", 6), dtype="f32", tau=0.1)
    d = layer.HcaDecode(cfg, cache(paged, R), device="cpu", groups=kw.pop("groups", None) or
                        paged.PrefixGroups.singles(R, device="cpu"), **kw)
    g = torch.Generator().manual_seed(3)
    d.pos.copy_(torch.randint(1, 60, d.pos.shape, generator=g))
    for t in (d.ring, d.carry):
        t.copy_(torch.randn(t.shape, generator=g))
    return d


@pytest.mark.parametrize("src,dst", [([0, 0], [1, 3]), ([2], [0]), ([], [])])
@pytest.mark.parametrize("made", [True, False])
def test_fork_copies_the_state_only_where_the_pages_were_forked(mods, monkeypatch, src, dst, made):
    _, ops, _ = mods
    d = decode(mods)
    calls = []

    def fork(s, t, n, *a):
        calls.append((s.tolist(), t.tolist(), n.tolist()))
        d.cache.ws[0] = len(t) if made else 0
    monkeypatch.setattr(ops, "kv_pages_fork", fork)
    before = [t.clone() for t in (d.pos, d.ring, d.carry)]
    d.cache.ws.fill_(0 if made else 7)
    d.fork(src, dst)
    assert calls == ([(src, dst, [int(before[0][i]) // 4 for i in src])] if dst else [])
    for t, b in zip((d.pos, d.ring, d.carry), before):
        want = b.clone()
        if made:
            want[dst] = b[src]
        assert torch.equal(t, want)


@pytest.mark.parametrize("src,dst", [([9], [1]), ([-1], [1]), ([0, 1], [2, 4]), ([0], [-3]), ([2 ** 31 - 1], [-2 ** 31])])
def test_fork_of_rows_out_of_range_reaches_the_cache(mods, monkeypatch, src, dst):
    """The cache refuses them (and records why); no indexing by them, which on a GPU
    would end the process."""
    _, ops, _ = mods
    d = decode(mods)
    calls = []
    monkeypatch.setattr(ops, "kv_pages_fork", lambda s, t, *a: (calls.append((s.tolist(), t.tolist())), d.cache.ws[:1].zero_()))
    before = [t.clone() for t in (d.pos, d.ring, d.carry)]
    d.fork(src, dst)
    assert calls == [(src, dst)]
    assert all(torch.equal(a, b) for a, b in zip((d.pos, d.ring, d.carry), before))


@pytest.mark.parametrize("nr", [False, True])
def test_a_step_tells_every_call_which_rows_are_idle(mods, monkeypatch, nr):
    layer, ops, paged = mods
    seen = {}

    def record(name):
        return lambda *a, **k: seen.update({name: (a, k)})
    for name in ("qk_norm_rope", "hca_paged_append", "hca_prefix_attn_fwd", "csa_ring_append", "csa_pos_advance"):
        monkeypatch.setattr(ops, name, record(name))
    groups = paged.PrefixGroups([([2, 0], 0)], 4, device="cpu")
    d = decode(mods, groups=groups, norm_rope=layer.NormRope() if nr else None)
    d.step({k: torch.zeros(4, 64) for k in ("a", "z", "kv_raw")} | {"q": torch.zeros(4, 2, 64)})
    live = groups.attended
    assert live.tolist() == [1, 0, 1, 0]
    assert seen["qk_norm_rope"][1]["lens"] is live and seen["hca_paged_append"][1]["lens"] is live
    assert seen["csa_pos_advance"][0][1] is live and "csa_ring_append" not in seen
    # every row attended: as before
    seen.clear()
    d.groups = paged.PrefixGroups.singles(4, device="cpu")
    d.step({k: torch.zeros(4, 64) for k in ("a", "z", "kv_raw")} | {"q": torch.zeros(4, 2, 64)})
    assert seen["hca_paged_append"][1]["lens"] is None and seen["csa_pos_advance"][0][1] == 1
    assert ("qk_norm_rope" if nr else "csa_ring_append") in seen


def test_advancing_by_rows_refusals(mods):
    _, ops, _ = mods
    f = 1 << 20
    assert ops.lib.csa_pos_advance_rows(None, 2, f, None) == 1 and ops.lib.csa_pos_advance_rows(f, 2, None, None) == 1
    assert ops.lib.csa_pos_advance_rows(f, -1, f, None) == 1 and ops.lib.csa_pos_advance_rows(f, 0, f, None) == 0
    with pytest.raises(ValueError):
        ops.csa_pos_advance(torch.zeros(2, dtype=torch.int32), torch.ones(2, dtype=torch.int32))


@pytest.mark.parametrize("nr", [False, True])
def test_without_a_window_there_is_no_ring_to_write(mods, monkeypatch, nr):
    layer, ops, _ = mods
    calls = []
    for name in ("qk_norm_rope", "hca_paged_append", "hca_prefix_attn_fwd", "csa_ring_append", "csa_pos_advance"):
        monkeypatch.setattr(ops, name, lambda *a, _n=name, **k: calls.append((_n, a)))
    d = decode(mods, W=0, norm_rope=layer.NormRope() if nr else None)
    d.load({k: torch.zeros(4, 5, 64) for k in ("a", "z", "kv_raw")})
    assert [c[0] for c in calls] == ["hca_paged_append"]
    calls.clear()
    d.step({k: torch.zeros(4, 64) for k in ("a", "z", "kv_raw")} | {"q": torch.zeros(4, 2, 64)})
    assert [c[0] for c in calls] == ["qk_norm_rope"] * nr + ["hca_paged_append", "hca_prefix_attn_fwd", "csa_pos_advance"]
    assert len(calls) == d.launches
    if nr:
        assert calls[0][1][1] is None and calls[0][1][3] is None


class _Lib:
    """Records calls of one entry point; nothing runs."""

    def __init__(self, monkeypatch, ops, name):
        self.calls = []
        monkeypatch.setattr(ops, "_home", lambda t: -1)
        monkeypatch.setattr(ops, "lib", type("L", (), {name: staticmethod(lambda *a: (self.calls.append(a), 0)[1])}))
        self.stream = type("S", (), {"cuda_stream": 0})


@pytest.mark.parametrize("H,kv,T,calls", [(0, 1, 3, 1), (2, 1, 3, 1), (0, 0, 3, 0), (0, 1, 0, 0), (2, 1, 0, 0)])
def test_a_key_beside_queries_of_no_heads_is_written(mods, monkeypatch, H, kv, T, calls):
    _, ops, _ = mods
    rec = _Lib(monkeypatch, ops, "qk_norm_rope")
    q, k = torch.zeros(2, T, H, 64), torch.zeros(2, T, 64) if kv else None
    ring = torch.zeros(2, 5, 64) if kv else None
    ops.qk_norm_rope(q, k, torch.zeros_like(q), ring, torch.zeros(2, dtype=torch.int32), stream=rec.stream)
    assert len(rec.calls) == calls
    if calls:
        a = rec.calls[0]
        assert a[9] == H and (a[0] is None) == (H == 0) and a[3] == k.data_ptr() and a[21] == ring.data_ptr()


@pytest.mark.parametrize("B,T,calls", [(0, 3, 0), (0, 0, 0), (2, 0, 1), (2, 3, 1)])
def test_append_of_an_empty_batch_is_no_call(mods, monkeypatch, B, T, calls):
    """No sequences: nothing to do (the library refuses null pointers); no tokens: the
    carry still goes on."""
    _, ops, _ = mods
    rec = _Lib(monkeypatch, ops, "hca_paged_append")
    a, i = torch.zeros(B, T, 64), torch.zeros(B, dtype=torch.int32)
    ops.hca_paged_append(a, a, i, torch.zeros(B, 2, 3, 64), torch.zeros(4, 2, 64), torch.zeros(B, 2, dtype=torch.int32), i, 4,
                         stream=rec.stream)
    assert len(rec.calls) == calls


def test_freed_rows_start_again(mods, monkeypatch):
    _, ops, _ = mods
    d = decode(mods)
    freed = []
    monkeypatch.setattr(ops, "kv_pages_free", lambda rows, *a: freed.append(rows.tolist()))
    before = d.pos.clone()
    d.free([2, 9, 0, 2])                      # (a cache takes lists of up to R rows)
    assert freed == [[2, 9, 0, 2]]
    before[[0, 2]] = 0
    assert torch.equal(d.pos, before)
    d.reset(torch.tensor([1, -1], dtype=torch.int32))
    assert d.pos.tolist()[1] == 0 and freed == [[2, 9, 0, 2]]
    d.free([])
    assert d.pos[3] == before[3]


def test_every_capture_holds_what_its_graph_reads(mods, monkeypatch):
    """Groups and inputs are the caller's to replace: a second capture must not release
    those of the first, whose graph may still be replayed."""
    import gc
    import weakref
    _, ops, paged = mods

    class Stream:
        def wait_stream(self, s):
            pass

    class Graph:
        pass
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(torch.cuda, "CUDAGraph", Graph)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "graph", lambda g, stream: contextlib.nullcontext())
    for name in ("qk_norm_rope", "hca_paged_append", "hca_prefix_attn_fwd", "csa_pos_advance"):
        monkeypatch.setattr(ops, name, lambda *a, **k: None)
    d = decode(mods)
    graphs, refs = [], []
    for b in range(2):
        d.groups = paged.PrefixGroups([([b], 0)], 4, device="cpu")
        x = {k: torch.zeros(4, 64) for k in ("a", "z", "kv_raw")} | {"q": torch.zeros(4, 2, 64)}
        graphs.append(d.capture(x))
        refs += [weakref.ref(d.groups), weakref.ref(x["q"])]
        del x
    d.groups = paged.PrefixGroups.singles(4, device="cpu")
    gc.collect()
    assert all(r() is not None for r in refs) and d.graph is graphs[1]
    del graphs[0]
    gc.collect()
    assert refs[0]() is None and refs[2]() is not None


@pytest.mark.parametrize("name", ["z", "kv_raw"])
def test_a_prompt_of_uneven_lengths_is_refused_untouched(mods, monkeypatch, name):
    """Positions advance by a's tokens: a window of more or fewer would be off."""
    _, ops, _ = mods
    calls = []
    for n in ("qk_norm_rope", "hca_paged_append"):
        monkeypatch.setattr(ops, n, lambda *a, **k: calls.append(a))
    d = decode(mods)
    before = d.pos.clone()
    x = {k: torch.zeros(4, 5, 64) for k in ("a", "z", "kv_raw")}
    x[name] = torch.zeros(4, 6, 64)
    with pytest.raises(ValueError):
        d.load(x)
    assert not calls and torch.equal(d.pos, before)


@pytest.mark.parametrize("B", [3, 5])
def test_groups_of_another_batch_are_refused_untouched(mods, monkeypatch, B):
    """Nothing of the step is done: a token pooled without its position would be pooled
    again by the next."""
    _, ops, paged = mods
    calls = []

    def attn(q, *a, **k):
        raise ValueError("groups must be those of the batch, on its device")
    monkeypatch.setattr(ops, "hca_prefix_attn_fwd", attn)
    for n in ("qk_norm_rope", "hca_paged_append", "csa_ring_append", "csa_pos_advance"):
        monkeypatch.setattr(ops, n, lambda *a, **k: calls.append(a))
    d = decode(mods)
    d.groups = paged.PrefixGroups.singles(B, device="cpu")
    with pytest.raises(ValueError):
        d.step({k: torch.zeros(4, 64) for k in ("a", "z", "kv_raw")} | {"q": torch.zeros(4, 2, 64)})
    assert not calls


@pytest.mark.parametrize("src,dst", [([0], []), ([], [1]), ([0, 1], [2])])
def test_fork_of_lists_of_unlike_lengths_is_refused(mods, monkeypatch, src, dst):
    _, ops, _ = mods
    monkeypatch.setattr(ops, "kv_pages_fork", lambda *a: pytest.fail("called"))
    d = decode(mods)
    before = d.pos.clone()
    with pytest.raises(ValueError):
        d.fork(src, dst)
    assert torch.equal(d.pos, before)
