"""The serving drivers where calls meet: side streams, refused calls, idle rows, layers
without a window, states that are taken up again."""
import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods(cuda_ok):
    from long_context_compressed_compress_b200 import build
    build.build()
    from long_context_compressed_compress_b200 import layer, ops, paged
    return layer, ops, paged


def np64(t):
    return t.detach().cpu().double().numpy()


def test_host_lists_on_a_busy_side_stream(mods):
    """The current stream takes and fills memory of the lists' size while the side stream
    has yet to read them."""
    _, _, paged = mods
    c = paged.PagedEntries(1, 64, 4, 8, 12, 60)
    m = serving.Pages(64, 4, 12, c.max_pages, c.pool.float().cpu().numpy())
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    keep = []
    for name, args in (("reserve", ([0, 3], [17, 8])), ("fork", ([0, 0, 3], [1, 2, 4], [17, 16, 5])), ("free", ([0, 2],)),
                       ("reserve", ([0, 1], [30, 40]))):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(20):                        # some milliseconds
                a = (a @ a).clamp(-1, 1)
        getattr(c, name)(*args, stream=s)
        getattr(m, name)(*args)
        keep += [torch.full((k,), 10 ** 9, dtype=torch.int32, device="cuda") for k in (1, 2, 3, 4) for _ in range(8)]
        torch.cuda.synchronize()
        assert c.status.item() == 0
        np.testing.assert_array_equal(c.held.cpu().numpy(), [len(r) for r in m.rows])
        np.testing.assert_array_equal(c.table.cpu().numpy(), m.table())
        np.testing.assert_array_equal(c.refcount.cpu().numpy(), m.ref)


def decode(mods, R=6, N=200, P=4, m=8, W=20, H=8, D=128, dt=torch.bfloat16, L=1, layer_at=0, cache=None, **kw):
    layer, _, paged = mods
    from long_context_compressed_compress_b200 import configs
    cfg = configs._hca(B=R, T=1024, H=H, D=D, m=m, W=W, dtype="bf16" if dt is torch.bfloat16 else "f32", tau=0.1)
    cache = cache or paged.PagedEntries(L, N, P, D, R, cfg.S, dtype=dt)
    return cache, layer.HcaDecode(cfg, cache, layer=layer_at, **kw)


def tokens(R, T, D=128, dt=torch.bfloat16, seed=0, H=8):
    g = torch.Generator().manual_seed(seed)
    x = {k: torch.randn(R, T, D, generator=g).to(dt).cuda() for k in ("a", "z", "kv_raw")}
    x["q"] = torch.randn(R, T, H, D, generator=g).to(dt).cuda()
    return x


def one(x, t=0):
    return {k: v[:, t].contiguous() for k, v in x.items()}


def state(d):
    c = d.cache
    return [t.clone() for t in (d.pos, d.ring, d.carry, c.held, c.table, c.refcount, c.pool)]


def same_state(d, want):
    assert all(torch.equal(a, b) for a, b in zip(state(d), want))


@pytest.mark.parametrize("why", ["dst is live", "no tail page", "src holds too few"])
def test_a_refused_fork_leaves_both_rows_alone(mods, why):
    c, d = decode(mods, N=20)
    c.reserve([0, 3], [60, 17] if why == "no tail page" else [32, 17])    # 15 + 5 or 8 + 5 of 20 pages
    d.load({k: v for k, v in tokens(6, 45).items() if k != "q"}, torch.tensor([45, 0, 0, 30, 0, 0], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert c.status.item() == 0
    if why == "src holds too few":
        c.free([3])
    before = state(d)
    src, dst = {"dst is live": ([0, 0], [1, 3]), "no tail page": ([0], [1]), "src holds too few": ([0, 3], [1, 2])}[why]
    d.fork(src, dst)
    torch.cuda.synchronize()
    assert c.status.item() == (6 if why == "no tail page" else 1) | 2 << 8
    same_state(d, before)
    # and the rows go on: a fork that can be made
    c.status.zero_()
    c.free([3])
    d.fork([0], [1])
    torch.cuda.synchronize()
    assert c.status.item() == 0 and d.pos[1].item() == 45 and c.held[1].item() == 2
    assert torch.equal(d.ring[1], before[1][0]) and torch.equal(d.carry[1], before[2][0])


def test_a_fork_for_two_layers_captured(mods):
    """The second layer's state goes by the same fork; in a graph, a replay that is
    refused changes neither."""
    c, d = decode(mods, L=2)
    _, e = decode(mods, cache=c, layer_at=1)
    c.reserve([0], [32])
    n = torch.tensor([45, 0, 0, 0, 0, 0], dtype=torch.int32).cuda()
    for k, lay in enumerate((d, e)):
        lay.load({k_: v for k_, v in tokens(6, 45, seed=k).items() if k_ != "q"}, n)
    src, dst = (torch.tensor(v, dtype=torch.int32).cuda() for v in ([0, 0], [1, 4]))

    def fork():
        d.fork(src, dst)
        e.copy_state(src.long(), dst.long(), c.forked())
    fork()
    torch.cuda.synchronize()
    assert c.status.item() == 0 and d.pos.tolist() == e.pos.tolist() == [45, 45, 0, 0, 45, 0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        fork()
    torch.cuda.current_stream().wait_stream(s)
    before = state(d), state(e)
    g.replay()                                         # rows 1 and 4 are live
    torch.cuda.synchronize()
    assert c.status.item() == 1 | 2 << 8
    same_state(d, before[0]), same_state(e, before[1])
    c.status.zero_()
    dst.copy_(torch.tensor([2, 5], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert c.status.item() == 0 and d.pos.tolist() == e.pos.tolist() == [45, 45, 45, 0, 45, 45]
    assert torch.equal(e.ring[5], e.ring[0]) and torch.equal(e.carry[2], e.carry[0])


@pytest.mark.parametrize("src,dst", [([9], [1]), ([-1], [1]), ([0, 1], [2, 6]), ([0], [-3]), ([2 ** 31 - 1], [-2 ** 31])])
def test_a_fork_of_rows_out_of_range_is_refused(mods, src, dst):
    c, d = decode(mods)
    c.reserve([0], [32])
    d.load({k: v for k, v in tokens(6, 20).items() if k != "q"}, torch.tensor([20, 0, 0, 0, 0, 0], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    before = state(d)
    d.fork(src, dst)
    torch.cuda.synchronize()
    assert c.status.item() == 1 | 2 << 8
    same_state(d, before)


def rope(layer, D=128, R=32):
    f = torch.tensor([10000.0 ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64)
    return layer.NormRope(inv_freq=f.cuda(), kv_weight=torch.linspace(0.5, 1.5, D).cuda())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nr", [False, True])
def test_idle_rows_stay_as_they_are(mods, nr, dt):
    """A freed row and an idle one that holds pages, over more steps than a block has
    tokens, some of them replayed: nothing is reported, their state, pages and outputs
    stay, and NaN in their input reaches nobody; the others go on as in a batch of
    their own."""
    layer, ops, paged = mods
    kw = dict(R=4, dt=dt, norm_rope=rope(layer) if nr else None)
    c, d = decode(mods, **kw)
    c2, e = decode(mods, **kw)
    x = {k: v for k, v in tokens(4, 37, dt=dt).items() if k != "q"}
    for cc, dd in ((c, d), (c2, e)):
        cc.reserve([0, 1, 2, 3], [40] * 4)
        dd.load(x)
    c.free([1])
    d.groups = paged.PrefixGroups([([3], 0), ([0], 0)], 4)           # 1 is freed, 2 idle
    idle = [1, 2]
    pages = c.table[2, :10].long()

    def kept():
        return [t[idle].clone() for t in (d.pos, d.ring, d.carry, d.out, c.table, c.held)] + [c.pool[:, pages].clone()]
    before = kept()
    static = {k: torch.zeros_like(v) for k, v in one(tokens(4, 1, dt=dt)).items()}
    y = tokens(4, 20, dt=dt, seed=5)
    for t in range(20):
        for k in static:
            static[k].copy_(y[k][:, t])
        want = e.step(static).clone()
        for k in static:
            static[k][idle] = float("nan")
        if t == 10:
            d.capture(static)
        got = d.step(static) if t < 10 else d.replay()
        assert torch.equal(got[[0, 3]], want[[0, 3]])
    torch.cuda.synchronize()
    assert c.status.item() == 0 and d.pos.tolist() == [57, 37, 37, 57]
    assert all(torch.equal(a, b) for a, b in zip(kept(), before))
    assert torch.equal(d.ring[[0, 3]], e.ring[[0, 3]]) and torch.equal(d.carry[[0, 3]], e.carry[[0, 3]])
    # and the idle one is taken up again where it was left
    d.groups = paged.PrefixGroups([([2], 0)], 4)
    c2, f = decode(mods, **kw)
    c2.reserve([0, 1, 2, 3], [40] * 4)
    f.load(x)
    for k in static:
        static[k].copy_(y[k][:, 0])
    assert torch.equal(d.step(static)[2], f.step(static)[2])


def test_positions_advance_by_rows(mods):
    _, ops, _ = mods
    p, n = torch.arange(700, dtype=torch.int32).cuda(), (torch.arange(700, dtype=torch.int32) % 3).cuda()
    want = p + n
    ops.csa_pos_advance(p, n)
    assert torch.equal(p, want)
    ops.csa_pos_advance(p, 2)
    assert torch.equal(p, want + 2)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nr", [False, True])
def test_decode_without_a_window(mods, nr, dt):
    """W = 0: a query sees its complete entries alone (none before the first, which gives
    0).  Tolerances are the decode driver's: 2e-2 absolute in bf16, 1e-5 in fp32; the
    logits of rounded entries are off by |q| |k| tau 2^-8 in bf16."""
    layer, _, paged = mods
    m, D, H = 8, 128, 8
    ropes = rope(layer) if nr else None
    c, d = decode(mods, R=3, m=m, W=0, dt=dt, norm_rope=ropes, with_lse=True)
    c.reserve([0, 1, 2], [8] * 3)
    x = tokens(3, 33, dt=dt, seed=2)
    lens = [25, 0, 7]
    d.load({k: v[:, :25].contiguous() for k, v in x.items() if k != "q"}, torch.tensor(lens, dtype=torch.int32).cuda())
    for step in range(4):
        out = d.step(one(x, 25 + step))
        torch.cuda.synchronize()
        for r in range(3):
            at = list(range(lens[r])) + list(range(25, 26 + step))
            n, q = len(at), np64(x["q"][r, 25 + step])
            ent, _ = serving.append(np64(x["z"][r, at]), np64(x["a"][r, at]), n, m)
            if nr:
                f = np64(ropes.inv_freq)
                q = serving.norm_rope(q, np.full(H, n - 1), f)
                ent = serving.norm_rope(ent, m * np.arange(len(ent)), f)
                q, ent = (np64(torch.tensor(v).to(dt)) for v in (q, ent))
            else:
                ent = np64(torch.tensor(ent).to(dt))
            ref, lse, _ = serving.attend(q, ent.reshape(-1, D), None, 0.1)
            if nr:
                ref = serving.norm_rope(ref, np.full(H, n - 1), f, norm=False, inverse=True)
            tol = 2e-2 if dt is torch.bfloat16 else 1e-5 * np.maximum(1, np.abs(ref))
            assert (np.abs(np64(out[r, 0]) - ref) <= tol).all()
            if n < m:
                assert (out[r] == 0).all() and (d.lse[r] == -float("inf")).all()
            else:
                assert np.abs(np64(d.lse[r, 0]) - lse).max() <= (0.05 if dt is torch.bfloat16 else 1e-4)
    assert c.status.item() == 0
    d.fork([0], [1])                                   # (row 1 holds pages: refused)
    assert c.status.item() == 1 | 2 << 8 and d.pos.tolist() == [29, 4, 11]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_key_beside_queries_of_no_heads(mods, dt):
    """q [B, T, 0, D] beside a key gives what the key alone gives."""
    layer, ops, _ = mods
    B, T, D = 2, 9, 64
    k = torch.randn(B, T, D, generator=torch.Generator().manual_seed(1)).to(dt).cuda()
    q = torch.empty(B, T, 0, D, dtype=dt, device="cuda")
    p = torch.tensor([5, 1000], dtype=torch.int32).cuda()
    f = rope(layer).inv_freq
    rings = [torch.full((B, 6, D), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    ops.qk_norm_rope(q, k, torch.empty_like(q), rings[0], p, inv_freq=f)
    ops.qk_norm_rope(None, k, None, rings[1], p, inv_freq=f)
    assert torch.equal(*rings) and not (rings[0] == 7.0).any()
    ops.qk_norm_rope(q, None, torch.empty_like(q), None, p, inv_freq=f)


def test_calls_on_an_empty_batch(mods):
    """No sequences, and no tokens: the calls return and write nothing (the carry of no
    tokens is the carry)."""
    _, ops, paged = mods
    pool = torch.full((4, 2, 128), 9.0, device="cuda")
    for B, T in ((0, 3), (2, 0)):
        a, i = torch.zeros(B, T, 128, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        tab = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
        carry = torch.randn(B, 2, 3, 128, device="cuda")
        out = torch.zeros_like(carry)
        ops.hca_paged_append(a, a, i, carry, pool, tab, i, 4, carry_out=out)
        assert torch.equal(out, carry)
        q = torch.zeros(B, T, 4, 128, device="cuda")
        ops.qk_norm_rope(q, a, torch.empty_like(q), torch.empty_like(a), i)
        ops.hca_prefix_attn_fwd(q, pool, tab, i, paged.PrefixGroups.singles(B), None, None, 1.0, 0, i, torch.empty_like(q), 4)
    torch.cuda.synchronize()
    assert (pool == 9.0).all()


@pytest.mark.parametrize("nr", [False, True])
def test_a_freed_row_takes_a_new_prompt(mods, nr):
    """A row that was freed in the middle of a block gives, with its next prompt, the bits
    of a row that was never used; in a second layer too."""
    layer, _, paged = mods
    kw = dict(R=2, L=2, m=8, norm_rope=rope(layer) if nr else None)
    c, d = decode(mods, **kw)
    _, e = decode(mods, cache=c, layer_at=1, **kw)
    c2, f = decode(mods, **kw)
    x = {k: v for k, v in tokens(2, 45).items() if k != "q"}
    y = tokens(2, 30, seed=9)
    c.reserve([0, 1], [8, 8])
    d.load(x), e.load(x)
    d.free([1]), e.reset([1])
    c.reserve([1], [8]), c2.reserve([0, 1], [8, 8])
    only = torch.tensor([0, 29], dtype=torch.int32).cuda()
    new = {k: v[:, :29].contiguous() for k, v in y.items() if k != "q"}
    d.load(new, only), e.load(new, only), f.load(new, only)
    for lay in (d, e, f):
        lay.groups = paged.PrefixGroups([([1], 0)], 2)
    outs = [lay.step(one(y, 29))[1].clone() for lay in (d, e, f)]
    torch.cuda.synchronize()
    assert c.status.item() == 0 and d.pos.tolist() == e.pos.tolist() == [45, 30]
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])


def test_two_captures_replayed_in_turn(mods):
    """The graph of an earlier capture goes on with its own groups and inputs, although
    nothing else holds them and their memory would be in use again."""
    layer, _, paged = mods
    c, d = decode(mods, R=4)
    c.reserve([0, 1, 2, 3], [16] * 4)
    d.load({k: v for k, v in tokens(4, 30).items() if k != "q"})
    d.step(one(tokens(4, 1, seed=1)))
    graphs = []
    for b in (2, 1):
        d.groups = paged.PrefixGroups([([b], 0)], 4)
        graphs.append(d.capture(one(tokens(4, 1, seed=2))))
    d.groups = paged.PrefixGroups.singles(4)
    keep = [torch.full((k,), -1, dtype=torch.int32, device="cuda") for k in (1, 2, 4) for _ in range(32)]
    for g, b in ((graphs[0], 2), (graphs[1], 1), (graphs[0], 2)):
        pos, out = d.pos.clone(), d.out.clone()
        g.replay()
        torch.cuda.synchronize()
        pos[b] += 1
        assert torch.equal(d.pos, pos)
        assert [not torch.equal(d.out[r], out[r]) for r in range(4)] == [r == b for r in range(4)]
    assert c.status.item() == 0 and len(keep) == 96


@pytest.mark.parametrize("dt,D,m,T", [("bf16", 128, 64, 700), ("bf16", 128, 128, 129), ("bf16", 128, 4, 333),
                                      ("f32", 64, 16, 90)])
def test_entries_of_a_prefill_are_those_of_a_decode(mods, dt, D, m, T):
    """A prompt's normalised, rotated entries: the same bits through HcaPrefill and
    HcaDecode.load, one rounding from the formula.  The pooled sums' error, relative
    to mean |a| (below 2 for these inputs): 2 (2 m + 64) half steps of fp32, over the
    row's rms; the norm and rotation 40 more, both times |w| of a pair; then half a step
    of the type."""
    layer, ops, paged = mods
    from long_context_compressed_compress_b200 import configs
    B, H = 2, 16
    cfg = configs._hca(B=B, T=T, H=H, D=D, m=m, W=20, dtype=dt, tau=0.1)
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    x = tokens(B, T, D=D, H=H, dt=t, seed=4) | {"sink": None}
    nr = rope(layer, D)
    nr.entry_weight = torch.linspace(1.5, 0.5, D).cuda()
    p = layer.HcaPrefill(cfg, norm_rope=nr)
    p.kv_c.fill_(9.0)
    p.run(x)
    cache = paged.PagedEntries(1, 2 * B * (T // m + 1), 1, D, B, T // m + 1, dtype=t)
    d = layer.HcaDecode(cfg, cache, norm_rope=nr)
    cache.reserve(list(range(B)), [T // m] * B)
    d.load({k: x[k] for k in ("a", "z", "kv_raw")})
    torch.cuda.synchronize()
    assert cache.status.item() == 0 and ops.device_status() == 0
    S = T // m
    got = cache.pool[0][cache.table[:, :S].long()].reshape(B, S, D)
    assert torch.equal(got, p.kv_c[:, :S])
    w = np64(nr.entry_weight)
    for b in range(B):
        ent, _ = serving.append(np64(x["z"][b]), np64(x["a"][b]), T, m)
        ref = serving.norm_rope(ent, m * np.arange(S), np64(nr.inv_freq), w)
        rms = np.sqrt((ent ** 2).mean(-1, keepdims=True))
        tol = (2 * (2 * m + 64) * 2 / rms + 40) * 2.0 ** -24 * 2 * w.max() * 3 + torch.finfo(t).eps / 2 * np.abs(ref) * 1.001
        assert (np.abs(np64(got[b]) - ref) <= tol).all()
