"""Host-side checks of the serving operators (no GPU needed): refusals of bad
calls before any launch, the group plan, and the float64 forms against torch."""
import numpy as np
import pytest
import torch

from oracle import serving

FAKE = 1 << 20       # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    from long_context_compressed_compress_b200 import build
    build.build()
    from long_context_compressed_compress_b200 import ops
    return ops.lib


def norm_rope(lib, **kw):
    a = dict(q=FAKE, qb=8192, qt=1024, kv=FAKE + (1 << 24), kb=1024, kt=128, dtype=1, B=1, T=8, H=8, D=128, pos=FAKE,
             lens=None, step=1, freq=FAKE, R=64, qw=None, kw=None, eps=1e-6, flags=1, qo=FAKE + (2 << 24),
             ko=FAKE + (3 << 24), cap=8)
    a.update(kw)
    return lib.qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(kv=None), 1), (dict(q=None, qo=None, kv=None, ko=None), 1), (dict(pos=None), 1),
    (dict(freq=None), 1), (dict(R=-16), 1), (dict(R=144), 1), (dict(cap=0), 1), (dict(dtype=2), 1),
    (dict(flags=8), 1), (dict(eps=-1.0), 1), (dict(B=-1), 1), (dict(qt=-1024), 1),
    (dict(D=96, R=32), 2), (dict(D=512), 2), (dict(R=24), 2),
    (dict(q=FAKE + 2), 3), (dict(ko=FAKE + (3 << 24) + 8), 3), (dict(qt=1028), 3), (dict(kb=1025), 3),
    (dict(qo=FAKE, qt=1152), 1),                       # in place, but not dense
    (dict(qo=FAKE + 4096), 1),                         # half over the input
    (dict(ko=FAKE + (1 << 24) + 256), 1),
    (dict(ko=FAKE), 1), (dict(ko=FAKE + (2 << 24)), 1),  # keys over the queries, in or out
    (dict(kv=FAKE + (3 << 24), cap=4), 1),              # in place into a ring
    (dict(B=0), 0), (dict(T=0), 0),
])
def test_norm_rope_refusals(lib, kw, want):
    assert norm_rope(lib, **kw) == want


def append(lib, **kw):
    a = dict(a=FAKE, z=FAKE, dtype=1, B=2, T=4, D=128, m=128, pos=FAKE, lens=None, ci=FAKE, co=FAKE, pool=FAKE, N=4,
             P=16, table=FAKE, held=FAKE, mp=2, w=None, eps=1e-6, freq=None, R=0, flags=0, status=FAKE)
    a.update(kw)
    return lib.hca_paged_append(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=None), 1), (dict(pool=None), 1), (dict(held=None), 1), (dict(ci=None), 1), (dict(m=0), 1), (dict(P=0), 1),
    (dict(mp=0), 1), (dict(T=-1), 1), (dict(R=64), 1), (dict(dtype=7), 1), (dict(flags=16), 1),
    (dict(co=FAKE + 4096), 1),                          # a carry half over itself
    (dict(D=32), 2), (dict(D=192), 2), (dict(R=8, freq=FAKE), 2),
    (dict(z=FAKE + 4), 3), (dict(co=FAKE + (1 << 22) + 4), 3), (dict(B=0), 0),
])
def test_append_refusals(lib, kw, want):
    assert append(lib, **kw) == want


def attn(lib, **kw):
    a = dict(q=FAKE, pool=FAKE, N=4, P=16, table=FAKE, held=FAKE, mp=2, off=FAKE, seq=FAKE, shared=FAKE, G=1, n=1,
             raw=FAKE, sink=None, tau=1.0, W=8, B=1, T=2, H=16, D=128, m=4, cap=9, pos=FAKE, out=FAKE, lse=None,
             dtype=1, status=FAKE)
    a.update(kw)
    return lib.hca_prefix_attn_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(off=None), 1), (dict(seq=None), 1), (dict(raw=None), 1), (dict(P=0), 1), (dict(m=0), 1),
    (dict(cap=8), 1),                                   # the ring is shorter than W + T - 1
    (dict(W=-1), 1), (dict(W=2 ** 31 - 1, T=2 ** 31 - 1, cap=2 ** 31 - 1), 1), (dict(dtype=3), 1), (dict(G=-1), 1),
    (dict(D=96), 2), (dict(H=1025), 2), (dict(P=1 << 20, mp=1 << 12), 2),
    (dict(pool=FAKE + 8), 3), (dict(out=FAKE + 2), 3), (dict(n=0), 0), (dict(T=0, cap=8), 0), (dict(H=0), 0),
])
def test_attention_refusals(lib, kw, want):
    assert attn(lib, **kw) == want


def test_page_refusals(lib):
    f, ws = FAKE, lib.kv_pages_workspace_size(100, 8)
    assert ws >= 4 * (3 * 100 + 8) and lib.kv_pages_workspace_size(-1, 2) == 0

    def reserve(rows=f, n=8, P=4, table=f, R=4, mp=2, N=100, w=f, wb=ws):
        return lib.kv_pages_reserve(rows, f, n, P, table, f, R, mp, f, N, w, wb, f, None)
    assert reserve(rows=None) == 1 and reserve(n=-1) == 1 and reserve(P=0) == 1 and reserve(table=None) == 1
    assert reserve(mp=0) == 1 and reserve(w=None) == 1 and reserve(wb=ws - 4) == 1 and reserve(w=f + 2) == 3
    assert reserve(N=(1 << 20) + 1) == 2 and reserve(n=0, w=None, wb=0) == 0

    def fork(src=f, n=8, P=4, pool=f, L=2, page=64, wb=ws, N=100):
        return lib.kv_pages_fork(src, f, f, n, P, f, f, 4, 2, f, N, pool, L, page, f, wb, f, None)
    assert fork(src=None) == 1 and fork(pool=None) == 1 and fork(L=0) == 1 and fork(page=0) == 1 and fork(wb=0) == 1
    assert fork(page=65) == 2 and fork(page=32) == 2 and fork(L=70000) == 2 and fork(pool=f + 4) == 3
    assert fork(n=0) == 0
    assert lib.kv_pages_free(None, 2, f, f, 4, 2, f, 100, f, None) == 1
    assert lib.kv_pages_free(f, 0, f, f, 4, 2, f, 100, f, None) == 0

    def compact(pool=f, page=64, out=f, live=f, wb=ws):
        return lib.kv_pages_compact(f, f, 4, 2, f, 100, pool, 1, page, out, f, live, f, wb, None)
    assert compact(pool=None) == 1 and compact(out=None) == 1 and compact(live=None) == 1 and compact(wb=16) == 1
    assert compact(page=40) == 2 and compact(pool=f + 8) == 3


def test_group_plan():
    from long_context_compressed_compress_b200 import paged
    g = paged.PrefixGroups([([2, 0], 64), ([3], 0)], 5, device="cpu")
    assert (g.G, g.n_seq, g.B) == (2, 3, 5)
    assert g.off.tolist() == [0, 2, 3] and g.seq.tolist() == [2, 0, 3] and g.shared.tolist() == [64, 0]
    assert paged.PrefixGroups.singles(3, device="cpu").off.tolist() == [0, 1, 2, 3]
    assert paged.PrefixGroups([], 2, device="cpu").n_seq == 0
    for bad in ([([0, 0], 1)], [([0], 1), ([0], 1)], [([5], 1)], [([-1], 1)], [([], 1)], [([0], -1)]):
        with pytest.raises(ValueError):
            paged.PrefixGroups(bad, 5, device="cpu")


def test_bindings_refuse_cpu_tensors_and_wrong_types():
    from long_context_compressed_compress_b200 import ops, paged
    q = torch.zeros(1, 2, 4, 64)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.qk_norm_rope(q, None, q, None, i)
    with pytest.raises(ValueError):
        ops.qk_norm_rope(q, None, None, None, i)
    with pytest.raises(ValueError):
        ops.hca_prefix_attn_fwd(q, q[0], i.view(1, 1), i, paged.PrefixGroups.singles(1, device="cpu"), None, None, 1.0, 0,
                                i, q, 4)
    with pytest.raises(ValueError):
        ops.hca_paged_append(q[0], q[0], i, q, q[0], i.view(1, 1), i, 4)
    with pytest.raises(ValueError):
        ops.kv_pages_free(i, i.view(1, 1), i, i)


# ---- pins of the float64 forms
def test_rotation_pins():
    """A rotation keeps lengths, composes, undoes itself and is the 2x2 matrix."""
    r = np.random.default_rng(0)
    x, f = r.standard_normal((5, 64)), np.array([10000.0 ** (-2.0 * i / 32) for i in range(16)])
    for inter in (True, False):
        y = serving.norm_rope(x, 7, f, norm=False, interleaved=inter)
        assert np.allclose((x ** 2).sum(-1), (y ** 2).sum(-1)) and (y[:, :32] == x[:, :32]).all()
        assert np.allclose(serving.norm_rope(y, 5, f, norm=False, interleaved=inter),
                           serving.norm_rope(x, 12, f, norm=False, interleaved=inter))
        assert np.allclose(serving.norm_rope(y, 7, f, norm=False, interleaved=inter, inverse=True), x)
        i, j = (32 + 6, 32 + 7) if inter else (32 + 3, 32 + 19)
        c, s = np.cos(7 * f[3]), np.sin(7 * f[3])
        assert np.allclose(y[:, i], x[:, i] * c - x[:, j] * s) and np.allclose(y[:, j], x[:, i] * s + x[:, j] * c)
    w = r.standard_normal(64)
    ref = torch.nn.functional.rms_norm(torch.tensor(x), (64,), torch.tensor(w), 1e-6)
    assert np.allclose(serving.norm_rope(x, 0, None, w), ref.numpy())


def test_append_pins():
    """The entries are the oracle's hca_compress; the parts join to the block."""
    import oracle
    r = np.random.default_rng(1)
    z, a = r.standard_normal((100, 8)), r.standard_normal((100, 8))
    e, parts = serving.append(z, a, 100, 32)
    assert np.allclose(e, oracle.hca_compress(a[None], z[None], 32)[0])
    assert (parts[0] == np.stack([np.full(8, serving.EMPTY), np.zeros(8), np.zeros(8)])).all()
    assert np.allclose(parts[1], serving.gate_state(z[96:], a[96:]))


def test_attend_pin():
    r = np.random.default_rng(2)
    q, k = r.standard_normal((3, 8)), r.standard_normal((9, 8))
    o, l, _ = serving.attend(q, k, None, 0.5)
    t = torch.softmax(torch.tensor(q @ k.T * 0.5), 1).numpy() @ k
    assert np.allclose(o, t)
    o2, l2, _ = serving.attend(q, k, l, 0.5)            # a sink as heavy as the keys
    assert np.allclose(o2, t / 2) and np.allclose(l, l2)


def test_pages_pins():
    p = serving.Pages(6, 2, 3, 4, np.arange(6 * 2.0).reshape(1, 6, 2, 1))
    p.reserve([0], [5])
    p.fork([0], [1], [3])
    assert p.rows[1] == [0, 3] and p.ref[:4] == [2, 1, 1, 1]
    assert p.pool[0, 3, 0, 0] == p.pool[0, 1, 0, 0] and p.pool[0, 3, 1, 0] == 7.0
    p.free([0])
    assert p.compact() == 2 and p.rows[1] == [0, 1] and p.ref == [1, 1, 0, 0, 0, 0]


def test_groups_say_who_is_attended():
    from long_context_compressed_compress_b200 import paged
    assert paged.PrefixGroups([([2, 0], 3), ([1], 0)], 3, device="cpu").attended is None
    assert paged.PrefixGroups([([3], 0), ([0], 5)], 5, device="cpu").attended.tolist() == [1, 0, 0, 1, 0]
    assert paged.PrefixGroups([], 2, device="cpu").attended.tolist() == [0, 0]
