"""The page operations against a host model of rows, counts and page contents:
every table, count and byte has to be equal."""
import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def paged(cuda_ok):
    from long_context_compressed_compress_b200 import build
    build.build()
    from long_context_compressed_compress_b200 import paged
    return paged


def pair(paged, L=2, N=40, P=4, D=8, R=12, max_entries=60, dtype=torch.bfloat16, seed=0):
    c = paged.PagedEntries(L, N, P, D, R, max_entries, dtype=dtype)
    c.pool.copy_(torch.randn(c.pool.shape, generator=torch.Generator().manual_seed(seed)))
    return c, serving.Pages(N, P, R, c.max_pages, c.pool.float().cpu().numpy())


def same(c, m, status=0):
    torch.cuda.synchronize()
    assert c.status.item() == status
    np.testing.assert_array_equal(c.held.cpu().numpy(), [len(r) for r in m.rows])
    np.testing.assert_array_equal(c.table.cpu().numpy(), m.table())
    np.testing.assert_array_equal(c.refcount.cpu().numpy(), m.ref)
    np.testing.assert_array_equal(c.pool.float().cpu().numpy(), m.pool)


def both(c, m, name, *args):
    getattr(c, name)(*args)
    getattr(m, name)(*args)


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 8), (torch.float32, 4), (torch.bfloat16, 128)])
def test_a_life_of_forks(paged, dtype, D):
    c, m = pair(paged, dtype=dtype, D=D)
    both(c, m, "reserve", [0, 3], [17, 8])
    same(c, m)
    both(c, m, "fork", [0, 0, 3, 0], [1, 2, 4, 5], [17, 16, 5, 0])      # partial, whole, from the middle, empty
    same(c, m)
    both(c, m, "reserve", [1, 2, 5, 0], [25, 16, 1, 3])                  # growing, enough already, first, shorter
    same(c, m)
    both(c, m, "fork", [1], [6], [23])                                   # a fork of a fork
    same(c, m)
    both(c, m, "free", [0, 4])
    same(c, m)
    both(c, m, "compact")
    same(c, m)
    assert c.n_live.item() == sum(r > 0 for r in m.ref)
    both(c, m, "compact")                                                # nothing left to move
    same(c, m)
    both(c, m, "free", [1, 2, 3, 5, 6, 7])
    same(c, m)
    assert c.refcount.abs().sum().item() == 0
    both(c, m, "compact")
    same(c, m)


def test_random_operations(paged):
    """200 random calls on a larger cache (page counts around the scan's chunk of
    1024, lists of one to all rows)."""
    r = np.random.default_rng(1)
    R, P = 40, 3
    c, m = pair(paged, L=1, N=2500, P=P, D=8, R=R, max_entries=300, seed=2)
    for _ in range(200):
        op = r.integers(0, 5)
        full = [i for i in range(R) if m.rows[i]]
        empty = [i for i in range(R) if not m.rows[i]]
        if op == 0:
            rows = r.permutation(R)[:r.integers(1, R)].tolist()
            n = [int(r.integers(0, 301)) for _ in rows]
            free = sum(v == 0 for v in m.ref)
            if sum(max(0, -(-e // P) - len(m.rows[i])) for i, e in zip(rows, n)) > free:
                continue
            both(c, m, "reserve", rows, n)
        elif op == 1 and full and empty:
            dst = empty[:r.integers(1, len(empty) + 1)]
            src = [int(r.choice(full)) for _ in dst]
            n = [int(r.integers(0, len(m.rows[s]) * P + 1)) for s in src]
            if sum(e % P != 0 for e in n) > sum(v == 0 for v in m.ref):
                continue
            both(c, m, "fork", src, dst, n)
        elif op == 2 and full:
            both(c, m, "free", [int(v) for v in r.permutation(full)[:r.integers(1, len(full) + 1)]])
        elif op == 3:
            both(c, m, "compact")
        same(c, m)


def test_lists_longer_than_a_block(paged):
    """1500 rows in one call."""
    n = 1500
    c, m = pair(paged, L=1, N=5000, P=2, D=8, R=n + 1, max_entries=8)
    both(c, m, "reserve", [n], [7])
    both(c, m, "fork", [n] * n, list(range(n)), [i % 8 for i in range(n)])
    same(c, m)
    both(c, m, "reserve", list(range(n)), [8] * n)
    same(c, m)
    both(c, m, "free", list(range(0, n, 2)))
    both(c, m, "compact")
    same(c, m)


@pytest.mark.parametrize("N", [8191, 8192, 8193, 20001])
def test_caches_around_a_sweep(paged, N):
    """Page counts around the 8192 that are gone through at once, nearly all of them
    in use and then few, far apart."""
    R = 9
    c, m = pair(paged, L=1, N=N, P=1, D=8, R=R, max_entries=N)
    both(c, m, "reserve", list(range(R)), [N // R] * R)
    both(c, m, "free", [1, 4, 7])
    both(c, m, "reserve", [4], [N // R + 100])
    same(c, m)
    both(c, m, "compact")
    same(c, m)
    both(c, m, "free", [0, 2, 3, 5, 6])
    both(c, m, "compact")
    same(c, m)


BAD = [
    ("reserve", ([12], [4]), 1 | 1 << 8),                       # row out of range
    ("reserve", ([-1, 2], [4, 4]), 1 | 1 << 8),
    ("reserve", ([1, 1], [4, 4]), 1 | 1 << 8),                  # listed twice
    ("reserve", ([1], [61]), 1 | 1 << 8),                       # longer than max_pages
    ("reserve", ([1], [-1]), 1 | 1 << 8),
    ("reserve", ([1, 2, 4], [60, 60, 60]), 6 | 1 << 8),         # too few free pages
    ("fork", ([0, 0], [1, 1], [4, 4]), 1 | 2 << 8),             # dst twice
    ("fork", ([0], [3], [4]), 1 | 2 << 8),                      # dst not empty
    ("fork", ([0], [0], [4]), 1 | 2 << 8),
    ("fork", ([0], [1], [21]), 1 | 2 << 8),                     # src holds too few
    ("fork", ([1], [2], [1]), 1 | 2 << 8),
    ("fork", ([0, 1], [1, 2], [4, 4]), 1 | 2 << 8),             # a chain within one call
    ("fork", ([99], [1], [4]), 1 | 2 << 8),
]


@pytest.mark.parametrize("op,args,want", BAD, ids=[f"{b[0]}{i}" for i, b in enumerate(BAD)])
def test_refused_calls_change_nothing(paged, op, args, want):
    c, m = pair(paged)
    both(c, m, "reserve", [0, 3], [17, 8])
    getattr(c, op)(*args)
    same(c, m, status=want)
    c.status.zero_()
    both(c, m, "fork", [0], [1], [17])                          # and the cache goes on
    same(c, m)


def test_fork_without_a_free_page(paged):
    c, m = pair(paged, N=5)
    both(c, m, "reserve", [0], [20])
    c.fork([0, 0], [1, 2], [16, 17])
    same(c, m, status=6 | 2 << 8)
    c.status.zero_()
    both(c, m, "fork", [0], [1], [16])                          # whole pages need none
    same(c, m)


def test_free_skips_bad_rows_and_frees_once(paged):
    c, m = pair(paged)
    both(c, m, "reserve", [0, 3], [17, 8])
    c.free([0, 12, 0, -4])
    m.free([0])
    same(c, m, status=1 | 3 << 8)


def test_metadata_apart_from_its_source(paged):
    """compact into other tensors: the source metadata stays, and the call can
    be made again from it."""
    from long_context_compressed_compress_b200 import ops
    c, m = pair(paged)
    both(c, m, "reserve", [0, 1, 2, 3], [17, 8, 30, 9])
    both(c, m, "free", [0, 2])
    t0, r0 = c.table.clone(), c.refcount.clone()
    for _ in range(2):
        t, rc = torch.zeros_like(c.table), torch.full_like(c.refcount, 5)
        ops.kv_pages_compact(c.pool, c.table, c.held, c.refcount, c.n_live, c.ws, table_out=t, refcount_out=rc)
        torch.cuda.synchronize()
        assert torch.equal(c.table, t0) and torch.equal(c.refcount, r0)
    m.compact()
    c.table, c.refcount = t, rc
    same(c, m)


def test_captured_with_attention_in_between(paged):
    """Reserve and fork captured in one graph replay with new lists in place."""
    c, m = pair(paged)
    both(c, m, "reserve", [0], [18])
    src, dst, n = (torch.tensor(v, dtype=torch.int32).cuda() for v in ([0, 0], [1, 2], [18, 7]))
    grow = torch.tensor([30, 9], dtype=torch.int32).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        c.fork(src, dst, n)
        c.reserve(dst, grow)
    torch.cuda.current_stream().wait_stream(s)
    for d in ([1, 2], [5, 4]):
        dst.copy_(torch.tensor(d, dtype=torch.int32))
        g.replay()
        m.fork([0, 0], d, [18, 7])
        m.reserve(d, [30, 9])
        same(c, m)
