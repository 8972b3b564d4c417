"""hca_prefix_attn_fwd against the softmax in float64 over each query's own
keys.

Tolerances.  With e the largest error of a row's logits (the fp32 dot product of
D terms on either unit: (D + 2) half steps of 2^-24 of tau sum |q k|, plus the
scaling) a weight is off by a factor within 1 +- (e + 4 * 2^-23), and, where P is
stored in bf16, another half step 2^-8 (numerator and denominator see the same
rounded weights).  So with d the sum of those, |out' - out| <= 2 d sum_j w_j |k_j
- out| + d' |out| for the sink's share; n terms of fp32 accumulation add n 2^-24
max |k|; then half a step of the stored type."""
import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def mods(cuda_ok):
    from long_context_compressed_compress_b200 import build
    build.build()
    from long_context_compressed_compress_b200 import ops, paged
    return ops, paged


def np64(t):
    return t.detach().cpu().double().numpy()


class Batch:
    """A random batch: ``groups`` lists (members, shared entries); n[b] is the
    number of entries sequence b sees at its first query."""

    def __init__(self, groups, n, T, H, D, m, P, W, dt, seed=0, cap=None, extra_pages=1, sink=True, scale=1.0,
                 max_pages=None):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        B = len(n)
        self.groups, self.n, self.T, self.H, self.D, self.m, self.P, self.W, self.dt = groups, n, T, H, D, m, P, W, dt
        self.pos = [(v * m - 1 + int(r.integers(0, m))) if v else int(r.integers(-1, max(1, m - T))) for v in n]
        need = {b: -(-((self.pos[b] + T) // m) // P) + extra_pages for b in range(B)}
        N = sum(need.values()) + 5
        ids = list(map(int, r.permutation(N)))
        self.rows = [[] for _ in range(B)]
        for ms, sh in groups:
            common = [ids.pop() for _ in range(sh // P)]
            for b in ms:
                self.rows[b] = common + [ids.pop() for _ in range(max(0, need[b] - len(common)))]
        mp = max_pages or max(1, max(len(x) for x in self.rows))
        tab = np.full((B, mp), -1, np.int32)
        for b, x in enumerate(self.rows):
            tab[b, :len(x)] = x
        self.table, self.held = torch.tensor(tab), torch.tensor([len(x) for x in self.rows], dtype=torch.int32)
        self.pool = torch.randn(N, P, D, generator=g).to(DT[dt])
        self.q = (torch.randn(B, T, H, D, generator=g) * scale).to(DT[dt])
        self.cap = cap or max(1, W + T - 1)
        self.ring = torch.randn(B, self.cap, D, generator=g).to(DT[dt])
        self.sink = torch.randn(H, generator=g) if sink else None
        self.tau = 1.0 / np.sqrt(D)

    def keys(self, b, t):
        p = self.pos[b] + t
        nv = min((p + 1) // self.m, len(self.rows[b]) * self.P) if p >= 0 else 0
        ent = self.pool[self.rows[b]].reshape(-1, self.D)[:nv] if self.rows[b] else self.pool[:0].reshape(-1, self.D)
        win = [j % self.cap for j in range(max(0, p - self.W + 1), p + 1)] if self.W else []
        return np64(torch.cat([ent, self.ring[b, win]]))

    def run(self, mods, groups=None, status=None, lse=True):
        ops, paged = mods
        B = len(self.n)
        out = torch.full((B, self.T, self.H, self.D), 3.0, dtype=DT[self.dt]).cuda()
        ls = torch.full((B, self.T, self.H), 3.0).cuda() if lse else None
        ops.hca_prefix_attn_fwd(self.q.cuda(), self.pool.cuda(), self.table.cuda(), self.held.cuda(),
                                paged.PrefixGroups(groups or self.groups, B), self.ring.cuda(),
                                None if self.sink is None else self.sink.cuda(), self.tau, self.W,
                                torch.tensor(self.pos, dtype=torch.int32).cuda(), out, self.m, lse=ls, status=status)
        torch.cuda.synchronize()
        return out, ls

    def check(self, out, lse, seqs=None):
        u = 2.0 ** -24
        for b in range(len(self.n)) if seqs is None else seqs:
            for t in range(self.T):
                k, q = self.keys(b, t), np64(self.q[b, t])
                ref, rl, spread = serving.attend(q, k, None if self.sink is None else np64(self.sink), self.tau)
                got = np64(out[b, t])
                if len(k) == 0:
                    assert (got == 0).all() and (np64(lse[b, t]) == -np.inf).all()
                    continue
                e = (self.D + 4) * u * (np.abs(q) @ np.abs(k).T).max() * abs(self.tau) + 8 * u * np.abs(rl).max()
                d = e + 8 * u + (2.0 ** -8 if self.dt == "bf16" else 0.0)
                tol = (2.05 * d * spread + 2.05 * d * np.abs(ref) * (self.sink is not None)
                       + (len(k) + 16) * u * np.abs(k).max() + torch.finfo(DT[self.dt]).eps / 2 * np.abs(ref) * 1.01)
                bad = np.abs(got - ref) > tol
                assert not bad.any(), (b, t, np.abs(got - ref).max(), tol.min())
                # lse: the log of a sum whose terms are off by e and the exponential's share (it
                # adds the weights before P is rounded)
                dl = e + 8 * u
                assert (np.abs(np64(lse[b, t]) - rl) <= 1.01 * dl + (len(k) + 16) * u + 2 * u * np.abs(rl)).all(), (b, t)


CASES = {
    # one short sequence, one key
    "one_key": dict(groups=[([0], 0)], n=[0], T=1, H=16, D=128, m=128, P=64, W=1, dt="bf16"),
    "short": dict(groups=[([0], 0)], n=[100], T=1, H=16, D=128, m=128, P=64, W=128, dt="bf16"),
    "shared_h128": dict(groups=[([2, 0, 1], 512)], n=[600, 530, 512], T=1, H=128, D=128, m=128, P=64, W=128, dt="bf16"),
    "shared_h16": dict(groups=[([4, 0, 7, 2, 9], 700), ([1], 0), ([3, 5, 6, 8, 10], 96)],
                       n=[720, 33, 704, 97, 1000, 100, 130, 701, 500, 705, 96], T=2, H=16, D=128, m=64, P=16, W=128,
                       dt="bf16"),
    "odd_heads": dict(groups=[([0, 1, 2], 130)], n=[131, 135, 140], T=3, H=40, D=128, m=4, P=10, W=17, dt="bf16"),
    "one_head": dict(groups=[([0, 1], 300)], n=[300, 301], T=2, H=1, D=128, m=8, P=100, W=5, dt="bf16"),
    "no_window": dict(groups=[([0, 1, 2, 3], 0)], n=[0, 1, 5, 260], T=1, H=64, D=128, m=16, P=32, W=0, dt="bf16"),
    "no_sink": dict(groups=[([0, 1], 128)], n=[0 + 128, 300], T=1, H=32, D=128, m=128, P=64, W=100, dt="bf16",
                    sink=False),
    "long": dict(groups=[([0], 0), ([1, 2], 4096)], n=[5000, 4097, 4200], T=1, H=64, D=128, m=128, P=64, W=128,
                 dt="bf16"),
    "odd_window": dict(groups=[([3, 0, 1, 4, 5, 2], 0)], n=[3, 0, 1, 5, 140, 2], T=1, H=16, D=128, m=128, P=16, W=100,
                       dt="bf16"),
    "wide_split": dict(groups=[([0, 1, 2], 64)], n=[64, 300, 77], T=3, H=8, D=128, m=128, P=64, W=300, dt="bf16",
                       max_pages=64),
    "many_groups": dict(groups=[([i], 0) for i in range(37)] + [([39, 37, 38], 64)], n=[(7 * i) % 50 for i in range(37)]
                        + [64, 70, 201], T=1, H=16, D=128, m=16, P=32, W=20, dt="bf16"),
    "wide_window": dict(groups=[([0, 1], 64)], n=[64, 80], T=2, H=16, D=128, m=128, P=64, W=700, dt="bf16"),
    "many_tokens": dict(groups=[([0, 1], 64)], n=[64, 70], T=37, H=8, D=128, m=4, P=16, W=30, dt="bf16"),
    "big_logits": dict(groups=[([0, 1, 2], 256)], n=[256, 500, 900], T=1, H=16, D=128, m=128, P=64, W=128, dt="bf16",
                       scale=30.0),
    "bf16_d64": dict(groups=[([0, 1], 32)], n=[40, 33], T=2, H=8, D=64, m=4, P=16, W=20, dt="bf16"),
    "bf16_h200": dict(groups=[([0, 1], 32)], n=[40, 33], T=1, H=200, D=128, m=4, P=16, W=20, dt="bf16"),
    "f32": dict(groups=[([0, 2], 48), ([1], 0)], n=[50, 61, 300], T=3, H=8, D=64, m=4, P=16, W=100, dt="f32"),
    "f32_d128": dict(groups=[([0, 1], 0)], n=[0, 70], T=1, H=5, D=128, m=2, P=7, W=3, dt="f32"),
}


@pytest.mark.parametrize("name", CASES)
def test_against_softmax(mods, name):
    b = Batch(**CASES[name], seed=len(name))
    out, lse = b.run(mods)
    b.check(out, lse)


@pytest.mark.parametrize("name", ["shared_h16", "shared_h128", "odd_heads", "f32", "odd_window", "one_head"])
def test_rows_do_not_depend_on_grouping_or_batch(mods, name):
    """Every grouping of the batch, and each sequence in a call of its own, gives
    the same bits."""
    c = CASES[name]
    b = Batch(**c, seed=1)
    out, lse = b.run(mods)
    B = len(b.n)
    o1, l1 = b.run(mods, groups=[([i], 0) for i in range(B)])
    assert torch.equal(out, o1) and torch.equal(lse, l1)
    o2, l2 = b.run(mods, groups=[(list(reversed(ms)), sh // 2) for ms, sh in c["groups"]])
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    o3, l3 = b.run(mods, groups=[([B - 1], 0)])
    assert torch.equal(out[B - 1], o3[B - 1]) and torch.equal(lse[B - 1], l3[B - 1])
    # sequences that no group lists are left as they were
    assert (o3[:B - 1] == 3.0).all() and (l3[:B - 1] == 3.0).all()


def test_nothing_visible_gives_zero(mods):
    """A position before the first token, and one without window or entries."""
    for W, dt, D in ((0, "bf16", 128), (4, "f32", 64), (4, "bf16", 128)):
        b = Batch([([0, 1, 2], 0)], [0, 0, 3], 1, 16, D, 8, 4, W, dt, seed=3)
        b.pos = [-1, -3 if W else 2, 24]
        out, lse = b.run(mods)
        assert (out[:2] == 0).all() and (lse[:2] == -float("inf")).all()
        b.check(out, lse)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f32", 64)])
def test_unseen_slots_may_hold_anything(mods, dt, D):
    """NaN and infinity in slots that no query sees (entries behind the last, free
    pages, ring slots outside the window) change nothing; in a sequence's own
    keys they stay in that sequence."""
    b = Batch([([0, 1, 2, 3], 32)], [32, 40, 65, 33], 1, 16, D, 8, 16, 5, dt, seed=4, cap=9)
    clean, cl = b.run(mods)
    pool, ring = b.pool.clone(), b.ring.clone()
    used = torch.zeros(pool.shape[:2], dtype=torch.bool)
    for i in range(4):
        for s in range((b.pos[i] + 1) // b.m):
            used[b.rows[i][s // b.P], s % b.P] = True
        keep = [j % b.cap for j in range(max(0, b.pos[i] - b.W + 1), b.pos[i] + 1)]
        rest = sorted(set(range(b.cap)) - set(keep))
        b.ring[i, rest] = float("nan")
    b.pool[~used] = float("inf")
    out, lse = b.run(mods)
    assert torch.equal(out, clean) and torch.equal(lse, cl)
    # sequence 2's own last entry and newest token
    b.pool[b.rows[2][64 // 16], 0] = float("nan")
    b.ring[2, b.pos[2] % b.cap] = float("inf")
    out, lse = b.run(mods)
    others = [0, 1, 3]
    assert torch.equal(out[others], clean[others]) and torch.equal(lse[others], cl[others])
    assert out[2].isnan().any()
    b.pool, b.ring = pool, ring


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_bad_pages_are_skipped(mods, dt):
    """Ids outside the pool and entries behind held are not followed."""
    b = Batch([([0, 1], 0)], [60, 50], 1, 16, 128, 8, 16, 4, dt, seed=5)
    b.table[0, 1] = 10 ** 6
    b.table[1, 2] = -7
    b.held[1] = 3
    keys = {}
    for i in range(2):
        rows = [x for x in b.rows[i]]
        n = (b.pos[i] + 1) // b.m
        ent = []
        for s in range(min(n, int(b.held[i]) * b.P)):
            pid = int(b.table[i, s // b.P])
            if 0 <= pid < b.pool.shape[0]:
                ent.append(b.pool[pid, s % b.P])
        win = [j % b.cap for j in range(max(0, b.pos[i] - b.W + 1), b.pos[i] + 1)]
        keys[i] = np64(torch.stack(ent + list(b.ring[i, win])))
        assert rows
    out, lse = b.run(mods)
    b.keys = lambda i, t: keys[i]
    b.check(out, lse)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_missing_shared_page_behind_nan(mods, dt):
    """A page that all lack, late enough that its place was first filled with another
    sequence's NaN."""
    b = Batch([([0, 1], 1024)], [1030, 1040], 1, 16, 128, 128, 64, 128, dt, seed=12, max_pages=20)
    b.ring[0] = float("nan")
    b.table[:, 13] = -1
    win = [j % b.cap for j in range(b.pos[1] - b.W + 1, b.pos[1] + 1)]
    ent = b.pool[b.rows[1]].reshape(-1, b.D)[:b.n[1]]
    keys = np64(torch.cat([ent[:13 * 64], ent[14 * 64:], b.ring[1, win]]))
    out, lse = b.run(mods)
    assert out[0].isnan().all()
    b.keys = lambda i, t: keys
    b.check(out, lse, seqs=[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_logits_far_below_zero(mods, dt):
    """All of a row's logits near -300: parts of the split that see none of its keys
    do not set its scale."""
    b = Batch([([0, 1], 128)], [700, 130], 1, 16, 128, 128, 64, 5, dt, seed=8, sink=False)
    k = torch.randn(128, generator=torch.Generator().manual_seed(1)) * 4
    b.pool[:] = (k + 0.05 * b.pool.float()).to(b.pool.dtype)
    b.ring[:] = (k + 0.05 * b.ring.float()).to(b.ring.dtype)
    b.q[:] = (-2 * k + 0.05 * b.q.float()).to(b.q.dtype)
    b.pool[b.rows[1][:2]] = b.pool[b.rows[0][:2]] = float("-inf")     # (never seen below)
    b.table[:, :2] = -1
    keys = {}
    for i in range(2):
        n = (b.pos[i] + 1) // b.m
        win = [j % b.cap for j in range(b.pos[i] - b.W + 1, b.pos[i] + 1)]
        ent = b.pool[b.rows[i]].reshape(-1, b.D)[128:n]
        keys[i] = np64(torch.cat([ent, b.ring[i, win]]))
    out, lse = b.run(mods)
    b.keys = lambda i, t: keys[i]
    assert lse.max() < -200
    b.check(out, lse)


@pytest.mark.parametrize("tau_sign", [1, -1])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_logits_that_grow_by_hundreds(mods, dt, tau_sign):
    """A key far behind the first outweighs all before it by e^500 for one head
    (and is outweighed for the others); so does a window token."""
    b = Batch([([0, 1, 2], 256)], [700, 260, 300], 1, 16, 128, 128, 64, 40, dt, seed=7, scale=4.0)
    b.tau *= tau_sign
    b.pool[b.rows[0][600 // 64], 600 % 64] = 3.0 * tau_sign * b.q[0, 0, 5]
    b.ring[1, b.pos[1] % b.cap] = 3.0 * tau_sign * b.q[1, 0, 9]
    out, lse = b.run(mods)
    b.check(out, lse)
    assert lse[0, 0, 5] > 400 and lse[1, 0, 9] > 400


def test_captured_in_a_graph_and_without_lse(mods):
    """A captured call replays on new positions and pages in the same buffers."""
    ops, paged = mods
    b = Batch([([0, 1, 2], 256)], [256, 300, 400], 1, 64, 128, 16, 16, 32, "bf16", seed=6, extra_pages=4)
    plan = paged.PrefixGroups(b.groups, 3)
    q, pool, tab, held, ring = (x.cuda() for x in (b.q, b.pool, b.table, b.held, b.ring))
    sink = b.sink.cuda()
    pos = torch.tensor(b.pos, dtype=torch.int32).cuda()
    out = torch.zeros_like(q)

    def call():
        ops.hca_prefix_attn_fwd(q, pool, tab, held, plan, ring, sink, b.tau, b.W, pos, out, b.m)
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    out.zero_()
    b.pos = [p + 19 for p in b.pos]
    pos += 19
    g.replay()
    torch.cuda.synchronize()
    _, lse = b.run(mods)
    b.check(out, lse)


def test_two_calls_at_once(mods):
    """Calls on two streams at once, each with its own output, give the bits of calls
    one after the other."""
    ops, paged = mods
    b = Batch([([0, 1, 2], 256)], [256, 300, 400], 1, 64, 128, 16, 16, 32, "bf16", seed=9)
    plan = paged.PrefixGroups(b.groups, 3)
    q, pool, tab, held, ring, sink = (x.cuda() for x in (b.q, b.pool, b.table, b.held, b.ring, b.sink))
    pos = torch.tensor(b.pos, dtype=torch.int32).cuda()
    first, _ = b.run(mods)
    outs = [[torch.zeros_like(q) for _ in range(8)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(8):
        for s, o in zip(streams, outs):
            with torch.cuda.stream(s):
                ops.hca_prefix_attn_fwd(q, pool, tab, held, plan, ring, sink, b.tau, b.W, pos, o[i], b.m)
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert torch.equal(o, first)


@pytest.mark.parametrize("max_pages", [4, 64])
def test_waits_that_run_out_are_reported(mods, max_pages):
    """With a limit of 1 ns the first wait gives up: the call returns, its status word
    says so, and the next call is right."""
    ops, _ = mods
    b = Batch([([0, 1], 64)], [100, 170], 1, 64, 128, 128, 64, 40, "bf16", seed=4, extra_pages=0, max_pages=max_pages)
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    assert ops.device_status() == 0
    ops.set_wait_timeout_ns(1)
    try:
        b.run(mods, status=status)
    finally:
        ops.set_wait_timeout_ns(0)
    assert int(status.item()) & 0xFF == 5, f"status {int(status.item()):#x}"
    assert ops.device_status() == 0
    status.zero_()
    out, lse = b.run(mods, status=status)
    assert int(status.item()) == 0
    b.check(out, lse)
