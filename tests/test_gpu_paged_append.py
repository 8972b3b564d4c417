"""hca_paged_append against the pooling in float64, and its bit-exactness
under any split of the tokens over calls.

Tolerances.  One entry is sum w a / sum w over n tokens.  A weight's exponent
d = z - M rounds by |d| 2^-24, expf by 2 steps of 2^-23; each of up to n - 1
further tokens (and n / 16 joins) rescales Z and A with one rounding and one
exponential each: relative error of numerator and denominator below
(2 n + 4 |d| + 16) 2^-24 each.  Then half a step of the stored type."""
import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ops(cuda_ok):
    from long_context_compressed_compress_b200 import build
    build.build()
    from long_context_compressed_compress_b200 import ops
    return ops


def np64(t):
    return t.detach().cpu().double().numpy()


class Cache:
    def __init__(self, B, D, m, P, total, dt, seed=0, N=None):
        n = max(1, -(-(total // m + 1) // P))
        self.N = N or B * n + 3
        perm = np.random.default_rng(seed).permutation(self.N)[:B * n].reshape(B, n)
        self.ids = perm
        self.table = torch.tensor(perm, dtype=torch.int32).cuda()
        self.held = torch.full((B,), n, dtype=torch.int32).cuda()
        self.pool = torch.full((self.N, P, D), 9.0, dtype=DT[dt]).cuda()
        self.carry = torch.full((B, 2, 3, D), float("nan")).cuda()    # not read before a block opens
        self.P = P

    def entries(self, b, n):
        e = self.pool[torch.tensor(self.ids[b]).cuda()].reshape(-1, self.pool.shape[2])
        return e[:n], e[n:]


def feed(ops, c, a, z, cuts, m, start=0, **kw):
    """The tokens of every sequence, in calls that end at ``cuts``."""
    B = a.shape[0]
    at = start
    for end in cuts:
        ops.hca_paged_append(a[:, at - start:end - start].contiguous(), z[:, at - start:end - start].contiguous(),
                             torch.full((B,), at, dtype=torch.int32).cuda(), c.carry, c.pool, c.table, c.held, m, **kw)
        at = end
    torch.cuda.synchronize()


CASES = [
    # B, total, D, m, P, dtype
    (2, 1, 128, 128, 64, "bf16"), (1, 128, 128, 128, 16, "f32"), (2, 777, 128, 128, 4, "bf16"),
    (3, 333, 64, 100, 16, "f32"), (1, 70, 256, 4, 16, "bf16"), (2, 515, 128, 64, 3, "f32"), (1, 9, 64, 1, 2, "f32"),
    (1, 700, 64, 300, 16, "f32"), (1, 40, 128, 17, 16, "bf16"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_whole_prompt_and_its_splits(ops, case):
    """One call against the formula; token by token, and in uneven pieces, the
    same bits."""
    B, total, D, m, P, dt = case
    g = torch.Generator().manual_seed(total)
    a = torch.randn(B, total, D, generator=g).to(DT[dt])
    z = (torch.randn(B, total, D, generator=g) * 1.5).to(DT[dt])
    ad, zd = a.cuda(), z.cuda()
    one = Cache(B, D, m, P, total, dt)
    feed(ops, one, ad, zd, [total], m)
    for b in range(B):
        ent, parts = serving.append(np64(z[b]), np64(a[b]), total, m)
        got, rest = one.entries(b, len(ent))
        assert (rest == 9.0).all()
        za, aa = np64(z[b]), np.abs(np64(a[b]))
        for i, e in enumerate(ent):
            zb = za[i * m:(i + 1) * m]
            d = (zb.max(0) - zb).max(0)
            w = np.exp(zb - zb.max(0))
            mean = (w * aa[i * m:(i + 1) * m]).sum(0) / w.sum(0)
            tol = 2 * (2 * m + 4 * d + 16) * 2.0 ** -24 * mean + torch.finfo(DT[dt]).eps / 2 * np.abs(e) * 1.001
            assert (np.abs(np64(got[i]) - e) <= tol).all()
        cr = np64(one.carry[b])
        assert (cr[:, 0] == parts[:, 0]).all()
        mag = serving.append(np64(z[b]), aa, total, m)[1]
        assert (np.abs(cr[:, 1:] - parts[:, 1:]) <= (2 * m + 64) * 2.0 ** -24 * mag[:, 1:]).all()
    rng = np.random.default_rng(total)
    cuts = sorted({int(v) for v in rng.integers(1, total + 1, size=7)} | {total})
    splits = [cuts]
    if total <= 200:
        splits.append(list(range(1, total + 1)))
    for sp in splits:
        two = Cache(B, D, m, P, total, dt)
        feed(ops, two, ad, zd, sp, m)
        assert torch.equal(one.pool, two.pool)
        assert torch.equal(one.carry, two.carry)


def test_padded_batch_lengths_and_separate_carry(ops):
    """Lengths of 0, 1, T and beyond; sequences at different positions; the carry
    given apart from its result, which stays as it was."""
    B, T, D, m, P = 4, 150, 128, 128, 16
    g = torch.Generator().manual_seed(5)
    a, z = torch.randn(B, 600, D, generator=g), torch.randn(B, 600, D, generator=g)
    pos, lens = [0, 127, 250, 300], [0, 1, 150, 999]
    c = Cache(B, D, m, P, 600, "f32")
    for b in range(B):        # what each has seen before
        if pos[b]:
            at = torch.zeros(B, dtype=torch.int32)
            ln = torch.zeros(B, dtype=torch.int32)
            ln[b] = pos[b]
            ops.hca_paged_append(a[:, :pos[b]].contiguous().cuda(), z[:, :pos[b]].contiguous().cuda(), at.cuda(), c.carry,
                                 c.pool, c.table, c.held, m, lens=ln.cuda())
    x = torch.stack([a[b, pos[b]:pos[b] + T] for b in range(B)]).cuda()
    y = torch.stack([z[b, pos[b]:pos[b] + T] for b in range(B)]).cuda()
    before = c.carry.clone()
    out = torch.zeros_like(c.carry)
    ops.hca_paged_append(x, y, torch.tensor(pos, dtype=torch.int32).cuda(), c.carry, c.pool, c.table, c.held, m,
                         carry_out=out, lens=torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.equal(before[1:], c.carry[1:])
    for b, n in enumerate([0, 1, 150, 150]):
        end = pos[b] + n
        ent, parts = serving.append(np64(z[b, :end]), np64(a[b, :end]), end, m)
        got, rest = c.entries(b, len(ent))
        assert (rest == 9.0).all()
        if len(ent):
            assert np.abs(np64(got) - ent).max() <= 2 * (2 * m + 64) * 2.0 ** -24 * np.abs(np64(a)).max()
        if n:
            assert (np64(out[b])[:, 0] == parts[:, 0]).all()
            mag = serving.append(np64(z[b, :end]), np.abs(np64(a[b, :end])), end, m)[1]
            assert (np.abs(np64(out[b]) - parts)[:, 1:] <= (2 * m + 64) * 2.0 ** -24 * mag[:, 1:]).all()


def test_gates_of_minus_infinity_and_the_lowest_value(ops):
    """A -inf gate drops its token, NaN and inf values behind it included; a block
    of them gives 0; gates at the type's lowest value weigh equally."""
    D, m = 64, 16
    g = torch.Generator().manual_seed(6)
    a, z = torch.randn(1, 64, D, generator=g), torch.randn(1, 64, D, generator=g)
    z[0, 3] = -float("inf")
    a[0, 3] = float("nan")
    z[0, 7], a[0, 7] = -float("inf"), float("inf")
    z[0, 16:32] = -float("inf")
    z[0, 32:48] = torch.finfo(torch.float32).min
    c = Cache(1, D, m, 2, 64, "f32")
    feed(ops, c, a.cuda(), z.cuda(), [5, 64], m)
    ent, _ = serving.append(np64(z[0]), np64(a[0]), 64, m)
    got = np64(c.entries(0, 4)[0])
    assert np.isfinite(got).all() and (got[1] == 0).all()
    assert np.abs(got - ent).max() <= 2 * (2 * m + 64) * 2.0 ** -24 * 5
    assert np.abs(got[2] - np64(a[0, 32:48]).mean(0)).max() <= 32 * 2.0 ** -24 * 5


def test_norm_and_rotation_of_entries(ops):
    """The entry is normalised and rotated at m * index, from the fp32 pooled
    value; the rotation's derived bound on top of the pooling's."""
    B, total, D, m, R = 2, 450, 128, 64, 64
    g = torch.Generator().manual_seed(7)
    a, z = torch.randn(B, total, D, generator=g), torch.randn(B, total, D, generator=g)
    w = torch.randn(D, generator=g)
    f = np.array([10000.0 ** (-2.0 * i / R) for i in range(R // 2)])
    for inter in (True, False):
        c = Cache(B, D, m, 4, total, "f32")
        feed(ops, c, a.cuda(), z.cuda(), [100, 300, total], m, norm=True, weight=w.cuda(),
             inv_freq=torch.tensor(f).cuda(), interleaved=inter)
        for b in range(B):
            ent, _ = serving.append(np64(z[b]), np64(a[b]), total, m)
            ref = serving.norm_rope(ent, m * np.arange(len(ent)), f, np64(w), interleaved=inter)
            got = np64(c.entries(b, len(ent))[0])
            rms = np.sqrt((ent ** 2).mean(-1, keepdims=True))
            # the pooling's relative error (of mean |a| < 2) over the row's rms, times |w| of the pair
            tol = (2 * (2 * m + 64) * 2 / rms + 40) * 2.0 ** -24 * 2 * np.abs(np64(w)).max() * 3
            assert (np.abs(got - ref) <= tol).all()


def test_entries_without_a_page_are_dropped_and_reported(ops):
    """Short held counts, ids outside the pool and a full table: the entry is not
    written, the status says so, the carry goes on."""
    B, D, m, P = 3, 64, 4, 2
    a = torch.randn(B, 16, D, generator=torch.Generator().manual_seed(8)).cuda()
    table = torch.tensor([[0, 1], [2, 99], [-5, 3]], dtype=torch.int32).cuda()
    held = torch.tensor([1, 2, 2], dtype=torch.int32).cuda()
    pool = torch.full((4, P, D), 9.0).cuda()
    carry = torch.zeros(B, 2, 3, D).cuda()
    st = torch.zeros(1, dtype=torch.int32).cuda()
    ops.hca_paged_append(a, a, torch.zeros(B, dtype=torch.int32).cuda(), carry, pool, table, held, m, status=st)
    torch.cuda.synchronize()
    assert st.item() == 6 | (1 << 8)
    assert (pool[1] == 9.0).all()                      # row 0 lists it but does not hold it
    assert (pool[0] != 9.0).any() and (pool[2] != 9.0).any() and (pool[3] != 9.0).any()


def test_negative_positions_only_copy_the_carry(ops):
    D = 64
    a = torch.randn(2, 8, D, generator=torch.Generator().manual_seed(9)).cuda()
    c = Cache(2, D, 4, 4, 8, "f32")
    c.carry = torch.randn(2, 2, 3, D, generator=torch.Generator().manual_seed(10)).cuda()
    out = torch.zeros_like(c.carry)
    ops.hca_paged_append(a, a, torch.tensor([-1, -8], dtype=torch.int32).cuda(), c.carry, c.pool, c.table, c.held, 4,
                         carry_out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, c.carry) and (c.pool == 9.0).all()
