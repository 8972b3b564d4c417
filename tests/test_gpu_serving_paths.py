"""Paths of the serving kernels that only larger calls, or rarer ones, take: against the
float64 forms."""
import numpy as np
import pytest
import torch

from oracle import serving
from test_gpu_norm_rope import close, freq
from test_gpu_prefix_attn import Batch

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


@pytest.mark.parametrize("dt,m,scale", [("f32", 128, 0.1), ("f32", 100, 1.0), ("bf16", 128, 0.03), ("f32", 16, 3.0)])
def test_gates_that_rise_token_by_token(mods, dt, m, scale):
    """Every token raises the maximum: n exponentials on the way of each sum.  Numerator
    and denominator are each off by (n + 4 u + 3 d + 5 n / 16 + 8) half steps of fp32 of
    their terms (u = n raises, gates within d), the quotient by one; then half a step of the
    type."""
    ops, _ = mods
    B, D, blocks = 2, 64, 3
    T = m * blocks
    g = torch.Generator().manual_seed(m)
    a = torch.randn(B, T, D, generator=g).to(DT[dt])
    z = (scale * torch.arange(T).view(1, T, 1) + 0.01 * scale * torch.rand(B, T, D, generator=g)).to(DT[dt])
    pool = torch.full((B * blocks, 1, D), 9.0, dtype=DT[dt], device="cuda")
    tab = torch.arange(B * blocks, dtype=torch.int32, device="cuda").view(B, blocks)
    ops.hca_paged_append(a.cuda(), z.cuda(), torch.zeros(B, dtype=torch.int32).cuda(), torch.empty(B, 2, 3, D).cuda(), pool, tab,
                         torch.full((B,), blocks, dtype=torch.int32).cuda(), m)
    got = np64(pool).reshape(B, blocks, D)
    for b in range(B):
        for i in range(blocks):
            zb, ab = np64(z[b, i * m:(i + 1) * m]), np64(a[b, i * m:(i + 1) * m])
            w = np.exp(zb - zb.max(0))
            ref, mean = (w * ab).sum(0) / w.sum(0), (w * np.abs(ab)).sum(0) / w.sum(0)
            d = zb.max(0) - zb.min(0)
            tol = (2 * (m + 4 * m + 3 * d + 5 * m / 16 + 8) + 2) * 2.0 ** -24 * mean + torch.finfo(DT[dt]).eps / 2 * np.abs(ref) * 1.001
            assert (np.abs(got[b, i] - ref) <= tol).all()


MAIN = [
    # B, T, H, D, R, dtype, interleaved, inverse: so many tokens that a warp goes through its rows in
    # several turns of loads
    (2, 650, 64, 128, 64, "bf16", True, False), (2, 650, 64, 128, 64, "bf16", False, False),
    (1, 1650, 16, 256, 256, "f32", True, True), (1, 1650, 16, 256, 64, "f32", False, False),
    (3, 801, 64, 64, 32, "bf16", True, False), (3, 801, 64, 64, 64, "f32", False, False),
    (1, 1300, 63, 128, 128, "f32", False, True),
]


@pytest.mark.parametrize("c", MAIN, ids=lambda c: "x".join(map(str, c)))
def test_norm_and_rotation_of_long_runs(mods, c):
    """Rows behind the first turn of loads: a padded batch, keys into a ring shorter than
    the call."""
    ops, _ = mods
    B, T, H, D, R, dt, inter, inv = c
    cap = T // 3
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(B, T, H + 1, D, generator=g).to(DT[dt])
    qw, kw = 1 + 0.3 * torch.randn(D, generator=g), torch.randn(D, generator=g)
    lens = [T - 5 * b for b in range(B)]
    pos = [1000 * b + 3 for b in range(B)]
    f = freq(R)
    xd = x.cuda()
    qo = torch.full((B, T, H, D), 7.0, dtype=DT[dt], device="cuda")
    ring = torch.full((B, cap, D), 7.0, dtype=DT[dt], device="cuda")
    ops.qk_norm_rope(xd[:, :, :H], xd[:, :, H], qo, ring, torch.tensor(pos, dtype=torch.int32).cuda(),
                     inv_freq=torch.tensor(f).cuda(), q_weight=qw.cuda(), kv_weight=kw.cuda(), interleaved=inter, inverse=inv,
                     lens=torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    for b in range(B):
        n, j = lens[b], pos[b] + np.arange(lens[b])
        xb = np64(x[b, :n])
        y = serving.norm_rope(xb[:, :H], 0, None, np64(qw))
        ref = serving.norm_rope(xb[:, :H], j[:, None], f, np64(qw), interleaved=inter, inverse=inv)
        close(np64(qo[b, :n]), ref, y, R, inter, dt)
        assert (qo[b, n:] == 7.0).all()
        last = slice(n - cap, n)
        y = serving.norm_rope(xb[last, H], 0, None, np64(kw))
        ref = serving.norm_rope(xb[last, H], j[last], f, np64(kw), interleaved=inter, inverse=inv)
        close(np64(ring[b, j[last] % cap]), ref, y, R, inter, dt)


def many_groups(count, seed):
    """``count`` groups of one to three sequences, in an order of their own."""
    r = np.random.default_rng(seed)
    sizes = r.integers(1, 4, size=count)
    ids = r.permutation(int(sizes.sum())).tolist()
    groups, n = [], [0] * len(ids)
    for s in sizes:
        ms = [ids.pop() for _ in range(s)]
        shared = 16 * int(r.integers(0, 3))
        for b in ms:
            n[b] = shared + int(r.integers(0, 20))
        groups.append((ms, shared))
    return groups, n


@pytest.mark.parametrize("count,T,H", [(129, 1, 16), (300, 2, 16), (513, 1, 64), (140, 3, 128)])
def test_more_groups_than_one_search_holds(mods, count, T, H):
    groups, n = many_groups(count, count)
    b = Batch(groups, n, T, H, 128, 16, 16, 20, "bf16", seed=count)
    out, lse = b.run(mods)
    b.check(out, lse)


@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("max_pages", [255, 256])
def test_many_heads_in_a_cache_of_many_entries(mods, H, max_pages):
    """Capacities on both sides of 16384 entries: four and eight ranks share a row."""
    b = Batch([([2, 0], 1024), ([1], 0)], [2300, 700, 1030], 1, H, 128, 16, 64, 128, "bf16", seed=H, max_pages=max_pages)
    out, lse = b.run(mods)
    b.check(out, lse)
    o1, l1 = b.run(mods, groups=[([i], 0) for i in range(3)])
    assert torch.equal(out, o1) and torch.equal(lse, l1)
