"""qk_norm_rope against its formula in float64.

Tolerances.  fp32 error of one output, relative to |y0| + |y1| of its rotated
pair: the sum of squares adds 8 terms a lane and up to 5 shuffle steps (13 half
steps, halved by the root), the root 2, the two products 2, cos and sin 3 each,
the rotation's two roundings: below 24 half steps of 2^-24.  The stored value
then rounds by half a step of its type."""
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


def freq(R, base=10000.0):
    return np.array([base ** (-2.0 * i / R) for i in range(R // 2)]) if R else None


def close(got, ref, y, R, interleaved, dt):
    """|got - ref| within the derived bound; y is the row before rotation."""
    pair = np.abs(y)
    if R:
        r = pair[..., -R:]
        if interleaved:
            s = r[..., 0::2] + r[..., 1::2]
            s = np.repeat(s, 2, -1)
        else:
            s = r[..., :R // 2] + r[..., R // 2:]
            s = np.concatenate([s, s], -1)
        pair = np.concatenate([pair[..., :-R], s], -1)
    tol = 24 * 2.0 ** -24 * pair + (torch.finfo(DT[dt]).eps / 2) * np.abs(ref) * 1.001 + 1e-30
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - ref).max())


def np64(t):
    return t.detach().cpu().double().numpy()


CASES = [
    # B, T, H, D, R, dtype, pos0, cap, interleaved, inverse, norm, step
    (1, 1, 16, 128, 64, "bf16", 1 << 20, 128, True, False, True, 1),
    (3, 1, 128, 128, 64, "bf16", 1000003, 100, True, False, True, 1),
    (2, 37, 8, 64, 32, "f32", 5, 37, False, False, True, 1),
    (1, 300, 1, 256, 256, "bf16", 0, 64, False, True, True, 1),
    (2, 5, 3, 64, 16, "bf16", 127, 4, True, False, True, 4),
    (1, 9, 5, 128, 128, "f32", 1 << 21, 9, True, True, False, 128),
    (1, 3, 7, 128, 0, "f32", 0, 3, True, False, True, 1),
    (2, 2, 40, 256, 240, "f32", 12345, 2, False, False, True, 1),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "x".join(map(str, c)))
def test_against_formula(ops, c):
    B, T, H, D, R, dt, pos0, cap, inter, inv, norm, step = c
    g = torch.Generator().manual_seed(hash(c[:5]) % 1000 + 1)
    q = (torch.randn(B, T, H, D, generator=g) * 3).to(DT[dt])
    kv = torch.randn(B, T, D, generator=g).to(DT[dt])
    qw, kw = torch.randn(D, generator=g), torch.randn(D, generator=g)
    p = torch.tensor([pos0 + 3 * b for b in range(B)], dtype=torch.int32)
    f = freq(R)
    q_out = torch.full((B, T, H, D), 7.0, dtype=DT[dt]).cuda()
    ring = torch.full((B, cap, D), 7.0, dtype=DT[dt]).cuda()
    ops.qk_norm_rope(q.cuda(), kv.cuda(), q_out, ring, p.cuda(), inv_freq=None if f is None else torch.tensor(f).cuda(),
                     q_weight=qw.cuda(), kv_weight=kw.cuda(), norm=norm, interleaved=inter, inverse=inv, pos_step=step)
    torch.cuda.synchronize()
    j = p.numpy()[:, None] + np.arange(T)
    kwargs = dict(norm=norm)
    yq = serving.norm_rope(np64(q), 0, None, np64(qw), **kwargs)
    yk = serving.norm_rope(np64(kv), 0, None, np64(kw), **kwargs)
    kwargs.update(interleaved=inter, inverse=inv)
    rq = serving.norm_rope(np64(q), (j * step)[..., None], f, np64(qw), **kwargs)
    rk = serving.norm_rope(np64(kv), j * step, f, np64(kw), **kwargs)
    close(np64(q_out), rq, yq, R, inter, dt)
    got = np64(ring)
    for b in range(B):
        live = range(max(0, T - cap), T)
        for t in live:
            close(got[b, j[b, t] % cap], rk[b, t], yk[b, t], R, inter, dt)
        other = sorted(set(range(cap)) - {int(j[b, t] % cap) for t in live})
        assert (got[b, other] == 7.0).all()


def test_padded_batch_from_a_fused_projection(ops):
    """q and kv are slices of one [B, T, (H + 1) D] tensor; tokens behind a
    row's length leave both outputs as they were (a length of 0 and one above T
    among them)."""
    B, T, H, D, R = 4, 11, 6, 64, 32
    x = torch.randn(B, T, H + 1, D, generator=torch.Generator().manual_seed(1)).cuda()
    lens = torch.tensor([0, 11, 4, 99], dtype=torch.int32).cuda()
    p = torch.tensor([3, 0, 250, 8], dtype=torch.int32).cuda()
    f = freq(R)
    qo, ko = torch.full((B, T, H, D), 5.0).cuda(), torch.full((B, T, D), 5.0).cuda()
    ops.qk_norm_rope(x[:, :, :H], x[:, :, H], qo, ko, p, inv_freq=torch.tensor(f).cuda(), lens=lens)
    torch.cuda.synchronize()
    xn, pn = np64(x), p.cpu().numpy()
    for b, n in enumerate([0, 11, 4, 11]):
        j = pn[b] + np.arange(n)
        ref = serving.norm_rope(xn[b, :n], j[:, None], f)
        y = serving.norm_rope(xn[b, :n], 0)
        close(np64(qo)[b, :n], ref[:, :H], y[:, :H], R, True, "f32")
        close(np64(ko)[b, j % T], ref[:, H], y[:, H], R, True, "f32")
        assert (qo[b, n:] == 5.0).all()
        rest = sorted(set(range(T)) - set((j % T).tolist()))
        assert (ko[b, rest] == 5.0).all()


def test_in_place_and_inverse_give_the_input_back(ops):
    """Rotating in place and back by the inverse gives the input up to the two
    roundings (kv in place keeps its rows where they are, whatever q_pos0)."""
    B, T, H, D = 2, 9, 4, 128
    g = torch.Generator().manual_seed(2)
    q0, k0 = torch.randn(B, T, H, D, generator=g).cuda(), torch.randn(B, T, D, generator=g).cuda()
    q, k = q0.clone(), k0.clone()
    f = torch.tensor(freq(64)).cuda()
    p = torch.tensor([77, 100001], dtype=torch.int32).cuda()
    ops.qk_norm_rope(q, k, q, k, p, inv_freq=f, norm=False)
    assert not torch.equal(q, q0) and not torch.equal(k, k0)
    ops.qk_norm_rope(q, k, q, k, p, inv_freq=f, norm=False, inverse=True)
    torch.cuda.synchronize()
    # two rotations, each a few half steps of the pair's magnitude
    for a, b in ((q, q0), (k, k0)):
        assert (a - b).abs().max().item() <= 16 * 2.0 ** -24 * 2 * b.abs().max().item()


def test_one_of_the_pair_alone_and_a_side_stream(ops):
    B, T, H, D = 2, 4, 8, 128
    g = torch.Generator().manual_seed(3)
    q, k = torch.randn(B, T, H, D, generator=g).bfloat16().cuda(), torch.randn(B, T, D, generator=g).bfloat16().cuda()
    p = torch.zeros(B, dtype=torch.int32).cuda()
    f = torch.tensor(freq(64)).cuda()
    q1, k1 = torch.empty_like(q), torch.empty_like(k)
    ops.qk_norm_rope(q, k, q1, k1, p, inv_freq=f)
    q2, k2 = torch.empty_like(q), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ops.qk_norm_rope(q, None, q2, None, p, inv_freq=f, stream=s)
    with torch.cuda.stream(s):
        ops.qk_norm_rope(None, k, None, k2, p, inv_freq=f)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(q1, q2) and torch.equal(k1, k2)


def test_nan_and_zero_rows_stay_in_their_rows(ops):
    B, T, H, D = 1, 2, 4, 64
    q = torch.ones(B, T, H, D).cuda()
    q[0, 0, 1] = 0.0
    q[0, 1, 2, 5] = float("nan")
    out = torch.empty_like(q)
    ops.qk_norm_rope(q, None, out, None, torch.zeros(1, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert (out[0, 0, 1] == 0).all() and out[0, 1, 2].isnan().all()
    keep = torch.ones(T, H, dtype=torch.bool)
    keep[1, 2] = False
    assert out[0][keep.cuda()].isfinite().all()


@pytest.mark.parametrize("R", [0, 16, "D"])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,H,kv", [(64, 0, 1), (64, 1, 1), (64, 1, 0), (64, 2, 0), (128, 0, 1), (128, 1, 0)])
def test_few_rows_a_token(ops, D, H, kv, dt, inter, R):
    """Tokens of one or two rows, several of them in a warp: an odd number, some behind
    their row's length, a ring shorter than the call."""
    B, T, cap = 3, 7, 5
    R = D if R == "D" else R
    lens, pos = [7, 0, 6], [1 << 20, 4, 250]
    g = torch.Generator().manual_seed(D + H)
    q = torch.randn(B, T, H, D, generator=g).to(DT[dt]) if H else None
    k = torch.randn(B, T, D, generator=g).to(DT[dt]) if kv else None
    qw, kw = torch.randn(D, generator=g), torch.randn(D, generator=g)
    qo = torch.full((B, T, H, D), 7.0, dtype=DT[dt]).cuda() if H else None
    ring = torch.full((B, cap, D), 7.0, dtype=DT[dt]).cuda() if kv else None
    f = freq(R)
    ops.qk_norm_rope(None if q is None else q.cuda(), None if k is None else k.cuda(), qo, ring,
                     torch.tensor(pos, dtype=torch.int32).cuda(), q_weight=qw.cuda(), kv_weight=kw.cuda(),
                     inv_freq=None if f is None else torch.tensor(f).cuda(), interleaved=inter,
                     lens=torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    for b in range(B):
        j, n = pos[b] + np.arange(T), lens[b]
        if H:
            y = serving.norm_rope(np64(q[b]), 0, None, np64(qw))
            close(np64(qo[b, :n]), serving.norm_rope(np64(q[b]), j[:, None], f, np64(qw), interleaved=inter)[:n], y[:n],
                  R, inter, dt)
            assert (np64(qo[b, n:]) == 7.0).all()
        if kv:
            y = serving.norm_rope(np64(k[b]), 0, None, np64(kw))
            ref = serving.norm_rope(np64(k[b]), j, f, np64(kw), interleaved=inter)
            live = range(max(0, n - cap), n)
            for t in live:
                close(np64(ring[b, j[t] % cap]), ref[t], y[t], R, inter, dt)
            other = sorted(set(range(cap)) - {int(j[t] % cap) for t in live})
            assert (np64(ring[b, other]) == 7.0).all()
