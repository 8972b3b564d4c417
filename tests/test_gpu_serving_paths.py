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
