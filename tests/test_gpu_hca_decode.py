"""The HCA decode driver, its calls run together: prompts loaded into pages,
rows forked, decode steps across block ends, forked rows attended as a group,
against the float64 forms of the same steps.  Tolerances are the layers' own:
2e-2 absolute in bf16 and 1e-5 relative in fp32."""
import math

import numpy as np
import pytest
import torch

from oracle import serving
from long_context_compressed_compress_b200 import configs, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods(cuda_ok):
    from long_context_compressed_compress_b200 import build
    build.build()
    from long_context_compressed_compress_b200 import layer, paged
    return layer, paged


def np64(t):
    return t.detach().cpu().double().numpy()


def bf(x, dt):
    return np64(torch.tensor(x).to(torch.bfloat16 if dt == "bf16" else torch.float32))


class Ref:
    """One row: every token's a, z, kv_raw so far."""

    def __init__(self, cfg, nr, w):
        self.cfg, self.nr, self.w = cfg, nr, w
        self.a, self.z, self.raw = [], [], []

    def feed(self, a, z, raw):
        self.a.append(a), self.z.append(z), self.raw.append(raw)

    def copy(self):
        r = Ref(self.cfg, self.nr, self.w)
        r.a, r.z, r.raw = list(self.a), list(self.z), list(self.raw)
        return r

    def attend(self, q, sink):
        """The attention of the newest token's query."""
        c, n = self.cfg, len(self.a)
        ent, _ = serving.append(np.array(self.z), np.array(self.a), n, c.m)
        raw = np.array(self.raw)
        if self.nr is not None:
            f = np64(self.nr.inv_freq)
            q = bf(serving.norm_rope(q, np.full(len(q), n - 1), f, self.w[0]), c.dtype)
            raw = bf(serving.norm_rope(raw, np.arange(n), f, self.w[1]), c.dtype)
            ent = serving.norm_rope(ent, c.m * np.arange(len(ent)), f, self.w[2])
        keys = np.concatenate([bf(ent, c.dtype), raw[max(0, n - c.W):]])
        out, lse, _ = serving.attend(q, keys, sink, c.tau)
        if self.nr is not None:
            out = serving.norm_rope(bf(out, c.dtype), np.full(len(out), n - 1), f, norm=False, inverse=True)
        return out, lse


def rope(D, R, seed):
    g = torch.Generator().manual_seed(seed)
    return dict(inv_freq=torch.tensor([10000.0 ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64),
                q_weight=1 + 0.1 * torch.randn(D, generator=g), kv_weight=1 + 0.1 * torch.randn(D, generator=g),
                entry_weight=1 + 0.1 * torch.randn(D, generator=g))


def drawn(cfg, R, T, seed):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    x = {k: torch.randn(R, T, cfg.D, generator=g).to(dt) for k in ("a", "kv_raw")}
    x["z"] = (torch.randn(R, T, cfg.D, generator=g) * math.sqrt(2.0)).to(dt)
    x["q"] = torch.randn(R, T, cfg.H, cfg.D, generator=g).to(dt)
    return x


def check(got, ref, dt):
    tol = 2e-2 if dt == "bf16" else 1e-5 * np.maximum(1, np.abs(ref))
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


CASES = [("bf16", 64, 128, 16, 40, False), ("bf16", 16, 128, 8, 128, True), ("f32", 8, 64, 4, 10, True),
         ("f32", 5, 128, 16, 33, False)]


@pytest.mark.parametrize("dt,H,D,m,W,nr", CASES, ids=lambda v: str(v))
def test_load_fork_and_decode(mods, dt, H, D, m, W, nr):
    """A prompt in two pieces of uneven lengths; two forks of it; five steps (crossing
    a block end) with a tokens of their own, as one group; a row freed and
    compacted away; a captured step replayed."""
    layer, paged = mods
    cfg = configs._hca(B=6, T=4096, H=H, D=D, m=m, W=W, dtype=dt, tau=1.0 / math.sqrt(D))
    R, P = cfg.B, 4
    cache = paged.PagedEntries(2, 400, P, D, R, cfg.S, dtype=torch.bfloat16 if dt == "bf16" else torch.float32)
    w = rope(D, 32, 3)
    ropes = layer.NormRope(**{k: v.cuda() for k, v in w.items()}) if nr else None
    sink = torch.randn(H, generator=torch.Generator().manual_seed(1))
    dec = layer.HcaDecode(cfg, cache, sink.cuda(), layer=1, norm_rope=ropes, with_lse=True)
    refs = [Ref(cfg, ropes, [np64(w[k]) for k in ("q_weight", "kv_weight", "entry_weight")]) for _ in range(R)]
    T = 40 * m + 3
    lens = [T, 7, 0, 0, 3 * m, 0]
    cache.reserve(list(range(R)), [n // m + 4 for n in lens])
    cache.free([2, 3, 5])                              # (rows to fork into hold nothing)
    for piece, part in enumerate((T // 3, T - T // 3)):
        x = drawn(cfg, R, part, 10 + piece)
        n = [min(max(v - piece * (T // 3), 0), part) for v in lens]
        dec.load({k: v.cuda() for k, v in x.items() if k != "q"}, torch.tensor(n, dtype=torch.int32).cuda())
        for r in range(R):
            for t in range(n[r]):
                refs[r].feed(*(np64(x[k][r, t]) for k in ("a", "z", "kv_raw")))
    dec.fork([0, 0], [2, 5])
    refs[2], refs[5] = refs[0].copy(), refs[0].copy()
    cache.reserve([2, 5], [T // m + 4, T // m + 4])
    shared = T // m // P * P
    dec.groups = paged.PrefixGroups([([0, 2, 5], shared), ([4], 0), ([1], 0)], R)     # row 3 is idle
    static = {k: torch.zeros_like(v[:, 0]).cuda() for k, v in drawn(cfg, R, 1, 0).items()}
    for step in range(5):
        x = drawn(cfg, R, 1, 100 + step)
        xs = {k: v[:, 0].contiguous() for k, v in x.items()}
        if step == 0:
            xs = {k: torch.cat([v[:2], v[:1], v[3:5], v[:1]]) for k, v in xs.items()}      # the forks repeat their parent
        for k in static:
            static[k].copy_(xs[k])
        if step == 3:
            cache.free([1])
            cache.compact()
        if step < 4:
            out = dec.step(static)
        else:
            dec.capture(static)
            out = dec.replay()
        torch.cuda.synchronize()
        assert cache.status.item() in ((0,) if step < 3 else (0, 6 | 1 << 8))
        for r in (0, 2, 4, 5) + ((1,) if step < 3 else ()):
            refs[r].feed(*(np64(xs[k][r]) for k in ("a", "z", "kv_raw")))
            ref, lse = refs[r].attend(np64(xs["q"][r]), np64(sink))
            check(np64(out[r, 0]), ref, dt)
            # (the logits of rounded entries: |q||k| tau 2^-8 in bf16)
            assert np.abs(np64(dec.lse[r, 0]) - lse).max() <= (0.05 if dt == "bf16" else 1e-4)
        assert (out[3] == 0).all()
        if step == 0:
            assert torch.equal(out[0], out[2]) and torch.equal(out[0], out[5])
            assert torch.equal(dec.lse[0], dec.lse[2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_continues_a_prefill(mods, dt):
    """The last rows of a prefill with norm and rotation, and the same tokens decoded
    behind its prompt: the layers' tolerance; the entries behind both are equal
    to half a step of their type."""
    layer, paged = mods
    D = 128 if dt == "bf16" else 64
    cfg = configs._hca(B=2, T=700, H=16, D=D, m=64, W=128, dtype=dt, tau=1.0 / math.sqrt(D), seed=9, z_std=math.sqrt(2.0))
    x = inputs.layer_inputs(cfg)
    xd = {k: v.cuda() for k, v in x.items()}
    nr = layer.NormRope(**{k: v.cuda() for k, v in rope(D, 64, 4).items()})
    full = layer.HcaPrefill(cfg, norm_rope=nr)
    want = full.run(xd)
    cache = paged.PagedEntries(1, 60, 4, D, 2, 64, dtype=xd["a"].dtype)
    dec = layer.HcaDecode(cfg, cache, xd["sink"], norm_rope=nr)
    cache.reserve([0, 1], [12, 12])
    T0 = 636
    dec.load({k: xd[k][:, :T0].contiguous() for k in ("a", "z", "kv_raw")})
    for t in range(T0, 644):
        out = dec.step({k: xd[k][:, t].contiguous() for k in ("a", "z", "kv_raw", "q")})
        check(np64(out[:, 0]), np64(want[:, t]), dt)
    torch.cuda.synchronize()
    assert cache.status.item() == 0 and dec.pos.tolist() == [644, 644]
    pages = cache.table[:, :3].long()
    got = cache.pool[0][pages].reshape(2, 12, D)[:, :10]
    a, b = np64(got), np64(full.kv_c[:, :10])
    # the pooled value's fp32 error (about 128 roundings of 2^-24), then one rounding each;
    # the prefill rounds its entry before it normalises it: half a step more of the row
    eps = torch.finfo(got.dtype).eps
    assert (np.abs(a - b) <= 1.5 * eps * (np.abs(a) + np.sqrt((a ** 2).mean(-1, keepdims=True)) * 3) + 1e-4 * (dt == "f32")).all()


def test_csa_prefill_with_norm_and_rotation(mods):
    """The CSA layer on normalised, rotated inputs equals the layer that is given
    them so, and its output is that layer's turned back."""
    layer, _ = mods
    from long_context_compressed_compress_b200 import ops
    cfg = configs.scaled(configs.CSA_PREFILL, T=1024, k=64, seed=8)
    xd = {k: v.cuda() for k, v in inputs.layer_inputs(cfg).items()}
    nr = layer.NormRope(**{k: v.cuda() for k, v in rope(cfg.D, 64, 5).items()})
    a = layer.CsaPrefill(cfg, norm_rope=nr)
    got = a.run(xd).clone()
    # the same by hand: entries in place, queries and keys apart
    b = layer.CsaPrefill(cfg)
    b.run(xd)
    idx = torch.empty((cfg.B, cfg.T, cfg.k), dtype=torch.int32, device="cuda")
    b.run(xd, keep_idx=idx)
    pos0 = torch.zeros(cfg.B, dtype=torch.int32, device="cuda")
    kv_c, q, raw = b.kv_c.clone(), torch.empty_like(xd["q"]), torch.empty_like(xd["kv_raw"])
    nr.entries(kv_c, cfg.m, pos0)
    nr.queries(xd["q"], xd["kv_raw"], q, raw, pos0)
    out = torch.empty_like(q)
    ops.sparse_attn_fwd(q, kv_c, idx, raw, xd["sink"], cfg.tau, cfg.W, pos0, out)
    nr.back(out, pos0)
    torch.cuda.synchronize()
    assert torch.equal(got, out)
    assert not torch.equal(got, b.out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_idle_rows_keep_their_outputs(mods, dt):
    """Rows that no group lists keep the output of their last step, rotation and all; a
    captured step goes on with the groups it was captured with."""
    layer, paged = mods
    cfg = configs._hca(B=4, T=256, H=8, D=128, m=16, W=40, dtype=dt, tau=0.1)
    cache = paged.PagedEntries(1, 40, 4, cfg.D, cfg.B, cfg.S, dtype=torch.bfloat16 if dt == "bf16" else torch.float32)
    ropes = layer.NormRope(**{k: v.cuda() for k, v in rope(cfg.D, 32, 3).items()})
    dec = layer.HcaDecode(cfg, cache, norm_rope=ropes)
    cache.reserve([0, 1, 2, 3], [cfg.S] * 4)
    x = drawn(cfg, 4, 50, 5)
    dec.load({k: v.cuda() for k, v in x.items() if k != "q"})
    static = {k: v[:, 0].contiguous().cuda() for k, v in drawn(cfg, 4, 1, 6).items()}
    first = dec.step(static).clone()
    dec.groups = paged.PrefixGroups([([2], 0), ([0], 0)], 4)
    second = dec.step(static).clone()
    assert torch.equal(second[[1, 3]], first[[1, 3]])
    assert not torch.equal(second[[0, 2]], first[[0, 2]])
    dec.capture(static)
    dec.groups = paged.PrefixGroups.singles(4)
    third = dec.replay().clone()
    torch.cuda.synchronize()
    assert cache.status.item() == 0
    assert torch.equal(third[[1, 3]], first[[1, 3]])
    assert not torch.equal(third[[0, 2]], second[[0, 2]])
