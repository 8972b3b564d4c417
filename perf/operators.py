"""Cases and plain forms of the HCA serving operators.

Four operators that together decode HCA layers for requests sharing a prefix:

``norm_rope``  queries and raw keys normalised per head and rotated by position
               in one pass; the keys go to their window-ring slots.
``append``     new tokens pooled into compressed entries, which are normalised,
               rotated and written to cache pages.
``attn``       attention of a batch over paged entries (leading pages shared by
               groups of sequences), the raw window and the sink.
``pages``      the cache's page operations: free + fork + reserve (``turnover``)
               and ``compact``.

``own`` selects the library's kernels; otherwise ``run`` computes the plain
form with elementary torch operations in 32 bits.  ``exact`` restates each
definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SUB = 16                     # tokens per sub-block of the append carry
_EMPTY = -3.4028234663852886e38   # carry maximum of an empty block


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one request's decode step, 16 heads: latency
        dict(name="norm_rope_decode_1x16", op="norm_rope", B=1, T=1, H=16, D=128, R=64, dtype="bf16",
             pos=1 << 20, cap=128, half=False, fused_qkv=False, ragged=False),
        # decode step of the 32-sequence, 128-head, 1M-context workload
        dict(name="norm_rope_decode_32x128", op="norm_rope", B=32, T=1, H=128, D=128, R=64, dtype="bf16",
             pos=1 << 20, cap=128, half=False, fused_qkv=False, ragged=False),
        # the 32K-token prefill of the 64-head layer
        dict(name="norm_rope_prefill_32k", op="norm_rope", B=1, T=32768, H=64, D=128, R=64, dtype="bf16",
             pos=0, cap=32768, half=False, fused_qkv=False, ragged=False),
        # fp32 layer shapes, a padded batch read in place from a fused q|kv projection
        dict(name="norm_rope_f32_ragged", op="norm_rope", B=3, T=333, H=8, D=64, R=32, dtype="f32",
             pos=700, cap=333, half=True, fused_qkv=True, ragged=True),
        # decode step: one token for each of 32 sequences, some completing a block
        dict(name="append_decode_32", op="append", B=32, T=1, D=128, m=128, P=64, R=64, dtype="bf16", pos=1 << 17),
        # prompts of up to 128K tokens into an empty cache, padded to one length
        dict(name="append_prefill_2x128k", op="append", B=2, T=131072, D=128, m=128, P=64, R=64, dtype="bf16",
             pos=0),
        # one short request, nothing shared
        dict(name="attn_1x16_12k", op="attn", B=1, T=1, H=16, D=128, m=128, P=64, W=128, dtype="bf16", G=1,
             shared=0, owned=100),
        # 32 sequences on one shared 1M-token prefix (8192 entries), 128 heads
        dict(name="attn_32x128_shared_1m", op="attn", B=32, T=1, H=128, D=128, m=128, P=64, W=128, dtype="bf16",
             G=1, shared=8192, owned=37),
        # three groups of 16-head sequences, two tokens a step, ragged suffixes, pages of 16
        dict(name="attn_47x16_3groups", op="attn", B=47, T=2, H=16, D=128, m=64, P=16, W=128, dtype="bf16", G=3,
             shared=2048, owned=300),
        # the fp32 layer's shapes
        dict(name="attn_f32_5x8", op="attn", B=5, T=3, H=8, D=64, m=4, P=16, W=100, dtype="f32", G=2, shared=200,
             owned=61),
        # 64 finished samples replaced by forks of four 8192-entry parents, two layers' pools
        dict(name="pages_turnover_64", op="pages", kind="turnover", parents=4, n=64, N=4096, P=64, D=128, L=2,
             entries=8192, extra=64, live=0.0),
        # half of a two-layer pool freed at random, then compacted
        dict(name="pages_compact_4096", op="pages", kind="compact", parents=0, n=64, N=4096, P=64, D=128, L=2,
             entries=0, extra=0, live=0.5),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attn", "pages"])
    if op == "norm_rope":
        f32 = rng.random() < 0.3
        D = rng.choice([64, 128, 256])
        H = rng.choice([1, 8, 16, 24, 32, 64, 128])
        B = _logint(rng, 1, 64)
        T = 1 if rng.random() < 0.3 else max(1, min(_logint(rng, 1, 32768), (1 << 28) // (B * H * D)))
        half = rng.random() < 0.5
        return dict(op=op, B=B, T=T, H=H, D=D, R=rng.choice([16, 32, D // 2, D]), dtype="f32" if f32 else "bf16",
                    pos=_logint(rng, 1, 1 << 21) - 1, cap=T if T > 1 else rng.choice([100, 128, 256]), half=half,
                    fused_qkv=rng.random() < 0.4, ragged=rng.random() < 0.4)
    if op == "append":
        B = _logint(rng, 1, 64)
        T = 1 if rng.random() < 0.4 else max(1, min(_logint(rng, 1, 131072), 262144 // B))
        return dict(op=op, B=B, T=T, D=rng.choice([64, 128]), m=rng.choice([4, 64, 100, 128]),
                    P=rng.choice([16, 32, 64]), R=rng.choice([0, 32, 64]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    pos=_logint(rng, 1, 1 << 17) - 1)
    if op == "attn":
        f32 = rng.random() < 0.25
        B = _logint(rng, 1, 12 if f32 else 64)
        H = rng.choice([1, 8, 16]) if f32 else rng.choice([8, 16, 32, 40, 64, 128])
        T = rng.choice([1, 1, 1, 2, 3, 4])
        cap = max(16, min(1024 if f32 else 8192, (1 << 25) // (B * H * T)))
        return dict(op=op, B=B, T=T, H=H, D=rng.choice([64, 128]) if f32 else 128, m=rng.choice([4, 64, 128]),
                    P=rng.choice([16, 32, 64]), W=rng.choice([0, 17, 128, 200]), dtype="f32" if f32 else "bf16",
                    G=rng.randint(1, min(B, 5)), shared=_logint(rng, 1, cap) - 1, owned=_logint(rng, 1, 400) - 1)
    P = rng.choice([16, 32, 64])
    L = rng.randint(1, 3)
    N = _logint(rng, 300, 4096 * 2 // L * 64 // P // 2)
    kind = rng.choice(["turnover", "compact"])
    if kind == "compact":
        return dict(op=op, kind=kind, parents=0, n=rng.randint(1, 64), N=N, P=P, D=128, L=L, entries=0, extra=0,
                    live=rng.uniform(0.05, 0.95))
    parents = rng.randint(1, 4)
    n = rng.randint(1, 64)
    extra = rng.randint(0, 2 * P)
    spare = N - n * (2 + (extra + P - 1) // P)
    while spare < parents:
        n, extra = max(1, n // 2), extra // 2
        spare = N - n * (2 + (extra + P - 1) // P)
    return dict(op=op, kind=kind, parents=parents, n=n, N=N, P=P, D=128, L=L,
                entries=_logint(rng, 1, max(2, min(8192, spare // parents * P))), extra=extra, live=0.0)


# --------------------------------------------------------------------- inputs
class _Draw:
    """Seeded draws on the GPU and on the host."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.r = np.random.default_rng(seed)

    def normal(self, shape, dtype, scale=1.0, mean=0.0):
        x = torch.randn(shape, generator=self.g, device="cuda", dtype=torch.float32)
        return x.mul_(scale).add_(mean).to(dtype)

    def ints(self, lo, hi, n):
        return [int(v) for v in self.r.integers(lo, hi, size=n)]


def _dev(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32).cuda()


def _inv_freq(R, base=10000.0):
    """Angle per position of each rotated pair, in 64 bits."""
    if R == 0:
        return None
    return torch.tensor([base ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64).cuda()


def _pages_for(d, need, P, N):
    """Page tables of sequences holding ``need`` pages each, ids scattered over the pool."""
    order = [int(v) for v in d.r.permutation(N)]
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n])
        at += n
    return rows


def _table(rows, maxp):
    t = np.full((len(rows), maxp), -1, np.int64)
    for i, r in enumerate(rows):
        t[i, :len(r)] = r
    return t


def _norm_rope_inputs(c, d):
    dt = _DT[c["dtype"]]
    B, T, H, D = c["B"], c["T"], c["H"], c["D"]
    s = {"c": c}
    if c["fused_qkv"]:
        # one projection's output [B, T, (H + 1) D]: H query heads, then the shared key
        x = d.normal((B, T, H + 1, D), dt, 1.7)
        s["q"], s["kv"] = x[:, :, :H], x[:, :, H]
    else:
        s["q"], s["kv"] = d.normal((B, T, H, D), dt, 1.7), d.normal((B, T, D), dt, 0.6)
    s["qw"] = d.normal((D,), torch.float32, 0.1, 1.0)
    s["kw"] = d.normal((D,), torch.float32, 0.1, 1.0)
    s["pos_h"] = [c["pos"] + v for v in (d.ints(0, 4000, B) if T == 1 else [0] * B)]
    s["lens_h"] = d.ints(1, T + 1, B) if c["ragged"] else [T] * B
    s["pos"] = _dev(s["pos_h"])
    s["lens"] = _dev(s["lens_h"]) if c["ragged"] else None
    s["freq"] = _inv_freq(c["R"])
    s["q_out"] = torch.zeros((B, T, H, D), dtype=dt, device="cuda")
    s["ring"] = torch.zeros((B, c["cap"], D), dtype=dt, device="cuda")
    return s


def _append_inputs(c, d):
    dt = _DT[c["dtype"]]
    B, T, D, m, P = c["B"], c["T"], c["D"], c["m"], c["P"]
    s = {"c": c, "a": d.normal((B, T, D), dt), "z": d.normal((B, T, D), dt, math.sqrt(2.0))}
    s["lens_h"] = d.ints(max(1, T - T // 8), T + 1, B)
    s["pos_h"] = [c["pos"] + v for v in (d.ints(0, m, B) if c["pos"] else [0] * B)]
    if T == 1 and B > 1:
        s["pos_h"][0] = (c["pos"] // m + 1) * m - 1    # one sequence completes its block
    s["pos"], s["lens"] = _dev(s["pos_h"]), _dev(s["lens_h"])
    # the carry of the tokens already in each sequence's open block
    o = torch.tensor([p % m for p in s["pos_h"]], device="cuda")
    za = d.normal((B, m, D), torch.float32, math.sqrt(2.0))
    aa = d.normal((B, m, D), torch.float32)
    t = torch.arange(m, device="cuda")[None, :, None]
    sub0 = (o // _SUB * _SUB)[:, None, None]
    parts = []
    for lo, hi in ((0 * sub0, sub0), (sub0, o[:, None, None])):
        w = (t >= lo) & (t < hi)
        M = torch.where(w, za, torch.full_like(za, _EMPTY)).amax(1)
        e = torch.where(w, torch.exp(za - M[:, None]), torch.zeros_like(za))
        parts.append(torch.stack([M, e.sum(1), (e * aa).sum(1)], 1))
    s["carry"] = torch.stack(parts, 1).contiguous()           # [B, 2, 3, D]
    s["carry_out"] = torch.zeros_like(s["carry"])
    total = [(p + n) // m for p, n in zip(s["pos_h"], s["lens_h"])]
    need = [(n + P - 1) // P for n in total]
    maxp = ((c["pos"] + m + T) // m + P - 1) // P
    N = B * maxp + 7
    s["rows_h"] = _pages_for(d, need, P, N)
    s["table"] = _dev(_table(s["rows_h"], maxp))
    s["held"] = _dev(need)
    s["pool"] = torch.zeros((N, P, D), dtype=dt, device="cuda")
    s["w"] = d.normal((D,), torch.float32, 0.1, 1.0)
    s["freq"] = _inv_freq(c["R"])
    return s


def _attn_inputs(c, d):
    dt = _DT[c["dtype"]]
    B, T, H, D, m, P, W = c["B"], c["T"], c["H"], c["D"], c["m"], c["P"], c["W"]
    s = {"c": c}
    perm = [int(v) for v in d.r.permutation(B)]
    cuts = sorted(int(v) for v in d.r.choice(np.arange(1, B), size=c["G"] - 1, replace=False)) if c["G"] > 1 else []
    members = [perm[a:b] for a, b in zip([0] + cuts, cuts + [B])]
    s["groups_h"] = []
    rows, pos = [None] * B, [0] * B
    need, shared_pages = [], []
    n_of = {}
    for g, ms in enumerate(members):
        sh = max(0, c["shared"] - (g * c["shared"]) // 3)
        shp = sh // P                       # whole pages are shared
        s["groups_h"].append((ms, shp * P))
        shared_pages.append(shp)
        need.append(shp)
        for b in ms:
            n_of[b] = sh + int(d.r.integers(0, c["owned"] + 1))
            need.append((n_of[b] + 1 + P - 1) // P + 1 - shp)
    N = sum(need) + 3
    got = _pages_for(d, need, P, N)
    at = 0
    for g, ms in enumerate(members):
        common = got[at]
        at += 1
        for b in ms:
            rows[b] = common + got[at]
            at += 1
            pos[b] = n_of[b] * m - 1 + int(d.r.integers(0, m)) if n_of[b] else int(d.r.integers(0, max(1, m - T)))
    s["pos_h"], s["rows_h"] = pos, rows
    s["pos"] = _dev(pos)
    s["table"] = _dev(_table(rows, max(len(r) for r in rows)))
    s["held"] = _dev([len(r) for r in rows])
    s["pool"] = d.normal((N, P, D), dt)
    s["q"] = d.normal((B, T, H, D), dt)
    s["cap"] = max(1, W + T - 1)
    s["ring"] = d.normal((B, s["cap"], D), dt)
    s["sink"] = d.normal((H,), torch.float32)
    s["tau"] = 1.0 / math.sqrt(D)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((B, T, H), dtype=torch.float32, device="cuda")
    # what the plain form indexes with
    s["plain"] = [(torch.tensor(ms).cuda(), sh, max((pos[b] + T) // m for b in ms) - sh)
                  for ms, sh in s["groups_h"]]
    if own:
        from long_context_compressed_compress_b200 import paged
        s["plan"] = paged.PrefixGroups(s["groups_h"], B)
    return s


def _pages_inputs(c, d):
    L, N, P, D = c["L"], c["N"], c["P"], c["D"]
    s = {"c": c, "pool": d.normal((L, N, P, D), torch.bfloat16)}
    if c["kind"] == "turnover":
        base = c["entries"]
        ents = [max(1, base - v) for v in d.ints(0, max(1, base // 8), c["parents"])]
        need = [(e + P - 1) // P for e in ents]
        par = _pages_for(d, need, P, N)
        s["src_h"] = d.ints(0, c["parents"], c["n"])
        s["dst_h"] = [c["parents"] + int(v) for v in d.r.permutation(c["n"])]
        s["len_h"] = [max(1, ents[p] - v) for p, v in zip(s["src_h"], d.ints(0, 3 * P, c["n"]))]
        s["grow_h"] = [n + v for n, v in zip(s["len_h"], d.ints(0, c["extra"] + 1, c["n"]))]
        maxp = (base + c["extra"] + P - 1) // P
        rows = par + [[] for _ in range(c["n"])]
        for k in ("src", "dst", "len", "grow"):
            s[k] = _dev(s[k + "_h"])
        # the forks whose last page is partial, for the plain form
        s["tail"] = torch.tensor([i for i, n in enumerate(s["len_h"]) if n % P], dtype=torch.long).cuda()
    else:
        live = max(1, int(N * c["live"]))
        per = live // c["n"]
        need = [per + (i < live % c["n"]) for i in range(c["n"])]
        for i in range(1, c["n"], 2):       # uneven lengths, some of them zero
            v = int(d.r.integers(0, need[i] + 1))
            need[i - 1], need[i] = need[i - 1] + v, need[i] - v
        rows = _pages_for(d, need, P, N)
        for i in range(1, c["n"]):          # a quarter of the rows share a neighbour's first pages
            if i % 4 == 0:
                k = len(rows[i - 1]) // 2
                rows[i] = rows[i - 1][:k] + rows[i]
        maxp = 3 * per + 4
    ref = np.zeros(N, np.int64)
    for r in rows:
        for p in r:
            ref[p] += 1
    s["rows_h"] = rows
    s["table"], s["held"], s["ref"] = _dev(_table(rows, maxp)), _dev([len(r) for r in rows]), _dev(ref)
    s["table_out"], s["ref_out"] = torch.zeros_like(s["table"]), torch.zeros_like(s["ref"])
    s["n_live"] = torch.zeros((1,), dtype=torch.int32, device="cuda")
    if own:
        from long_context_compressed_compress_b200 import ops
        s["ws"] = torch.empty((ops.kv_pages_workspace_size(N, max(1, c["n"])) // 4,), dtype=torch.int32,
                              device="cuda")
    return s


def prepare(case, seed):
    d = _Draw(seed)
    make = {"norm_rope": _norm_rope_inputs, "append": _append_inputs, "attn": _attn_inputs, "pages": _pages_inputs}
    return make[case["op"]](case, d)


# ---------------------------------------------------------------- plain forms
def _rope_plain(y, angle, R, half, dim):
    """Rotate the last R of y's dims; angle [..., R/2] broadcasts against them."""
    if R == 0:
        return y
    cs, sn = torch.cos(angle).float(), torch.sin(angle).float()
    x = y[..., dim - R:]
    if half:
        x0, x1 = x[..., :R // 2], x[..., R // 2:]
        r = torch.cat([x0 * cs - x1 * sn, x0 * sn + x1 * cs], -1)
    else:
        x0, x1 = x[..., 0::2], x[..., 1::2]
        r = torch.stack([x0 * cs - x1 * sn, x0 * sn + x1 * cs], -1).flatten(-2)
    return torch.cat([y[..., :dim - R], r], -1)


def _norm_plain(x, w, eps=1e-6):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def _norm_rope_plain(s):
    c = s["c"]
    B, T, D, R, cap = c["B"], c["T"], c["D"], c["R"], c["cap"]
    j = s["pos"].long()[:, None] + torch.arange(T, device="cuda")
    ang = j.double()[..., None] * s["freq"]
    q = _rope_plain(_norm_plain(s["q"], s["qw"]), ang[:, :, None], R, c["half"], D).to(s["q_out"].dtype)
    k = _rope_plain(_norm_plain(s["kv"], s["kw"]), ang, R, c["half"], D).to(s["ring"].dtype)
    if s["lens"] is None:
        s["q_out"].copy_(q)
        s["ring"].scatter_(1, (j % cap)[..., None].expand(B, T, D), k)
    else:
        ok = torch.arange(T, device="cuda") < s["lens"][:, None]
        s["q_out"].copy_(torch.where(ok[..., None, None], q, s["q_out"]))
        at = (j % cap)[..., None].expand(B, T, D)
        s["ring"].scatter_(1, at, torch.where(ok[..., None], k, s["ring"].gather(1, at)))
    return s["q_out"], s["ring"]


def _join(x, y):
    """(M, Z, A) of the union of two token sets, stacked on dim -2."""
    M = torch.maximum(x[..., 0, :], y[..., 0, :])
    ex, ey = torch.exp(x[..., 0, :] - M), torch.exp(y[..., 0, :] - M)
    return torch.stack([M, x[..., 1, :] * ex + y[..., 1, :] * ey, x[..., 2, :] * ex + y[..., 2, :] * ey], -2)


def _join_over(part, dim, ok=None):
    """(M, Z, A) of the union along ``dim`` (of the sets that ``ok`` keeps)."""
    if ok is not None:
        empty = torch.zeros_like(part)
        empty[..., 0, :] = _EMPTY
        part = torch.where(ok, part, empty)
    M = part[..., 0, :].amax(dim, keepdim=True)
    e = torch.exp(part[..., 0, :] - M)
    return torch.stack([M.squeeze(dim), (part[..., 1, :] * e).sum(dim), (part[..., 2, :] * e).sum(dim)], -2)


def _append_plain(s):
    c = s["c"]
    B, T, D, m, P, R = c["B"], c["T"], c["D"], c["m"], c["P"], c["R"]
    nsub = (m + _SUB - 1) // _SUB
    nb = (T + 2 * m - 2) // m + 1             # blocks any sequence's tokens can touch, and the open one
    o = s["pos"].long() % m
    slot = torch.arange(nb, device="cuda")[:, None] * m + torch.arange(nsub * _SUB, device="cuda")
    inblk = (torch.arange(nsub * _SUB, device="cuda") < m)[None, None]
    t = slot[None] - o[:, None, None]
    ok = (t >= 0) & (t < s["lens"].long()[:, None, None]) & inblk
    t = t.clamp(0, T - 1).reshape(B, -1, 1).expand(-1, -1, D)
    z = s["z"].gather(1, t).float().view(B, nb, nsub, _SUB, D)
    a = s["a"].gather(1, t).float().view(B, nb, nsub, _SUB, D)
    ok = ok.view(B, nb, nsub, _SUB, 1)
    M = torch.where(ok, z, torch.full_like(z, _EMPTY)).amax(3)
    e = torch.where(ok, torch.exp(z - M[:, :, :, None]), torch.zeros_like(z))
    part = torch.stack([M, e.sum(3), (e * a).sum(3)], 3)          # [B, nb, nsub, 3, D]
    # the carry joins the first block
    first = torch.arange(nsub, device="cuda")[None] == (o // _SUB)[:, None]
    part[:, 0] = torch.where(first[:, :, None, None], _join(part[:, 0], s["carry"][:, 1:2]), part[:, 0])
    whole = _join_over(part, 2)
    whole[:, 0] = _join(whole[:, 0], s["carry"][:, 0])
    # the entries of the completed blocks
    y = whole[..., 2, :] / whole[..., 1, :].clamp_min(1e-30)
    blk = s["pos"].long()[:, None] // m + torch.arange(nb, device="cuda")
    end = s["pos"].long() + s["lens"].long()
    done = (blk + 1) * m <= end[:, None]
    y = _norm_plain(y, s["w"])
    if R:
        y = _rope_plain(y, (blk * m).double()[..., None] * s["freq"], R, False, D)
    y = y.to(s["pool"].dtype)
    maxp = s["table"].shape[1]
    page = s["table"].long().gather(1, (blk // P).clamp(max=maxp - 1))
    flat = s["pool"].view(-1, D)
    # entries that are not complete go to the last slot's old value
    at = torch.where(done, page * P + blk % P, torch.full_like(page, -1))
    keep = torch.cat([flat, flat.new_zeros((1, D))])
    keep.index_put_((torch.where(at < 0, torch.full_like(at, flat.shape[0]), at),), y)
    flat.copy_(keep[:-1])
    # the carry after the last token: the open block's complete sub-blocks, and the open sub-block
    eo = end % m
    last = (end // m - s["pos"].long() // m)
    p_last = part[torch.arange(B, device="cuda"), last]            # [B, nsub, 3, D]
    i = torch.arange(nsub, device="cuda")[None, :, None, None]
    at = (eo // _SUB)[:, None, None, None]
    blkst = _join_over(p_last, 1, i < at)
    blkst = torch.where((last == 0)[:, None, None], _join(blkst, s["carry"][:, 0]), blkst)
    sub = _join_over(p_last, 1, i == at)
    s["carry_out"].copy_(torch.stack([blkst, sub], 1))
    return (s["pool"], *s["carry_out"].unbind(2))


def _attn_plain(s):
    c = s["c"]
    B, T, H, D, m, P, W = c["B"], c["T"], c["H"], c["D"], c["m"], c["P"], c["W"]
    for ms, sh, n_own in s["plain"]:
        n = ms.numel()
        q = s["q"][ms].float() * s["tau"]                                   # [n, T, H, D]
        p = s["pos"].long()[ms][:, None] + torch.arange(T, device="cuda")     # [n, T]
        logits, values = [], []
        if sh:
            tab = s["table"][ms[0], :sh // P].long()
            k = s["pool"][tab].view(-1, D).float()                            # [sh, D]
            logits.append(q.reshape(-1, D) @ k.t())
            values.append(lambda w, k=k: w @ k)
        if n_own > 0:
            e = sh + torch.arange(n_own, device="cuda")
            pid = s["table"][ms].long()[:, e // P]
            k = s["pool"][pid, e % P].float()                                 # [n, n_own, D]
            lg = q.reshape(n, T * H, D) @ k.transpose(1, 2)
            ok = (e < ((p + 1) // m)[..., None])[:, :, None].expand(n, T, H, n_own).reshape(n, T * H, n_own)
            logits.append(torch.where(ok, lg, torch.full_like(lg, -math.inf)).view(n * T * H, -1))
            values.append(lambda w, k=k: (w.view(n, T * H, -1) @ k).view(-1, D))
        if W:
            j = p[..., None] - torch.arange(W, device="cuda")                 # [n, T, W]
            k = s["ring"][ms[:, None, None], j.clamp_min(0) % s["cap"]].float()
            lg = q @ k.transpose(2, 3)
            lg = torch.where((j >= 0)[:, :, None], lg, torch.full_like(lg, -math.inf))
            logits.append(lg.view(n * T * H, -1))
            values.append(lambda w, k=k: (w.view(n, T, H, -1) @ k).view(-1, D))
        sg = s["sink"].repeat(n * T)
        M = sg
        for lg in logits:
            M = torch.maximum(M, lg.amax(1))
        den, acc = torch.zeros_like(M), torch.zeros((n * T * H, D), device="cuda")
        for lg, val in zip(logits, values):
            w = torch.exp(lg - M[:, None])
            den = den + w.sum(1)
            acc = acc + val(w)
        o = acc / (den + torch.exp(sg - M))[:, None]
        s["out"][ms] = o.view(n, T, H, D).to(s["out"].dtype)
        s["lse"][ms] = (M + torch.log(den)).view(n, T, H)
    return s["out"], s["lse"]


def _turnover_plain(s):
    c = s["c"]
    P, n = c["P"], c["n"]
    table, held, ref = s["table"], s["held"], s["ref"]
    maxp, N = table.shape[1], ref.shape[0]
    col = torch.arange(maxp, device="cuda")
    dst, src = s["dst"].long(), s["src"].long()

    def count(rows, upto, sign):
        ok = col < upto[:, None]
        ids = torch.where(ok, table[rows].long(), torch.zeros_like(ok, dtype=torch.long))
        ref.index_add_(0, ids.view(-1), (ok * sign).int().view(-1))

    # free
    count(dst, held[dst], -1)
    table[dst] = -1
    held[dst] = 0
    # fork: whole pages shared, the tail copied to the lowest free pages
    whole, tail = s["len"].long() // P, s["len"].long() % P
    free = torch.argsort((ref > 0).int(), stable=True)
    part = tail > 0
    new = free[(torch.cumsum(part.int(), 0) - 1).clamp_min(0)]
    row = torch.where(col < whole[:, None], table[src].long(), torch.full((n, maxp), -1, device="cuda"))
    row = torch.where((col == whole[:, None]) & part[:, None], new[:, None], row)
    table[dst] = row.int()
    held[dst] = (whole + part).int()
    i = s["tail"]
    if i.numel():
        old = table[src[i], whole[i]].long()
        rows = torch.arange(P, device="cuda") < tail[i][:, None]
        s["pool"][:, new[i]] = torch.where(rows[..., None], s["pool"][:, old], s["pool"][:, new[i]])
    count(dst, held[dst], 1)
    # reserve
    want = (s["grow"].long() + P - 1) // P
    add = (want - held[dst]).clamp_min(0)
    free = torch.argsort((ref > 0).int(), stable=True)
    at = torch.cumsum(add, 0) - add
    more = (col >= held[dst][:, None]) & (col < want[:, None])
    ids = free[(at[:, None] + col - held[dst][:, None]).clamp(0, N - 1)]
    row = torch.where(more, ids, table[dst].long())
    table[dst] = row.int()
    ref.index_add_(0, torch.where(more, row, torch.zeros_like(row)).view(-1), more.int().view(-1))
    held[dst] = torch.maximum(held[dst], want.int())
    return s["pool"], table, held, ref


def _compact_plain(s):
    ref, table, pool = s["ref"], s["table"], s["pool"]
    N = ref.shape[0]
    live = ref > 0
    n_live = live.sum()
    ids = torch.arange(N, device="cuda")
    mover = live & (ids >= n_live)
    hole = ~live & (ids < n_live)
    holes = torch.argsort((~hole).int(), stable=True)              # holes first, ascending
    movers = torch.argsort((~mover).int(), stable=True)
    new = torch.where(mover, holes[(torch.cumsum(mover.int(), 0) - 1).clamp_min(0)], ids)
    src = torch.where(hole, movers[(torch.cumsum(hole.int(), 0) - 1).clamp_min(0)], ids)
    pool.copy_(pool[:, src])
    s["table_out"].copy_(torch.where(table >= 0, new[table.long().clamp_min(0)].int(), table))
    s["ref_out"].copy_(torch.where(ids < n_live, ref[src], torch.zeros_like(ref)))
    s["n_live"].copy_(n_live.view(1))
    return pool, s["table_out"], s["ref_out"], s["n_live"]


def _run_own(s):
    from long_context_compressed_compress_b200 import ops
    c = s["c"]
    if c["op"] == "norm_rope":
        ops.qk_norm_rope(s["q"], s["kv"], s["q_out"], s["ring"], s["pos"], inv_freq=s["freq"], q_weight=s["qw"],
                         kv_weight=s["kw"], eps=1e-6, interleaved=not c["half"], lens=s["lens"])
        return s["q_out"], s["ring"]
    if c["op"] == "append":
        ops.hca_paged_append(s["a"], s["z"], s["pos"], s["carry"], s["pool"], s["table"], s["held"], c["m"],
                             carry_out=s["carry_out"], lens=s["lens"], norm=True, weight=s["w"], eps=1e-6,
                             inv_freq=s["freq"])
        return (s["pool"], *s["carry_out"].unbind(2))
    if c["op"] == "attn":
        ops.hca_prefix_attn_fwd(s["q"], s["pool"], s["table"], s["held"], s["plan"], s["ring"], s["sink"], s["tau"],
                                c["W"], s["pos"], s["out"], c["m"], lse=s["lse"])
        return s["out"], s["lse"]
    if c["kind"] == "turnover":
        ops.kv_pages_free(s["dst"], s["table"], s["held"], s["ref"])
        ops.kv_pages_fork(s["src"], s["dst"], s["len"], s["pool"], s["table"], s["held"], s["ref"], s["ws"])
        ops.kv_pages_reserve(s["dst"], s["grow"], c["P"], s["table"], s["held"], s["ref"], s["ws"])
        return s["pool"], s["table"], s["held"], s["ref"]
    ops.kv_pages_compact(s["pool"], s["table"], s["held"], s["ref"], s["n_live"], s["ws"], table_out=s["table_out"],
                         refcount_out=s["ref_out"])
    return s["pool"], s["table_out"], s["ref_out"], s["n_live"]


def run(state):
    if own:
        return _run_own(state)
    op = state["c"]["op"]
    if op == "norm_rope":
        return _norm_rope_plain(state)
    if op == "append":
        return _append_plain(state)
    if op == "attn":
        return _attn_plain(state)
    return _turnover_plain(state) if state["c"]["kind"] == "turnover" else _compact_plain(state)


# ----------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "pages":
        page = c["P"] * c["D"] * 2 * c["L"]
        if c["kind"] == "turnover":
            # half a tail page per fork, read and written; the new rows' ids
            pages = c["entries"] // c["P"] + 1
            return {"bytes": c["n"] * page + 8 * c["n"] * pages + 4 * c["N"], "flops": 0}
        live = int(c["N"] * c["live"])
        moved = live * (c["N"] - live) / c["N"]
        return {"bytes": int(2 * moved * page + 8 * c["N"] + 8 * live), "flops": 0}
    es = 4 if c["dtype"] == "f32" else 2
    B, T, D = c["B"], c["T"], c["D"]
    if c["op"] == "norm_rope":
        f = 0.5 if c["ragged"] else 1.0
        el = f * B * T * (c["H"] + 1) * D
        return {"bytes": int(2 * es * el), "flops": int(5 * el)}
    if c["op"] == "append":
        el = (1.0 if T == 1 else 15.0 / 16.0) * B * T * D
        return {"bytes": int(es * (2 * el + el / c["m"]) + 2 * 24 * B * D), "flops": int(6 * el)}
    H, W, G = c["H"], c["W"], c["G"]
    sh = [max(0, c["shared"] - (g * c["shared"]) // 3) for g in range(G)]
    mean = sum(sh) / G
    rows = mean + c["owned"] / 2 + W
    byt = es * (2 * B * T * H * D + D * (sum(sh) + B * (c["owned"] / 2 + W + T - 1))) + 4 * B * T * H
    return {"bytes": int(byt), "flops": int(4 * D * H * B * T * rows)}


# ---------------------------------------------------------------------- exact
def _rope64(y, pos, freq, half):
    """y [n, D] in 64 bits rotated at positions pos [n] as complex numbers."""
    if freq is None:
        return y
    h = freq.numel()
    x = y[:, -2 * h:]
    z = torch.complex(x[:, :h], x[:, h:]) if half else torch.view_as_complex(x.reshape(-1, h, 2).contiguous())
    ang = pos.double()[:, None] * freq
    z = z * torch.polar(torch.ones_like(ang), ang)
    r = torch.cat([z.real, z.imag], 1) if half else torch.view_as_real(z).reshape(-1, 2 * h)
    return torch.cat([y[:, :-2 * h], r], 1)


def _unit64(x, w, eps=1e-6):
    x = x.double()
    return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + eps) * w.double()


def _norm_rope_exact(s):
    c = s["c"]
    B, T, H, D = c["B"], c["T"], c["H"], c["D"]
    q = torch.zeros((B, T, H, D), dtype=torch.float64, device="cuda")
    ring = torch.zeros((B, c["cap"], D), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 24) // (H * D))
    for b in range(B):
        for t0 in range(0, s["lens_h"][b], step):
            t1 = min(t0 + step, s["lens_h"][b])
            j = torch.arange(t0, t1, device="cuda") + s["pos_h"][b]
            x = _unit64(s["q"][b, t0:t1], s["qw"]).reshape(-1, D)
            q[b, t0:t1] = _rope64(x, j.repeat_interleave(H), s["freq"], c["half"]).view(-1, H, D)
            ring[b, j % c["cap"]] = _rope64(_unit64(s["kv"][b, t0:t1], s["kw"]), j, s["freq"], c["half"])
    return q, ring


def _append_exact(s):
    c = s["c"]
    B, D, m, P = c["B"], c["D"], c["m"], c["P"]
    pool = s["pool"].double()
    carry = torch.zeros((B, 2, 3, D), dtype=torch.float64, device="cuda")
    carry[:, :, 0] = _EMPTY
    for b in range(B):
        p0, n = s["pos_h"][b], s["lens_h"][b]
        z, a = s["z"][b, :n].double(), s["a"][b, :n].double()
        old = s["carry"][b].double()

        def pooled(lo, hi, with_old):
            """(M, Z, A) of the tokens at positions [lo, hi), and of the carry's parts."""
            zz, aa = z[lo - p0:hi - p0], a[lo - p0:hi - p0]
            tops = ([zz.amax(0)] if hi > lo else []) + [o[0] for o in with_old]
            M = torch.stack(tops).amax(0) if tops else torch.full((D,), _EMPTY, dtype=torch.float64, device="cuda")
            e = torch.exp(zz - M)
            Z, A = e.sum(0), (e * aa).sum(0)
            for o in with_old:
                Z, A = Z + o[1] * torch.exp(o[0] - M), A + o[2] * torch.exp(o[0] - M)
            return M, Z, A

        end = p0 + n
        first, last = p0 // m, end // m
        blocks = list(range(first, last))
        rest = blocks
        out = []
        if blocks and p0 % m:
            M, Z, A = pooled(p0, (first + 1) * m, [old[0], old[1]])
            out.append(A[None] / Z[None])
            rest = blocks[1:]
        if rest:
            lo = rest[0] * m - p0
            zb, ab = (v[lo:lo + len(rest) * m].view(-1, m, D) for v in (z, a))
            out.append((torch.softmax(zb, 1) * ab).sum(1))
        if blocks:
            e = _unit64(torch.cat(out), s["w"])
            blk = torch.tensor(blocks, device="cuda")
            e = _rope64(e, blk * m, s["freq"], False)
            pid = torch.tensor([s["rows_h"][b][i // P] for i in blocks], device="cuda")
            pool[pid, blk % P] = e
        lo = max(p0, last * m)
        mid = last * m + (end - last * m) // _SUB * _SUB
        cur = last == first                                   # the carry's block is still open
        sub_open = cur and p0 >= mid                          # and so is its sub-block
        if mid > last * m:
            carry[b, 0] = torch.stack(pooled(lo, max(lo, mid), [old[0]] + ([] if sub_open else [old[1]]) if cur else []))
        if end > mid:
            carry[b, 1] = torch.stack(pooled(max(lo, mid), end, [old[1]] if sub_open else []))
    return (pool, *carry.unbind(2))


def _attn_exact(s):
    c = s["c"]
    B, T, H, D, m, P, W = c["B"], c["T"], c["H"], c["D"], c["m"], c["P"], c["W"]
    out = torch.zeros((B, T, H, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, T, H), dtype=torch.float64, device="cuda")
    sink = s["sink"].double()
    for b in range(B):
        pages = torch.tensor(s["rows_h"][b], device="cuda")
        ent = s["pool"][pages].reshape(-1, D)
        for t in range(T):
            p = s["pos_h"][b] + t
            win = torch.tensor([j % s["cap"] for j in range(max(0, p - W + 1), p + 1)] if W else [], dtype=torch.long,
                               device="cuda")
            k = torch.cat([ent[:(p + 1) // m], s["ring"][b, win]]).double()
            lg = s["q"][b, t].double() @ k.t() * s["tau"]
            lse[b, t] = torch.logsumexp(lg, 1)
            out[b, t] = torch.softmax(torch.cat([lg, sink[:, None]], 1), 1)[:, :-1] @ k
    return out, lse


def _turnover_exact(s):
    P, N = s["c"]["P"], s["c"]["N"]
    rows = [list(r) for r in s["rows_h"]]
    pool = s["pool"].double()
    ref = np.zeros(N, np.int64)
    for r in rows:
        for p in r:
            ref[p] += 1

    def take():
        p = int(np.argmax(ref == 0))
        ref[p] = 1
        return p

    tails = []
    for a, b, n in zip(s["src_h"], s["dst_h"], s["len_h"]):
        rows[b] = rows[a][:n // P]
        tails.append((rows[a][n // P], n % P) if n % P else None)
        for p in rows[b]:
            ref[p] += 1
    for b, t in zip(s["dst_h"], tails):
        if t:
            p = take()
            pool[:, p, :t[1]] = pool[:, t[0], :t[1]]
            rows[b].append(p)
    for b, n in zip(s["dst_h"], s["grow_h"]):
        while len(rows[b]) * P < n:
            rows[b].append(take())
    t = _dev(_table(rows, s["table"].shape[1])).long()
    return pool, t, _dev([len(r) for r in rows]).long(), _dev(ref).long()


def _compact_exact(s):
    N = s["c"]["N"]
    ref = s["ref"].cpu().numpy().astype(np.int64)
    n_live = int((ref > 0).sum())
    holes = iter([i for i in range(n_live) if ref[i] == 0])
    new = {i: (i if i < n_live else next(holes)) for i in range(N) if ref[i] > 0}
    pool = s["pool"].double()
    out = np.zeros(N, np.int64)
    for i, k in new.items():
        out[k] = ref[i]
    moved = [(i, k) for i, k in new.items() if i != k]
    if moved:
        a, b = torch.tensor(moved, device="cuda").t()
        pool[:, b] = pool[:, a]
    rows = [[new[p] for p in r] for r in s["rows_h"]]
    return (pool, _dev(_table(rows, s["table"].shape[1])).long(), _dev(out).long(),
            torch.tensor([n_live], device="cuda"))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _norm_rope_exact(s)
    if case["op"] == "append":
        return _append_exact(s)
    if case["op"] == "attn":
        return _attn_exact(s)
    return _turnover_exact(s) if case["kind"] == "turnover" else _compact_exact(s)
