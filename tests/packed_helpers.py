"""Random caches and 64-bit references of the packed-batch operators.

The reference reads the cache's planes (codes, scales, minima, dense values) as stored and
restates the definitions in float64 numpy, loops over sequences and KV heads; it shares
nothing with the CUDA path.
"""

import math

import numpy as np
import torch

# half a step of each type, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def logical(t, table):
    """[pool, Hkv, page, ...] in logical order [B, Hkv, T_cap, ...] (or as it is)."""
    if table is None:
        return t
    B, P = table.shape
    g = t[table.reshape(-1).long()].reshape((B, P) + tuple(t.shape[1:])).transpose(1, 2)
    return g.reshape((B, t.shape[1], P * t.shape[2]) + tuple(t.shape[3:]))


class Cache:
    """A cache with random contents: `hq` the framework's handle, `planes` its tensors."""

    def __init__(self, seed, B, Hkv, T_cap, d, r, vmode="dense", v_dtype=torch.bfloat16, page=0,
                 kmode="token", spread=1.0, device="cuda"):
        from bit_decode_attention_sm_b200 import headq
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.d, self.r, self.vmode, self.kmode = B, Hkv, d, r, vmode, kmode
        self.table = None
        lead = (B, Hkv, T_cap)
        if page:
            per = -(-T_cap // page)
            pool = B * per + 3
            self.table = torch.from_numpy(rng.permutation(pool)[:B * per].reshape(B, per).astype(np.int32))
            lead = (pool, Hkv, page)
        ng = d // min(32, d)
        ks = lead + (ng,) if kmode == "token" else lead[:2] + (lead[2] // 64, d)

        def codes(w):
            return torch.randint(0, 256, lead + (w,), generator=g, dtype=torch.uint8)

        def scales(shape, mul):
            return mul * torch.exp(0.4 * torch.randn(shape, generator=g))

        p = dict(k_codes=codes(d // 4), k_scale=scales(ks, 0.8 * spread))
        p["k_min"] = -1.5 * p["k_scale"] + 0.3 * spread * torch.randn(ks, generator=g)
        if r:
            z = codes(r // 2)
            p["z_codes"] = torch.where((z & 0xF) == 8, z ^ 0x8, z)          # level -8 is unused
            p["z_codes"] = torch.where((p["z_codes"] >> 4) == 8, p["z_codes"] ^ 0x80, p["z_codes"])
            p["z_scale"] = scales(lead, 0.15 * spread)
        if vmode == "2bit":
            p["v_codes"] = codes(d // 4)
            p["v_scale"] = scales(lead + (ng,), 0.7)
            p["v_min"] = -1.5 * p["v_scale"] + 0.2 * torch.randn(lead + (ng,), generator=g)
        else:
            p["v"] = torch.randn(lead + (d,), generator=g).to(v_dtype)
        self.planes = {n: t.to(device) for n, t in p.items()}
        if self.table is not None:
            self.table = self.table.to(device)
        self.U = torch.from_numpy(np.stack([np.linalg.qr(rng.standard_normal((d, max(r, 1))))[0]
                                            for _ in range(Hkv)])[:, :, :r].astype(np.float32).copy()).to(device)
        self.hq = headq.HeadQCache.from_planes(kmode=kmode, block_table=self.table, **self.planes)

    def parts(self):
        """(base keys, z^, values, U), float64 in logical order [B, Hkv, T_cap, .]."""
        p = {n: t for n, t in self.planes.items()}
        d = self.d
        gs = min(32, d)

        def two_bit(codes, scale, mn, channel=False):
            c = logical(codes, self.table).cpu().numpy()
            s, m = (logical(x, self.table).cpu().numpy().astype(np.float64) for x in (scale, mn))
            ch = np.arange(d)
            code = (c[..., ch // 4] >> (2 * (ch % 4))) & 3
            if channel:  # one row of d per block of 64 tokens
                blk = np.arange(c.shape[2]) // 64
                return m[:, :, blk] + code * s[:, :, blk]
            return m[..., ch // gs] + code * s[..., ch // gs]

        k = two_bit(p["k_codes"], p["k_scale"], p["k_min"], self.kmode == "channel")
        if self.r:
            zc = logical(p["z_codes"], self.table).cpu().numpy().astype(np.int64)
            i = np.arange(self.r)
            w = (zc[..., i // 2] >> (4 * (i % 2))) & 15
            w = np.where(w > 7, w - 16, w)
            z = w * logical(p["z_scale"], self.table).cpu().numpy().astype(np.float64)[..., None]
        else:
            z = np.zeros(k.shape[:3] + (0,))
        if self.vmode == "2bit":
            v = two_bit(p["v_codes"], p["v_scale"], p["v_min"])
        else:
            v = logical(p["v"], self.table).double().cpu().numpy()
        return k, z, v, self.U.double().cpu().numpy()


def spans(counts, lens):
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return torch.from_numpy(cu).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def tree_masks(rng, B, n):
    """Random draft trees: every node sees itself and its ancestors."""
    m = np.zeros((B, n, n), bool)
    for b in range(B):
        for i in range(n):
            p = rng.integers(-1, i) if i else -1
            if p >= 0:
                m[b, i] = m[b, p]
            m[b, i, i] = True
    return m


def tensor_core(cache, q_dtype):
    """Whether headq_tree_attn documents the tensor-core path for these shapes."""
    return (q_dtype == torch.bfloat16 and cache.d in (64, 128) and cache.r in (0, 8, 16)
            and (cache.vmode == "2bit" or cache.planes["v"].dtype == torch.bfloat16))


def ref_tree(cache, q, counts, lens, mask, sm=None, sigma=1.0):
    """(out, lse, tolerance of out, tolerance of lse), float64, [rows, Hq, .].

    The tolerances count the roundings that the operator documents, to first order in each
    and doubled: with weights w and |v| the readout moves by at most
        sum_j w_j (|ds_j| + sum_i w_i |ds_i|) |v_j|   for logit errors ds,
        e_p sum_j w_j |v_j|                           for weights rounded by e_p,
        e_v sum_j w_j |v_j|                           for values rounded by e_v,
    and is then rounded to its type."""
    k, z, v, U = cache.parts()
    qn = q.double().cpu().numpy()
    rows, Hq, d = qn.shape
    G = Hq // cache.Hkv
    sm = 1.0 / math.sqrt(d) if sm is None else sm
    mma = tensor_core(cache, q.dtype)
    f16, f32 = 2.0 ** -11, 2.0 ** -24
    out, lse = np.zeros((rows, Hq, d)), np.full((rows, Hq), -np.inf)
    tol, tl = np.zeros((rows, Hq, d)), np.full((rows, Hq), 1e-6)
    r0 = 0
    for b, (c, T) in enumerate(zip(counts, lens)):
        if c <= T:
            see = np.ones((c, T), bool)
            see[:, T - c:] = np.tril(np.ones((c, c), bool)) if mask is None else mask[b][:c, :c]
            for h in range(Hq if c else 0):
                kv = h // G
                qh = qn[r0:r0 + c, h]
                with np.errstate(invalid="ignore"):
                    qu = qh @ U[kv]
                    s = sm * (qh @ k[b, kv, :T].T + sigma * (qu @ z[b, kv, :T].T))
                    base = abs(sm) * (np.abs(qh) @ np.abs(k[b, kv, :T]).T)
                    side = abs(sigma * sm) * (np.abs(qh) @ np.abs(U[kv]) @ np.abs(z[b, kv, :T]).T)
                ds = (d + cache.r + 16) * f32 * (base + side) + 4 * f32 * np.abs(s)
                if mma:
                    ds = ds + f16 * base + 2 * f16 * side
                e_p = 2.0 ** -7 if mma else (T + 16) * f32
                e_v = HALF[torch.bfloat16] if mma and cache.vmode == "2bit" else 2 * f32
                for i in range(c):
                    j = np.flatnonzero(see[i])
                    if not len(j):
                        continue
                    x = s[i, j]
                    m = x.max()
                    w = np.exp(x - m)
                    tot = w.sum()
                    lse[r0 + i, h] = m + np.log(tot)
                    w = w / tot
                    vj, dj = v[b, kv, j], ds[i, j]
                    o = w @ vj
                    out[r0 + i, h] = o
                    a = w @ np.abs(vj)
                    first = (w * dj) @ np.abs(vj) + (w @ dj) * a + (e_p + e_v) * a
                    tol[r0 + i, h] = 2 * first + HALF[q.dtype] * np.abs(o) + 1e-30
                    tl[r0 + i, h] = 2 * (w @ dj) + (T + 16) * f32 + f32 * abs(lse[r0 + i, h]) + 2.0 ** -20
        r0 += c
    return out, lse, tol, tl


def check_tree(got, lse, ref, rows=None):
    out, rl, tol, tl = ref
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - out) <= tol)
    assert not bad.any(), "out: %d of %d outside, worst %.3g times its tolerance" % (
        bad.sum(), bad.size, np.nanmax(np.abs(g - out) / tol))
    if lse is not None:
        l = lse.double().cpu().numpy()
        fin = np.isfinite(rl)
        assert (l[~fin] == rl[~fin]).all()
        assert (np.abs(l - rl)[fin] <= tl[fin]).all(), np.max((np.abs(l - rl) / tl)[fin])
