"""Speculative decoding over a HeadQ cache: what each operator computes and what it is timed on.

Three operators, in the order a serving loop runs them on one layer:

  write   the new tokens of every sequence (a packed batch of ragged length, optionally
          gathered: the accepted nodes of a draft tree) are encoded into the cache at each
          sequence's own positions; then read back, which is what prefill attention sees
  read    a span of cached tokens of every sequence is decoded to dense keys and values
  tree    every drafted token attends over its sequence's cached prefix and over those
          drafted tokens that its row of the tree mask names

`run` computes them in plain torch where `own` is false, and through the package's entry
points where it is true.  Sequence b's tokens are rows cu[b] .. cu[b+1] of the packed
tensors and lie at the last cu[b+1] - cu[b] of its lens[b] cached positions.
"""

import math

import numpy as np
import torch

own = False

# Layers of the repository's workloads (bit_decode_attention_sm_b200/configs.py)
_LAYERS = {
    "tiny": dict(B=1, Hq=16, Hkv=1, d=64, T=512, r=8, kv="f32", vmode="dense"),
    "mha": dict(B=8, Hq=12, Hkv=12, d=64, T=2048, r=8, kv="bf16", vmode="dense"),
    "gqa": dict(B=16, Hq=28, Hkv=4, d=128, T=8192, r=16, kv="bf16", vmode="dense"),
    "longctx": dict(B=1, Hq=32, Hkv=8, d=128, T=131072, r=16, kv="bf16", vmode="dense"),
    "fullkv2bit": dict(B=64, Hq=28, Hkv=4, d=128, T=4096, r=16, kv="bf16", vmode="2bit"),
}


def _case(op, layer, n, **kw):
    c = dict(op=op, n=n, ragged=False, page=0, gather=False, **_LAYERS[layer])
    c.update(kw)
    return c


def listed():
    return [
        # an 8-token draft on the small fp32 layer: latency
        dict(name="tree_tiny_fp32", **_case("tree", "tiny", 8)),
        # drafts of up to 11 tokens, sequences and drafts of different lengths
        dict(name="tree_mha_ragged", **_case("tree", "mha", 11, ragged=True)),
        # no draft: the single new token of each sequence
        dict(name="tree_gqa_single", **_case("tree", "gqa", 1)),
        # a 16-node draft tree per sequence on pages of 256 tokens
        dict(name="tree_gqa_16_paged", **_case("tree", "gqa", 16, page=256)),
        # a 32-node tree per sequence over 2-bit keys and values
        dict(name="tree_fullkv2bit_32", **_case("tree", "fullkv2bit", 32)),
        # one long sequence verified with a 64-node tree: the largest
        dict(name="tree_longctx_64", **_case("tree", "longctx", 64)),
        # after verification: the accepted tokens of 32-node trees, picked out of the draft
        dict(name="write_accepted", **_case("write", "fullkv2bit", 32, ragged=True, gather=True)),
        # chunked prefill of prompts of different lengths into pages
        dict(name="write_ragged_paged", **_case("write", "gqa", 2048, ragged=True, page=64)),
        # a prefill chunk at the end of a long sequence
        dict(name="write_longctx_chunk", **_case("write", "longctx", 8192)),
        # the tail of every sequence, for a check or a transfer
        dict(name="read_mha_tail", **_case("read", "mha", 37)),
        # whole prefixes of different lengths, 2-bit keys and values
        dict(name="read_fullkv2bit_ragged", **_case("read", "fullkv2bit", 4096, ragged=True)),
        # a whole long sequence, for dense attention over a reused prefix
        dict(name="read_longctx", **_case("read", "longctx", 131072)),
    ]


def draw(rng):
    """A case of the same ranges, never dearer than the largest listed one of its kind."""
    op = rng.choice(["tree", "tree", "write", "read"])
    layer = rng.choice(["tiny", "mha", "gqa", "longctx", "fullkv2bit"])
    L = _LAYERS[layer]

    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    T = log(64, L["T"])
    top = {"tree": 64 if layer == "longctx" else 32, "write": 65536 // (L["B"] * L["Hkv"]), "read": T}[op]
    c = _case(op, layer, min(T, log(1, min(T, top))), T=T, ragged=rng.random() < 0.5,
              page=rng.choice([0, 0, 64, 128, 256]))
    if op == "write":
        c["gather"] = c["n"] <= 64 and rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs

def _up(x, m):
    return (x + m - 1) // m * m


def _dtype(case):
    return torch.float32 if case["kv"] == "f32" else torch.bfloat16


def _spans(case):
    """lens[b] cached tokens and counts[b] <= n new ones of each sequence: the case's, whatever the seed."""
    B, T, n = case["B"], case["T"], case["n"]
    rs = np.random.RandomState(1000 * n + T + B)
    if not case["ragged"]:
        return [T] * B, [n] * B
    counts = [int(c) for c in rs.randint(1, n + 1, B)]
    counts[rs.randint(B)] = n
    lens = [int(rs.randint(max(c, T // 2), T + 1)) for c in counts]
    if B > 2:
        i, j = rs.choice(B, 2, replace=False)
        lens[i] = counts[i]     # a sequence that has its new tokens only
        counts[j] = 0           # one that takes no part in this call
    return lens, counts


def _keys(shape, stats, gen):
    """Keys as the workloads draw them: per-channel mean and spread, 4 outlier channels."""
    mu, sigma = stats
    return torch.randn(shape, generator=gen, device="cuda").mul_(sigma).add_(mu)


def _stats(Hkv, d, gen):
    mu = torch.randn(Hkv, 1, d, generator=gen, device="cuda")
    sigma = torch.exp(0.5 * torch.randn(Hkv, 1, d, generator=gen, device="cuda"))
    out = torch.rand(Hkv, 1, d, generator=gen, device="cuda").argsort(-1) < 4
    mult = torch.where(out, 10.0, 1.0)
    return mu * mult, sigma * mult


def _divided(x, by):
    """x / by as one rounded division: with a Python number torch multiplies by 1/by instead."""
    return x / torch.full_like(x, by)


def _group_code(x):
    """Base code of the last axis: (packed codes, scale, minimum, decoded values)."""
    xs = x.unflatten(-1, (-1, 32))
    lo, hi = xs.amin(-1) + 0.0, xs.amax(-1) + 0.0
    scale = _divided(hi - lo, 3.0)
    div = torch.where(scale == 0, 1.0, scale).unsqueeze(-1)
    code = torch.round((xs - lo.unsqueeze(-1)) / div).clamp_(0, 3)
    code = torch.where(scale.unsqueeze(-1) == 0, 0.0, code)
    back = lo.unsqueeze(-1) + code * scale.unsqueeze(-1)
    c = code.to(torch.uint8).flatten(-2).unflatten(-1, (-1, 4))
    packed = c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6)
    return packed, scale, lo, back.flatten(-2)


def _side_code(y):
    """4-bit side code of y [..., r]: (packed nibbles, scale, decoded values)."""
    s = _divided(y.abs().amax(-1), 7.0)
    div = torch.where(s == 0, 1.0, s).unsqueeze(-1)
    w = torch.where(s.unsqueeze(-1) == 0, 0.0, torch.round(y / div).clamp_(-7, 7))
    u = w.to(torch.int32) & 15
    return (u[..., 0::2] | (u[..., 1::2] << 4)).to(torch.uint8), s, w * s.unsqueeze(-1)


def prepare(case, seed):
    B, Hq, Hkv, d, T, r, n = (case[k] for k in ("B", "Hq", "Hkv", "d", "T", "r", "n"))
    gen = torch.Generator("cuda").manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    dt = _dtype(case)
    lens, counts = _spans(case)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(starts[-1])
    st = dict(case=case, rows=rows,
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              cu=torch.from_numpy(starts).cuda())

    # the query-PCA basis: an orthonormal basis of the space the queries lie in
    A = torch.randn(Hkv, d, r, generator=gen, device="cuda")
    st["U"] = torch.linalg.qr(A)[0].contiguous()

    # the cache: pages in a shuffled pool, or one run per sequence
    if case["page"]:
        ps = case["page"]
        per = _up(T, ps) // ps
        pool = B * per + 3
        st["table"] = torch.from_numpy(rs.permutation(pool)[:B * per].reshape(B, per).astype(np.int32)).cuda()
        lead = (pool, Hkv, ps)
    else:
        lead = (B, Hkv, _up(T, 16))
    stats = _stats(Hkv, d, gen)
    planes = dict(k_codes=torch.zeros(*lead, d // 4, dtype=torch.uint8, device="cuda"),
                  k_scale=torch.zeros(*lead, d // 32, device="cuda"),
                  k_min=torch.zeros(*lead, d // 32, device="cuda"),
                  z_codes=torch.zeros(*lead, r // 2, dtype=torch.uint8, device="cuda"),
                  z_scale=torch.zeros(*lead, device="cuda"))
    if case["vmode"] == "2bit":
        for name, like in (("v_codes", "k_codes"), ("v_scale", "k_scale"), ("v_min", "k_min")):
            planes[name] = torch.zeros_like(planes[like])
    else:
        planes["v"] = torch.zeros(*lead, d, dtype=dt, device="cuda")
    if case["op"] != "write":  # a filled cache
        step = max(1, (1 << 25) // (lead[1] * lead[2] * d))
        for i in range(0, lead[0], step):
            j = min(lead[0], i + step)
            x = _keys((j - i,) + lead[1:] + (d,), stats, gen).to(dt).float()
            planes["k_codes"][i:j], planes["k_scale"][i:j], planes["k_min"][i:j], back = _group_code(x)
            y = torch.matmul(x - back, st["U"])
            planes["z_codes"][i:j], planes["z_scale"][i:j], _ = _side_code(y)
            v = torch.randn(x.shape, generator=gen, device="cuda").to(dt).float()
            if case["vmode"] == "2bit":
                planes["v_codes"][i:j], planes["v_scale"][i:j], planes["v_min"][i:j], _ = _group_code(v)
            else:
                planes["v"][i:j] = v
    st["planes"] = planes

    if case["op"] == "write":
        # keys and values of the new tokens, side by side as a projection leaves them
        src_rows = B * n if case["gather"] else rows
        kv = torch.randn(src_rows, 2 * Hkv, d, generator=gen, device="cuda")
        kv[:, :Hkv] = kv[:, :Hkv] * stats[1].squeeze(1) + stats[0].squeeze(1)
        st["kv"] = kv.to(dt)
        if case["gather"]:  # an ascending path through each sequence's n drafted tokens
            st["src"] = torch.from_numpy(np.concatenate(
                [b * n + np.sort(rs.choice(n, c, replace=False)) for b, c in enumerate(counts)]
            ).astype(np.int32)).cuda()
    if case["op"] in ("write", "read"):
        st["k_out"] = torch.zeros(rows, Hkv, d, dtype=dt, device="cuda")
        st["v_out"] = torch.zeros(rows, Hkv, d, dtype=dt, device="cuda")
    if case["op"] == "tree":
        g = torch.randn(rows, Hkv, Hq // Hkv, r, generator=gen, device="cuda")
        q = torch.einsum("nkgr,kdr->nkgd", g, A).reshape(rows, Hq, d)
        q = q + 0.1 * torch.randn(q.shape, generator=gen, device="cuda")
        st["q"] = q.to(dt)
        mask = np.zeros((B, n, n), bool)  # each node sees itself and its ancestors
        for b in range(B):
            for i in range(n):
                p = rs.randint(-1, i) if i else -1
                if p >= 0:
                    mask[b, i] = mask[b, p]
                mask[b, i, i] = True
        st["mask"] = torch.from_numpy(mask).cuda()
        st["out"] = torch.zeros(rows, Hq, d, dtype=dt, device="cuda")
    return st


# ---------------------------------------------------------------- the plain forms

def _place(st):
    """For every packed row: its sequence, its index in the span, its position."""
    cu, lens = st["cu"].long(), st["lens"].long()
    row = torch.arange(st["rows"], device="cuda")
    b = torch.searchsorted(cu, row, right=True) - 1
    i = row - cu[b]
    return b, i, lens[b] - (cu[b + 1] - cu[b]) + i


def _slots(st, b, t):
    """Slab and offset of tokens t of sequences b in the planes."""
    if "table" not in st:
        return b, t
    ps = st["case"]["page"]
    return st["table"].long()[b, t // ps], t % ps


def _unpack2(codes, scale, mn):
    c = torch.stack([(codes >> s) & 3 for s in (0, 2, 4, 6)], -1).flatten(-2).float()
    return (mn.unsqueeze(-1) + c.unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2)


def _unpack4(codes, scale):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return torch.where(c >= 8, c - 16, c) * scale.unsqueeze(-1)


def _decoded(st, pick, U):
    """Keys (with the side code's correction) and values of the planes' picked rows, fp32."""
    p = st["planes"]
    k = _unpack2(pick(p["k_codes"]), pick(p["k_scale"]), pick(p["k_min"]))
    z = _unpack4(pick(p["z_codes"]), pick(p["z_scale"]))
    k = k + torch.matmul(z.transpose(-3, -2), U.transpose(-1, -2)).transpose(-3, -2)
    if "v" in p:
        return k, pick(p["v"]).float()
    return k, _unpack2(pick(p["v_codes"]), pick(p["v_scale"]), pick(p["v_min"]))


def _plain_read(st):
    b, _, t = _place(st)
    slab, off = _slots(st, b, t)
    k, v = _decoded(st, lambda p: p[slab, :, off], st["U"])
    st["k_out"].copy_(k)
    st["v_out"].copy_(v)
    return st["k_out"], st["v_out"]


def _plain_write(st):
    p, U = st["planes"], st["U"]
    Hkv, d = U.shape[:2]
    kv = st["kv"][st["src"].long()] if "src" in st else st["kv"]
    k, v = kv[:, :Hkv].float(), kv[:, Hkv:]
    b, _, t = _place(st)
    slab, off = _slots(st, b, t)
    codes, scale, mn, back = _group_code(k)
    e = k - back
    # the projection is defined channel by channel, a rounded product and then a rounded sum,
    # so that side codes are the same bits everywhere: the order is part of the result
    y = torch.zeros(e.shape[:-1] + (U.shape[2],), device=e.device)
    for c in range(d):
        y += e[..., c, None] * U[:, c]
    zc, zs, _ = _side_code(y)
    for name, x in (("k_codes", codes), ("k_scale", scale), ("k_min", mn), ("z_codes", zc), ("z_scale", zs)):
        p[name][slab, :, off] = x
    if "v" in p:
        p["v"][slab, :, off] = v
    else:
        for name, x in zip(("v_codes", "v_scale", "v_min"), _group_code(v.float())):
            p[name][slab, :, off] = x
    return _plain_read(st)


def _plain_tree(st):
    case, rows, n = st["case"], st["rows"], st["case"]["n"]
    B, Hq, Hkv, d, T = (case[k] for k in ("B", "Hq", "Hkv", "d", "T"))
    G = Hq // Hkv
    if "table" in st:
        def pick(p):  # [pool, Hkv, page, ...] -> [B, T, Hkv, ...]
            return p[st["table"].long()].transpose(2, 3).flatten(1, 2)[:, :T]
    else:
        def pick(p):
            return p[:, :, :T].transpose(1, 2)
    k, v = _decoded(st, pick, st["U"])                               # [B, T, Hkv, d]
    b, i, _ = _place(st)
    q = torch.zeros(B, n, Hq, d, device="cuda")
    q[b, i] = st["q"].float()
    q = q.view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))  # [B, Hkv, n*G, T]
    lens = st["lens"].long().view(B, 1, 1)
    count = (st["cu"][1:] - st["cu"][:-1]).long().view(B, 1, 1)
    j = torch.arange(T, device="cuda").view(1, 1, T)
    a = j - (lens - count)                                           # index among the new tokens
    seen = torch.gather(st["mask"], 2, a.clamp(0, n - 1).expand(B, n, T))
    seen = (a < 0) | (seen & (a < count))
    s = s.view(B, Hkv, n, G, T).masked_fill_(~seen.view(B, 1, n, 1, T), float("-inf"))
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, Hkv, n * G, T), v.transpose(1, 2)).view(B, Hkv, n, G, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d)
    st["out"].copy_(o[b, i])
    return st["out"]


# ---------------------------------------------------------------- the framework's calls

def _cache(st):
    """The handles that a user's program keeps beside its planes."""
    if "cache" not in st:
        from bit_decode_attention_sm_b200 import headq

        case = st["case"]
        st["cache"] = headq.HeadQCache.from_planes(block_table=st.get("table"), **st["planes"])
        if case["op"] == "tree":
            st["ws"] = headq.tree_workspace(st["cache"], case["Hq"], case["n"], T=case["T"])
    return st["cache"]


def _own(st):
    from bit_decode_attention_sm_b200 import headq

    case, cache = st["case"], _cache(st)
    span = dict(seq_lens=st["lens"], cu=st["cu"], n=case["n"], T=case["T"])
    if case["op"] == "tree":
        return headq.headq_tree_attn(cache, st["q"], st["U"], mask=st["mask"], out=st["out"], ws=st["ws"], **span)
    if case["op"] == "write":
        Hkv = case["Hkv"]
        headq.headq_cache_write_ragged(cache, st["kv"][:, :Hkv], st["kv"][:, Hkv:], st["U"], src=st.get("src"), **span)
    return headq.headq_cache_read(cache, st["U"], k_out=st["k_out"], v_out=st["v_out"], **span)


def run(state):
    op = state["case"]["op"]
    if own:
        out = _own(state)
    else:
        out = {"tree": _plain_tree, "write": _plain_write, "read": _plain_read}[op](state)
    if op == "tree":
        return {"out": out}
    res = {"k": out[0], "v": out[1]}
    if op == "write":  # the planes' scales and minima too; the codes are in what was read back
        res.update({n: t for n, t in state["planes"].items() if t.dtype == torch.float32 and n != "v"})
    return res


def work(case):
    B, Hq, Hkv, d, r, n = (case[k] for k in ("B", "Hq", "Hkv", "d", "r", "n"))
    e = 4 if case["kv"] == "f32" else 2
    token = d // 4 + d // 4 + r // 2 + 4 + (d * e if case["vmode"] == "dense" else d // 2)
    lens, counts = _spans(case)
    tokens = sum(counts) * Hkv
    if case["op"] == "tree":
        pairs = sum(c * t for c, t in zip(counts, lens)) * Hq
        cached = sum(t for t, c in zip(lens, counts) if c) * Hkv
        return {"bytes": cached * token + 2 * sum(counts) * Hq * d * e, "flops": pairs * (4 * d + 2 * r)}
    both = 2 * d * e  # a dense key and value
    if case["op"] == "read":
        return {"bytes": tokens * (token + both), "flops": tokens * 2 * d * r}
    # the new tokens read, their rows of the planes written, and read back
    return {"bytes": tokens * (2 * both + 2 * token), "flops": tokens * 4 * d * r}


# ---------------------------------------------------------------- 64 bits

def _codes_as_stored(x):
    """Base code of x [N, d] by its definition, which is in 32-bit steps; values in 64."""
    N, d = x.shape
    x = x.astype(np.float32).reshape(N, d // 32, 32)
    mn, mx = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    sc = ((mx - mn) / np.float32(3)).astype(np.float32)
    with np.errstate(all="ignore"):
        c = np.where(sc == 0, np.float32(0), np.clip(np.rint((x - mn) / sc), 0, 3)).astype(np.float32)
    res = x - (mn + c * sc)
    val = mn.astype(np.float64) + c.astype(np.float64) * sc
    return val.reshape(N, d), sc[..., 0], mn[..., 0] + np.float32(0), res.reshape(N, d)


def _exact_write(case, st):
    Hkv, d = case["Hkv"], case["d"]
    U = st["U"].cpu().numpy()
    kv = st["kv"].float().cpu().numpy()
    if "src" in st:
        kv = kv[st["src"].cpu().numpy()]
    b, _, t = (x.cpu().numpy() for x in _place_by_hand(st))
    ks, vs = np.empty((len(b), Hkv, d)), np.empty((len(b), Hkv, d))
    planes = {n: x.cpu().numpy().copy() for n, x in st["planes"].items() if x.dtype == torch.float32 and n != "v"}
    if "table" in st:
        tab = st["table"].cpu().numpy()
        slab, off = tab[b, t // case["page"]], t % case["page"]
    else:
        slab, off = b, t
    for h in range(Hkv):
        val, sc, mn, res = _codes_as_stored(kv[:, h])
        planes["k_scale"][slab, h, off], planes["k_min"][slab, h, off] = sc, mn
        y = np.zeros((len(b), U.shape[2]), np.float32)
        for c in range(d):
            y = y + (res[:, c:c + 1] * U[h, c][None]).astype(np.float32)
        s = (np.abs(y).max(-1) / np.float32(7)).astype(np.float32)
        planes["z_scale"][slab, h, off] = s
        with np.errstate(all="ignore"):
            w = np.where(s[:, None] == 0, 0, np.clip(np.rint(y / s[:, None]), -7, 7))
        ks[:, h] = val + (w.astype(np.float64) * s[:, None]) @ U[h].astype(np.float64).T
        if case["vmode"] == "2bit":
            vs[:, h], sc, mn, _ = _codes_as_stored(kv[:, Hkv + h])
            planes["v_scale"][slab, h, off], planes["v_min"][slab, h, off] = sc, mn
        else:
            vs[:, h] = kv[:, Hkv + h]
    return {"k": ks, "v": vs, **{n: x.astype(np.float64) for n, x in planes.items()}}


def _place_by_hand(st):
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    got = [(b, i, lens[b] - (cu[b + 1] - cu[b]) + i) for b in range(len(lens)) for i in range(cu[b + 1] - cu[b])]
    return [torch.tensor(x, dtype=torch.long) for x in zip(*got)] if got else [torch.zeros(0, dtype=torch.long)] * 3


def _token_values(st, b, h, t0, t1):
    """Keys and values of tokens [t0, t1) of one sequence and KV head, in 64 bits."""
    def rows(p):
        if "table" not in st:
            return p[b, h, t0:t1]
        t = torch.arange(t0, t1, device="cuda")
        return p[st["table"][b].long()[t // st["case"]["page"]], h, t % st["case"]["page"]]

    def two_bit(c, s, m):
        c = rows(c).int()
        ch = torch.arange(c.shape[-1] * 4, device="cuda")
        code = (c[:, ch // 4] >> (2 * (ch % 4))) & 3
        return rows(m).double()[:, ch // 32] + code.double() * rows(s).double()[:, ch // 32]

    p = st["planes"]
    k = two_bit(p["k_codes"], p["k_scale"], p["k_min"])
    zc = rows(p["z_codes"]).int()
    i = torch.arange(zc.shape[-1] * 2, device="cuda")
    w = (zc[:, i // 2] >> (4 * (i % 2))) & 15
    w = w - 16 * (w > 7).int()
    k = k + (w.double() * rows(p["z_scale"]).double()[:, None]) @ st["U"][h].double().T
    v = rows(p["v"]).double() if "v" in p else two_bit(p["v_codes"], p["v_scale"], p["v_min"])
    return k, v


def exact(case, seed):
    st = prepare(case, seed)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "write":
        return _exact_write(case, st)
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    if case["op"] == "read":
        k = torch.zeros(st["rows"], Hkv, d, dtype=torch.float64, device="cuda")
        v = torch.zeros_like(k)
        for b in range(case["B"]):
            for h in range(Hkv):
                k[cu[b]:cu[b + 1], h], v[cu[b]:cu[b + 1], h] = _token_values(
                    st, b, h, lens[b] - (cu[b + 1] - cu[b]), lens[b])
        return {"k": k, "v": v}
    out = torch.zeros(st["rows"], Hq, d, dtype=torch.float64, device="cuda")
    G = Hq // Hkv
    for b in range(case["B"]):
        c = cu[b + 1] - cu[b]
        if c == 0:
            continue
        see = torch.ones(c, lens[b], dtype=torch.bool, device="cuda")
        see[:, lens[b] - c:] = st["mask"][b, :c, :c]
        for h in range(Hkv):
            k, v = _token_values(st, b, h, 0, lens[b])
            q = st["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double()
            x = torch.einsum("igd,td->git", q, k) / math.sqrt(d)
            x = torch.where(see[None], x, -math.inf)
            out[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.einsum("git,td->igd", torch.softmax(x, -1), v)
    return {"out": out}
