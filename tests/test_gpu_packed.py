"""Packed-batch operators against 64-bit references: headq_cache_write_ragged (bit for bit
against the oracle's codec), headq_cache_read, headq_tree_attn, and the three as a
speculative-decoding step uses them."""

import numpy as np
import pytest
import torch

import oracle
from packed_helpers import (HALF, Cache, check_tree, logical, ref_tree, spans, tensor_core, tree_masks)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def hq():
    from bit_decode_attention_sm_b200 import headq
    return headq


# ---------------------------------------------------------------- write

def new_tokens(rng, rows, Hkv, d, dt):
    """k and v as strided halves of one tensor, with constant and tie-rich groups among them."""
    kv = rng.standard_normal((rows, 2 * Hkv, d)).astype(np.float32)
    kv[:, :, : d // 2] *= 4
    if rows > 2:
        kv[1, 0] = 0.75                                          # scale 0
        kv[2, 0] = np.round(kv[2, 0] * 2) / 2                    # exact ties
    t = torch.from_numpy(kv).cuda().to(dt)
    return t[:, :Hkv], t[:, Hkv:]


def expected_planes(c, k, v, counts, lens, src=None):
    """The cache's planes after the write: everything else as it was."""
    want = {n: logical(t, c.table).clone() for n, t in c.planes.items()}
    r0 = 0
    for b, (n, T) in enumerate(zip(counts, lens)):
        for i in range(n if n <= T else 0):
            row = r0 + i if src is None else int(src[r0 + i])
            if not 0 <= row < k.shape[0]:
                continue
            kk = k[row].float().cpu().numpy()[None, :, None]     # [1, Hkv, 1, d]
            vv = v[row].float().cpu().numpy()[None, :, None]
            pl = oracle.cache_write(kk, c.U.cpu().numpy(), v=vv, vmode=c.vmode)
            t = T - n + i
            names = dict(kc="k_codes", ks="k_scale", km="k_min")
            if c.r:
                names.update(zc="z_codes", zs="z_scale")
            if c.vmode == "2bit":
                names.update(vc="v_codes", vs="v_scale", vm="v_min")
            else:
                want["v"][b, :, t] = v[row].to(want["v"].dtype)
            for a, name in names.items():
                want[name][b, :, t] = torch.from_numpy(np.ascontiguousarray(pl[a][0, :, 0])).cuda()
        r0 += n
    return want


WRITES = [  # B, Hkv, T_cap, d, r, vmode, v dtype, input dtype, page, counts, lens
    (3, 4, 512, 128, 16, "dense", BF, BF, 0, [5, 0, 70], [5, 100, 389]),
    (4, 2, 256, 128, 16, "2bit", BF, BF, 64, [1, 64, 65, 130], [64, 64, 200, 256]),
    (2, 12, 128, 64, 8, "dense", BF, BF, 0, [1, 1], [1, 128]),
    (2, 1, 128, 64, 8, "dense", F32, F32, 128, [33, 7], [100, 7]),
    (2, 2, 128, 32, 6, "dense", BF, F32, 0, [9, 40], [60, 128]),
    (2, 2, 64, 256, 32, "2bit", BF, F32, 64, [3, 17], [64, 17]),
    (1, 3, 64, 8, 2, "dense", F32, BF, 0, [13], [40]),
    (2, 2, 64, 16, 0, "2bit", BF, BF, 0, [5, 6], [64, 6]),
]


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@pytest.mark.parametrize("i", range(len(WRITES)))
def test_write_ragged(i, gather):
    B, Hkv, T_cap, d, r, vmode, vd, dt, page, counts, lens = WRITES[i]
    rng = np.random.default_rng(i)
    c = Cache(i, B, Hkv, T_cap, d, r, vmode, vd, page)
    rows = sum(counts)
    k, v = new_tokens(rng, rows + 11 if gather else rows, Hkv, d, dt)
    src = None
    if gather:
        src = torch.from_numpy(rng.integers(0, rows + 11, rows).astype(np.int32))
        if rows > 3:
            src[1], src[3] = -1, rows + 11                        # not written
        src = src.cuda()
    want = expected_planes(c, k, v, counts, lens, src)
    cu, sl = spans(counts, lens)
    hq().headq_cache_write_ragged(c.hq, k, v, c.U, seq_lens=sl, cu=cu, n=max(counts), src=src)
    for name, t in c.planes.items():
        got = logical(t, c.table)
        assert torch.equal(got.view(torch.uint8), want[name].view(torch.uint8)), name


def test_write_matches_the_dense_write():
    c, e = Cache(5, 2, 4, 640, 128, 16), Cache(5, 2, 4, 640, 128, 16)
    rng = np.random.default_rng(0)
    k = torch.from_numpy(rng.standard_normal((2, 4, 600, 128)).astype(np.float32)).cuda().to(BF)
    v = torch.from_numpy(rng.standard_normal((2, 4, 600, 128)).astype(np.float32)).cuda().to(BF)
    hq().headq_cache_write(c.hq, k, v, c.U, t0=40)
    flat = [x.transpose(1, 2).reshape(1200, 4, 128) for x in (k, v)]
    hq().headq_cache_write_ragged(e.hq, *flat, e.U, T=640)        # uniform: no cu, no lengths
    for name in c.planes:
        assert torch.equal(c.planes[name].view(torch.uint8), e.planes[name].view(torch.uint8)), name


def test_write_leaves_values_alone_without_v():
    c = Cache(6, 1, 2, 64, 64, 8)
    before = c.planes["v"].clone()
    codes = c.planes["k_codes"].clone()
    k, _ = new_tokens(np.random.default_rng(1), 5, 2, 64, BF)
    hq().headq_cache_write_ragged(c.hq, k, None, c.U, T=20)
    assert torch.equal(c.planes["v"], before)
    assert not torch.equal(c.planes["k_codes"][:, :, 15:20], codes[:, :, 15:20])


def test_spans_that_take_no_part():
    """More new rows than cached tokens, an empty sequence, descending and overlong cu."""
    c = Cache(7, 4, 2, 64, 64, 8)
    want = {n: t.clone() for n, t in c.planes.items()}
    k, v = new_tokens(np.random.default_rng(1), 12, 2, 64, BF)
    cu = torch.tensor([0, 6, 3, 3, 40], dtype=torch.int32, device="cuda")
    sl = torch.tensor([5, 10, 0, 64], dtype=torch.int32, device="cuda")
    hq().headq_cache_write_ragged(c.hq, k, v, c.U, seq_lens=sl, cu=cu, n=8)
    for n, t in c.planes.items():
        assert torch.equal(t, want[n]), n
    ko, vo = (torch.full((12, 2, 64), 7.0, dtype=BF, device="cuda") for _ in "kv")
    hq().headq_cache_read(c.hq, c.U, seq_lens=sl, cu=cu, n=8, k_out=ko, v_out=vo)
    assert (ko == 7).all() and (vo == 7).all()
    q = torch.randn(12, 4, 64, device="cuda").to(BF)
    out = torch.full((12, 4, 64), 7.0, dtype=BF, device="cuda")
    lse = torch.full((12, 4), 7.0, device="cuda")
    hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl, cu=cu, n=8, out=out, lse=lse)
    assert (out[:6] == 0).all() and (out[6:] == 7).all()
    assert (lse[:6] == -float("inf")).all() and (lse[6:] == 7).all()


# ---------------------------------------------------------------- read

READS = [  # B, Hkv, T_cap, d, r, vmode, v dtype, kmode, page, counts, lens
    (3, 4, 512, 128, 16, "dense", BF, "token", 0, [5, 0, 70], [5, 100, 389]),
    (2, 8, 256, 128, 16, "2bit", BF, "token", 64, [200, 33], [256, 65]),
    (2, 12, 128, 64, 8, "dense", BF, "token", 0, [1, 128], [77, 128]),
    (2, 2, 128, 128, 8, "dense", F32, "channel", 64, [100, 7], [128, 71]),
    (1, 3, 128, 64, 16, "2bit", BF, "channel", 0, [128], [128]),
    (2, 2, 64, 128, 0, "dense", BF, "token", 0, [9, 40], [60, 64]),
    (2, 2, 64, 256, 32, "2bit", BF, "token", 64, [3, 17], [64, 17]),
    (2, 2, 64, 8, 2, "dense", F32, "token", 0, [13, 2], [40, 50]),
    (1, 2, 64, 32, 6, "dense", BF, "channel", 0, [33], [64]),
]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(READS)))
def test_read(i, dt):
    B, Hkv, T_cap, d, r, vmode, vd, kmode, page, counts, lens = READS[i]
    c = Cache(i, B, Hkv, T_cap, d, r, vmode, vd, page, kmode)
    k, z, v, U = c.parts()
    rows = sum(counts)
    cu, sl = spans(counts, lens)
    for sigma in (1, 0, -1):
        kv = torch.full((rows + 4, 2 * Hkv + 1, d), 7.0, dtype=dt, device="cuda")  # strided, rows behind
        ko, vo = kv[:, :Hkv], kv[:, Hkv:2 * Hkv]
        hq().headq_cache_read(c.hq, c.U, seq_lens=sl, cu=cu, n=max(counts), corr_sign=sigma, k_out=ko, v_out=vo)
        assert (kv[rows:] == 7).all() and (kv[:, 2 * Hkv:] == 7).all()
        r0 = 0
        for b, (n, T) in enumerate(zip(counts, lens)):
            for h in range(Hkv):
                zz = z[b, h, T - n:T]
                kr = k[b, h, T - n:T] + sigma * zz @ U[h].T
                # r + 4 roundings of fp32 in sums whose terms are these, then the output's
                mag = np.abs(k[b, h, T - n:T]) * 4 + np.abs(zz) @ np.abs(U[h]).T
                tol = (r + 4) * 2.0 ** -24 * mag + HALF[dt] * np.abs(kr) + 1e-30
                got = ko[r0:r0 + n, h].double().cpu().numpy()
                assert (np.abs(got - kr) <= tol).all()
                vr = v[b, h, T - n:T]
                gv = vo[r0:r0 + n, h].double().cpu().numpy()
                assert (np.abs(gv - vr) <= 2.0 ** -22 * (np.abs(vr) + 4) + HALF[dt] * np.abs(vr)).all()
            r0 += n


def test_read_one_of_the_two_and_new_tensors():
    c = Cache(3, 2, 2, 64, 64, 8)
    k, v = hq().headq_cache_read(c.hq, c.U, n=10, T=30)
    assert k.shape == v.shape == (20, 2, 64) and k.dtype == BF
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    hq().headq_cache_read(c.hq, c.U, n=10, T=30, k_out=ko)
    hq().headq_cache_read(c.hq, None, n=10, T=30, v_out=vo)
    assert torch.equal(ko, k) and torch.equal(vo, v)


@pytest.mark.parametrize("d,r", [(128, 16), (32, 4)])
def test_bad_page_reads_zero_and_is_reported(d, r):
    c = Cache(4, 2, 2, 128, d, r, page=64)
    c.table[1, 1] = 99999
    ws = hq().tree_workspace(c.hq, 2, 1)
    k, v = hq().headq_cache_read(c.hq, c.U, n=128, T=128, ws=ws)
    with pytest.raises(hq().HeadQError):
        hq().headq_workspace_status(ws)
    hq().headq_workspace_status(ws)
    assert (k[192:] == 0).all() and (v[192:] == 0).all()
    assert (k[:192] != 0).any(-1).all()
    kk, vv = new_tokens(np.random.default_rng(1), 256, 2, d, BF)
    want = {n: t.clone() for n, t in c.planes.items()}
    hq().headq_cache_write_ragged(c.hq, kk, vv, c.U, T=128)       # the bad page's tokens are dropped
    free = [p for p in range(c.planes["k_codes"].shape[0]) if p not in c.table.reshape(-1).tolist()]
    for n, t in c.planes.items():
        assert torch.equal(t[free], want[n][free]), n
    q = torch.randn(256, 2, d, device="cuda").to(BF)
    hq().headq_tree_attn(c.hq, q, c.U, T=128, ws=hq().tree_workspace(c.hq, 2, 128))


# ---------------------------------------------------------------- tree attention

TREES = [  # B, Hq, Hkv, T_cap, d, r, vmode, v dtype, q dtype, page, counts, lens
    (3, 28, 4, 512, 128, 16, "dense", BF, BF, 0, [5, 0, 16], [5, 100, 389]),
    (2, 32, 8, 1024, 128, 16, "dense", BF, BF, 256, [64, 33], [1000, 1024]),
    (3, 28, 4, 512, 128, 16, "2bit", BF, BF, 64, [32, 1, 7], [512, 1, 130]),
    (2, 12, 12, 256, 64, 8, "dense", BF, BF, 0, [11, 3], [256, 129]),
    (1, 8, 2, 512, 64, 16, "2bit", BF, BF, 128, [17], [401]),
    (2, 4, 4, 384, 128, 0, "dense", BF, BF, 0, [1, 1], [383, 128]),
    (1, 16, 1, 640, 128, 8, "dense", BF, BF, 0, [70], [600]),
    (2, 6, 2, 512, 128, 16, "2bit", BF, BF, 0, [140, 200], [400, 512]),
    (1, 16, 1, 512, 64, 8, "dense", F32, F32, 0, [8], [512]),
    (2, 6, 2, 128, 128, 16, "2bit", BF, F32, 64, [20, 3], [97, 128]),
    (2, 4, 2, 128, 32, 6, "dense", BF, BF, 0, [9, 2], [77, 128]),
    (1, 4, 1, 128, 256, 32, "dense", F32, F32, 0, [5], [100]),
    (1, 2, 2, 64, 8, 2, "2bit", BF, F32, 0, [4], [60]),
    (1, 2, 1, 64, 16, 0, "dense", F32, F32, 0, [3], [3]),
]


def tree_case(i, seed=0):
    B, Hq, Hkv, T_cap, d, r, vmode, vd, qd, page, counts, lens = TREES[i]
    rng = np.random.default_rng(100 * seed + i)
    c = Cache(i + 50 * seed, B, Hkv, T_cap, d, r, vmode, vd, page)
    q = torch.from_numpy(rng.standard_normal((sum(counts), Hq, d)).astype(np.float32) * 1.5).cuda().to(qd)
    return c, q, counts, lens, tree_masks(rng, B, max(counts))


@pytest.mark.parametrize("sigma", [1, 0, -1])
@pytest.mark.parametrize("i", range(len(TREES)))
def test_tree(i, sigma):
    c, q, counts, lens, mask = tree_case(i)
    ref = ref_tree(c, q, counts, lens, mask, sigma=float(sigma))
    cu, sl = spans(counts, lens)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    kw = dict(seq_lens=sl, cu=cu, n=max(counts), corr_sign=sigma)
    m = torch.from_numpy(mask).cuda()
    ws = hq().tree_workspace(c.hq, q.shape[1], max(counts))
    out = hq().headq_tree_attn(c.hq, q, c.U, mask=m, lse=lse, ws=ws, **kw)
    hq().headq_workspace_status(ws)
    check_tree(out, lse, ref)
    again = hq().headq_tree_attn(c.hq, q, c.U, mask=m, ws=ws, **kw)
    assert torch.equal(out, again)


@pytest.mark.parametrize("i", [0, 2, 8, 10])
def test_tree_without_a_mask_is_a_run(i):
    c, q, counts, lens, _ = tree_case(i, 1)
    cu, sl = spans(counts, lens)
    out = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl, cu=cu, n=max(counts))
    check_tree(out, None, ref_tree(c, q, counts, lens, None))


@pytest.mark.parametrize("i", [0, 2, 3, 8])
def test_rows_that_see_nothing(i):
    c, q, counts, lens, mask = tree_case(i, 2)
    lens = [n for n in counts]                     # no prefix at all
    mask[:, ::2] = False
    cu, sl = spans(counts, lens)
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = hq().headq_tree_attn(c.hq, q, c.U, mask=torch.from_numpy(mask).cuda(), seq_lens=sl, cu=cu,
                               n=max(counts), lse=lse)
    ref = ref_tree(c, q, counts, lens, mask)
    check_tree(out, lse, ref)
    assert (ref[1] == -np.inf).any() and (out[0] == 0).all()


@pytest.mark.parametrize("poison", ["nan", "inf", "huge"])
@pytest.mark.parametrize("i", [0, 2, 3, 7, 8, 10])
def test_what_is_not_seen_is_not_felt(i, poison):
    """Tokens past a sequence's end, and drafted tokens that a row does not see, hold NaN,
    infinities or values of the type's size; the row that sees such a token feels it."""
    c, q, counts, lens, mask = tree_case(i, 3)
    b = int(np.argmax(counts))
    n, T = counts[b], lens[b]
    j = n - 1
    mask[b, :n - 1, j] = False                     # the last new token is seen by itself alone
    clean = ref_tree(c, q, counts, lens, mask)
    x = {"nan": float("nan"), "inf": float("inf"), "huge": 3e38}[poison]
    T_cap = c.hq.T_cap
    for t in [T - 1] + list(range(T, T_cap)):
        slab, off = (b, t) if c.table is None else (int(c.table[b, t // c.hq.page_size]), t % c.hq.page_size)
        for name in ("k_scale", "k_min", "z_scale", "v", "v_scale", "v_min"):
            if name in c.planes:
                c.planes[name][slab, :, off] = x
    cu, sl = spans(counts, lens)
    out = hq().headq_tree_attn(c.hq, q, c.U, mask=torch.from_numpy(mask).cuda(), seq_lens=sl, cu=cu,
                               n=max(counts))
    row = sum(counts[:b]) + j
    keep = np.ones(q.shape[0], bool)
    keep[row] = False
    check_tree(out[torch.from_numpy(keep).cuda()], None, [a[keep] for a in clean])
    if poison != "huge":
        assert not torch.isfinite(out[row]).any()


@pytest.mark.parametrize("vmode", ["dense", "2bit"])
@pytest.mark.parametrize("n", [100, 200, 300])
def test_first_seen_token_late(n, vmode):
    """Rows whose first visible token lies in a later tile than the call's first."""
    c = Cache(21, 2, 2, 512, 128, 16, vmode)
    rng = np.random.default_rng(n)
    q = torch.from_numpy(rng.standard_normal((2 * n, 4, 128)).astype(np.float32)).cuda().to(BF)
    mask = np.zeros((2, n, n), bool)
    for i in range(n):
        mask[:, i, i] = i % 3 > 0            # itself, or nothing
        mask[:, i, max(0, i - 5):i] = i % 2 > 0
    lens = [n, n]
    cu, sl = spans([n, n], lens)
    lse = torch.zeros(2 * n, 4, device="cuda")
    out = hq().headq_tree_attn(c.hq, q, c.U, mask=torch.from_numpy(mask).cuda(), seq_lens=sl, cu=cu, n=n, lse=lse)
    check_tree(out, lse, ref_tree(c, q, [n, n], lens, mask))


def test_strided_queries_and_outputs():
    c, q, counts, lens, mask = tree_case(0, 4)
    rows, Hq, d = q.shape
    big = torch.full((rows + 5, Hq + 8, d), 7.0, dtype=BF, device="cuda")
    big[:rows, :Hq] = q
    outs = torch.full((rows + 5, Hq, 2 * d), 7.0, dtype=BF, device="cuda")
    cu, sl = spans(counts, lens)
    hq().headq_tree_attn(c.hq, big[:, :Hq], c.U, mask=torch.from_numpy(mask).cuda(), seq_lens=sl, cu=cu,
                         n=max(counts), out=outs[:, :, d:])
    check_tree(outs[:rows, :, d:], None, ref_tree(c, q, counts, lens, mask))
    assert (outs[rows:] == 7).all() and (outs[:, :, :d] == 7).all()


@pytest.mark.parametrize("mag", [(1e-3, 1.0), (300.0, 1e-2), (1e4, 1e-4), (1.0, 1e3)])
@pytest.mark.parametrize("i", [0, 4])
def test_magnitudes(i, mag):
    """Queries and keys far from 1: operands keep their relative precision."""
    c, q, counts, lens, mask = tree_case(i, 5)
    for n in ("k_scale", "k_min", "z_scale"):
        c.planes[n] *= mag[1]
    q = (q.float() * mag[0]).to(BF)
    cu, sl = spans(counts, lens)
    out = hq().headq_tree_attn(c.hq, q, c.U, mask=torch.from_numpy(mask).cuda(), seq_lens=sl, cu=cu,
                               n=max(counts))
    check_tree(out, None, ref_tree(c, q, counts, lens, mask))


@pytest.mark.parametrize("sm", [0.0, -0.1, 0.3])
def test_other_logit_scales(sm):
    c, q, counts, lens, mask = tree_case(0, 6)
    cu, sl = spans(counts, lens)
    out = hq().headq_tree_attn(c.hq, q, c.U, mask=torch.from_numpy(mask).cuda(), seq_lens=sl, cu=cu,
                               n=max(counts), sm_scale=sm)
    check_tree(out, None, ref_tree(c, q, counts, lens, mask, sm=sm))


def test_one_tree_for_all():
    c, q, counts, lens, mask = tree_case(3, 7)
    cu, sl = spans(counts, lens)
    kw = dict(seq_lens=sl, cu=cu, n=max(counts))
    m = torch.from_numpy(mask[0]).cuda()
    a = hq().headq_tree_attn(c.hq, q, c.U, mask=m, **kw)
    b = hq().headq_tree_attn(c.hq, q, c.U, mask=m.to(torch.uint8)[None].repeat(len(counts), 1, 1), **kw)
    assert torch.equal(a, b)


def test_long_sequence():
    c = Cache(9, 1, 2, 20000, 128, 16, spread=0.5)
    q = torch.randn(9, 8, 128, generator=torch.Generator().manual_seed(1)).cuda().to(BF)
    mask = tree_masks(np.random.default_rng(9), 1, 9)
    out = hq().headq_tree_attn(c.hq, q, c.U, mask=torch.from_numpy(mask).cuda(), T=19993)
    check_tree(out, None, ref_tree(c, q, [9], [19993], mask))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("vmode", ["dense", "2bit"])
def test_speculative_step(vmode):
    """Draft, verify, accept: the tree's rows are what plain decoding of each path gives, and
    the accepted path re-written in order leaves the cache that plain decoding would."""
    rng = np.random.default_rng(3)
    B, Hq, Hkv, d, r, n = 2, 28, 4, 128, 16, 12
    lens0, T_cap = [300, 77], 512
    a, e = (Cache(11, B, Hkv, T_cap, d, r, vmode) for _ in range(2))
    mask = tree_masks(rng, B, n)
    k, v = new_tokens(rng, B * n, Hkv, d, BF)
    q = torch.from_numpy(rng.standard_normal((B * n, Hq, d)).astype(np.float32)).cuda().to(BF)
    sl = torch.tensor([t + n for t in lens0], dtype=torch.int32, device="cuda")
    hq().headq_cache_write_ragged(a.hq, k, v, a.U, seq_lens=sl, n=n)
    out = hq().headq_tree_attn(a.hq, q, a.U, mask=torch.from_numpy(mask).cuda(), seq_lens=sl, n=n)
    tol = ref_tree(a, q, [n] * B, [t + n for t in lens0], mask)[2]
    paths = [np.flatnonzero(mask[b, mask[b].sum(1).argmax()]) for b in range(B)]
    # plain decoding of the deepest path, one token at a time
    for step in range(max(map(len, paths))):
        rows = [b * n + paths[b][min(step, len(paths[b]) - 1)] for b in range(B)]
        now = torch.tensor([lens0[b] + step + 1 if step < len(paths[b]) else 0 for b in range(B)],
                           dtype=torch.int32, device="cuda")
        o, _ = hq().headq_decode_append(e.hq, k[rows].contiguous(), v[rows].contiguous(),
                                        q[rows].contiguous(), e.U, T=T_cap, seq_lens=now)
        for b in range(B):
            if step < len(paths[b]):
                d_o = (out[rows[b]].double() - o[b].double()).abs().cpu().numpy()
                lim = tol[rows[b]] + 2e-3 * o[b].double().abs().amax(-1, keepdim=True).cpu().numpy()
                assert (d_o <= lim).all()
    # accept the paths: gathered from the draft, written in order over the tree
    counts = [len(p) for p in paths]
    src = torch.from_numpy(np.concatenate([b * n + p for b, p in enumerate(paths)]).astype(np.int32)).cuda()
    cu, ends = spans(counts, [lens0[b] + counts[b] for b in range(B)])
    hq().headq_cache_write_ragged(a.hq, k, v, a.U, seq_lens=ends, cu=cu, n=max(counts), src=src)
    ka, va = hq().headq_cache_read(a.hq, a.U, seq_lens=ends, cu=cu, n=max(counts), rows=sum(counts))
    ke, ve = hq().headq_cache_read(e.hq, e.U, seq_lens=ends, cu=cu, n=max(counts), rows=sum(counts))
    assert torch.equal(ka, ke) and torch.equal(va, ve)


def test_streams_and_graphs():
    """A step captured once and replayed on new inputs, beside eager calls on another stream
    with their own workspace."""
    c, q, counts, lens, mask = tree_case(1, 8)
    cu, sl = spans(counts, lens)
    m = torch.from_numpy(mask).cuda()
    n = max(counts)
    ws, ws2 = (hq().tree_workspace(c.hq, q.shape[1], n) for _ in range(2))
    out = torch.zeros_like(q)
    kw = dict(mask=m, seq_lens=sl, cu=cu, n=n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hq().headq_tree_attn(c.hq, q, c.U, out=out, ws=ws, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hq().headq_tree_attn(c.hq, q, c.U, out=out, ws=ws, **kw)
    for step in range(3):
        q.copy_(torch.randn(q.shape, device="cuda"))
        sl.copy_(torch.tensor([lens[0] - step, lens[1] - 7 * step], dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        eager = hq().headq_tree_attn(c.hq, q, c.U, ws=ws2, stream=side, out=torch.zeros_like(q), **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        check_tree(out, None, ref_tree(c, q, counts, sl.tolist(), mask))
