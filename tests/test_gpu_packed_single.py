"""headq_tree_attn of single tokens, one workspace under calls of many sizes, calls in a row."""

import numpy as np
import pytest
import torch

from packed_helpers import Cache, check_tree, ref_tree, spans, tree_masks

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def hq():
    from bit_decode_attention_sm_b200 import headq
    return headq


SINGLES = [  # B, Hq, Hkv, T_cap, d, r, vmode, page, lens
    (4, 28, 4, 1024, 128, 16, "dense", 0, [1024, 1, 65, 700]),
    (3, 8, 1, 2048, 128, 16, "2bit", 256, [2000, 64, 1]),
    (3, 32, 8, 512, 64, 8, "dense", 64, [512, 63, 130]),
    (2, 4, 4, 512, 128, 0, "dense", 0, [511, 2]),
    (2, 6, 2, 256, 64, 16, "2bit", 0, [256, 17]),
    (2, 5, 1, 256, 128, 8, "2bit", 64, [200, 256]),
    (2, 16, 1, 512, 128, 16, "dense", 0, [512, 129]),      # more query heads than the decode takes
    (2, 4, 2, 256, 128, 0, "2bit", 0, [255, 3]),           # a shape only the tree kernel takes
]


def single_case(i, seed=0):
    B, Hq, Hkv, T_cap, d, r, vmode, page, lens = SINGLES[i]
    rng = np.random.default_rng(1000 * seed + i)
    c = Cache(i + 70 * seed, B, Hkv, T_cap, d, r, vmode, BF, page)
    q = torch.from_numpy(rng.standard_normal((B, Hq, d)).astype(np.float32) * 1.5).cuda().to(BF)
    return c, q, lens


@pytest.mark.parametrize("sigma", [1, 0, -1])
@pytest.mark.parametrize("i", range(len(SINGLES)))
def test_single(i, sigma):
    c, q, lens = single_case(i)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    ws = hq().tree_workspace(c.hq, q.shape[1], 1)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = dict(seq_lens=sl, corr_sign=sigma, ws=ws)
    out = hq().headq_tree_attn(c.hq, q, c.U, lse=lse, **kw)
    hq().headq_workspace_status(ws)
    check_tree(out, lse, ref_tree(c, q, [1] * len(lens), lens, None, sigma=float(sigma)))
    assert torch.equal(out, hq().headq_tree_attn(c.hq, q, c.U, **kw))


@pytest.mark.parametrize("i", range(len(SINGLES)))
def test_some_sequences_have_a_token_and_some_see_themselves(i):
    c, q, lens = single_case(i, 1)
    B = len(lens)
    counts = [b % 2 for b in range(B)][::-1]                # the last sequence has one
    cu, sl = spans(counts, lens)
    for see in (False, True):
        mask = np.full((1, 1), see)
        big = torch.full((B, q.shape[1], q.shape[2] + 8), 7.0, dtype=BF, device="cuda")
        lse = torch.full((B, q.shape[1]), 7.0, device="cuda")
        hq().headq_tree_attn(c.hq, q, c.U, mask=torch.from_numpy(mask).cuda(), seq_lens=sl, cu=cu, n=1,
                             out=big[:, :, 8:], lse=lse)
        rows = sum(counts)
        ref = ref_tree(c, q[:rows], counts, lens, np.broadcast_to(mask, (B, 1, 1)))
        check_tree(big[:rows, :, 8:], lse[:rows], ref)
        assert (big[rows:] == 7).all() and (big[:, :, :8] == 7).all() and (lse[rows:] == 7).all()


@pytest.mark.parametrize("i", [0, 1, 2, 4])
def test_single_rows_that_see_nothing(i):
    """No cached token at all, a sequence of its own unseen token, one with more new tokens
    than n, and one with more than it has cached."""
    c, q, _ = single_case(i, 2)
    B, Hq, d = q.shape
    lens = [0, 1, 5, 3][:B]
    counts = [1, 1, 3, 4][:B]
    cu, sl = spans(counts, lens)
    rows = sum(counts)
    qq = torch.randn(rows, Hq, d, device="cuda").to(BF)
    out, lse = torch.full_like(qq, 7.0), torch.full((rows, Hq), 7.0, device="cuda")
    mask = torch.zeros(1, 1, dtype=torch.bool, device="cuda")
    hq().headq_tree_attn(c.hq, qq, c.U, mask=mask, seq_lens=sl, cu=cu, n=1, out=out, lse=lse)
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all()
    if B > 2:                                              # its first row sees the two before it
        first = ref_tree(c, qq[2:3].repeat(B, 1, 1), [1] * B, [0, 0, 2, 0][:B], np.ones((B, 1, 1), bool))
        check_tree(out[2:3], lse[2:3], [a[2:3] for a in first])
        assert (out[3:5] == 7).all() and (lse[3:5] == 7).all()
    if B > 3:
        assert (out[5] == 0).all() and (lse[5] == -np.inf).all() and (out[6:] == 7).all()


@pytest.mark.parametrize("poison", ["nan", "inf", "huge"])
@pytest.mark.parametrize("i", range(len(SINGLES)))
def test_what_lies_behind_a_sequence_is_not_felt(i, poison):
    c, q, lens = single_case(i, 3)
    clean = ref_tree(c, q, [1] * len(lens), lens, None)
    x = {"nan": float("nan"), "inf": float("inf"), "huge": 3e38}[poison]
    for b, T in enumerate(lens):
        for t in range(T, c.hq.T_cap):
            slab, off = (b, t) if c.table is None else (int(c.table[b, t // c.hq.page_size]), t % c.hq.page_size)
            for name in ("k_scale", "k_min", "z_scale", "v", "v_scale", "v_min"):
                if name in c.planes:
                    c.planes[name][slab, :, off] = x
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    check_tree(hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl), None, clean)


@pytest.mark.parametrize("mag", [(1e-3, 1.0), (300.0, 1e-2), (1e4, 1e-4), (1.0, 1e3)])
@pytest.mark.parametrize("i", [0, 1])
def test_single_magnitudes(i, mag):
    c, q, lens = single_case(i, 4)
    q = (q.float() * mag[0]).to(BF)
    for n in ("k_scale", "k_min", "z_scale"):
        c.planes[n] *= mag[1]
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl, lse=lse)
    check_tree(out, lse, ref_tree(c, q, [1] * len(lens), lens, None))


@pytest.mark.parametrize("qd", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (28, 4), (16, 1)])
def test_one_workspace_for_smaller_calls(Hq, Hkv, qd):
    """A workspace serves every call of fewer new tokens and shorter sequences, in any order,
    whatever an earlier call of another shape left in it."""
    c = Cache(31, 2, Hkv, 4096, 128, 16)
    L = hq().lib()
    ws = hq().tree_workspace(c.hq, Hq, 260)
    rng = np.random.default_rng(5)
    for n, T in [(260, 4096), (1, 4096), (129, 4096), (128, 900), (1, 64), (37, 3000), (1, 4096), (2, 129)]:
        assert L.headq_tree_workspace_bytes(c.hq.struct(), Hq, n, T) <= ws.numel()
        q = torch.from_numpy(rng.standard_normal((2 * n, Hq, 128)).astype(np.float32)).cuda().to(qd)
        lens = [T, max(n, T // 3)]
        mask = tree_masks(rng, 2, min(n, 8))
        if n > 8:
            mask = np.broadcast_to(np.tril(np.ones((n, n), bool)), (2, n, n)).copy()
            mask[:, ::3, :n // 2] = False
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        out = hq().headq_tree_attn(c.hq, q, c.U, mask=torch.from_numpy(mask).cuda(), seq_lens=sl, n=n, T=T, ws=ws)
        fresh = hq().headq_tree_attn(c.hq, q, c.U, mask=torch.from_numpy(mask).cuda(), seq_lens=sl, n=n, T=T)
        assert torch.equal(out, fresh)
        if n <= 37:
            check_tree(out, None, ref_tree(c, q, [n, n], lens, mask))
    hq().headq_workspace_status(ws)


def test_workspace_bounds():
    """The bytes grow with n and T, so that a workspace holds every smaller call's."""
    L = hq().lib()
    for B, Hq, Hkv in [(1, 8, 8), (3, 28, 4), (16, 40, 40), (200, 8, 1), (1, 16, 1)]:
        c = Cache(1, B, Hkv, 64, 128, 16)
        s = c.hq.struct()
        size = [[L.headq_tree_workspace_bytes(s, Hq, n, T) for T in (1, 100, 1000, 4096, 9999, 50000, 131072)]
                for n in (1, 2, 16, 18, 19, 64, 127, 128, 129, 500)]
        size = np.array(size, dtype=np.float64)
        assert (size > 0).all() and (np.diff(size, axis=0) >= 0).all() and (np.diff(size, axis=1) >= 0).all()


def test_single_captured_and_replayed():
    c, q, lens = single_case(0, 6)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws, ws2 = (hq().tree_workspace(c.hq, q.shape[1], 1) for _ in range(2))
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl, out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl, out=out, ws=ws)
    for step in range(3):
        q.copy_(torch.randn(q.shape, device="cuda"))
        sl.copy_(torch.tensor([n - (step if n > 9 else 0) for n in lens], dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        eager = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl, ws=ws2, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        check_tree(out, None, ref_tree(c, q, [1] * len(lens), sl.tolist(), None))


def test_allocations_follow_the_stream():
    """Outputs and workspaces that a call makes are made on the stream it runs on."""
    c, q, lens = single_case(0, 7)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl)
    k0, v0 = hq().headq_cache_read(c.hq, c.U, seq_lens=sl, n=1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    x = torch.randn(4096, 4096, device="cuda")
    for _ in range(5):                                     # work that the current stream is busy with
        x = (x @ x).clamp_(-1, 1)
    got = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl, stream=side)
    k1, v1 = hq().headq_cache_read(c.hq, c.U, seq_lens=sl, n=1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(k0, k1) and torch.equal(v0, v1)


@pytest.mark.parametrize("name", ["k_scale", "k_min", "v", "v_scale"])
@pytest.mark.parametrize("i", range(len(SINGLES)))
def test_a_seen_token_that_is_not_a_number_is_felt(i, name):
    c, q, lens = single_case(i, 8)
    if name not in c.planes:
        return
    clean = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    t = lens[0] // 2                                       # one token of the first sequence
    slab, off = (0, t) if c.table is None else (int(c.table[0, t // c.hq.page_size]), t % c.hq.page_size)
    c.planes[name][slab, :, off] = float("nan")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl)
    assert out[0].isnan().all() and torch.equal(out[1:], clean[1:])


@pytest.mark.parametrize("n,qd,Hq", [(1, BF, 8), (1, BF, 32), (6, BF, 8), (70, BF, 8), (6, F32, 8)])
def test_a_query_that_is_not_a_number_spoils_its_own_row(n, qd, Hq):
    c = Cache(41, 2, 2, 512, 128, 16)
    rng = np.random.default_rng(n)
    q = torch.from_numpy(rng.standard_normal((2 * n, Hq, 128)).astype(np.float32)).cuda().to(qd)
    sl = torch.tensor([500, 201], dtype=torch.int32, device="cuda")
    clean = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl, n=n)
    q[n, 3, 5] = float("nan")
    q[0, 1, 9] = float("inf")
    out = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl, n=n)
    assert out[n, 3].isnan().all() and not torch.isfinite(out[0, 1]).any()
    out[n, 3] = clean[n, 3]
    out[0, 1] = clean[0, 1]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("vmode,B", [("dense", 33), ("2bit", 65)])
def test_offsets_past_32_bits(vmode, B):
    """The last sequence of a cache whose planes pass 2^32 elements (dense values) and 2^31
    bytes (codes): written, read and attended to as in a cache of its own."""
    Hkv, T, d, r = 8, 131072, 128, 16
    rows = B * Hkv * T
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    assert rows * (d if vmode == "dense" else d // 4) > (1 << 32 if vmode == "dense" else 1 << 31)
    kw = dict(vmode=vmode)
    big = hq().HeadQCache(B, Hkv, T, d, r, **kw)
    one = Cache(51, 1, Hkv, 512, d, r, vmode)
    rng = np.random.default_rng(7)
    kv = torch.from_numpy(rng.standard_normal((40, 2 * Hkv, d)).astype(np.float32)).cuda().to(BF)
    for name, t in one.planes.items():
        getattr(big, name).view(B, Hkv, T, -1)[B - 1, :, T - 512:] = t.view(1, Hkv, 512, -1)[0]
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[B] = 40
    hq().headq_cache_write_ragged(one.hq, kv[:, :Hkv], kv[:, Hkv:], one.U)
    hq().headq_cache_write_ragged(big, kv[:, :Hkv], kv[:, Hkv:], one.U, cu=cu, n=40)
    for name, t in one.planes.items():
        assert torch.equal(getattr(big, name).view(B, Hkv, T, -1)[B - 1, :, T - 512:], t.view(1, Hkv, 512, -1)[0]), name
    cu[B] = 512
    for x, y in zip(hq().headq_cache_read(big, one.U, cu=cu, n=512, rows=512),
                    hq().headq_cache_read(one.hq, one.U, n=512)):
        assert torch.equal(x, y)
    # attention: the other tokens' keys are minus infinity's stand-in, so only the last 512 count
    big.k_min[B - 1, :, :T - 512] = 0.0
    big.k_scale[B - 1, :, :T - 512] = 0.0
    big.z_scale[B - 1, :, :T - 512] = 0.0
    for n, q_dtype in [(1, BF), (40, BF), (5, F32)]:
        U0 = torch.zeros_like(one.U)                       # no correction: a logit is q . k^base
        q = torch.full((n, Hkv, d), 0.0, device="cuda", dtype=q_dtype)
        q[..., 0] = 1.0
        base = hq().headq_cache_read(one.hq, U0, n=512, dtype=F32)[0][..., 0]
        one.planes["k_min"][..., 0] += 200.0 - base.min()  # channel 0 of the last 512 is at least 200
        big.k_min.view(B, Hkv, T, -1)[B - 1, :, T - 512:] = one.planes["k_min"][0]
        cu[B] = n
        got = hq().headq_tree_attn(big, q, U0, cu=cu, n=n, sm_scale=1.0)
        check_tree(got, None, ref_tree(one, q, [n], [512], None, sm=1.0, sigma=0.0))


@pytest.mark.parametrize("Hq,Hkv,d,r,n,vmode,qd", [
    (12, 12, 64, 8, 11, "dense", BF), (28, 4, 128, 16, 32, "dense", BF), (28, 4, 128, 16, 32, "2bit", BF),
    (28, 4, 128, 16, 1, "dense", BF), (8, 2, 128, 16, 7, "dense", F32), (4, 4, 64, 0, 3, "dense", BF)])
def test_steps_in_a_row_on_one_workspace(Hq, Hkv, d, r, n, vmode, qd):
    """Write, attend, read, over and over with nothing between: the kernels of a step that start
    early see the cache, queries and workspace as the steps before them left these."""
    B, T, steps = 3, 2048, 24
    rng = np.random.default_rng(n)
    kvs = [torch.from_numpy(rng.standard_normal((B * n, 2 * Hkv, d)).astype(np.float32)).cuda().to(BF)
           for _ in range(steps)]
    qs = [torch.from_numpy(rng.standard_normal((B * n, Hq, d)).astype(np.float32)).cuda().to(qd) for _ in range(steps)]
    lens = [torch.tensor([T - 3 * k, n + 5 * k, 700 + k], dtype=torch.int32, device="cuda") for k in range(steps)]

    def run(sync):
        c = Cache(61, B, Hkv, T, d, r, vmode)
        ws = hq().tree_workspace(c.hq, Hq, n)
        q, kv, sl = torch.empty_like(qs[0]), torch.empty_like(kvs[0]), torch.empty_like(lens[0])
        outs, rows = [], []
        for k in range(steps):
            q.copy_(qs[k])
            kv.copy_(kvs[k])
            sl.copy_(lens[k])
            hq().headq_cache_write_ragged(c.hq, kv[:, :Hkv], kv[:, Hkv:], c.U, seq_lens=sl, n=n)
            outs.append(hq().headq_tree_attn(c.hq, q, c.U, seq_lens=sl, n=n, ws=ws))
            rows.append(hq().headq_cache_read(c.hq, c.U, seq_lens=sl, n=n))
            if sync:
                torch.cuda.synchronize()
        hq().headq_workspace_status(ws)
        return outs, rows

    a, b = run(True), run(False)
    for x, y in zip(a[0], b[0]):
        assert torch.equal(x, y)
    for (k0, v0), (k1, v1) in zip(a[1], b[1]):
        assert torch.equal(k0, k1) and torch.equal(v0, v1)
