"""The packed-batch operators where numbers leave the ordinary range, or pages the pool."""

import numpy as np
import pytest
import torch

from packed_helpers import Cache, check_tree, logical, ref_tree
from test_gpu_packed import expected_planes, new_tokens

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def hq():
    from bit_decode_attention_sm_b200 import headq
    return headq


def slot(c, b, t):
    """Slab and offset of token t of sequence b in the planes."""
    return (b, t) if c.table is None else (int(c.table[b, t // c.hq.page_size]), t % c.hq.page_size)


def lens_of(lens):
    return torch.tensor(lens, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- not a number

DECODES = [  # Hq, Hkv, d, r, vmode, page: single tokens on either decode kernel
    (8, 2, 128, 16, "dense", 0), (2, 2, 64, 8, "2bit", 64), (6, 2, 64, 16, "2bit", 0), (4, 1, 128, 0, "dense", 128),
    (14, 2, 128, 16, "dense", 0), (10, 2, 64, 8, "2bit", 0),
]


@pytest.mark.parametrize("name", ["k_min", "z_scale"])
@pytest.mark.parametrize("i", range(len(DECODES)))
def test_a_split_of_tokens_that_are_not_numbers_is_felt(i, name):
    """The only token of a sequence's last split, and every token of a split in its middle:
    the row is not a number, as it is where such a token has neighbours."""
    Hq, Hkv, d, r, vmode, page = DECODES[i]
    T = 2048
    c = Cache(80 + i, 3, Hkv, T, d, r, vmode, BF, page)
    if name not in c.planes:
        return
    splits, chunk, _, _ = hq().decode_plan(c.hq, Hq, T)
    assert splits > 3
    lens = [2 * chunk + 1, T, T - 3]
    rng = np.random.default_rng(i)
    q = torch.from_numpy(rng.standard_normal((3, Hq, d)).astype(np.float32)).cuda().to(BF)
    ref = ref_tree(c, q, [1, 1, 1], lens, None)
    for b, ts in [(0, [2 * chunk]), (1, range(chunk, 2 * chunk))]:
        for t in ts:
            slab, off = slot(c, b, t)
            c.planes[name][slab, :, off] = float("nan")
    lse = torch.zeros(3, Hq, device="cuda")
    out = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=lens_of(lens), lse=lse)
    assert out[:2].isnan().all() and lse[:2].isnan().all()
    check_tree(out[2:], lse[2:], [a[2:] for a in ref])
    # the decode call itself: no row with such a token passes for a finite one
    o, l = hq().headq_decode_attn(c.hq, q, c.U, seq_lens=lens_of(lens))
    assert not torch.isfinite(l[:2]).any() and torch.isfinite(o[2]).all() and torch.isfinite(l[2]).all()


# ---------------------------------------------------------------- far from zero

FORMS = [  # Hq, Hkv, d, r, vmode, n, query dtype: every kernel of the tree attention
    (8, 2, 128, 16, "dense", 1, BF), (2, 2, 64, 8, "2bit", 1, BF), (14, 2, 128, 16, "dense", 1, BF),
    (10, 2, 64, 8, "2bit", 1, BF), (8, 2, 128, 16, "dense", 3, BF), (14, 2, 64, 8, "2bit", 40, BF),
    (8, 2, 128, 16, "dense", 2, F32), (4, 2, 32, 0, "2bit", 1, BF),
]


def same_keys(c, x):
    """Every cached key has `x` in all channels, without a side code."""
    c.planes["k_scale"].zero_()
    c.planes["k_min"].fill_(x)
    if c.r:
        c.planes["z_scale"].zero_()


@pytest.mark.parametrize("i", range(len(FORMS)))
def test_rows_whose_logits_are_all_minus_infinity(i):
    """q . k beyond the range of fp32: such a row gives 0 and minus infinity in every form."""
    Hq, Hkv, d, r, vmode, n, qd = FORMS[i]
    c = Cache(90 + i, 2, Hkv, 512, d, r, vmode)
    same_keys(c, -1e25)
    q = torch.full((2 * n, Hq, d), 1e25, device="cuda", dtype=qd)
    lse = torch.zeros(2 * n, Hq, device="cuda")
    out = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=lens_of([500, n]), n=n, lse=lse)
    assert (out == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_rows_whose_logits_are_equal_and_huge(i, sign):
    """Equal logits near -1e34 or 1e34: the mean of the values that a row sees."""
    Hq, Hkv, d, r, vmode, n, qd = FORMS[i]
    c = Cache(90 + i, 2, Hkv, 512, d, r, vmode)
    same_keys(c, sign * 2.0 ** 50)
    q = torch.full((2 * n, Hq, d), 2.0 ** 60, device="cuda", dtype=qd)
    lens = [500, n]
    lse = torch.zeros(2 * n, Hq, device="cuda")
    out = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=lens_of(lens), n=n, lse=lse)
    v = c.parts()[2]
    if vmode == "2bit":
        vmin = c.planes["v_min"].double().cpu().numpy()[..., np.arange(d) // 32]
    logit = sign * 2.0 ** 110 * np.sqrt(d)
    for b in range(2):
        for j in range(n):
            seen = v[b, :, :lens[b] - n + j + 1]                         # [Hkv, tokens, d]
            m, a = seen.mean(1)[:, None], np.abs(seen).mean(1)[:, None]
            got = out[b * n + j].double().cpu().numpy().reshape(Hkv, -1, d)
            # equal weights are exact; each value is rounded to bf16 (half a step, 2^-8 of it: the
            # mean moves by 2^-8 of the mean size), 500 fp32 sums, and the output is rounded once
            tol = (2.0 ** -8 + 512 * 2.0 ** -23) * a + 2.0 ** -8 * np.abs(m) * 1.01
            if n == 1 and vmode == "2bit":
                # the decode sums scale * code apart from the minima, the scale to fp16 (2^-11 of it)
                steps = np.abs(seen - vmin[b, :, :lens[b] - n + j + 1]).mean(1)[:, None]
                tol = tol + (2.0 ** -11 + 512 * 2.0 ** -23) * steps + 512 * 2.0 ** -23 * (a + steps)
            assert (np.abs(got - m) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() / logit - 1) <= 2.0 ** -18).all()


@pytest.mark.parametrize("e", [-100, -60, 60, 120])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_keys_and_queries_of_opposite_magnitudes(i, e):
    """Keys times 2^e against queries times 2^-e: the same logits, whatever either's size."""
    Hq, Hkv, d, r, vmode, n, qd = FORMS[i]
    c = Cache(130 + i, 2, Hkv, 512, d, r, vmode)
    rng = np.random.default_rng(i)
    q = torch.from_numpy(rng.standard_normal((2 * n, Hq, d)).astype(np.float32) * 1.5).cuda().to(qd)
    lens = [500, 300]
    ref = ref_tree(c, q, [n, n], lens, None)
    for name in ("k_scale", "k_min", "z_scale"):
        if name in c.planes:
            c.planes[name] *= 2.0 ** e
    q = (q.float() * 2.0 ** -e).to(qd)
    lse = torch.zeros(2 * n, Hq, device="cuda")
    out = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=lens_of(lens), n=n, lse=lse)
    check_tree(out, lse, ref)


@pytest.mark.parametrize("mag", [1e-27, 2.0 ** -64, 1e-9, 1e9, 1e30])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_value_magnitudes(i, mag):
    """Values far from 1 keep their relative precision: from 2^-66 up where several tokens run
    on the tensor cores, everywhere else in every form."""
    Hq, Hkv, d, r, vmode, n, qd = FORMS[i]
    if mag < 2.0 ** -66 and n > 1 and qd == BF:
        return
    c = Cache(100 + i, 2, Hkv, 512, d, r, vmode)
    for name in ("v", "v_scale", "v_min"):
        if name in c.planes:
            c.planes[name].copy_(c.planes[name].float() * mag)
    rng = np.random.default_rng(i)
    q = torch.from_numpy(rng.standard_normal((2 * n, Hq, d)).astype(np.float32)).cuda().to(qd)
    lens = [500, 300]
    out = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=lens_of(lens), n=n)
    assert out.abs().max() > 0.01 * mag
    ref = ref_tree(c, q, [n, n], lens, None)
    # in units of the magnitude, so that the tolerances' absolute parts stay negligible
    check_tree(out.double() / mag, None, [ref[0] / mag, None, (ref[2] - 1e-30) / mag + 1e-30, None])


# ---------------------------------------------------------------- dequantised, bit for bit

@pytest.mark.parametrize("kmode", ["token", "channel"])
@pytest.mark.parametrize("d,r,page", [(128, 16, 0), (64, 8, 64), (128, 0, 0), (32, 4, 0)])
def test_read_rounds_the_product_before_the_sum(d, r, page, kmode):
    """Base keys and 2-bit values read in fp32 are min + code * scale with the product rounded
    first, as the write forms them when it takes the residual."""
    c = Cache(110, 2, 3, 128, d, r, "2bit", F32, page, kmode)
    ch = np.arange(d)
    gs = min(32, d)

    def base(codes, scale, mn, channel):
        c8 = logical(codes, c.table).cpu().numpy()
        s, m = (logical(x, c.table).cpu().numpy() for x in (scale, mn))
        code = ((c8[..., ch // 4] >> (2 * (ch % 4))) & 3).astype(np.float32)
        if channel:
            blk = np.arange(128) // 64
            return m[:, :, blk] + (code * s[:, :, blk]).astype(np.float32)
        return m[..., ch // gs] + (code * s[..., ch // gs]).astype(np.float32)

    p = c.planes
    k = base(p["k_codes"], p["k_scale"], p["k_min"], kmode == "channel")
    v = base(p["v_codes"], p["v_scale"], p["v_min"], False)
    # keys and values by CTAs of their own, and in one CTA
    for kw in (dict(), dict(k_out=0), dict(v_out=0)):
        kw = {n: torch.empty(256, 3, d, device="cuda") for n in kw}
        kg, vg = hq().headq_cache_read(c.hq, c.U, n=128, corr_sign=0, dtype=F32, **kw)
        for got, want in ((kg, k), (vg, v)):
            if got is not None:
                assert np.array_equal(got.cpu().numpy(), want.transpose(0, 2, 1, 3).reshape(256, 3, d))


@pytest.mark.parametrize("d,r", [(128, 16), (64, 8), (32, 4)])
def test_a_lone_token_is_its_value(d, r):
    """fp32 queries that see one token: its dequantised value, bit for bit."""
    c = Cache(111, 5, 3, 64, d, r, "2bit")
    q = torch.randn(5, 6, d, generator=torch.Generator().manual_seed(1)).cuda()
    out = hq().headq_tree_attn(c.hq, q, c.U, T=1)
    v = hq().headq_cache_read(c.hq, c.U, n=1, T=1, dtype=F32)[1]
    assert torch.equal(out, v.repeat_interleave(2, 1))


# ---------------------------------------------------------------- bad pages

@pytest.mark.parametrize("Hq,d,r,n", [(4, 128, 16, 1), (14, 128, 16, 1), (4, 128, 16, 5), (4, 128, 16, 100),
                                      (4, 32, 4, 3)])
def test_a_bad_page_is_reported_and_touches_its_own_sequence_only(Hq, d, r, n):
    c = Cache(120, 3, 2, 192, d, r, page=64)
    good = [b for b in range(3) if b != 1]
    lens = [192, 180, 150]
    kk, vv = new_tokens(np.random.default_rng(2), 3 * n, 2, d, BF)
    want = expected_planes(c, kk, vv, [n] * 3, lens)
    table = c.table.clone()
    for bad in (-1, 99999):
        c.table.copy_(table)
        c.table[1, 1 if n > 1 else 2] = bad
        q = torch.randn(3 * n, Hq, d, generator=torch.Generator().manual_seed(n)).cuda().to(BF)
        hq().headq_cache_write_ragged(c.hq, kk, vv, c.U, seq_lens=lens_of(lens), n=n)
        for name, t in c.planes.items():
            assert torch.equal(logical(t, table)[good].view(torch.uint8), want[name][good].view(torch.uint8)), name
        ws = hq().tree_workspace(c.hq, Hq, n)
        lse = torch.zeros(3 * n, Hq, device="cuda")
        out = hq().headq_tree_attn(c.hq, q, c.U, seq_lens=lens_of(lens), n=n, ws=ws, lse=lse)
        with pytest.raises(hq().HeadQError):
            hq().headq_workspace_status(ws)
        hq().headq_workspace_status(ws)
        c.table.copy_(table)
        ref = ref_tree(c, q, [n] * 3, lens, None)
        rows = [b * n + i for b in good for i in range(n)]
        check_tree(out[rows], lse[rows], [a[rows] for a in ref])
        hq().headq_tree_attn(c.hq, q, c.U, seq_lens=lens_of(lens), n=n, ws=ws)
        hq().headq_workspace_status(ws)                    # nothing left of it


# ---------------------------------------------------------------- nothing

def test_batches_without_rows():
    """No sequence takes part: every call returns, whatever strides the empty tensors have."""
    c = Cache(140, 2, 2, 64, 64, 8)
    before = {n: t.clone() for n, t in c.planes.items()}
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    empty = torch.from_numpy(np.empty((0, 2, 64), np.float32)).cuda().to(BF)
    sliced = torch.empty(3, 64, 2, dtype=BF, device="cuda").transpose(1, 2)[:0]
    for t in (empty, sliced):
        hq().headq_cache_write_ragged(c.hq, t, t, c.U, cu=cu, n=3)
        k, v = hq().headq_cache_read(c.hq, c.U, cu=cu, n=3, k_out=t, v_out=t)
        out = hq().headq_tree_attn(c.hq, t, c.U, cu=cu, n=3, out=t)
        assert k.shape == v.shape == out.shape == (0, 2, 64)
    assert hq().headq_tree_attn(c.hq, empty, c.U).shape == (0, 2, 64)
    assert hq().headq_cache_read(c.hq, c.U, n=0)[0].shape == (0, 2, 64)
    for n, t in c.planes.items():
        assert torch.equal(t, before[n]), n
