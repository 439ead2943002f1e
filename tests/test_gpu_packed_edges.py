"""The packed-batch operators where numbers leave the ordinary range."""

import numpy as np
import pytest
import torch

from packed_helpers import Cache, check_tree, ref_tree

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
