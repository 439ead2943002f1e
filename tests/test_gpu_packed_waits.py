"""headq_tree_attn on the tensor cores with a cold cache: values that arrive after the codes of
later tiles change nothing."""

import numpy as np
import pytest
import torch

from packed_helpers import Cache, check_tree, ref_tree, spans

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

CASES = [  # Hq, Hkv, d, r, vmode, page, counts, lens: few tiles, the last with new tokens
    (16, 4, 128, 0, "dense", 64, [1, 70, 1, 33], [376, 600, 400, 512]),      # two row blocks a CTA
    (16, 2, 128, 16, "dense", 64, [16, 3, 1], [500, 1000, 390]),             # one, in two lanes
    (8, 4, 64, 8, "dense", 0, [5, 11, 2, 64], [385, 700, 1023, 520]),
    (28, 4, 128, 16, "2bit", 64, [5, 60, 2], [385, 700, 1023]),
]


@pytest.mark.parametrize("copies", [1, 12], ids=["split", "whole"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_late_values(i, copies):
    """copies: more sequences make for fewer splits, and so for more tiles to a CTA."""
    from bit_decode_attention_sm_b200 import headq
    Hq, Hkv, d, r, vmode, page, counts, lens = CASES[i]
    B = len(counts)
    c = Cache(200 + i, B * copies, Hkv, 1024, d, r, vmode, BF, page)
    counts, lens = counts * copies, lens * copies
    rng = np.random.default_rng(i)
    q = torch.from_numpy(rng.standard_normal((sum(counts), Hq, d)).astype(np.float32) * 1.5).cuda().to(BF)
    cu, sl = spans(counts, lens)
    kw = dict(seq_lens=sl, cu=cu, n=max(counts))
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")     # larger than L2
    outs = []
    for k in range(40):
        flush.fill_(k)
        outs.append(headq.headq_tree_attn(c.hq, q, c.U, **kw))
    ref = ref_tree(c, q, counts, lens, None)
    check_tree(outs[0], None, ref)
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("Hq,Hkv,d,r,vmode", [(28, 4, 128, 16, "dense"), (14, 2, 64, 8, "2bit"), (8, 2, 128, 0, "dense")])
def test_late_tiles_of_single_tokens(Hq, Hkv, d, r, vmode):
    """The decode kernels' warps, not all of which have a part in every tile."""
    from bit_decode_attention_sm_b200 import headq
    B, T = 24, 2048
    c = Cache(230, B, Hkv, T, d, r, vmode, BF, 64)
    rng = np.random.default_rng(1)
    q = torch.from_numpy(rng.standard_normal((B, Hq, d)).astype(np.float32) * 1.5).cuda().to(BF)
    lens = [int(x) for x in rng.integers(T // 2, T + 1, B)]
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    outs = []
    for k in range(40):
        flush.fill_(k)
        outs.append(headq.headq_tree_attn(c.hq, q, c.U, seq_lens=sl))
    check_tree(outs[0], None, ref_tree(c, q, [1] * B, lens, None))
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
