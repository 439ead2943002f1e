"""How near headq_tree_attn comes to 64 bits: no further than the roundings it documents."""

import math

import numpy as np
import pytest
import torch

from packed_helpers import Cache, tree_masks

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rounded(x, bits):
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2.0 ** bits), e - bits)


def attend(c, q, T, mask, b, keys=lambda x: x, weights=lambda x: x, values=lambda x: x):
    """Rows of sequence b in float64, with keys, weights and values passed through roundings."""
    k, z, v, U = (torch.from_numpy(x).cuda() for x in c.parts())
    n, Hq, d = q.shape
    G = Hq // c.Hkv
    see = torch.ones(n, T, dtype=torch.bool, device="cuda")
    see[:, T - n:] = torch.from_numpy(mask[b]).cuda()
    out = torch.empty(n, Hq, d, dtype=torch.float64, device="cuda")
    for h in range(Hq):
        kv = h // G
        x = q[:, h].double()
        s = (x @ keys(k[b, kv, :T]).T + (x @ U[kv]) @ z[b, kv, :T].T) / math.sqrt(d)
        s = s.masked_fill(~see, -math.inf)
        w = weights(torch.exp(s - s.amax(1, keepdim=True)))
        out[:, h] = w @ values(v[b, kv, :T]) / w.sum(1, keepdim=True)
    return out


@pytest.mark.parametrize("Hq,Hkv,d,r,vmode,n,T", [
    (28, 4, 128, 16, "2bit", 32, 4096), (32, 8, 128, 16, "dense", 16, 6000), (12, 12, 64, 8, "dense", 11, 2048)])
def test_error_against_64_bits(Hq, Hkv, d, r, vmode, n, T):
    """Logits of a standard deviation near 12, the side code's part among them: base keys to 11
    bits, weights to 8, 2-bit values to 8, the output to 8, and nothing else that shows."""
    c = Cache(3, 2, Hkv, T // 16 * 16, d, r, vmode, spread=2.0)
    if r:  # a side code as large as the base code
        c.planes["z_scale"] *= 12.0
    rng = np.random.default_rng(3)
    q = torch.from_numpy(rng.standard_normal((2, n, Hq, d)).astype(np.float32) * 2.0).cuda().to(BF)
    mask = tree_masks(rng, 2, n)
    T = c.hq.T_cap
    from bit_decode_attention_sm_b200 import headq
    got = headq.headq_tree_attn(c.hq, q.view(2 * n, Hq, d), c.U, mask=torch.from_numpy(mask).cuda()).view(q.shape)
    err = told = 0.0
    for b in range(2):
        exact = attend(c, q[b], T, mask, b)
        model = attend(c, q[b], T, mask, b, lambda x: rounded(x, 11), lambda x: rounded(x, 8),
                       (lambda x: rounded(x, 8)) if vmode == "2bit" else (lambda x: x)).to(BF).double()
        err += ((got[b].double() - exact) ** 2).sum().item()
        told += ((model - exact) ** 2).sum().item()
    # both are sums over 10^4 to 10^5 outputs of the same independent roundings: their ratio is
    # within a few per cent of 1
    assert err <= 1.1 ** 2 * told, (err / told) ** 0.5
