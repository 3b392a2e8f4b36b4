"""Full attention and its cache where calls meet, end or are padded: bounds from attn_ref."""
import pytest
import torch

import attn_ref as R
from test_gpu_attn import api, cu_of, inputs, spans_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv", [(16, 8), (16, 16)])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_many_short_items_follow_one_another(d, Hq, Hkv):
    """Items of one or two steps, ten to a CTA, whose products follow one another closely: no
    wait runs out in any of the calls, and all give the same bits."""
    attn = api()
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(1, 200, (200,), generator=g).tolist()
    q, k, v, _ = inputs(40, sum(lens), Hq, Hkv, d, torch.bfloat16)
    cu, ws = cu_of(lens), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    o, lse = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu, workspace=ws)
    assert attn.kda_attn_status(ws) == (0, 0)
    ro, rl, to, tl = R.attn_fwd(q[0], k[0], v[0], spans_of(lens), d ** -0.5)
    R.close(o[0], ro, to)
    R.close(lse[0], rl, tl)
    for _ in range(50):
        again = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu, workspace=ws)
        assert attn.kda_attn_status(ws) == (0, 0)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
