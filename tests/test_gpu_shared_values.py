"""Values, scores and steps at which attention behind shared prefixes can go wrong, on the GPU."""
import pytest
import torch

import gated_deltanet_linear_core_gb300 as gdn
from test_gpu_shared import BF, F, INF, NAN, shared_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("D,hkv", [(8, 8), (64, 4), (256, 2)])
def test_non_finite_new_tokens_reach_every_row_that_sees_them(D, hkv):
    """Rows in all four warps' quarters of a block, several segments to a CTA, every other sequence with a new
    token's value that is not finite: it spoils its dim of the rows that see it at every call, and nothing else."""
    B, K, group, page = 96, 16, 8, 16
    x = shared_inputs([(256, [16 + 5 * (b % 40) for b in range(B)])], K, group * hkv, hkv, D, page, BF, 60 + D)
    clean = gdn.gdn_attn_decode_shared(**x)
    want = torch.zeros_like(clean, dtype=torch.bool)
    for b in range(0, B, 2):
        back, h, d = b % K, (b // 2) % hkv, (7 * b) % D  # `back` tokens before the newest
        at = int(x["seq_lens"][b]) - 1 - back
        x["v_cache"][int(x["page_table"][b, at // page]), h, at % page, d] = NAN if b % 4 else INF
        if back < K - 1:  # (all rows see the first new token)
            want[b, K - 1 - back:, group * h:group * (h + 1), d] = True
        else:
            want[b, :, group * h:group * (h + 1), d] = True
    for _ in range(50):
        out = gdn.gdn_attn_decode_shared(**x)
        assert torch.equal(~torch.isfinite(out), want)
        assert torch.equal(out[~want], clean[~want])
