"""Values, scores and steps at which attention behind shared prefixes can go wrong, on the GPU."""
import pytest
import torch

import gated_deltanet_linear_core_gb300 as gdn
import serving_ref as ref
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


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,hq,hkv", [(64, 8, 2), (256, 16, 2), (128, 64, 4)])
@pytest.mark.parametrize("low", [-INF, -1e30, -1e4])
@pytest.mark.parametrize("pages,gone", [(64, 64), (64, 32), (64, 1), (1250, 700)])
def test_keys_far_out_of_sight_leave_the_rest(pages, gone, low, D, hq, hkv, dtype):
    """The first `gone` of the prefix's pages of 16 hold keys whose scores are -inf, or finite and so low that their
    weights vanish in 64 bits as well: what remains is attention over the tokens behind them."""
    x = shared_inputs([(16 * pages, [9, 60, 200, 140])], 2, hq, hkv, D, 16, dtype, 8)
    x["q"] = x["q"].abs() + 0.5
    x["k_cache"][x["page_table"][0, :gone].long()] = low
    out, lse = gdn.gdn_attn_decode_shared(**x, return_lse=True)
    rest = ref.attention(x["q"], x["k_cache"], x["v_cache"], x["page_table"][:, gone:].contiguous(), x["seq_lens"] - 16 * gone)
    ref.check_attention(out, lse, rest, dtype)
    del x["prefix_lens"], x["cu_groups"]
    ref.check_attention(*gdn.gdn_attn_decode(**x, return_lse=True), rest, dtype)


def alike(shift, dtype, n=20000):
    """Inputs whose rows' scores are each the same number, the outputs and the log of the count, and what the outputs
    may be off by.  (The queries are powers of two and one dim of the keys holds the number: the products are exact.)"""
    x = shared_inputs([(n, [9, 60, 200, 140])], 3, 8, 2, 64, 16, dtype, 9)
    x["k_cache"].zero_()
    x["q"] = torch.pow(2.0, torch.randint(-3, 4, x["q"].shape, generator=torch.Generator().manual_seed(1)).float()).to(dtype).cuda()
    want, count, _ = ref.attention(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"])
    x["k_cache"][..., 5] = shift
    # the weights as in ref.attention(), where scores of 0 are exact: 2 (2^-21 + 2^-16 + (n / 128 + 256) 2^-24) |v|
    err = 2 * (2.0 ** -21 + 2.0 ** -16 + (n / 128 + 258) * 2.0 ** -24) * x["v_cache"].double().nan_to_num().abs().max()
    score = x["q"][..., 5].double() * x["k_cache"][0, 0, 0, 5].double() / 8
    return x, want, score + count, ref.HALF_STEP[dtype] * want.abs() + err, 2.0 ** -20 * (1 + score.abs()) + 1e-4


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("shift", [-3e35, -1e30, -1e12, -3e7, 1e5, 3e7, 1e12, 1e30, 3e35])
@pytest.mark.parametrize("shared", [True, False])
def test_scores_that_are_alike_and_large(shared, shift, dtype):
    """However large: the weights are all 1 / n, over many tiles; and so in gdn_attn_decode."""
    x, want, want_lse, tol, lse_tol = alike(shift, dtype)
    if shared:
        out, lse = gdn.gdn_attn_decode_shared(**x, return_lse=True)
    else:
        del x["prefix_lens"], x["cu_groups"]
        out, lse = gdn.gdn_attn_decode(**x, return_lse=True)
    assert bool(((out.double() - want).abs() <= tol).all())
    assert bool(((lse.double() - want_lse).abs() <= lse_tol).all())


@pytest.mark.parametrize("K,hq,hkv,D", [(1, 8, 8, 64), (3, 16, 2, 64), (8, 8, 2, 128), (16, 16, 2, 256), (16, 16, 2, 64), (1, 48, 1, 256)])
@pytest.mark.parametrize("shift", [-1e30, 1e12, 1e30])
def test_large_scores_at_every_number_of_rows(shift, K, hq, hkv, D):
    """gdn_attn_decode's forms for 16 to 128 rows: alternate rows have huge scores that are alike, and ordinary ones."""
    x = shared_inputs([(3000, [16, 60])], K, hq, hkv, D, 16, BF, 10, hidden=0.0)
    del x["prefix_lens"], x["cu_groups"]
    x["q"][:, :, ::2] = 0
    x["q"][:, :, ::2, 5] = 2.0
    x["k_cache"][..., 5] = 0
    want, lse, bound = ref.attention(**{k: x[k] for k in ("q", "k_cache", "v_cache")}, table=x["page_table"], lens=x["seq_lens"])
    x["q"][:, :, 1::2, 5] = 0
    want[:, :, 1::2], lse[:, :, 1::2], bound[:, :, 1::2] = (
        t[:, :, 1::2] for t in ref.attention(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"]))
    x["k_cache"][..., 5] = shift
    score = torch.zeros_like(lse)
    score[:, :, ::2] = 2 * x["k_cache"][0, 0, 0, 5].double() * D ** -0.5
    out, e = gdn.gdn_attn_decode(**x, return_lse=True)
    assert bool(((out.double() - want).abs() <= ref.HALF_STEP[BF] * want.abs() + bound).all())
    assert bool(((e.double() - lse - score).abs() <= 2.0 ** -20 * (1 + score.abs() + lse.abs()) + 1e-4).all())


@pytest.mark.parametrize("hq,hkv,D,n", [(16, 8, 16, 105570), (14, 7, 64, 90000), (8, 4, 128, 70000), (8, 2, 256, 60000)])
def test_f32_sums_over_long_prefixes(hq, hkv, D, n):
    """A rounding of f32 is off by 2.5e-8 of the value (rms).  A sum of n terms of either sign: 2.5e-8 sqrt(n / 2), as its
    parts are smaller before.  Of a tile's 64 tokens 1.4e-7, of the up to 90 tiles that a CTA has 1.7e-7, of D products
    in a score at most 2.8e-7 of it (D = 256; as many parts as a thread holds are added up apart), of sums of weights
    below these; the weights' exponentials 5e-8, averaged over.  Together 3.6e-7; twice that."""
    x = shared_inputs([(n, [9, 60, 200, 140, 33])], 1, hq, hkv, D, 16, F, 21)
    out, lse = gdn.gdn_attn_decode_shared(**x, return_lse=True)
    want, want_lse, _ = ref.attention(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"])
    assert float((out.double() - want).norm() / want.norm()) <= 7.2e-7
    assert float((lse.double() - want_lse).norm() / want_lse.norm()) <= 2e-7
