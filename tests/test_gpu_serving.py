"""Paged-cache attention of the newest tokens, cache append and drafted-token
acceptance on the GPU, against their definitions in 64 bits."""
import pytest
import torch

import gated_deltanet_linear_core_gb300 as gdn
import serving_ref as ref
import workloads as W

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def attn_inputs(lens, K, hq, hkv, D, page, dtype, seed, gate=False, hidden=NAN):
    g = torch.Generator().manual_seed(seed)
    kc, vc, table, ln = ref.make_cache(lens, page, hkv, D, dtype, g, "cuda", hidden=hidden)
    q = torch.randn((len(lens), K, hq, D), generator=g).to(dtype).cuda()
    gt = torch.randn((len(lens), K, hq, D), generator=g).to(dtype).cuda() if gate else None
    return q, kc, vc, table, ln, gt


def run_attn(x, **kw):
    q, kc, vc, table, ln, gt = x
    return gdn.gdn_attn_decode(q, kc, vc, table, ln, gate=gt, return_lse=True, **kw)


def check(x, dtype, **kw):
    q, kc, vc, table, ln, gt = x
    out, lse = run_attn(x, **kw)
    gdn.gdn_sync_status()
    scale = kw.get("scale") or None
    r = ref.attention(q, kc, vc, table, ln, scale=scale, gate=gt)
    ref.check_attention(out, lse, r, dtype)
    return out, lse


# lengths, K, H_q, H_kv, D, page, gate: one token, empty sequences, rows that see nothing, tiles and
# pages that end inside one another, odd sizes, one to 512 rows per key-value head
SHAPES = [
    ([1], 1, 1, 1, 16, 16, False),
    ([0, 5, 0, 1, 0], 1, 4, 2, 64, 8, True),
    ([3, 1, 0, 2, 16], 4, 8, 2, 128, 16, True),
    ([127, 128, 129, 255, 256, 257], 1, 16, 2, 256, 16, True),
    ([31, 32, 33, 63, 64, 65], 3, 6, 3, 128, 32, False),
    ([700, 1, 333], 1, 15, 3, 80, 24, False),
    ([501, 100, 99, 101], 2, 6, 2, 96, 100, True),
    ([77, 200, 13], 2, 4, 2, 72, 7, False),
    ([300, 45], 5, 16, 2, 256, 48, True),
    ([1000, 129], 16, 32, 4, 128, 128, False),
    ([260, 515], 16, 16, 2, 256, 64, True),
    ([150, 131, 16], 16, 32, 1, 64, 16, False),
    ([40, 41], 4, 5, 5, 8, 4, False),
    ([520, 9], 8, 12, 2, 200, 256, True),
    ([5000], 1, 16, 2, 256, 64, True),
    ([9000, 17, 4000], 5, 16, 2, 256, 16, True),
    ([6001], 6, 6, 1, 192, 1, False),
    ([3000, 250, 129, 5, 1200], 5, 16, 2, 256, 8, True),
    ([2500, 40, 1111], 16, 16, 2, 256, 16, False),
    ([2500, 40, 1111], 16, 16, 2, 128, 8, True),
    ([900] * 40, 8, 8, 1, 256, 4, False),
    ([130] * 300, 3, 8, 1, 256, 12, True),
    ([4000, 4000], 2, 40, 4, 104, 40, True),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention_matches_its_definition(i, dtype):
    lens, K, hq, hkv, D, page, gate = SHAPES[i]
    check(attn_inputs(lens, K, hq, hkv, D, page, dtype, 100 + i, gate), dtype)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_many_sequences_of_all_lengths(dtype):
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 700, (301,), generator=g).tolist()
    check(attn_inputs(lens, 2, 4, 2, 64, 16, dtype, 6), dtype)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_a_new_token_does_not_reach_the_rows_before_it(dtype, bad):
    """Keys and values of a later new token, non-finite ones too, leave earlier rows alone."""
    for lens, K, hq, hkv, D, page in [([130], 4, 8, 2, 128, 16), ([4], 4, 8, 2, 256, 16), ([300], 16, 16, 2, 256, 64),
                                      ([2049], 3, 2, 2, 64, 32)]:
        x = attn_inputs(lens, K, hq, hkv, D, page, dtype, 9)
        out0, lse0 = run_attn(x)
        q, kc, vc, table, ln, _ = x
        n = lens[0]
        pg = int(table[0, (n - 1) // page])
        kc[pg, :, (n - 1) % page] = bad
        vc[pg, :, (n - 1) % page] = bad
        out1, lse1 = run_attn(x)
        assert torch.equal(out0[:, :K - 1], out1[:, :K - 1])
        assert torch.equal(lse0[:, :K - 1], lse1[:, :K - 1])


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_a_non_finite_value_reaches_the_rows_that_see_it(dtype):
    x = attn_inputs([130], 4, 8, 2, 128, 16, dtype, 9)
    q, kc, vc, table, ln, _ = x
    for pos, first_row in ((50, 0), (127, 1), (129, 3)):
        v2 = vc.clone()
        v2[int(table[0, pos // 16]), 1, pos % 16, 77] = INF
        out = gdn.gdn_attn_decode(q, kc, v2, table, ln)
        hit = torch.isinf(out)
        want = torch.zeros_like(hit)
        want[0, first_row:, 4:, 77] = True
        assert torch.equal(hit, want)


# K new tokens that lie on both sides of a border of 128 tokens, in sequences of several tiles, several per
# SM: 24, 40, 64 and 128 rows per key-value head
STRADDLING = [(3, 16, 2, 256, 8), (3, 16, 2, 256, 64), (5, 16, 2, 256, 16), (5, 16, 2, 256, 64), (8, 16, 2, 200, 64),
              (16, 16, 2, 256, 8), (16, 16, 2, 256, 64), (16, 32, 4, 128, 16)]


def straddling_inputs(K, hq, hkv, D, page, dtype):
    lens = [128 * (3 + b % 4) + 1 + b // 4 % (K - 1) for b in range(120)]
    return lens, attn_inputs(lens, K, hq, hkv, D, page, dtype, 700 + K + page)


def new_token(table, lens, K, i, page):
    """Page and place in it of every sequence's new token i."""
    pos = torch.tensor(lens, device="cuda") - (K - i)
    return table[torch.arange(len(lens), device="cuda"), pos // page].long(), pos % page


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("K,hq,hkv,D,page", STRADDLING)
def test_new_tokens_across_a_tile_border_do_not_reach_the_rows_before_them(K, hq, hkv, D, page, dtype):
    lens, (q, kc, vc, table, ln, _) = straddling_inputs(K, hq, hkv, D, page, dtype)
    for i in range(1, K) if K <= 5 else (1, 2, K // 2, K - 1):
        pg, at = new_token(table, lens, K, i, page)
        old = kc[pg, :, at].clone(), vc[pg, :, at].clone()
        got = []
        for bad in (0.0, NAN, INF, -INF):
            kc[pg, :, at] = bad
            vc[pg, :, at] = bad
            got.append([t[:, :i].clone() for t in run_attn((q, kc, vc, table, ln, None))])
        for out, lse in got[1:]:
            assert torch.equal(got[0][0], out) and torch.equal(got[0][1], lse), f"token {i}"
        kc[pg, :, at], vc[pg, :, at] = old
    gdn.gdn_sync_status()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("K,hq,hkv,D,page", STRADDLING)
def test_a_value_across_a_tile_border_reaches_the_rows_that_see_it(K, hq, hkv, D, page, dtype):
    lens, (q, kc, vc, table, ln, _) = straddling_inputs(K, hq, hkv, D, page, dtype)
    for i in range(K) if K <= 5 else (0, 1, K // 2, K - 1):
        pg, at = new_token(table, lens, K, i, page)
        old = vc[pg, 1, at].clone()
        vc[pg, 1, at, 77] = -INF
        hit = torch.isneginf(gdn.gdn_attn_decode(q, kc, vc, table, ln))
        want = torch.zeros_like(hit)
        want[:, i:, hq // hkv:2 * (hq // hkv), 77] = True
        assert torch.equal(hit, want), f"token {i}"
        vc[pg, 1, at] = old
    check((q, kc, vc, table, ln, None), dtype)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_rows_that_see_nothing_are_zero_whatever_their_gate_holds(dtype, bad):
    """Padding rows: out 0 and lse -inf, in sequences without a token and in those with fewer than the new ones."""
    for lens, K, hq, hkv, D, page in [([0, 3, 1, 700, 2], 5, 16, 2, 256, 16), ([3], 8, 4, 1, 64, 16),
                                      ([2, 0], 16, 16, 2, 128, 64), ([1, 2, 0], 3, 4, 2, 72, 7)]:
        x = attn_inputs(lens, K, hq, hkv, D, page, dtype, 23, gate=True)
        seen = torch.tensor([[n - (K - 1 - i) > 0 for i in range(K)] for n in lens], device="cuda")
        want, lse0 = check(x, dtype)
        x[5][~seen] = bad
        out, lse = run_attn(x)
        assert torch.equal(out, want) and torch.equal(lse, lse0)
        assert (out[~seen] == 0).all() and torch.isneginf(lse[~seen]).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_scale_and_peaked_scores(dtype):
    x = attn_inputs([700, 90], 2, 8, 2, 128, 16, dtype, 21)
    check(x, dtype, scale=0.5)
    # scores that grow along the sequence, so that the running maximum moves at every tile
    q, kc, vc, table, ln, _ = x
    q.fill_(1.0)
    for b, n in enumerate([700, 90]):
        for t in range(n):
            kc[int(table[b, t // 16]), :, t % 16] = t / 64.0
    check(x, dtype)
    for b, n in enumerate([700, 90]):
        for t in range(n):
            kc[int(table[b, t // 16]), :, t % 16] = -t / 64.0
    check(x, dtype)


@pytest.mark.parametrize("low", [-1e7, -3e38, -INF])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_scores_far_below_the_others_change_nothing(dtype, low):
    """Keys whose scores are lower than the others' by so much that their weights are 0: the outputs are
    those over the other keys, to the same bound, wherever the low ones lie."""
    page = 64
    for B, K, hq, hkv, D, lo, hi in [(200, 1, 8, 2, 128, 0, 128), (100, 5, 16, 2, 256, 0, 256),
                                     (100, 5, 16, 2, 256, 448, 576), (60, 16, 16, 2, 128, 0, 128)]:
        x = attn_inputs([640] * B, K, hq, hkv, D, page, dtype, 51)
        q, kc, vc, table, ln, _ = x
        q[..., 0] = 1.0
        kc[table[:, lo // page:hi // page].flatten().long(), :, :, 0] = low
        out, lse = run_attn(x)
        others = torch.cat([table[:, :lo // page], table[:, hi // page:]], 1)
        ref.check_attention(out, lse, ref.attention(q, kc, vc, others, ln - (hi - lo)), dtype)


# lengths, K, H_q, H_kv, D, page, gate
DIGITS = [([5000], 1, 16, 2, 256, 64, True), ([3000, 2501, 1201], 5, 16, 2, 256, 16, True),
          ([900 + b for b in range(40)], 1, 4, 4, 16, 32, False), ([20000], 1, 8, 1, 64, 16, False),
          ([2500, 1111], 16, 16, 2, 128, 8, True), ([1500] * 8, 2, 6, 2, 72, 7, False)]


@pytest.mark.parametrize("i", range(len(DIGITS)))
def test_f32_is_held_in_32_bits(i):
    """Elementwise to the bound without any rounding to fewer bits, and in the mean: the errors of the weights are
    independent and mostly of 2^-22 or less (scores, exponentials), so rel-L2 stays below 2^-19; weights cut to 16
    bits would leave 2^-18 (2^-16 of uniform error, less by sqrt(12) in the mean)."""
    lens, K, hq, hkv, D, page, gate = DIGITS[i]
    x = attn_inputs(lens, K, hq, hkv, D, page, F, 300 + i, gate)
    q, kc, vc, table, ln, gt = x
    out, _ = run_attn(x)
    r_out, _, _ = ref.attention(q, kc, vc, table, ln, gate=gt)
    # the largest value of any position in use: pages hold NaN elsewhere
    top = torch.nan_to_num(vc, nan=0.0).abs().max().double()
    tol = 2.0 ** -20 * r_out.abs() + 2 * ref.weight_error(q, kc, table, ln).unsqueeze(-1) * top
    err = (out.double() - r_out).abs()
    assert bool((err <= tol).all()), f"{(err / tol).max().item():.2f} times its bound off"
    rel = (err.norm() / r_out.norm()).item()
    assert rel <= 2.0 ** -19, f"rel-L2 {rel:.2e}"


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(DIGITS)))
def test_lse_is_held_in_32_bits(i, dtype):
    """To the error of the weights (sums are f32 whatever the type), and three roundings on the way out."""
    lens, K, hq, hkv, D, page, _ = DIGITS[i]
    x = attn_inputs(lens, K, hq, hkv, D, page, dtype, 400 + i)
    q, kc, vc, table, ln, _ = x
    _, lse = run_attn(x)
    _, r_lse, _ = ref.attention(q, kc, vc, table, ln)
    err = (lse.double() - r_lse).abs()
    tol = ref.weight_error(q, kc, table, ln) + 2.0 ** -21 * (1 + r_lse.abs())
    assert bool((err <= tol).all()), f"{(err / tol).max().item():.2f} times its bound off"


def test_lengths_and_pages_are_clamped():
    """A length beyond the table, a negative one, and pages that do not exist."""
    x = attn_inputs([64, 64, 64], 1, 4, 2, 128, 16, BF, 3)
    q, kc, vc, table, ln, _ = x
    want = ref.attention(q, kc, vc, table, ln)
    out, lse = gdn.gdn_attn_decode(q, kc, vc, table, torch.tensor([1000, -7, 64], dtype=torch.int32, device="cuda"),
                                   return_lse=True)
    torch.testing.assert_close(out[0].double(), want[0][0], rtol=2 ** -8, atol=1e-3)
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    bad = table.clone()
    bad[1, 2] = kc.shape[0] + 5
    bad[2, 1] = -3
    out = gdn.gdn_attn_decode(q, kc, vc, bad, ln)
    gdn.gdn_sync_status()
    torch.testing.assert_close(out[0].double(), want[0][0], rtol=2 ** -8, atol=1e-3)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_repeated_calls_agree_bit_for_bit_and_write_nothing_else(dtype):
    x = attn_inputs([3000, 1, 700, 0], 3, 8, 2, 128, 16, dtype, 33, gate=True)
    q, kc, vc, table, ln, gt = x
    out, lse = run_attn(x)
    keep = [t.clone() for t in (q, kc, vc, table, ln, gt)]
    need = gdn.gdn_attn_decode_workspace_size(4, 3, 8, 2, 128, 16, dtype)
    for fill in (0, 255):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        o2 = torch.full((6,) + q.shape[1:], 7.0, dtype=dtype, device="cuda")
        l2 = torch.full((6,) + q.shape[1:3], 7.0, device="cuda")
        gdn.gdn_attn_decode(q, kc, vc, table, ln, gate=gt, out=o2[1:5], lse=l2[1:5], workspace=ws[:need])
        assert torch.equal(o2[1:5], out) and torch.equal(l2[1:5], lse)
        assert (o2[[0, 5]] == 7).all() and (l2[[0, 5]] == 7).all() and (ws[need:] == fill).all()
    for a, b in zip(keep, (q, kc, vc, table, ln, gt)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_sequence_alone_matches_itself_in_a_batch():
    lens = [900, 30, 1500, 64]
    x = attn_inputs(lens, 2, 16, 2, 256, 16, BF, 44)
    q, kc, vc, table, ln, _ = x
    whole = gdn.gdn_attn_decode(q, kc, vc, table, ln)
    for b in range(4):
        r = ref.attention(q[b:b + 1], kc, vc, table[b:b + 1], ln[b:b + 1])
        one, lse = gdn.gdn_attn_decode(q[b:b + 1], kc, vc, table[b:b + 1].contiguous(), ln[b:b + 1], return_lse=True)
        ref.check_attention(one, lse, r, BF)
        ref.check_attention(whole[b:b + 1], None, r, BF)


def test_cache_beyond_32_bit_offsets():
    """Pages past 2^31 elements and past 2^32 bytes."""
    page, hkv, D = 64, 8, 256
    n_pages = (1 << 31) // (page * hkv * D) + 40
    g = torch.Generator().manual_seed(8)
    kc = torch.zeros((n_pages, hkv, page, D), dtype=BF, device="cuda")
    vc = torch.zeros((n_pages, hkv, page, D), dtype=BF, device="cuda")
    ids = torch.tensor([[n_pages - 1, 3, n_pages - 17, n_pages - 30, n_pages - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([290], dtype=torch.int32, device="cuda")
    k = torch.randn((290, hkv, D), generator=g).to(BF).cuda()
    v = torch.randn((290, hkv, D), generator=g).to(BF).cuda()
    gdn.gdn_kv_append(k, v, kc, vc, ids, lens)
    got = kc[ids[0].long()].transpose(1, 2).reshape(-1, hkv, D)[:290]
    assert torch.equal(got, k)
    q = torch.randn((1, 2, 16, D), generator=g).to(BF).cuda()
    out, lse = gdn.gdn_attn_decode(q, kc, vc, ids, lens, return_lse=True)
    ref.check_attention(out, lse, ref.attention(q, kc, vc, ids, lens), BF)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("hkv,D,page", [(2, 256, 16), (3, 80, 24), (1, 8, 1), (5, 128, 100)])
def test_append_is_a_bit_copy_and_touches_nothing_else(hkv, D, page, dtype):
    g = torch.Generator().manual_seed(hkv)
    lens = [1, 0, 257, 33, 64]
    kc, vc, table, ln = ref.make_cache(lens, page, hkv, D, dtype, g, "cuda", hidden=NAN)
    for cu in ([0, 1, 1, 258, 270, 270], [0, 0, 0, 57, 57, 121]):
        k = torch.randn((cu[-1], hkv, D), generator=g).to(dtype).cuda()
        v = torch.randn((cu[-1], hkv, D), generator=g).to(dtype).cuda()
        k.view(-1)[5] = NAN
        rk, rv = ref.append(k, v, kc, vc, table, ln, cu)
        gdn.gdn_kv_append(k, v, kc, vc, table, ln, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert torch.equal(kc.view(torch.uint8), rk.view(torch.uint8))
        assert torch.equal(vc.view(torch.uint8), rv.view(torch.uint8))
    # the same number of tokens each, more than some sequences have positions for
    k = torch.randn((5 * 3, hkv, D), generator=g).to(dtype).cuda()
    v = torch.randn((5 * 3, hkv, D), generator=g).to(dtype).cuda()
    rk, rv = ref.append(k, v, kc, vc, table, ln, [0, 3, 6, 9, 12, 15])
    gdn.gdn_kv_append(k, v, kc, vc, table, ln)
    assert torch.equal(kc.view(torch.uint8), rk.view(torch.uint8))
    assert torch.equal(vc.view(torch.uint8), rv.view(torch.uint8))


def test_append_leaves_out_what_has_no_place():
    g = torch.Generator().manual_seed(1)
    kc, vc, table, ln = ref.make_cache([40, 40, 40], 16, 2, 64, BF, g, "cuda")
    table[1, 1] = kc.shape[0]
    table[2, 2] = -1
    ln = torch.tensor([400, 40, 40], dtype=torch.int32, device="cuda")
    cu = [0, 390, 430, 470]  # sequence 0: positions 10..399 of 48
    k = torch.randn((480, 2, 64), generator=g).to(BF).cuda()
    v = torch.randn((480, 2, 64), generator=g).to(BF).cuda()
    rk, rv = ref.append(k, v, kc, vc, table, ln, cu)
    gdn.gdn_kv_append(k, v, kc, vc, table, ln, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    gdn.gdn_sync_status()
    assert torch.equal(kc, rk) and torch.equal(vc, rv)


def test_append_of_prompts():
    g = torch.Generator().manual_seed(2)
    lens = [3000, 1, 5111, 700]
    kc, vc, table, ln = ref.make_cache(lens, 64, 2, 256, BF, g, "cuda")
    cu = [0, 3000, 3001, 8112, 8812]
    k = torch.randn((8812, 2, 256), generator=g).to(BF).cuda()
    v = torch.randn((8812, 2, 256), generator=g).to(BF).cuda()
    gdn.gdn_kv_append(k, v, kc, vc, table, ln, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // 64)].long()
        assert torch.equal(kc[ids].transpose(1, 2).reshape(-1, 2, 256)[:n], k[cu[b]:cu[b + 1]])
        assert torch.equal(vc[ids].transpose(1, 2).reshape(-1, 2, 256)[:n], v[cu[b]:cu[b + 1]])


# ------------------------------------------------------------------ acceptance
def accept_inputs(B, K, V, dtype, seed, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((B, K + 1, V), generator=g) * sharp
    p = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits[:, :K] + 0.5 * torch.randn((B, K, V), generator=g), -1).to(dtype)
    draft = torch.zeros((B, K), dtype=torch.int32)
    if K:
        draft = torch.multinomial(q.float().reshape(B * K, V), 1, generator=g).reshape(B, K).to(torch.int32)
    u = torch.rand((B, K + 1), generator=g)
    slots = torch.randint(0, 1000, (B, K + 2), generator=g).to(torch.int32)
    return p, q, draft, u, slots


def check_accept(p, q, draft, u, n_draft=None, slots=None):
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    n, tokens, ns = gdn.gdn_draft_accept(c(p), c(q), c(draft), c(u), n_draft=c(n_draft), slots=c(slots))
    gdn.gdn_sync_status()
    rn, rt = ref.accept(p, q, draft, u, n_draft)
    assert n.tolist() == rn
    assert tokens.tolist() == rt
    if slots is not None:
        assert ns.tolist() == [int(slots[b, m + 1]) for b, m in enumerate(rn)]
    else:
        assert ns is None
    return rn


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,K,V", [(1, 3, 32000), (5, 0, 1), (7, 1, 2), (3, 15, 1023), (3, 4, 1024), (3, 4, 1025),
                                   (64, 4, 5001), (9, 7, 8192), (2, 2, 131072), (2, 2, 131071), (1, 1, 300007),
                                   (3, 2, 8200), (2, 3, 20004)])
def test_acceptance_matches_its_definition(B, K, V, dtype):
    p, q, draft, u, slots = accept_inputs(B, K, V, dtype, B + K + V)
    check_accept(p, q, draft, u, slots=slots)
    check_accept(p, None, draft, u)
    g = torch.Generator().manual_seed(3)
    n_draft = torch.randint(-1, K + 2, (B,), generator=g).to(torch.int32)
    check_accept(p, q, draft, u, n_draft, slots)
    check_accept(p, None, draft, u, n_draft)


def test_acceptance_over_the_largest_vocabulary():
    """Sums over 2^24 values, of which the last ones decide."""
    V = 1 << 24
    p = torch.full((2, 1, V), 2.0 ** -24)
    p[0, 0, :-3] = 0
    u = torch.tensor([[0.999], [1 - 2.0 ** -24]])
    check_accept(p, None, torch.zeros((2, 0), dtype=torch.int32), u)


def test_acceptance_borders():
    V = 4100
    p, q, draft, u, slots = accept_inputs(6, 3, V, F, 12)
    # u q(d) == p(d) exactly: not held; one step of u below: held
    d = draft[:, 0].long()
    b = torch.arange(6)
    p[b, 0, d] = 0.25 * q[b, 0, d]
    u[:, 0] = 0.25
    u[1::2, 0] = 0.25 * (1 - 2.0 ** -24)
    n = check_accept(p, q, draft, u, slots=slots)
    assert all(m == 0 for m in n[::2]) and all(m >= 1 for m in n[1::2])
    # uniforms at the ends pick the first and the last value with weight
    for end in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0):
        u2 = u.clone()
        u2[:, 3] = end
        check_accept(p, q, draft, u2, slots=slots)
    # weight at single values only, in the first, a middle and the last place
    for at in (0, 1, 1023, 1024, 2048, V - 1):
        one = torch.zeros((6, 4, V))
        one[:, :, at] = 0.7
        check_accept(one, q, draft, u, slots=slots)
        check_accept(one, None, draft, u)


def test_acceptance_without_weight():
    """Rows without a positive value, tokens outside the vocabulary, equal distributions, NaN."""
    V = 3001
    p, q, draft, u, slots = accept_inputs(4, 2, V, F, 13)
    check_accept(torch.zeros_like(p), q, draft, u, slots=slots)
    check_accept(p, p[:, :2].clone(), draft, torch.ones_like(u) * 0.999, slots=slots)
    # p <= q everywhere: the failed draft leaves nothing over, p itself is drawn from
    check_accept(p * 0.5, p[:, :2].clone(), draft, torch.full_like(u, 0.9), slots=slots)
    far = draft.clone()
    far[0, 0], far[1, 1], far[2, 0] = -1, V, 2 ** 31 - 1
    check_accept(p, q, far, u, slots=slots)
    check_accept(p, None, far, u)
    bad = p.clone()
    bad[0], bad[1, :, 5], bad[2, :, 7] = NAN, NAN, INF
    n, tokens, ns = gdn.gdn_draft_accept(bad.cuda(), q.cuda(), draft.cuda(), u.cuda(), slots=slots.cuda())
    t = tokens.cpu()
    assert ((t >= -1) & (t < V)).all() and ((n >= 0) & (n <= 2)).all()


def test_acceptance_of_the_smallest_probabilities():
    """Rows of subnormal values, whose sums times a uniform fall between two of them: the token is picked all the
    same, as the definition in 64 bits has it."""
    V = 3001
    g = torch.Generator().manual_seed(14)
    us = [0.0, 0.3, 0.4999, 0.5, 0.5001, 0.9, 0.999, 1 - 2.0 ** -24]
    tiny = 2.0 ** -149
    for steps in (1, 3, 40, 1 << 14):  # values of 0 to this many smallest steps
        few = torch.randint(0, V, (len(us), 3), generator=g)
        p = torch.zeros((len(us), 2, V))
        p[:, 0] = (torch.randint(0, steps + 1, (len(us), V), generator=g).double() * tiny).float()
        p[:, 1].scatter_(1, few, steps * tiny)
        assert (p[:, 1] > 0).any(-1).all()
        u = torch.tensor(us).view(-1, 1).repeat(1, 2)
        draft = few[:, :1].to(torch.int32)
        none = torch.zeros((len(us), 0), dtype=torch.int32)
        for row in (0, 1):
            check_accept(p[:, row:row + 1].contiguous(), None, none, u[:, :1].contiguous())
        check_accept(p, None, draft, u)
        q = p[:, :1] * 0.5  # what is left over after the draft fails is smaller still
        q.scatter_(2, draft.long().view(-1, 1, 1), 1.0)
        check_accept(p, q, draft, u)


def test_acceptance_does_not_depend_on_the_split_of_a_row():
    """Values over many magnitudes: the running sums keep what f32 would lose."""
    V = 50000
    g = torch.Generator().manual_seed(4)
    p = torch.exp2(-40 * torch.rand((8, 1, V), generator=g))
    p[:, :, 100] = 3e4
    u = torch.rand((8, 1), generator=g)
    u[0] = 1 - 2.0 ** -24
    run = p.double().cumsum(-1)
    for b in range(1, 8):  # borders inside the small values' range
        u[b, 0] = float((run[b, 0, 1000 * b] / run[b, 0, -1]).float())
    check_accept(p, None, torch.zeros((8, 0), dtype=torch.int32), u)


# ------------------------------------------------------------------ streams, graphs
def test_other_streams_and_graphs():
    x = attn_inputs([3000, 500], 2, 16, 2, 256, 16, BF, 50, gate=True)
    q, kc, vc, table, ln, gt = x
    p, pq, draft, u, slots = (t.cuda() for t in accept_inputs(2, 1, 5000, F, 51))
    k = torch.randn((4, 2, 256), device="cuda").to(BF)
    v = torch.randn((4, 2, 256), device="cuda").to(BF)

    def step(stream=None):
        gdn.gdn_kv_append(k, v, kc, vc, table, ln, stream=stream)
        out, lse = gdn.gdn_attn_decode(q, kc, vc, table, ln, gate=gt, return_lse=True, stream=stream)
        n, tok, ns = gdn.gdn_draft_accept(p, pq, draft, u, slots=slots, stream=stream)
        return out, lse, n, tok, ns

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = step(s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got = step()
        graphs.append((gr, got))
    for rounds in range(3):
        for gr, got in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for gr, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(want, got))
    # the captured call follows the lengths and the page table
    ln.copy_(torch.tensor([129, 2], dtype=torch.int32))
    for gr, got in graphs:
        gr.replay()
        torch.cuda.synchronize()
        r = ref.attention(q, kc, vc, table, ln, gate=gt)
        ref.check_attention(got[0], got[1], r, BF)


def test_inputs_dropped_after_a_call_on_another_stream():
    """Inputs given up right after the call are not reused before the stream has run it."""
    side = torch.cuda.Stream()
    g = torch.Generator().manual_seed(52)
    kc, vc, table, ln = ref.make_cache([2000, 1500], 16, 2, 256, BF, g, "cuda")
    q0 = torch.randn((2, 1, 16, 256), generator=g).to(BF).cuda()
    want = gdn.gdn_attn_decode(q0, kc, vc, table, ln)
    torch.cuda.synchronize()
    for _ in range(20):
        q = q0.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        got = gdn.gdn_attn_decode(q, kc, vc, table, ln, stream=side)
        del q
        junk = [torch.full_like(q0, 3.0) for _ in range(4)]  # would land in q's memory
        side.synchronize()
        assert torch.equal(got, want)
        del junk


def test_two_calls_at_once():
    xs = [attn_inputs([4000, 100], 1, 16, 2, 256, 16, BF, 60 + i) for i in range(2)]
    want = [run_attn(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        got = [run_attn(x, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


# ------------------------------------------------------------------ a wait that runs out
@pytest.mark.parametrize("stop_at", [0, 1, 4])
@pytest.mark.parametrize("K,hq,hkv,D,page", [(1, 16, 2, 256, 16), (5, 16, 2, 256, 64), (16, 16, 2, 256, 16),
                                             (16, 32, 4, 128, 64)])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(K, hq, hkv, D, page, stop_at):
    """The MMAs of every CTA that has so many tiles stop: the call returns, gdn_sync_status reports it once,
    and the context goes on."""
    lens = [900 + 17 * b for b in range(90)]
    x = attn_inputs(lens, K, hq, hkv, D, page, BF, 65)
    q, kc, vc, table, ln, _ = x
    want, _ = run_attn(x)
    gdn.gdn_sync_status()
    lib, out = gdn._lib.load(), torch.empty_like(q)
    ws = torch.zeros(gdn.gdn_attn_decode_workspace_size(len(lens), K, hq, hkv, D, page, BF), dtype=torch.uint8,
                     device="cuda")

    def stopped(at):
        return lib.gdn_selftest_attn_decode(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), table.data_ptr(), ln.data_ptr(),
                                            out.data_ptr(), len(lens), K, hq, hkv, D, page, kc.shape[0], table.shape[1],
                                            ws.data_ptr(), ws.numel(), at, torch.cuda.current_stream().cuda_stream)

    assert stopped(stop_at) == 0
    with pytest.raises(gdn.GDNError, match="TIMEOUT"):
        gdn.gdn_sync_status()
    gdn.gdn_sync_status()  # cleared
    assert stopped(10 ** 6) == 0  # no CTA has that many
    gdn.gdn_sync_status()
    assert torch.equal(out, want)
    assert torch.equal(run_attn(x)[0], want)


# ------------------------------------------------------------------ refusals
def test_refusals():
    q, kc, vc, table, ln, _ = attn_inputs([64, 64], 2, 4, 2, 128, 16, BF, 70)
    with pytest.raises(ValueError, match="q: shape"):
        gdn.gdn_attn_decode(q[:1], kc, vc, table, ln)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.gdn_attn_decode(q.transpose(1, 2), kc, vc, table, ln)
    with pytest.raises(ValueError, match="both alike"):
        gdn.gdn_attn_decode(q, kc, vc[:1], table, ln)
    with pytest.raises(TypeError, match="dtype"):
        gdn.gdn_attn_decode(q, kc.float(), vc, table, ln)
    with pytest.raises(TypeError, match="dtype"):
        gdn.gdn_attn_decode(q, kc, vc, table.long(), ln)
    with pytest.raises(ValueError, match="different devices"):
        gdn.gdn_attn_decode(q, kc, vc, table, ln.cpu())
    with pytest.raises(gdn.GDNError, match="WORKSPACE"):
        gdn.gdn_attn_decode(q, kc, vc, table, ln, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gdn.GDNError, match="INVALID_ARG"):
        gdn.gdn_attn_decode(q, kc, vc, table, ln, scale=-1.0)
    with pytest.raises(gdn.GDNError, match="INVALID_ARG"):  # 3 query heads, 2 key-value heads
        gdn.gdn_attn_decode(q[:, :, :3].contiguous(), kc, vc, table, ln)
    with pytest.raises(gdn.GDNError, match="ALIGN"):
        buf = torch.empty(q.numel() + 1, dtype=BF, device="cuda")
        gdn.gdn_attn_decode(buf[1:].view(q.shape), kc, vc, table, ln)
    with pytest.raises(TypeError, match="unsupported activation dtype"):
        gdn.gdn_attn_decode(q.half(), kc.half(), vc.half(), table, ln)
    with pytest.raises(gdn.GDNError, match="UNSUPPORTED"):  # head dim not a multiple of 8
        gdn.gdn_attn_decode(q[..., :12].contiguous(), kc[..., :12].contiguous(), vc[..., :12].contiguous(), table, ln)
    k = torch.zeros((5, 2, 128), dtype=BF, device="cuda")
    with pytest.raises(gdn.GDNError, match="INVALID_ARG"):  # 5 tokens, 2 sequences
        gdn.gdn_kv_append(k, k, kc, vc, table, ln)
    with pytest.raises(ValueError, match="v: shape"):
        gdn.gdn_kv_append(k[:4], k, kc, vc, table, ln)
    p, pq, draft, u, slots = (t.cuda() for t in accept_inputs(2, 1, 100, F, 71))
    with pytest.raises(ValueError, match="draft_tokens: shape"):
        gdn.gdn_draft_accept(p, pq, draft[:1], u)
    with pytest.raises(gdn.GDNError, match="INVALID_ARG"):  # too many drafts
        z = torch.zeros((1, 17, 8), device="cuda")
        gdn.gdn_draft_accept(z, None, torch.zeros((1, 16), dtype=torch.int32, device="cuda"),
                             torch.zeros((1, 17), device="cuda"))
    with pytest.raises(gdn.GDNError, match="INVALID_ARG"):  # next_slot without slots
        gdn.gdn_draft_accept(p, pq, draft, u, next_slot=torch.zeros(2, dtype=torch.int32, device="cuda"))
    # nothing to do
    e = torch.zeros((0, 1, 4, 128), dtype=BF, device="cuda")
    assert gdn.gdn_attn_decode(e, kc, vc, table[:0], ln[:0]).shape == e.shape
    gdn.gdn_kv_append(k[:0], k[:0], kc, vc, table, ln)
    gdn.gdn_sync_status()


# ------------------------------------------------------------------ together
def test_speculative_serving_steps():
    """A softmax layer and a linear layer of a hybrid model through several speculative steps, as a
    server runs them: append the last sampled token and the drafts, attend, run the linear layer's
    verification pass, accept, continue from the accepted slot.  The accepted tokens' outputs and the
    states carried on equal a token-by-token run over the same tokens."""
    g = torch.Generator().manual_seed(80)
    B, K, V, page, hq, hkv, D = 5, 3, 600, 16, 16, 2, 256
    s = W.GDNShape(2, 4, 128, 128)
    dims = gdn.GDNDims(2, 4, 128, 128)
    cap = 160
    lens = torch.tensor([100, 1, 37, 64, 15], dtype=torch.int32)
    per = cap // page
    kc = torch.randn((B * per, hkv, page, D), generator=g).to(BF).cuda()
    vc = torch.randn((B * per, hkv, page, D), generator=g).to(BF).cuda()
    table = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per).cuda()
    kc1, vc1 = kc.clone(), vc.clone()
    par = {k: v.cuda() for k, v in W.layer_params(s, BF, 81).items()}
    n_slots = B * (K + 2)
    state = 0.02 * torch.randn((n_slots, 4, 128, 128), generator=g).cuda()
    conv = torch.randn((n_slots, s.conv_dim, 3), generator=g).to(BF).cuda()
    slots = torch.arange(n_slots, dtype=torch.int32).view(B, K + 2)
    state1, conv1 = state[slots[:, 0].long()].clone(), conv[slots[:, 0].long()].clone()

    def rand(*shape):
        return torch.randn(shape, generator=g).to(BF).cuda()

    total = 0
    for step in range(4):
        N = K + 1
        q, gate = rand(B, N, hq, D), rand(B, N, hq, D)
        k, v = rand(B, N, hkv, D), rand(B, N, hkv, D)
        x, z, a, b = rand(B, N, s.conv_dim), rand(B, N, 512), rand(B, N, 4), rand(B, N, 4)
        p, pq, draft, u, _ = accept_inputs(B, K, V, F, 90 + step)
        after = (lens + N).cuda()
        gdn.gdn_kv_append(k.view(B * N, hkv, D), v.view(B * N, hkv, D), kc, vc, table, after)
        attn = gdn.gdn_attn_decode(q, kc, vc, table, after, gate=gate)
        lin = gdn.gdn_decode_verify(x, z, a, b, par["conv_w"], par["A_log"], par["dt_bias"], par["norm_w"], dims,
                                    state, conv, slots.cuda())
        n, tokens, nxt = gdn.gdn_draft_accept(p.cuda(), pq.cuda(), draft.cuda(), u.cuda(), slots=slots.cuda())
        gdn.gdn_sync_status()
        rn, rt = ref.accept(p, pq, draft, u)
        assert n.tolist() == rn and tokens.tolist() == rt
        # token by token over what was accepted
        for i in range(N):
            live = [j for j in range(B) if i <= rn[j]]
            if not live:
                break
            ix = torch.tensor(live, device="cuda")
            ln1 = (lens[live] + i + 1).cuda()
            t1 = table[ix].contiguous()
            gdn.gdn_kv_append(k[ix, i].contiguous(), v[ix, i].contiguous(), kc1, vc1, t1, ln1)
            o1, e1 = gdn.gdn_attn_decode(q[ix, i:i + 1].contiguous(), kc1, vc1, t1, ln1,
                                         gate=gate[ix, i:i + 1].contiguous(), return_lse=True)
            r = ref.attention(q[ix, i:i + 1], kc1, vc1, t1, ln1, gate=gate[ix, i:i + 1])
            ref.check_attention(o1, e1, r, BF)
            ref.check_attention(attn[ix, i:i + 1], None, r, BF)
            st, cs = state1[ix].contiguous(), conv1[ix].contiguous()
            l1 = gdn.gdn_decode_step(x[ix, i].contiguous(), z[ix, i].contiguous(), a[ix, i].contiguous(),
                                     b[ix, i].contiguous(), par["conv_w"], par["A_log"], par["dt_bias"],
                                     par["norm_w"], dims, st, cs)
            state1[ix], conv1[ix] = st, cs
            assert torch.equal(l1, lin[ix, i])
        at = nxt.long()
        assert torch.equal(state[at], state1) and torch.equal(conv[at], conv1)
        # continue: the accepted slot comes first in the next row
        cur = nxt.cpu()
        for j in range(B):
            row = slots[j].tolist()
            row.remove(int(cur[j]))
            slots[j] = torch.tensor([int(cur[j])] + row, dtype=torch.int32)
        lens = lens + torch.tensor(rn, dtype=torch.int32) + 1
        total += sum(rn)
    assert 0 < total < 4 * B * K
