"""Attention behind shared prefixes on the GPU, against the attention's definition in
64 bits (over every sequence's whole table row), and a serving loop that uses it."""
import pytest
import torch

import gated_deltanet_linear_core_gb300 as gdn
import rotary_ref as rot
import serving_ref as ref
from gated_deltanet_linear_core_gb300 import _lib

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def shared_inputs(groups, K, hq, hkv, D, page, dtype, seed, gate=False, hidden=NAN):
    """groups: [(prefix length, [own lengths])].  A group's sequences have the pages that lie wholly in the
    prefix in common and their own copy of the page that it ends in."""
    g = torch.Generator().manual_seed(seed)
    lens = [p + n if n >= 0 else 0 for p, own in groups for n in own]  # own length -1: an empty sequence
    B = len(lens)
    counts = []
    for p, own in groups:
        counts += [p // page] + [-(-(p + n) // page) - p // page if n >= 0 else 0 for n in own]
    total = sum(counts) + 2
    order = torch.randperm(total, generator=g).to(torch.int32)
    width = max(max(-(-n // page) for n in lens), 1)
    table = torch.full((B, width), -1, dtype=torch.int32)
    k = torch.randn((total, hkv, page, D), generator=g).to(dtype)
    v = torch.randn((total, hkv, page, D), generator=g).to(dtype)
    used = torch.zeros((total, page), dtype=torch.bool)
    at, b = 0, 0
    for p, own in groups:
        common = order[at:at + p // page]
        at += p // page
        used[common.long()] = True
        last = None
        for n in own:
            if n >= 0:
                mine = order[at:at + -(-(p + n) // page) - p // page]
                at += mine.numel()
                row = torch.cat([common, mine])
                table[b, :row.numel()] = row
                if p % page and mine.numel():
                    if last is not None:
                        k[mine[0], :, :p % page] = k[last, :, :p % page]
                        v[mine[0], :, :p % page] = v[last, :, :p % page]
                    last = int(mine[0])
                for t in range(p // page * page, p + n, page):
                    used[table[b, t // page], :min(page, p + n - t)] = True
            b += 1
    if hidden is not None:
        free = ~used.view(total, 1, page, 1)
        k.masked_fill_(free, hidden)
        v.masked_fill_(free, hidden)
    cu = torch.zeros(len(groups) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor([len(own) for _, own in groups]).cumsum(0)
    q = torch.randn((B, K, hq, D), generator=g).to(dtype).cuda()
    gt = torch.randn((B, K, hq, D), generator=g).to(dtype).cuda() if gate else None
    return dict(q=q, k_cache=k.cuda(), v_cache=v.cuda(), page_table=table.cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                prefix_lens=torch.tensor([p for p, _ in groups], dtype=torch.int32, device="cuda"), cu_groups=cu.cuda(), gate=gt)


def definition(x, scale=None):
    return ref.attention(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], scale=scale, gate=x["gate"])


def check(x, **kw):
    out, lse = gdn.gdn_attn_decode_shared(**x, return_lse=True, **kw)
    gdn.gdn_sync_status()
    ref.check_attention(out, lse, definition(x, kw.get("scale") or None), x["q"].dtype)
    return out, lse


# groups (prefix, own lengths), K, H_q, H_kv, D, page, gate: prefixes below, at and behind a tile, inside a page, of 0;
# groups of none and one; rows that fill, just pass and do not fill a block; empty sequences; every kind of page
CASES = [
    ([(128, [1, 1])], 1, 1, 1, 16, 16, False),
    ([(127, [5, 9])], 1, 4, 2, 64, 8, True),
    ([(300, [1, 2, 60])], 1, 16, 2, 256, 16, True),
    ([(1000, [7, 1, 33, 16])], 1, 16, 2, 256, 16, True),
    ([(256, [1, 1, 1]), (0, [40, 3]), (513, [200]), (640, [128, 5, -1, 129])], 1, 8, 2, 128, 32, False),
    ([(1290, [5, 30, 17])], 5, 15, 3, 80, 24, False),
    ([(2000, [16, 400])], 16, 32, 4, 128, 128, True),
    ([(700, [4, -1, 9]), (400, [-1, -1]), (900, [-1, 50, -1])], 4, 8, 2, 64, 64, True),
    ([(3000, [1] * 64)], 1, 16, 2, 256, 64, True),
    ([(4100, [3] * 43)], 3, 6, 2, 200, 20, False),
    ([(640, [2] * 65)], 2, 2, 1, 72, 4, True),
    ([(900, [1, 8])], 1, 5, 5, 8, 7, False),
    ([(1400, [6, 100, 6])], 6, 6, 1, 192, 1, True),
    ([(20000, [1, 700])], 1, 16, 2, 256, 64, True),
    ([(6000, [17, 130, 16])], 16, 64, 2, 96, 256, False),
    ([(260 + 8 * i, [1 + i % 3] * (1 + i % 5)) for i in range(70)], 1, 4, 2, 64, 8, True),
    ([(2600, [9] * 20)], 8, 24, 8, 128, 40, True),
    ([(5000, [2, 3, 4]), (7000, [1] * 30)], 1, 40, 8, 104, 48, False),
    ([(300, [9, 40, 300]), (100, [500])], 8, 48, 8, 16, 100, True),
    ([(520, [3, 70, 131])], 3, 3, 1, 8, 4, True),
    ([(400, [16, 700, 64])], 16, 66, 2, 128, 32, True),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_shared_attention_matches_its_definition(i, dtype):
    groups, K, hq, hkv, D, page, gate = CASES[i]
    check(shared_inputs(groups, K, hq, hkv, D, page, dtype, 900 + i, gate))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_without_groups_and_with_a_scale(dtype):
    x = shared_inputs([(800, [1, 20, 300])], 1, 8, 2, 128, 16, dtype, 3, True)
    want, _ = gdn.gdn_attn_decode_shared(**x, return_lse=True, scale=0.03)
    x["cu_groups"] = None
    out, _ = check(x, scale=0.03)
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_prefix_lengths_that_reach_too_far_or_nowhere(dtype):
    """A prefix is shared only as far as every new token sees it, whatever its length says; sequences of no group
    and groups of one are on their own."""
    x = shared_inputs([(640, [9, 300, 30]), (256, [8]), (300, [12, 13])], 4, 8, 2, 64, 16, dtype, 4)
    r = definition(x)
    for prefix in ([640, 256, 300], [10 ** 9, 256, 300], [-5, 2 ** 31 - 1, 0]):
        # (beyond the common 640 tokens the sequences differ: not claimed as shared)
        y = dict(x, prefix_lens=torch.tensor([min(prefix[0], 640)] + prefix[1:], dtype=torch.int32, device="cuda"))
        if prefix[0] > 640:
            y["prefix_lens"][0] = 10 ** 9
            y["seq_lens"] = x["seq_lens"].clone()
            y["seq_lens"][0] = 643  # the first new token sees 640: 512 are shared, all of them common
            ref_y = definition(y)
        else:
            ref_y = r
        out, lse = gdn.gdn_attn_decode_shared(**y, return_lse=True)
        ref.check_attention(out, lse, ref_y, dtype)
    y = dict(x, prefix_lens=x["prefix_lens"][:1].clone(), cu_groups=torch.tensor([1, 3], dtype=torch.int32, device="cuda"))
    out, lse = gdn.gdn_attn_decode_shared(**y, return_lse=True)
    ref.check_attention(out, lse, r, dtype)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_a_sequence_shorter_than_the_prefix(dtype):
    x = shared_inputs([(640, [9, 300, 30])], 4, 8, 2, 64, 16, dtype, 5)
    for n in (0, 1, 3, 4, 5, 127, 128, 131, 132, 133, 640, 641):
        x["seq_lens"][1] = n
        check(x)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_non_finite_values(dtype, bad):
    x = shared_inputs([(512, [3, 200, 7])], 2, 8, 2, 128, 16, dtype, 6)
    out0, _ = check(x)
    page, place = int(x["page_table"][0, 10]), 5  # in the prefix: every row sees it
    x["v_cache"][page, 1, place, 77] = bad
    out = gdn.gdn_attn_decode_shared(**x)
    hit = ~torch.isfinite(out)
    want = torch.zeros_like(hit)
    want[:, :, 4:, 77] = True
    assert torch.equal(hit, want) and torch.equal(out[~want], out0[~want])
    x["v_cache"][page, 1, place, 77] = 0
    n = int(x["seq_lens"][1])  # the last new token of one sequence: its last row alone sees it
    x["v_cache"][int(x["page_table"][1, (n - 1) // 16]), 0, (n - 1) % 16, 3] = bad
    hit = ~torch.isfinite(gdn.gdn_attn_decode_shared(**x))
    want = torch.zeros_like(hit)
    want[1, 1, :4, 3] = True
    assert torch.equal(hit, want)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_scores_of_all_sizes(dtype):
    """Rows whose maximum moves at every tile, far up and far down, and weights that vanish."""
    x = shared_inputs([(1024, [5, 60, 200])], 2, 8, 2, 64, 16, dtype, 7)
    ramp = torch.linspace(0.02, 3.0, x["k_cache"].shape[0], device="cuda")
    order = torch.argsort(x["page_table"][0, :64])
    for up in (True, False):
        y = dict(x, k_cache=x["k_cache"].clone(), q=(x["q"].float() * 4).to(dtype))
        for i, pg in enumerate(x["page_table"][0, :64].tolist()):
            y["k_cache"][pg] = (y["k_cache"][pg].float() * ramp[i if up else 63 - i]).to(dtype)
        check(y)
    assert order.numel() == 64
    x["k_cache"][x["page_table"][0, :64].long()] = -INF  # the whole prefix out of sight, as scores go
    x["q"] = x["q"].abs()
    out, lse = gdn.gdn_attn_decode_shared(**x, return_lse=True)
    z = dict(x, k_cache=x["k_cache"].clone())
    z["k_cache"][x["page_table"][0, :64].long()] = torch.finfo(dtype).min / 8
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    out2, lse2 = gdn.gdn_attn_decode_shared(**z, return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_pages_that_do_not_exist_read_as_zeros(dtype):
    x = shared_inputs([(640, [9, 300])], 1, 8, 2, 64, 16, dtype, 8)
    bad = dict(x, page_table=x["page_table"].clone())
    bad["page_table"][:, 3] = x["k_cache"].shape[0]
    bad["page_table"][:, 20] = -7
    zero = dict(x, k_cache=x["k_cache"].clone(), v_cache=x["v_cache"].clone())
    for pg in (x["page_table"][0, 3], x["page_table"][0, 20]):
        zero["k_cache"][pg] = 0
        zero["v_cache"][pg] = 0
    assert torch.equal(gdn.gdn_attn_decode_shared(**bad), gdn.gdn_attn_decode_shared(**zero))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_repeats_bit_for_bit_and_ignores_its_workspace(dtype):
    x = shared_inputs([(3000, [5, 70, 300, 9]), (900, [5] * 9)], 3, 16, 2, 128, 16, dtype, 9, True)
    out, lse = gdn.gdn_attn_decode_shared(**x, return_lse=True)
    n = gdn.gdn_attn_decode_shared_workspace_size(13, 3, 16, 2, 128, 16, dtype, groups=2)
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        o = torch.empty_like(out)
        o2, l2 = gdn.gdn_attn_decode_shared(**x, out=o, return_lse=True, workspace=ws)
        assert o2 is o and torch.equal(o, out) and torch.equal(l2, lse)


def test_capture_follows_lengths_groups_and_prefixes():
    x = shared_inputs([(900, [40, 33, 60, 50])], 1, 16, 2, 256, 16, BF, 10, True)
    x["prefix_lens"] = torch.tensor([900, 0], dtype=torch.int32, device="cuda")
    x["cu_groups"] = torch.tensor([0, 4, 4], dtype=torch.int32, device="cuda")
    gdn.gdn_attn_decode_shared(**x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        out, lse = gdn.gdn_attn_decode_shared(**x, return_lse=True)
    torch.cuda.current_stream().wait_stream(s)
    for lens, prefix, cu in (([940, 933, 960, 950], [900, 0], [0, 4, 4]), ([930, 901, 940, 0], [512, 300], [0, 2, 4]),
                             ([0, 0, 0, 0], [900, 900], [0, 1, 4]), ([905, 933, 901, 910], [130, 899], [1, 1, 4])):
        x["seq_lens"].copy_(torch.tensor(lens))
        x["prefix_lens"].copy_(torch.tensor(prefix))
        x["cu_groups"].copy_(torch.tensor(cu))
        graph.replay()
        torch.cuda.synchronize()
        ref.check_attention(out, lse, definition(x), BF)


def test_two_calls_at_once_on_two_streams():
    xs = [shared_inputs([(5000, [30] * 20)], 1, 16, 2, 256, 16, BF, 20 + i, True) for i in range(2)]
    want = [gdn.gdn_attn_decode_shared(**x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [gdn.gdn_attn_decode_shared(**x, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gives_up_in_time_and_recovers():
    x = shared_inputs([(3000, [30] * 6)], 1, 16, 2, 256, 16, BF, 30)
    want = gdn.gdn_attn_decode_shared(**x)
    n_ws = gdn.gdn_attn_decode_shared_workspace_size(6, 1, 16, 2, 256, 16, BF)
    ws, out = torch.empty(n_ws, dtype=torch.uint8, device="cuda"), torch.empty_like(want)
    p = {k: t.data_ptr() for k, t in x.items() if t is not None}
    st = _lib.load().gdn_selftest_attn_decode_shared(
        p["q"], p["k_cache"], p["v_cache"], p["page_table"], p["seq_lens"], p["prefix_lens"], out.data_ptr(), 6, 1, 16, 2,
        256, 16, x["k_cache"].shape[0], x["page_table"].shape[1], ws.data_ptr(), n_ws, 0,
        torch.cuda.current_stream().cuda_stream)
    assert st == _lib.GDN_OK
    with pytest.raises(gdn.GDNError) as e:
        gdn.gdn_sync_status()
    assert e.value.status == _lib.GDN_ERR_TIMEOUT
    gdn.gdn_sync_status()
    assert torch.equal(gdn.gdn_attn_decode_shared(**x), want)


def test_caches_past_32_bits_of_elements():
    D, hkv, page, n_pages = 256, 8, 128, 8300
    g = torch.Generator(device="cuda").manual_seed(1)
    kc = torch.zeros((n_pages, hkv, page, D), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    assert kc.numel() > 2 ** 31
    used = torch.tensor([n_pages - 1, n_pages - 2, 3, n_pages - 3, n_pages - 4, n_pages - 5])
    for c in (kc, vc):
        c[used] = torch.randn((6, hkv, page, D), generator=g, device="cuda", dtype=BF)
    table = torch.tensor([[n_pages - 1, n_pages - 2, 3, n_pages - 3], [n_pages - 1, n_pages - 2, 3, n_pages - 4],
                          [n_pages - 1, n_pages - 2, 3, n_pages - 5]], dtype=torch.int32, device="cuda")
    q = torch.randn((3, 2, 32, D), generator=g, device="cuda", dtype=BF)
    check(dict(q=q, k_cache=kc, v_cache=vc, page_table=table, gate=None, cu_groups=None,
               seq_lens=torch.tensor([400, 500, 386], dtype=torch.int32, device="cuda"),
               prefix_lens=torch.tensor([384], dtype=torch.int32, device="cuda")))


def test_serving_samples_of_one_prompt():
    """A prompt goes into the cache once, with head norms and positions of three axes; six samples
    continue it, each with pages of its own behind the whole ones of the prompt, one to four tokens
    a step.  Every step is held to the definitions in 64 bits."""
    hq, hkv, D, R, page, B, P = 8, 2, 128, 64, 16, 6, 700
    g = torch.Generator().manual_seed(77)
    whole, width = P // page, -(-(P + 16) // page)
    n_pages = whole + B * (width - whole)
    table = torch.cat([torch.arange(whole).expand(B, whole),
                       whole + torch.arange(B * (width - whole)).view(B, width - whole)], 1).to(torch.int32).cuda()
    kc = torch.full((n_pages, hkv, page, D), NAN, dtype=BF, device="cuda")
    vc = torch.full_like(kc, NAN)
    f = (1e4 ** (-torch.arange(R // 2, dtype=torch.float64) / (R // 2))).float().cuda()
    axes = (torch.arange(R // 2) % 3).to(torch.int32).cuda()
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    rope = dict(axes=axes, q_norm_w=qw, k_norm_w=kw)

    def tokens(n):
        row = torch.randn((n, (2 * hq + 2 * hkv) * D), generator=g).to(BF).cuda()
        q, k, v = row.split([2 * hq * D, hkv * D, hkv * D], 1)
        q, gate = q.view(n, hq, 2, D).unbind(2)
        return q, k.view(n, hkv, D), v.view(n, hkv, D), gate

    # the prompt, through the first sample's row; then the page that it ends in for the others
    q, k, v, _ = tokens(P)
    pos = torch.stack([torch.arange(P), torch.arange(P) // 7, torch.arange(P) % 7]).to(torch.int32).cuda()
    lens = torch.tensor([P], dtype=torch.int32, device="cuda")
    gdn.gdn_rope_kv_append(q, k, v, kc, vc, table[:1], lens, f, positions=pos, **rope)
    rot.check_rope(kc[:whole].transpose(1, 2).reshape(-1, hkv, D),
                   tuple(t[:whole * page] for t in rot.rope(k, f, pos, axes, kw)), BF)
    for c in (kc, vc):
        c[table[1:, whole].long()] = c[table[0, whole].long()].clone()
    lens = torch.full((B,), P, dtype=torch.int32, device="cuda")
    prefix = torch.tensor([P], dtype=torch.int32, device="cuda")
    for K in (1, 4, 2, 1, 3):
        lens += K
        q, k, v, gate = tokens(B * K)
        at = (lens.view(B, 1) - K + torch.arange(K, device="cuda")).flatten().to(torch.int32)
        pos = at.expand(3, B * K).contiguous()
        q = gdn.gdn_rope_kv_append(q, k, v, kc, vc, table, lens, f, positions=pos, **rope).view(B, K, hq, D)
        x = dict(q=q, k_cache=kc, v_cache=vc, page_table=table, seq_lens=lens, prefix_lens=prefix, cu_groups=None,
                 gate=gate.reshape(B, K, hq, D).contiguous())
        out, lse = check(x)
        o, e = gdn.gdn_attn_decode(q, kc, vc, table, lens, gate=x["gate"], return_lse=True)
        # each is off by its own roundings: a step of bf16 in all
        assert bool(((out.double() - o.double()).abs() <= 2.0 ** -7 * o.double().abs() + 2.0 ** -13).all())


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_more_sequences_and_groups_than_the_plan_holds_at_once(dtype):
    """1100 groups of one to three sequences, 2200 sequences, some of them empty; then all in one group."""
    g = torch.Generator().manual_seed(12)
    groups = [(int(torch.randint(0, 300, (1,), generator=g)), [int(n) for n in torch.randint(-1, 20, (1 + i % 3,), generator=g)])
              for i in range(1100)]
    x = shared_inputs(groups, 1, 2, 1, 16, 16, dtype, 13)
    check(x)
    x = shared_inputs([(260, [1 + i % 7 if i % 11 else -1 for i in range(2100)])], 1, 2, 1, 16, 16, dtype, 14)
    check(x)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("K,hq,hkv,D,page", [(1, 16, 2, 256, 16), (16, 16, 1, 64, 8), (3, 4, 4, 8, 4)])
def test_one_sequence(dtype, K, hq, hkv, D, page):
    for n in (K, 130, 1000):
        check(shared_inputs([(500, [n])], K, hq, hkv, D, page, dtype, 40 + n, True))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_a_query_that_is_not_finite_spoils_its_own_row(dtype):
    x = shared_inputs([(700, [9, 300, 30])], 2, 8, 2, 64, 16, dtype, 41)
    want = gdn.gdn_attn_decode_shared(**x)
    x["q"][1, 0, 3, 5] = NAN
    out = gdn.gdn_attn_decode_shared(**x)
    assert bool(torch.isnan(out[1, 0, 3]).all())
    out[1, 0, 3] = want[1, 0, 3]
    assert torch.equal(out, want)


def test_two_graphs_of_one_batch():
    """Captured with workspaces of their own, replayed in turns and beside one another."""
    x = shared_inputs([(2000, [40] * 12)], 1, 16, 2, 256, 16, BF, 42, True)
    y = dict(x, q=x["q"].flip(0).contiguous(), gate=None)
    want = [gdn.gdn_attn_decode_shared(**x), gdn.gdn_attn_decode_shared(**y)]
    s, graphs, outs = torch.cuda.Stream(), [], []
    s.wait_stream(torch.cuda.current_stream())
    for z in (x, y):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            outs.append(gdn.gdn_attn_decode_shared(**z))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, o, w in zip(graphs, outs, want):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, w)
    other = torch.cuda.Stream()
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    graphs[0].replay()
    with torch.cuda.stream(other):
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_the_binding_refuses_what_does_not_fit():
    x = shared_inputs([(300, [9, 30])], 1, 8, 2, 64, 16, BF, 43)
    for bad, error in ((dict(cu_groups=None, prefix_lens=x["prefix_lens"].repeat(2)), ValueError),
                       (dict(cu_groups=x["cu_groups"][:1]), ValueError), (dict(prefix_lens=x["prefix_lens"].view(1, 1)), ValueError),
                       (dict(prefix_lens=x["prefix_lens"].long()), TypeError), (dict(q=x["q"][:1]), ValueError),
                       (dict(gate=x["q"][:, :, :4]), ValueError), (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
                                                                   gdn.GDNError), (dict(scale=-1.0), gdn.GDNError)):
        with pytest.raises(error):
            gdn.gdn_attn_decode_shared(**dict(x, **bad))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("B", [127, 128, 129])
def test_as_many_sequences_as_a_small_plan_takes(B, dtype):
    """Three sequences to a group; 43 groups, the last of what is left."""
    own = [[1 + (3 * i + j) % 20 for j in range(min(3, B - 3 * i))] for i in range(43)]
    check(shared_inputs([(128 if i % 2 == 0 else 40, n) for i, n in enumerate(own)], 1, 4, 2, 64, 16, dtype, B))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("more", [32, 96])
def test_padded_batches(more, i, dtype):
    """The same with empty sequences behind them: batches of other sizes are planned in other ways."""
    groups, K, hq, hkv, D, page, gate = CASES[i]
    check(shared_inputs(groups + [(0, [-1] * more)], K, hq, hkv, D, page, dtype, 900 + i, gate))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("G,B", [(1, 31), (1, 32), (7, 24), (8, 24), (8, 25), (9, 23), (9, 9), (31, 1), (8, 3), (3, 62),
                                  (2, 63), (1, 95), (1, 96), (8, 88), (8, 89)])
def test_as_many_groups_and_sequences_as_a_warp_plans(G, B, dtype):
    own = [[1 + (5 * g + j) % 30 for j in range((B * (g + 1)) // G - B * g // G)] for g in range(G)]
    check(shared_inputs([(150 + 100 * (g % 3), n) for g, n in enumerate(own)], 2, 8, 2, 64, 16, dtype, 70 + G, True))
