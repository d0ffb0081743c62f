"""Rotary positions, alone and on the way into the paged cache, on the GPU against
their definition in 64 bits."""
import pytest
import torch

import gated_deltanet_linear_core_gb300 as gdn
import rotary_ref as rot
import serving_ref as ref

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def freqs(R, base=1e4):
    return (base ** (-torch.arange(R // 2, dtype=torch.float64) / (R // 2))).float().cuda()


def inputs(T, H, D, R, n_axes, dtype, seed, layout="dense", norm=False, far=5000):
    g = torch.Generator().manual_seed(seed)
    if layout == "dense":
        x = torch.randn((T, H, D), generator=g).to(dtype).cuda()
    elif layout == "fused":  # among other heads of a token
        x = torch.randn((T, H + 3, D), generator=g).to(dtype).cuda()[:, 2:2 + H]
    elif layout == "gated":  # beside a gate
        x = torch.randn((T, H, 2, D), generator=g).to(dtype).cuda()[:, :, 1]
    else:  # heads outside
        x = torch.randn((H, T, D), generator=g).to(dtype).cuda().transpose(0, 1)
    pos = torch.randint(-far, far, (n_axes, T) if n_axes > 1 else (T,), generator=g, dtype=torch.int32).cuda()
    axes = torch.randint(0, n_axes, (R // 2,), generator=g, dtype=torch.int32).cuda() if n_axes > 1 else None
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda() if norm else None
    return x, freqs(R), pos, axes, w


SHAPES = [  # T, H, D, R, axes, layout, norm, interleaved
    (1, 1, 8, 2, 1, "dense", False, False),
    (1, 16, 256, 64, 3, "gated", True, False),
    (2, 1, 16, 16, 1, "dense", True, True),
    (37, 3, 8, 8, 2, "dense", True, False),
    (130, 5, 72, 36, 2, "fused", True, True),
    (130, 5, 72, 72, 3, "fused", False, False),
    (1000, 16, 80, 80, 3, "fused", False, False),
    (301, 7, 96, 96, 1, "heads", True, False),
    (99, 2, 128, 126, 2, "dense", True, False),
    (99, 2, 128, 126, 2, "dense", True, True),
    (64, 33, 200, 50, 4, "gated", True, False),
    (65, 9, 256, 254, 1, "dense", True, True),
    (65, 9, 256, 254, 1, "gated", True, False),
    (65, 9, 256, 2, 16, "dense", True, False),
    (2500, 4, 256, 256, 3, "heads", True, False),
    (7000, 3, 64, 64, 1, "dense", False, True),
    (40000, 2, 128, 128, 3, "fused", True, False),
    (17, 300, 24, 12, 2, "dense", True, False),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_rotation_matches_its_definition(i, dtype):
    T, H, D, R, n_axes, layout, norm, inter = SHAPES[i]
    x, f, pos, axes, w = inputs(T, H, D, R, n_axes, dtype, 50 + i, layout, norm)
    before = x.clone()
    y = gdn.gdn_rope(x, f, pos, axes=axes, norm_w=w, interleaved=inter, mscale=1.25 if i % 2 else 1.0)
    assert y.shape == x.shape and y.is_contiguous() and torch.equal(x, before)
    rot.check_rope(y, rot.rope(x, f, pos, axes, w, mscale=1.25 if i % 2 else 1.0, interleaved=inter), dtype)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_far_positions_and_odd_frequencies(dtype):
    g = torch.Generator().manual_seed(1)
    x = torch.randn((600, 2, 64), generator=g).to(dtype).cuda()
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (600,), generator=g, dtype=torch.int64).to(torch.int32).cuda()
    pos[0], pos[1], pos[2] = 2 ** 31 - 1, -2 ** 31, 0
    f = freqs(64).clone()
    f[3], f[4], f[5], f[6], f[7] = 0.0, -0.37, 1e-30, -1e-30, 2.5
    y = gdn.gdn_rope(x, f, pos)
    rot.check_rope(y, rot.rope(x, f, pos), dtype)


def test_angles_keep_their_digits_where_f32_has_none():
    """One position past a million in 64 steps of the fastest frequency: neighbours differ as they should."""
    x = torch.zeros((64, 1, 16), device="cuda")
    x[:, :, 0] = 1
    pos = torch.arange(2 ** 30, 2 ** 30 + 64, dtype=torch.int32, device="cuda")
    f = torch.tensor([1.0, 0.1, 0.01, 0.001], device="cuda")
    y = gdn.gdn_rope(x, f, pos)[:, 0].double()
    want = torch.cos(pos.double())
    assert (y[:, 0] - want).abs().max() < 2.0 ** -20
    assert (y[:, 4] - torch.sin(pos.double())).abs().max() < 2.0 ** -20


@pytest.mark.parametrize("layout", ["dense", "fused", "gated", "heads"])
def test_in_place_and_strided_outputs(layout):
    x, f, pos, axes, w = inputs(77, 6, 128, 64, 3, BF, 3, layout, True)
    want = gdn.gdn_rope(x, f, pos, axes=axes, norm_w=w)
    wide = torch.full((77, 8, 128), 7.0, dtype=BF, device="cuda")
    gdn.gdn_rope(x, f, pos, axes=axes, norm_w=w, out=wide[:, 1:7])
    assert torch.equal(wide[:, 1:7], want) and bool((wide[:, 0] == 7).all()) and bool((wide[:, 7] == 7).all())
    y = gdn.gdn_rope(x, f, pos, axes=axes, norm_w=w, out=x)
    assert y is x and torch.equal(x, want)


def test_an_input_that_repeats_rows_and_an_axis_that_is_none():
    x = torch.randn((1, 4, 64), generator=torch.Generator().manual_seed(2)).to(BF).cuda().expand(50, 4, 64)
    f, pos = freqs(64), torch.arange(50, dtype=torch.int32, device="cuda")
    axes = torch.tensor([0, 1, -1, 7] * 8, dtype=torch.int32, device="cuda")
    two = torch.stack([pos, 3 * pos])
    y = gdn.gdn_rope(x, f, two, axes=axes)
    rot.check_rope(y, rot.rope(x, f, two, axes), BF)
    assert torch.equal(y[:, :, 2::4], x[:, :, 2::4]) and torch.equal(y[:, :, 3::4], x[:, :, 3::4])


def test_non_finite_inputs_stay_in_their_row():
    x, f, pos, _, w = inputs(33, 4, 128, 64, 1, BF, 4, "dense", True)
    want = gdn.gdn_rope(x, f, pos, norm_w=w)
    x[5, 2, 100] = float("nan")
    x[6, 1, 3] = float("inf")
    y = gdn.gdn_rope(x, f, pos, norm_w=w)
    assert bool(torch.isnan(y[5, 2]).all())
    y[5, 2], y[6, 1] = want[5, 2], want[6, 1]
    assert torch.equal(y, want)
    x[6, 1, 100] = float("inf")  # a dim that is not rotated, without the norm
    y = gdn.gdn_rope(x, f, pos)
    assert torch.equal(y[:, :, 64:].view(torch.int16), x[:, :, 64:].view(torch.int16))
    f[0] = float("nan")
    y = gdn.gdn_rope(want, f, pos)
    assert bool(torch.isnan(y[:, :, 0]).all()) and bool(torch.isfinite(y[:, :, 1:32]).all())


# ------------------------------------------------------------------ into the cache
def append_inputs(lens, new, hq, hkv, D, page, dtype, seed, fused=True):
    g = torch.Generator().manual_seed(seed)
    kc, vc, table, ln = ref.make_cache(lens, page, hkv, D, dtype, g, "cuda")
    T = sum(new)
    if fused:
        row = torch.randn((T, (2 * hq + 2 * hkv) * D), generator=g).to(dtype).cuda()
        q, k, v = row.split([2 * hq * D, hkv * D, hkv * D], 1)
        q, k, v = q.view(T, hq, 2, D)[:, :, 0], k.view(T, hkv, D), v.view(T, hkv, D)
    else:
        q, k, v = (torch.randn((T, h, D), generator=g).to(dtype).cuda() for h in (hq, hkv, hkv))
    cu = torch.zeros(len(new) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(new).cumsum(0)
    return q, k, v, kc, vc, table, ln, cu.cuda()


def check_append(x, f, pos, axes, qw, kw, inter, dtype, cu, per=None, **kw_call):
    q, k, v, kc, vc, table, ln, cu_dev = x
    B, page = ln.numel(), kc.shape[2]
    place = torch.cat([torch.arange(int(ln[b]) - (cu[b + 1] - cu[b]), int(ln[b])) for b in range(B)]).to(torch.int32).cuda()
    at = place if pos is None else pos
    rq = rot.rope(q, f, at, axes, qw, interleaved=inter)
    rk = rot.rope(k, f, at, axes, kw, interleaved=inter)
    want_k, bound_k = kc.double(), torch.zeros_like(kc, dtype=torch.float64)
    _, want_v = ref.append(k, v, kc, vc, table, ln, cu)
    touched = torch.zeros(kc.shape[:3], dtype=torch.bool, device="cuda")
    cap = table.shape[1] * page
    for t, p in enumerate(place.tolist()):
        b = next(i for i in range(B) if cu[i] <= t < cu[i + 1])
        if 0 <= p < cap and 0 <= int(table[b, p // page]) < kc.shape[0]:
            pg = int(table[b, p // page])
            want_k[pg, :, p % page], bound_k[pg, :, p % page] = rk[0][t], rk[1][t]
            touched[pg, :, p % page] = True
    kc0 = kc.clone()
    out = gdn.gdn_rope_kv_append(q, k, v, kc, vc, table, ln, f, positions=pos, axes=axes, q_norm_w=qw, k_norm_w=kw,
                                 interleaved=inter, cu_seqlens=None if per else cu_dev, **kw_call)
    rot.check_rope(out, rq, dtype)
    assert torch.equal(vc, want_v)
    rot.check_rope(kc, (want_k, bound_k), dtype)
    assert torch.equal(kc[~touched], kc0[~touched])
    return out


APPENDS = [  # lens, new, hq, hkv, D, R, page, axes, norm, interleaved, fused
    ([1], [1], 1, 1, 8, 8, 1, 1, False, False, False),
    ([5, 1, 200], [1, 1, 1], 16, 2, 256, 64, 16, 3, True, False, True),
    ([64, 65, 300, 5], [5, 5, 5, 5], 4, 2, 128, 128, 16, 0, True, False, True),
    ([10, 0, 700, 33], [10, 0, 650, 1], 6, 3, 96, 96, 24, 0, False, True, True),
    ([40, 700], [40, 131], 5, 5, 72, 36, 7, 2, True, True, False),
    ([3000, 20], [2999, 20], 16, 2, 256, 64, 64, 3, True, False, True),
    ([3, 2, 20], [5, 5, 5], 8, 1, 64, 32, 8, 0, True, False, True),  # more new tokens than places
    ([9] * 200, [2] * 200, 2, 1, 80, 80, 12, 0, False, False, True),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append_with_rotation(i, dtype):
    lens, new, hq, hkv, D, R, page, n_axes, norm, inter, fused = APPENDS[i]
    x = append_inputs(lens, new, hq, hkv, D, page, dtype, 300 + i, fused)
    _, f, pos, axes, w = inputs(sum(new), 1, D, R, max(n_axes, 1), dtype, 400 + i, norm=norm)
    cu = x[7].tolist()
    check_append(x, f, pos if n_axes else None, axes if n_axes else None, w, None if w is None else w.flip(0), inter, dtype,
                 cu, per=len(set(new)) == 1)


def test_append_equals_rope_then_kv_append():
    x = append_inputs([100, 7], [40, 7], 4, 2, 128, 16, BF, 8)
    q, k, v, kc, vc, table, ln, cu = x
    f = freqs(128)
    place = torch.cat([torch.arange(60, 100), torch.arange(0, 7)]).to(torch.int32).cuda()
    k2, v2 = kc.clone(), vc.clone()
    gdn.gdn_kv_append(gdn.gdn_rope(k, f, place), v.contiguous(), k2, v2, table, ln, cu_seqlens=cu)
    out = gdn.gdn_rope_kv_append(q, k, v, kc, vc, table, ln, f, cu_seqlens=cu)
    assert torch.equal(out, gdn.gdn_rope(q, f, place)) and torch.equal(kc, k2) and torch.equal(vc, v2)


def test_tokens_and_pages_that_do_not_exist_are_left_out():
    q, k, v, kc, vc, table, ln, cu = append_inputs([40, 20, 9], [4, 4, 4], 4, 2, 64, 8, BF, 11)
    table[0, 4] = -1                 # places 32..39 of sequence 0
    table[1, 2] = kc.shape[0]        # places 16..23 of sequence 1
    ln[2] = 10 ** 6                  # behind the table
    kc0, vc0 = kc.clone(), vc.clone()
    out = torch.full((14, 4, 64), 3.0, dtype=BF, device="cuda")
    more = [torch.cat([t, t[:2]]) for t in (q, k, v)]
    cu = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device="cuda")  # tokens 12 and 13 belong to none
    got = gdn.gdn_rope_kv_append(*more, kc, vc, table, ln, freqs(64), cu_seqlens=cu, q_out=out)
    assert got is out and torch.equal(kc, kc0) and torch.equal(vc, vc0)
    assert bool((out[12:] == 3).all())
    place = torch.tensor([36, 37, 38, 39, 16, 17, 18, 19] + list(range(10 ** 6 - 4, 10 ** 6)), dtype=torch.int32, device="cuda")
    rot.check_rope(out[:12], rot.rope(q, freqs(64), place), BF)


def test_capture_follows_lengths_and_positions():
    q, k, v, kc, vc, table, ln, cu = append_inputs([40, 20], [1, 1], 4, 2, 64, 8, BF, 12)
    pos = torch.tensor([7, 9], dtype=torch.int32, device="cuda")
    f, out = freqs(64), torch.empty((2, 4, 64), dtype=BF, device="cuda")
    call = lambda: gdn.gdn_rope_kv_append(q, k, v, kc, vc, table, ln, f, positions=pos, q_out=out)  # noqa: E731
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    pos += 100
    ln -= 3
    k2, v2 = kc.clone(), vc.clone()
    graph.replay()
    torch.cuda.synchronize()
    gdn.gdn_kv_append(gdn.gdn_rope(k, f, pos), v.contiguous(), k2, v2, table, ln)
    assert torch.equal(out, gdn.gdn_rope(q, f, pos)) and torch.equal(kc, k2) and torch.equal(vc, v2)


def test_on_a_named_stream():
    x, f, pos, axes, w = inputs(5000, 8, 128, 128, 3, BF, 13)
    want = gdn.gdn_rope(x, f, pos, axes=axes)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gdn.gdn_rope(x, f, pos, axes=axes, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_caches_and_inputs_past_32_bits_of_elements():
    """The last page of a cache of more than 2^32 bytes and 2^31 elements; a token stride past them too."""
    D, hkv, page, n_pages = 256, 8, 128, 8300
    kc = torch.zeros((n_pages, hkv, page, D), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    assert kc.numel() > 2 ** 31
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    ln = torch.tensor([128], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn((2, hkv, D), generator=g).to(BF).cuda() for _ in range(2))
    big = torch.empty(2 ** 31 + 4096, dtype=BF, device="cuda")
    q = big.as_strided((2, 4, D), (2 ** 31, D, 1))
    q.copy_(torch.randn((2, 4, D), generator=g).to(BF))
    out = gdn.gdn_rope_kv_append(q, k, v, kc, vc, table, ln, freqs(D))
    place = torch.tensor([126, 127], dtype=torch.int32, device="cuda")
    assert torch.equal(out, gdn.gdn_rope(q.contiguous(), freqs(D), place))
    assert torch.equal(kc[-1].transpose(0, 1)[126:], gdn.gdn_rope(k, freqs(D), place))
    assert torch.equal(vc[-1].transpose(0, 1)[126:], v) and not bool(kc[:-1].any())


def test_append_with_queries_in_place():
    q, k, v, kc, vc, table, ln, cu = append_inputs([900, 300], [700, 299], 6, 2, 128, 16, BF, 21, fused=False)
    f, w = freqs(96), (1 + 0.1 * torch.randn(128, generator=torch.Generator().manual_seed(1))).cuda()
    k2, v2 = kc.clone(), vc.clone()
    want = gdn.gdn_rope_kv_append(q, k, v, k2, v2, table, ln, f, q_norm_w=w, cu_seqlens=cu)
    got = gdn.gdn_rope_kv_append(q, k, v, kc, vc, table, ln, f, q_norm_w=w, cu_seqlens=cu, q_out=q)
    assert got is q and torch.equal(q, want) and torch.equal(kc, k2) and torch.equal(vc, v2)


@pytest.mark.parametrize("T", [4000, 12000, 20001])
def test_prompts_of_many_tokens(T):
    """More tokens than warps: several of a warp at once, the last ones fewer."""
    x, f, pos, axes, w = inputs(T, 3, 64, 32, 3, BF, 22, "gated", True)
    rot.check_rope(gdn.gdn_rope(x, f, pos, axes=axes, norm_w=w), rot.rope(x, f, pos, axes, w), BF)
    rot.check_rope(gdn.gdn_rope(x, f, pos, axes=axes), rot.rope(x, f, pos, axes), BF)
    a = append_inputs([T // 2, T], [T // 2, T - T // 2], 2, 1, 64, 16, BF, 23)
    check_append(a, f, pos, axes, w, None, False, BF, a[7].tolist())


def test_the_binding_refuses_what_does_not_fit():
    x, f, pos, axes, w = inputs(9, 4, 64, 32, 3, BF, 24)
    for bad, error in ((dict(positions=pos[:, :5]), ValueError), (dict(positions=pos.long()), TypeError),
                       (dict(inv_freq=f[:7]), ValueError), (dict(inv_freq=f.double()), TypeError), (dict(axes=axes[:3]), ValueError),
                       (dict(norm_w=x[0, 0].float()[:9]), ValueError), (dict(out=x.float()), TypeError), (dict(x=x.half()), TypeError),
                       (dict(x=x[:, :, ::2]), ValueError), (dict(norm_w=torch.ones(64, device="cuda"), norm_eps=0.0), gdn.GDNError),
                       (dict(out=x[:, :, :].transpose(0, 1).contiguous().transpose(0, 1)[:, :2]), ValueError)):
        with pytest.raises(error):
            gdn.gdn_rope(**dict(dict(x=x, inv_freq=f, positions=pos, axes=axes), **bad))
