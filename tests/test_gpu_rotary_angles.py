"""The angles of the rotary operators by themselves: a pair (0, 1) turns into (-sin, cos), without
any other rounding but the output's."""
import pytest
import torch

import gated_deltanet_linear_core_gb300 as gdn
import rotary_ref as rot

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def turned(f, pos, dtype, interleaved, cached):
    """(-sin, cos) [T, len(f)] in 64 bits, of positions `pos` (and as a key's on its way into the cache)."""
    T, half = pos.numel(), f.numel()
    D = -(-2 * half // 8) * 8
    x = torch.zeros((T, 2, D), dtype=dtype, device="cuda")
    a = torch.arange(half, device="cuda") * (2 if interleaved else 1)
    b = a + (1 if interleaved else half)
    x[:, :, b] = 1
    if cached:
        kc = torch.zeros((1, 2, T, D), dtype=dtype, device="cuda")
        one = torch.tensor([[0]], dtype=torch.int32, device="cuda")
        y = gdn.gdn_rope_kv_append(x, x, x, kc, kc.clone(), one, one[0] + T, f, positions=pos, interleaved=interleaved)
        assert torch.equal(kc[0].transpose(0, 1), y)
    else:
        y = gdn.gdn_rope(x, f, pos, interleaved=interleaved)
    assert torch.equal(y[:, 0], y[:, 1])
    return y[:, 0, a].double(), y[:, 0, b].double()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_slow_pairs_keep_their_digits(dtype, interleaved):
    """Sines relatively, of frequencies down to 1e-9.  The angle: |p f| 2^-52 + |p| 2^-62, that is 2^-32 of it at 1e-9.
    The sine of an f32 argument: 2^-22 (of one that the rest next to it halves: 2^-21), and few roundings of 2^-24:
    2^-20 in all, then the output's own half step."""
    f = torch.tensor([3e-3, 1e-4, 1.65e-7, 1e-6, 1e-7, 3.7e-8, 1e-8, 1e-9, -1e-7], device="cuda")
    pos = torch.tensor([1, -1, 2, -2, 3, 7, -7, 100, -100, 4097, -4097], dtype=torch.int32, device="cuda")
    for cached in (False, True):
        s, c = turned(f, pos, dtype, interleaved, cached)
        g = pos.double().view(-1, 1) * f.double()
        tol = 2.0 ** -20 + (2.0 ** -8 if dtype is BF else 0.0)
        assert bool(((s + torch.sin(g)).abs() <= tol * torch.sin(g).abs()).all())
        assert bool(((c - torch.cos(g)).abs() <= tol).all())


@pytest.mark.parametrize("cached", [False, True])
def test_cosines_are_as_near_as_those_of_angles_in_64_bits(cached):
    """f32, |p f| up to 2^15: the function is good to a step (2^-24 below 1), making the rounding of its argument good
    rounds once more (2^-25); what is left of second order, and the angle's own 2^-37, are below 2^-30."""
    g = torch.Generator().manual_seed(11)
    f = torch.cat([torch.rand(20, generator=g), 1e4 ** (-torch.arange(20, dtype=torch.float64) / 20).float()]).cuda()
    pos = torch.randint(-2 ** 15, 2 ** 15, (20000,), generator=g, dtype=torch.int32).cuda()
    s, c = turned(f, pos, F, False, cached)
    angle = pos.double().view(-1, 1) * f.double()
    tol = 2.0 ** -24 + 2.0 ** -25 + 2.0 ** -30
    assert float((s + torch.sin(angle)).abs().max()) <= tol
    assert float((c - torch.cos(angle)).abs().max()) <= tol


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_quarter_half_and_whole_turns(dtype):
    """Frequencies that are, to 64 bits, fractions of a turn: positions at and next to where the fraction's sign changes."""
    f = torch.tensor([0.5, 0.25, 0.125, 1 / 3, 1.0, 0.75, 1 - 2.0 ** -20, 2.0 ** -31], dtype=torch.float64)
    f = (f * 2 * torch.pi).float().cuda()
    pos = torch.tensor([0, 1, -1, 2, -2, 3, 4, 5, 1000, -1001, 2 ** 20, -2 ** 20], dtype=torch.int32, device="cuda")
    s, c = turned(f, pos, dtype, False, False)
    angle = pos.double().view(-1, 1) * f.double()
    # (f32 frequencies are off the fractions by up to 2^-25 of them: the angles here are those of the f32 values)
    tol = 2.0 ** -22 + angle.abs() * 2.0 ** -51 + (2.0 ** -8 if dtype is BF else 0.0)
    assert bool(((s + torch.sin(angle)).abs() <= tol).all()) and bool(((c - torch.cos(angle)).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,D,R", [(16, 2, 256, 64), (7, 1, 72, 36), (5, 9, 24, 24), (64, 3, 16, 8)])
def test_tokens_come_out_alike_however_many_warps_share_them(dtype, hq, hkv, D, R):
    """A few tokens' heads are spread over warps, of which some have query heads and no key heads; of many
    tokens a warp takes several whole ones: the same bits."""
    g = torch.Generator().manual_seed(5)
    most = 5000
    q, k, v = (torch.randn((most, h, D), generator=g).to(dtype).cuda() for h in (hq, hkv, hkv))
    w = [(1 + 0.1 * torch.randn(D, generator=g)).cuda() for _ in range(2)]
    f = (1e4 ** (-torch.arange(R // 2, dtype=torch.float64) / (R // 2))).float().cuda()
    pos = torch.arange(most, dtype=torch.int32, device="cuda") + 77
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")

    def run(T):
        kc, vc = (torch.zeros((1, hkv, most, D), dtype=dtype, device="cuda") for _ in range(2))
        lens = torch.tensor([T], dtype=torch.int32, device="cuda")
        out = gdn.gdn_rope_kv_append(q[:T], k[:T], v[:T], kc, vc, table, lens, f, positions=pos[:T], q_norm_w=w[0], k_norm_w=w[1])
        return out, kc, vc

    out, kc, vc = run(most)
    assert torch.equal(vc[0].transpose(0, 1), v)
    for T in (1, 2, 3, 37, 151, 152, 153, 303, 608, 809, 1215, 1216, 1217, 2431, 2432, 2433, 3040, 3041):
        o, kt, vt = run(T)
        assert torch.equal(o, out[:T]) and torch.equal(kt[:, :, :T], kc[:, :, :T]) and torch.equal(vt[:, :, :T], vc[:, :, :T])
        assert not kt[:, :, T:].any() and not vt[:, :, T:].any()


@pytest.mark.parametrize("T,H,D,R,n_axes,interleaved", [(130, 5, 72, 72, 3, False), (1000, 16, 80, 80, 3, False), (700, 3, 64, 64, 1, True),
                                                        (99, 2, 128, 126, 2, True), (500, 4, 256, 64, 16, False), (9, 1, 8, 2, 1, False)])
def test_f32_rotations_without_a_norm(T, H, D, R, n_axes, interleaved):
    """The cosine and the sine are off by 1.5 steps of 2^-24 (see above) and are rounded once more with mscale; a
    product and a sum round once each: (|a| + |b|) mscale 4.5 2^-24 in all, and the output is one of those roundings."""
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H, D), generator=g).cuda()
    f = (1e4 ** (-torch.arange(R // 2, dtype=torch.float64) / (R // 2))).float().cuda()
    pos = torch.randint(-30000, 30000, (n_axes, T), generator=g, dtype=torch.int32).cuda()
    axes = torch.randint(0, n_axes, (R // 2,), generator=g, dtype=torch.int32).cuda()
    for mscale in (1.0, 1.25, -0.7):
        y = gdn.gdn_rope(x, f, pos, axes=axes, mscale=mscale, interleaved=interleaved).double()
        want, _ = rot.rope(x, f, pos, axes, mscale=mscale, interleaved=interleaved)
        j = torch.arange(R // 2, device="cuda")
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)
        size = (x[:, :, a].abs() + x[:, :, b].abs()).double() * abs(mscale) * 4.5 * 2.0 ** -24 + 1e-30
        assert bool(((y - want)[:, :, a].abs() <= size).all()) and bool(((y - want)[:, :, b].abs() <= size).all())
        assert torch.equal(y[:, :, R:], want[:, :, R:])
