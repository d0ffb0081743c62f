"""64-bit forms of the serving operators (paged-cache attention, cache append,
drafted-token acceptance) and the error bounds their outputs are held to."""
from __future__ import annotations

import torch

EPS_F32 = 2.0 ** -24  # half a step, relative
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS_F32}


def make_cache(lens, page, hkv, D, dtype, gen, device, extra=2, hidden=None):
    """A cache whose sequences' pages lie scattered, and its page table.  `hidden`
    fills every position that belongs to no sequence (NaN, say)."""
    B = len(lens)
    pages = [-(-n // page) for n in lens]
    total = sum(pages) + extra
    order = torch.randperm(total, generator=gen)
    width = max(max(pages), 1)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    k = torch.randn((total, hkv, page, D), generator=gen).to(dtype)
    v = torch.randn((total, hkv, page, D), generator=gen).to(dtype)
    if hidden is not None:
        used = torch.zeros((total, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            for t in range(0, n, page):
                used[table[b, t // page], :min(page, n - t)] = True
        free = ~used.view(total, 1, page, 1)
        k.masked_fill_(free, hidden)
        v.masked_fill_(free, hidden)
    return k.to(device), v.to(device), table.to(device), torch.tensor(lens, dtype=torch.int32, device=device)


def attention(q, k_cache, v_cache, table, lens, scale=None, gate=None):
    """(out, lse, bound): the outputs in 64 bits and an elementwise bound of what a
    kernel in f32 arithmetic may be off by before it rounds its output.

    A score is a sum of D products in f32: off by at most (D + 2) 2^-24 scale
    |q| |k| (Cauchy-Schwarz over the terms; + 2 for scaling into the log2 domain
    and subtracting the maximum).  exp2 of it adds 2^-21 (the special-function
    unit's error and the argument's rounding at moderate arguments), the weights
    may be held as two bf16 (2^-16), and sums of n weights run over tiles: at most
    (n / 128 + 256) 2^-24.  Twice the sum of these relative errors (numerator and
    denominator) times the largest |v| bounds the output's error."""
    B, K, hq, D = q.shape
    hkv, page = k_cache.shape[1:3]
    G = hq // hkv
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros((B, K, hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((B, K, hq), -torch.inf, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(lse)
    cap = table.shape[1] * page
    for b, n in enumerate(lens.tolist()):
        n = min(max(n, 0), cap)
        ids = table[b, :-(-n // page)].long()
        for h in range(hkv):
            k = k_cache[ids, h].reshape(-1, D)[:n].double()
            v = v_cache[ids, h].reshape(-1, D)[:n].double()
            for i in range(K):
                m = n - (K - 1 - i)
                if m <= 0:
                    continue
                qr = q[b, i, h * G:(h + 1) * G].double()
                s = qr @ k[:m].t() * scale
                out[b, i, h * G:(h + 1) * G] = torch.softmax(s, -1) @ v[:m]
                lse[b, i, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
                d_s = (D + 2) * EPS_F32 * scale * qr.norm(dim=-1) * k[:m].norm(dim=-1).max()
                rel = d_s + 2.0 ** -21 + 2.0 ** -16 + (m / 128 + 256) * EPS_F32
                bound[b, i, h * G:(h + 1) * G] = 2 * rel * v[:m].abs().max()
    if gate is not None:
        out = out * torch.sigmoid(gate.double())
    return out, lse, bound.unsqueeze(-1)


def check_attention(out, lse, ref, dtype):
    r_out, r_lse, bound = ref
    # the gate and the division round to f32 a few times
    tol = (HALF_STEP[dtype] + 2.0 ** -20) * r_out.abs() + bound
    err = (out.double() - r_out).abs()
    assert torch.isfinite(out).all(), "non-finite output"
    worst = (err / tol.clamp(min=1e-300)).max().item()
    assert bool((err <= tol).all()), f"output {worst:.2f} times its bound off"
    rel = (err.norm() / r_out.norm().clamp(min=1e-300)).item()
    assert rel <= HALF_STEP[dtype] + 1e-4 * (dtype == torch.bfloat16) + 1e-5, f"rel-L2 {rel:.2e}"
    if lse is not None:
        dead = r_lse == -torch.inf
        assert torch.equal(torch.isneginf(lse), dead), "lse of empty rows"
        e = (lse.double() - r_lse).abs()[~dead]
        # bound holds the relative error of a weight (times |v|max >= ...); lse adds one rounding
        if e.numel():
            lim = 2.0 ** -20 * (1 + r_lse.abs()[~dead]) + 1e-4
            assert bool((e <= lim).all()), f"lse off by {e.max().item():.2e}"


def weight_error(q, k_cache, table, lens, scale=None):
    """[B, K, H_q] f64: by how much a weight of a row may be off, relatively, where nothing is held in fewer
    than 32 bits; the log of a row's sum may then be off by as much.

    The score's error as in attention(); five exponentials of 2^-21 each that multiply into a weight (its own,
    one move of the running maximum, and the joins of warps, of groups of parts and of parts); the sum over
    tiles at most (n / 128 + 256) 2^-24."""
    B, K, hq, D = q.shape
    hkv, page = k_cache.shape[1:3]
    G = hq // hkv
    scale = D ** -0.5 if scale is None else scale
    err = torch.zeros((B, K, hq), dtype=torch.float64, device=q.device)
    for b, n in enumerate(lens.tolist()):
        ids = table[b, :-(-n // page)].long()
        for h in range(hkv):
            far = k_cache[ids, h].reshape(-1, D)[:n].double().norm(dim=-1).max()
            d_s = (D + 2) * EPS_F32 * scale * q[b, :, h * G:(h + 1) * G].double().norm(dim=-1) * far
            err[b, :, h * G:(h + 1) * G] = d_s + 5 * 2.0 ** -21 + (n / 128 + 256) * EPS_F32
    return err


def append(k, v, k_cache, v_cache, table, lens, cu):
    """Token by token; returns new caches."""
    kc, vc = k_cache.clone(), v_cache.clone()
    page, cap = kc.shape[2], table.shape[1] * kc.shape[2]
    for b, n in enumerate(lens.tolist()):
        for t in range(cu[b], cu[b + 1]):
            pos = n - (cu[b + 1] - t)
            if not 0 <= pos < cap:
                continue
            pg = int(table[b, pos // page])
            if 0 <= pg < kc.shape[0]:
                kc[pg, :, pos % page] = k[t]
                vc[pg, :, pos % page] = v[t]
    return kc, vc


def accept(p, q, draft, u, n_draft=None):
    """(n_accept, tokens): lists, from the definition in 64 bits."""
    B, K = p.shape[0], p.shape[1] - 1
    V = p.shape[2]
    p, u = p.double().cpu(), u.double().cpu()
    q = None if q is None else q.double().cpu()
    ns, toks = [], []
    for b in range(B):
        m = K if n_draft is None else min(max(int(n_draft[b]), 0), K)
        n = 0
        while n < m:
            d = int(draft[b, n])
            if not 0 <= d < V:
                break
            qd = 1.0 if q is None else float(q[b, n, d])
            if not float(u[b, n]) * qd < float(p[b, n, d]):
                break
            n += 1
        row = p[b, n].clone()
        if n < m:
            if q is not None:
                row -= q[b, n]
            elif 0 <= int(draft[b, n]) < V:
                row[int(draft[b, n])] -= 1.0
        row = row.clamp(min=0)
        if not row.sum() > 0:
            row = p[b, n].clamp(min=0)
        run = torch.cumsum(row, 0)
        total = float(run[-1])
        if total > 0:
            border = min(max(float(u[b, K]) * total, 0.0), total * (1 - 2.0 ** -52))
            hit = torch.nonzero((run > border) & (row > 0))
            tok = int(hit[0]) if hit.numel() else int(torch.nonzero(row > 0)[-1])
        else:
            tok = 0
        ns.append(n)
        toks.append([int(x) for x in draft[b, :n]] + [tok] + [-1] * (K - n))
    return ns, toks
