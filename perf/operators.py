"""Cases of the serving operators that stand beside the layer core's decode and
verification calls: the paged key-value cache of the softmax-attention layers
of the hybrid models, the attention of the newest tokens that reads it, and the
acceptance of drafted tokens.

`run` makes one call of an operator: in its plain form (elementary torch
operations in 32 bits, 64 where a border is decided), or, with `own`, through
the package.  `exact` computes the same outputs in 64 bits, sequence by
sequence.
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # --- attention of the newest tokens over the paged cache
        # one user, a short chat, head layout of the hybrid models' softmax layers: latency
        dict(name="attn_one_short", op="attn", B=1, K=1, hq=16, hkv=2, D=256, page=16, lo=201, hi=201,
             gate=True, dtype="bf16"),
        # one user at the longest context of the long-context workload: the split over the length
        dict(name="attn_one_262144", op="attn", B=1, K=1, hq=16, hkv=2, D=256, page=64, lo=262144, hi=262144,
             gate=True, dtype="bf16"),
        # the decode batch of 64 sequences, ragged lengths as in the packed prefill workload
        dict(name="attn_batch64", op="attn", B=64, K=1, hq=16, hkv=2, D=256, page=64, lo=512, hi=8192,
             gate=True, dtype="bf16"),
        # its verification pass: the last sampled token and 4 drafts per sequence
        dict(name="attn_batch64_verify5", op="attn", B=64, K=5, hq=16, hkv=2, D=256, page=16, lo=512, hi=8192,
             gate=True, dtype="bf16"),
        # the widest verification pass: 16 tokens of 8 query heads per key-value head
        dict(name="attn_verify16_d128", op="attn", B=16, K=16, hq=32, hkv=4, D=128, page=128, lo=1024, hi=16384,
             gate=False, dtype="bf16"),
        # odd everything: heads, head dim, page size that is no power of two, lengths down to K
        dict(name="attn_odd", op="attn", B=7, K=3, hq=15, hkv=3, D=80, page=24, lo=3, hi=3001,
             gate=False, dtype="bf16"),
        # the all-f32 path
        dict(name="attn_f32", op="attn", B=8, K=1, hq=16, hkv=4, D=128, page=32, lo=100, hi=4096,
             gate=False, dtype="f32"),
        # --- acceptance of drafted tokens
        # one user, 3 drafts
        dict(name="accept_one", op="accept", B=1, K=3, V=32000, drafts="sampled", dtype="f32"),
        # the batch of 64, 4 drafts, a large vocabulary
        dict(name="accept_batch64", op="accept", B=64, K=4, V=131072, drafts="sampled", dtype="f32"),
        # deterministic drafts (no draft probabilities), odd vocabulary, ragged draft counts, bf16
        dict(name="accept_fixed_odd", op="accept", B=33, K=7, V=50021, drafts="fixed", dtype="bf16"),
        # --- writing new keys and values into their pages
        # one verification pass of the batch
        dict(name="append_batch64", op="append", B=64, K=5, hkv=2, D=256, page=16, lo=512, hi=8192, dtype="bf16"),
        # prompts: 8 packed sequences of 32768 tokens in all
        dict(name="append_prompts", op="append", B=8, K=0, hkv=2, D=256, page=64, lo=512, hi=8192, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(2.0 ** rng.uniform(torch.log2(torch.tensor(float(lo))).item(),
                                        torch.log2(torch.tensor(float(hi))).item())))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "accept", "append"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "accept":
        while True:
            c = dict(op=op, B=_log_int(rng, 1, 64), K=rng.randint(0, 15), V=_log_int(rng, 500, 200000),
                     drafts=rng.choice(["sampled", "fixed"]), dtype=dtype)
            if c["B"] * (2 * c["K"] + 1) * c["V"] <= 64 * 9 * 131072:
                return c
    while True:
        hkv = rng.randint(1, 8)
        D = rng.choice([16, 64, 80, 96, 128, 128, 192, 256, 256])
        page = rng.choice([8, 16, 16, 24, 32, 48, 64, 100, 128, 256])
        B = _log_int(rng, 1, 64)
        K = rng.choice([1, 1, 1, 2, 4, 5, 8, 16])
        hi = _log_int(rng, 32, 131072)
        lo = min(hi, max(K, _log_int(rng, 32, hi)))
        es = 2 if dtype == "bf16" else 4
        cache = 2 * es * hkv * D * B * hi
        if op == "append":
            if cache <= 1 << 29:
                return dict(op=op, B=B, K=rng.choice([0, K]), hkv=hkv, D=D, page=page, lo=lo, hi=hi, dtype=dtype)
            continue
        group = rng.randint(1, 8)
        # padded 32-bit scores and caches of the plain form stay below the largest listed case's
        if cache <= 1 << 29 and B * hi * hkv * group * K <= 1 << 26 and (dtype == "bf16" or K <= 5):
            return dict(op=op, B=B, K=K, hq=group * hkv, hkv=hkv, D=D, page=page, lo=lo, hi=hi,
                        gate=rng.random() < 0.5, dtype=dtype)


def _lengths(case):
    """Sequence lengths after the new tokens: spread over lo..hi by the case alone."""
    r = random.Random("%d %d %d" % (case["B"], case["lo"], case["hi"]))
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    n[-1] = case["hi"]  # the longest is among them
    return n


def _accepted(case):
    """How many drafts there are and how many hold, per sequence, by the case alone."""
    r = random.Random("%d %d %d" % (case["B"], case["K"], case["V"]))
    drafts = [case["K"] if case["drafts"] == "sampled" else r.randint(0, case["K"]) for _ in range(case["B"])]
    return drafts, [min(n, r.randint(0, case["K"] + 1)) for n in drafts]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    B, K = case["B"], case["K"]
    if case["op"] == "accept":
        # a rejected sequence needs the target's and the draft's row, an accepted one the target's
        drafts, held = _accepted(case)
        rows = sum(1 if h == n or case["drafts"] == "fixed" else 2 for n, h in zip(drafts, held))
        return {"bytes": rows * case["V"] * es + B * (K * (4 + 4 + 8) + 24), "flops": 3 * rows * case["V"]}
    n = _lengths(case)
    if case["op"] == "append":
        T = B * K if K else sum(n)
        return {"bytes": 4 * T * case["hkv"] * case["D"] * es + 8 * B, "flops": 0}
    cached = 2 * sum(n) * case["hkv"] * case["D"] * es
    rows = B * K * case["hq"]
    seen = sum(x * K - K * (K - 1) // 2 for x in n) * case["hq"]
    return {"bytes": cached + rows * (case["D"] * es * (3 if case["gate"] else 2) + 4) + 4 * sum(-(-x // case["page"]) for x in n),
            "flops": 4 * seen * case["D"]}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    B, K = case["B"], case["K"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dt)

    if case["op"] == "accept":
        return _prepare_accept(case, gen, dt)
    n = _lengths(case)
    page = case["page"]
    pages = [-(-x // page) for x in n]
    width, total = max(pages), sum(pages) + 3
    # every sequence's pages lie scattered over the cache; entries past them are never used
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor([sum(pages[:b]) for b in range(B)], device="cuda").view(B, 1)
    col = torch.arange(width, device="cuda").view(1, width)
    used = col < torch.tensor(pages, device="cuda").view(B, 1)
    table = torch.where(used, order[(first + col).clamp(max=total - 1)], 0).to(torch.int32)
    s = {"case": case, "table": table, "lens": torch.tensor(n, dtype=torch.int32, device="cuda"),
         "k_cache": normal(total, case["hkv"], page, case["D"]),
         "v_cache": normal(total, case["hkv"], page, case["D"])}
    if case["op"] == "append":
        T = B * K if K else sum(n)
        s["k"], s["v"] = normal(T, case["hkv"], case["D"]), normal(T, case["hkv"], case["D"])
        s["cu"] = None
        if not K:
            s["cu"] = torch.tensor([sum(n[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        return s
    s["q"] = normal(B, K, case["hq"], case["D"])
    s["gate"] = normal(B, K, case["hq"], case["D"]) if case["gate"] else None
    return s


def _prepare_accept(case, gen, dt):
    """Rows of softmax probabilities, drafts sampled from the draft's rows, and uniforms under which
    the planned number of drafts holds."""
    B, K, V = case["B"], case["K"], case["V"]
    drafts, held = _accepted(case)
    logits = torch.randn((B, K + 1, V), generator=gen, device="cuda").mul_(2.5)
    p = torch.softmax(logits, -1).to(dt)
    q = torch.softmax(logits[:, :K] + torch.randn((B, K, V), generator=gen, device="cuda"), -1).to(dt)
    del logits
    u = torch.rand((B, K + 1), generator=gen, device="cuda").clamp_(max=1 - 2.0 ** -20)
    n_draft = torch.tensor(drafts, dtype=torch.int32, device="cuda")
    n_held = torch.tensor(held, device="cuda").view(B, 1)
    if K:
        token = torch.multinomial(q.float().view(B * K, V), 1, generator=gen).view(B, K)
        if case["drafts"] == "fixed":
            token = p[:, :K].float().argmax(-1)
        # the draft that fails is one the draft model likes better than the target
        worst = (q.float() - p[:, :K].float()).argmax(-1)
        at = torch.arange(K, device="cuda").view(1, K)
        token = torch.where(at == n_held, worst, token)
        ratio = p[:, :K].gather(-1, token.unsqueeze(-1)).squeeze(-1).float()
        if case["drafts"] == "sampled":
            ratio = ratio / q.gather(-1, token.unsqueeze(-1)).squeeze(-1).float()
        ratio = ratio.clamp(max=1.0)
        u[:, :K] = torch.where(at < n_held, u[:, :K] * ratio * 0.99, ratio + (1 - ratio) * (0.01 + 0.98 * u[:, :K]))
        token = token.to(torch.int32)
    else:
        token = torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    slots = torch.randperm(B * (K + 2), generator=gen, device="cuda").to(torch.int32).view(B, K + 2)
    return {"case": case, "p": p, "q": q if case["drafts"] == "sampled" else None, "token": token, "u": u,
            "n_draft": n_draft if case["drafts"] == "fixed" else None, "slots": slots}


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if op == "attn":
        return _run_attn(state)
    return _run_append(state) if op == "append" else _run_accept(state)


def _run_attn(s):
    if own:
        import gated_deltanet_linear_core_gb300 as gdn
        out, lse = gdn.gdn_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], gate=s["gate"],
                                       return_lse=True)
        return {"out": out, "lse": lse}
    q, lens = s["q"], s["lens"]
    B, K, hq, D = q.shape
    hkv, page = s["k_cache"].shape[1], s["k_cache"].shape[2]
    L = s["table"].shape[1] * page

    def gathered(cache):  # [B, hkv, L, D] in 32 bits
        return cache[s["table"].long()].transpose(1, 2).reshape(B, hkv, L, D).float()

    rows = q.float().view(B, K, hkv, hq // hkv, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, K * (hq // hkv), D)
    score = torch.matmul(rows, gathered(s["k_cache"]).transpose(2, 3)) * D ** -0.5
    score = score.view(B, hkv, K, hq // hkv, L)
    # token i of the K newest sees the cache up to itself
    end = lens.view(B, 1) - (K - 1 - torch.arange(K, device=q.device)).view(1, K)
    hidden = torch.arange(L, device=q.device).view(1, 1, L) >= end.view(B, K, 1)
    score = score.masked_fill(hidden.view(B, 1, K, 1, L), float("-inf"))
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - top)
    total = weight.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    out = torch.matmul((weight / total).view(B, hkv, -1, L), gathered(s["v_cache"]))
    out = out.view(B, hkv, K, hq // hkv, D).permute(0, 2, 1, 3, 4).reshape(B, K, hq, D)
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].float()))
    return {"out": out.to(q.dtype), "lse": lse.permute(0, 2, 1, 3).reshape(B, K, hq)}


def _run_append(s):
    if own:
        import gated_deltanet_linear_core_gb300 as gdn
        gdn.gdn_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], cu_seqlens=s["cu"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    T, B, page = s["k"].shape[0], s["lens"].shape[0], s["k_cache"].shape[2]
    t = torch.arange(T, device=s["k"].device)
    if s["cu"] is None:
        seq, end = t // (T // B), (t // (T // B) + 1) * (T // B)
    else:
        seq = torch.searchsorted(s["cu"], t, right=True) - 1
        end = s["cu"][seq + 1]
    pos = s["lens"][seq] - (end - t)
    at = s["table"][seq, (pos // page).long()].long()
    s["k_cache"][at, :, pos % page] = s["k"]
    s["v_cache"][at, :, pos % page] = s["v"]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _run_accept(s):
    if own:
        import gated_deltanet_linear_core_gb300 as gdn
        n, tokens, slot = gdn.gdn_draft_accept(s["p"], s["q"], s["token"], s["u"], n_draft=s["n_draft"],
                                               slots=s["slots"])
        return {"n_accept": n, "tokens": tokens, "next_slot": slot}
    p, q, token, u = s["p"], s["q"], s["token"].long(), s["u"].double()
    B, K, V = p.shape[0], token.shape[1], p.shape[2]
    at = torch.arange(K, device=p.device).view(1, K)
    # a draft holds when u q(d) < p(d) and every draft before it holds
    pd = p[:, :K].gather(-1, token.unsqueeze(-1)).squeeze(-1).double()
    qd = torch.ones_like(pd) if q is None else q.gather(-1, token.unsqueeze(-1)).squeeze(-1).double()
    drafts = torch.full((B, 1), K, device=p.device) if s["n_draft"] is None else s["n_draft"].long().view(B, 1)
    good = (u[:, :K] * qd < pd) & (at < drafts)
    n = good.long().cumprod(1).sum(1, keepdim=True)
    # the next token: from (p - q)+ after a draft that failed, else from the target's next row
    b = torch.arange(B, device=p.device).view(B, 1)
    row = p[b, n].squeeze(1).double()
    failed = n < drafts
    if K:
        last = n.clamp(max=K - 1)
        if q is None:
            less = torch.zeros_like(row).scatter_(1, token.gather(1, last), 1.0)
        else:
            less = q[b, last].squeeze(1).double()
        row = torch.where(failed, (row - less).clamp(min=0), row)
    total = row.cumsum(-1)
    picked = torch.searchsorted(total, u[:, K:] * total[:, -1:], right=True).clamp(max=V - 1)
    wide = torch.arange(K + 1, device=p.device).view(1, K + 1)
    padded = torch.cat([token, torch.zeros((B, 1), dtype=torch.long, device=p.device)], 1)
    tokens = torch.where(wide < n, padded, torch.where(wide == n, picked, -1))
    return {"n_accept": n.view(B).to(torch.int32), "tokens": tokens.to(torch.int32),
            "next_slot": s["slots"].gather(1, n + 1).view(B)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_accept(s)


def _exact_attn(s):
    q = s["q"].double()
    B, K, hq, D = q.shape
    hkv, page = s["k_cache"].shape[1:3]
    group = hq // hkv
    out, lse = torch.zeros_like(q), torch.zeros((B, K, hq), dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["lens"].tolist()):
        ids = s["table"][b, :-(-n // page)].long()
        for h in range(hkv):
            k = s["k_cache"][ids, h].reshape(-1, D)[:n].double()
            v = s["v_cache"][ids, h].reshape(-1, D)[:n].double()
            x = q[b, :, h * group:(h + 1) * group].reshape(K * group, D)
            a = x @ k.t() / D ** 0.5
            for i in range(K - 1):
                a[i * group:(i + 1) * group, n - (K - 1 - i):] = -torch.inf
            lse[b, :, h * group:(h + 1) * group] = torch.logsumexp(a, -1).view(K, group)
            out[b, :, h * group:(h + 1) * group] = (torch.softmax(a, -1) @ v).view(K, group, D)
    if s["gate"] is not None:
        out *= torch.sigmoid(s["gate"].double())
    return {"out": out, "lse": lse}


def _exact_append(s):
    lens = s["lens"].tolist()
    B, page, T = len(lens), s["k_cache"].shape[2], s["k"].shape[0]
    cu = s["cu"].tolist() if s["cu"] is not None else [b * (T // B) for b in range(B + 1)]
    result = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    for b in range(B):
        new = cu[b + 1] - cu[b]
        pos = torch.arange(lens[b] - new, lens[b], device=s["k"].device)
        ids = s["table"][b].long()[pos // page]
        for name, x in (("k_cache", s["k"]), ("v_cache", s["v"])):
            result[name][ids, :, pos % page] = x[cu[b]:cu[b + 1]].double()
    return result


def _exact_accept(s):
    p, u, token, slots = s["p"], s["u"].double().cpu(), s["token"].tolist(), s["slots"].tolist()
    B, K = p.shape[0], p.shape[1] - 1
    n_accept, tokens, slot = [], [], []
    for b in range(B):
        drafts = K if s["n_draft"] is None else int(s["n_draft"][b])
        n = 0
        while n < drafts:
            d = token[b][n]
            like = 1.0 if s["q"] is None else float(s["q"][b, n, d])
            if not float(u[b, n]) * like < float(p[b, n, d]):
                break
            n += 1
        row = p[b, n].double().cpu()
        if n < drafts:
            if s["q"] is None:
                row[token[b][n]] -= 1.0
            else:
                row -= s["q"][b, n].double().cpu()
            row = row.clamp(min=0)
        total = torch.cumsum(row, 0)
        picked = int((total <= u[b, K] * total[-1]).sum())
        n_accept.append(n)
        tokens.append(token[b][:n] + [min(picked, row.numel() - 1)] + [-1] * (K - n))
        slot.append(slots[b][n + 1])
    return {"n_accept": torch.tensor(n_accept), "tokens": torch.tensor(tokens), "next_slot": torch.tensor(slot)}
