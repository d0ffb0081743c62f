"""Cases of the rotary and shared-prefix serving operators of the softmax-attention
layers: rotary positions of one to three axes with the head norms before them, the
same on the way into the paged key-value cache, and the attention of the newest
tokens of sequences that share a long prefix.

`run` makes one call of an operator: in its plain form (elementary torch
operations in 32 bits, angles in 64), or, with `own`, through the package.
`exact` computes the same outputs in 64 bits, in another way.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # --- rotary positions alone
        # one user's decode step: the queries of one token, three axes in turns over the first 64 of 256 dims; latency
        dict(name="rope_one", op="rope", T=1, H=16, D=256, R=64, axes="turns", layout="gated", norm=True, pairs="halves",
             base=1e7, dtype="bf16"),
        # a video's patches (21 x 40 x 39) in a vision tower: queries taken out of the fused projection, all dims rotated
        dict(name="rope_video", op="rope", T=32760, H=16, D=80, R=80, axes="sections", layout="fused", norm=False,
             pairs="halves", base=1e4, dtype="bf16"),
        # odd everything, f32: part of an odd head, neighbouring dims paired, one axis
        dict(name="rope_odd_f32", op="rope", T=5003, H=7, D=72, R=36, axes="one", layout="dense", norm=False,
             pairs="neighbours", base=1e4, dtype="f32"),
        # --- into the cache
        # a verification pass of the batch of 64: positions are the cache's own
        dict(name="rope_append_batch64", op="append", B=64, K=5, hq=16, hkv=2, D=256, R=64, page=16, lo=512, hi=8192,
             axes="cache", layout="gated", norm=True, pairs="halves", base=1e7, dtype="bf16"),
        # prompts with images: 8 packed sequences of some 32000 tokens in all, three axes
        dict(name="rope_append_prompts", op="append", B=8, K=0, hq=16, hkv=2, D=256, R=64, page=64, lo=512, hi=8192,
             axes="turns", layout="gated", norm=True, pairs="halves", base=1e7, dtype="bf16"),
        # far positions in f32, odd heads, pages that are no power of two
        dict(name="rope_append_far_f32", op="append", B=3, K=4, hq=6, hkv=3, D=96, R=96, page=24, lo=100000, hi=131072,
             axes="cache", layout="fused", norm=False, pairs="halves", base=1e4, dtype="f32"),
        # --- attention over a shared prefix
        # four samples of one short chat: latency
        dict(name="shared_four_short", op="shared", B=4, groups=1, K=1, hq=16, hkv=2, D=256, page=16, plo=1000, phi=1000,
             lo=1, hi=60, gate=True, dtype="bf16"),
        # the decode batch of 64 behind one long document
        dict(name="shared_batch64", op="shared", B=64, groups=1, K=1, hq=16, hkv=2, D=256, page=64, plo=32768, phi=32768,
             lo=16, hi=1024, gate=True, dtype="bf16"),
        # the verification pass of 48 sequences in 6 groups of their own system prompts
        dict(name="shared_groups_verify5", op="shared", B=48, groups=6, K=5, hq=16, hkv=2, D=256, page=16, plo=512,
             phi=8192, lo=5, hi=2000, gate=True, dtype="bf16"),
        # the widest verification pass: 32 sequences with 16 new tokens each, 4096 rows per key-value head
        dict(name="shared_verify16_d128", op="shared", B=32, groups=1, K=16, hq=32, hkv=4, D=128, page=128, plo=16384,
             phi=16384, lo=16, hi=512, gate=False, dtype="bf16"),
        # eight samples at the longest context
        dict(name="shared_eight_262144", op="shared", B=8, groups=1, K=1, hq=16, hkv=2, D=256, page=64, plo=262000,
             phi=262000, lo=1, hi=144, gate=True, dtype="bf16"),
        # the all-f32 path, odd heads, head dim and pages
        dict(name="shared_odd_f32", op="shared", B=9, groups=2, K=3, hq=15, hkv=3, D=80, page=24, plo=100, phi=5000,
             lo=3, hi=300, gate=False, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "shared", "shared", "shared"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op != "shared":
        D = rng.choice([16, 64, 72, 80, 96, 128, 128, 192, 256, 256])
        c = dict(op=op, D=D, R=rng.choice([D, D, 2 * rng.randint(1, D // 2)]), layout=rng.choice(["dense", "fused", "gated"]),
                 norm=rng.random() < 0.5, pairs=rng.choice(["halves", "halves", "neighbours"]),
                 base=rng.choice([1e4, 1e6, 1e7]), dtype=dtype)
        if op == "rope":
            while True:
                c.update(T=_log_int(rng, 1, 40000), H=_log_int(rng, 1, 64), axes=rng.choice(["one", "sections", "turns"]))
                if c["T"] * c["H"] * D <= 1 << 26:
                    return c
        while True:
            hkv = rng.randint(1, 8)
            c.update(B=_log_int(rng, 1, 64), K=rng.choice([0, 1, 1, 2, 5, 16]), hkv=hkv, hq=hkv * rng.randint(1, 8),
                     page=rng.choice([8, 16, 16, 24, 32, 64, 100, 128]), axes=rng.choice(["cache", "one", "sections", "turns"]))
            c["hi"] = _log_int(rng, 32, 131072)
            c["lo"] = min(c["hi"], max(c["K"], _log_int(rng, 32, c["hi"])))
            tokens = c["B"] * (c["K"] or c["hi"])
            if 4 * hkv * D * c["B"] * c["hi"] <= 1 << 28 and tokens * (c["hq"] + 2 * hkv) * D <= 1 << 27:
                return c
    while True:
        hkv = rng.randint(1, 8)
        c = dict(op=op, B=_log_int(rng, 2, 64), K=rng.choice([1, 1, 1, 2, 4, 5, 8, 16]), hq=hkv * rng.randint(1, 8), hkv=hkv,
                 D=rng.choice([16, 64, 80, 96, 128, 128, 192, 256, 256]), page=rng.choice([8, 16, 16, 24, 32, 48, 64, 100, 128, 256]),
                 gate=rng.random() < 0.5, dtype=dtype)
        c["groups"] = min(c["B"], rng.choice([1, 1, 2, 3, 7]))
        c["phi"] = _log_int(rng, 64, 131072)
        c["plo"] = _log_int(rng, 64, c["phi"])
        c["hi"] = _log_int(rng, 32, 2048)
        c["lo"] = min(c["hi"], max(c["K"], _log_int(rng, 1, c["hi"])))
        es = 2 if dtype == "bf16" else 4
        cache = 2 * es * hkv * c["D"] * (c["groups"] * c["phi"] + c["B"] * c["hi"])
        rows = c["B"] * c["K"] * c["hq"]
        flops = 4 * rows * (c["phi"] + c["hi"]) * c["D"]
        # no more than the largest listed cases: the cache's bytes, the products, the 32-bit scores of the plain form
        if cache <= 1 << 29 and flops <= (1.3e11 if dtype == "bf16" else 1e10) and rows * max(c["phi"], c["hi"]) <= 1 << 28:
            return c


def _rng(case, what):
    return random.Random("%s %s" % (what, sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """Lengths (behind the prefix, for shared ones), spread over lo..hi by the case alone."""
    r = _rng(case, "lengths")
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    n[-1] = case["hi"]  # the longest is among them
    return n


def _groups(case):
    """(first sequence of each group and the end, prefix lengths)."""
    r = _rng(case, "groups")
    cuts = sorted(r.sample(range(1, case["B"]), case["groups"] - 1))
    prefix = [r.randint(case["plo"], case["phi"]) for _ in range(case["groups"])]
    prefix[-1] = case["phi"]
    return [0] + cuts + [case["B"]], prefix


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    D = case["D"]
    if case["op"] == "rope":
        n = case["T"] * case["H"] * D
        return {"bytes": 2 * n * es + 4 * case["T"] * (1 if case["axes"] == "one" else 3), "flops": 3 * n}
    if case["op"] == "append":
        T = case["B"] * case["K"] if case["K"] else sum(_lengths(case))
        n = T * (case["hq"] + 2 * case["hkv"]) * D
        at = {"cache": 0, "one": 1}.get(case["axes"], 3)
        return {"bytes": 2 * n * es + 4 * T * at + 8 * case["B"], "flops": 3 * T * (case["hq"] + case["hkv"]) * D}
    own_n, (first, prefix) = _lengths(case), _groups(case)
    K, rows = case["K"], case["B"] * case["K"] * case["hq"]
    cached = 2 * (sum(own_n) + sum(prefix)) * case["hkv"] * D * es
    seen = 0
    for g, p in enumerate(prefix):
        for n in own_n[first[g]:first[g + 1]]:
            seen += ((p + n) * K - K * (K - 1) // 2) * case["hq"]
    return {"bytes": cached + rows * (D * es * (3 if case["gate"] else 2) + 4), "flops": 4 * seen * D}


# ------------------------------------------------------------------ inputs
def _rotation(case, T, gen, first=None):
    """Frequencies, the axis of each, and the positions of T tokens (None: the cache's own)."""
    half = case["R"] // 2
    j = torch.arange(half, device="cuda", dtype=torch.float64)
    inv_freq = (case["base"] ** (-j / half)).float()
    if case["axes"] in ("one", "cache"):
        if case["axes"] == "cache":
            return inv_freq, None, None
        start = torch.randint(0, 100000, (1,), generator=gen, device="cuda", dtype=torch.int32)
        return inv_freq, None, torch.arange(T, device="cuda", dtype=torch.int32) + start
    if case["axes"] == "turns":  # time, height, width, time, ..
        axis = torch.arange(half, device="cuda", dtype=torch.int32) % 3
    else:  # a quarter for time, then height and width
        cut = [half // 4, half // 4 + (half - half // 4 + 1) // 2]
        axis = (torch.arange(half, device="cuda").view(-1, 1) >= torch.tensor(cut, device="cuda")).sum(1).to(torch.int32)
    # frames of 40 x 39 patches one after another, from some position on
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    at = torch.stack([t // 1560, t // 39 % 40, t % 39])
    return inv_freq, axis, (at + torch.randint(0, 2000, (3, 1), generator=gen, device="cuda", dtype=torch.int32)).contiguous()


def _taken(case, T, heads, gen):
    """[T, h, D] for each of `heads`, as the projection before leaves them: fused (all heads of a token in one
    row), gated (each query head next to its gate besides), or tensors of their own."""
    dt, D = DTYPES[case["dtype"]], case["D"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dt)

    if case["layout"] == "dense":
        return [normal(T, h, D) for h in heads]
    wide = 2 if case["layout"] == "gated" else 1
    width = [heads[0] * wide] + list(heads[1:])
    if len(heads) == 1 and wide == 1:
        width += [heads[0], heads[0]]  # the keys and values that lie beside a tower's queries
    row = normal(T, sum(width) * D)
    parts = [p.view(T, n, D) for p, n in zip(row.split([n * D for n in width], 1), width)][:len(heads)]
    parts[0] = parts[0].view(T, heads[0], wide, D)[:, :, 0]
    return parts


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "shared":
        return _prepare_shared(case, gen)
    dt, D = DTYPES[case["dtype"]], case["D"]
    s = {"case": case}

    def weight():
        return 1 + 0.1 * torch.randn(D, generator=gen, device="cuda") if case["norm"] else None

    if case["op"] == "rope":
        s["x"], = _taken(case, case["T"], [case["H"]], gen)
        s["w"] = weight()
        s["inv_freq"], s["axis"], s["pos"] = _rotation(case, case["T"], gen)
        return s
    B, K, page, n = case["B"], case["K"], case["page"], _lengths(case)
    T = B * K if K else sum(n)
    s["q"], s["k"], s["v"] = _taken(case, T, [case["hq"], case["hkv"], case["hkv"]], gen)
    s["qw"], s["kw"] = weight(), weight()
    s["inv_freq"], s["axis"], s["pos"] = _rotation(case, T, gen)
    s["cu"] = None
    if not K:
        s["cu"] = torch.tensor([sum(n[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    # every sequence's pages lie scattered over the cache
    pages = [-(-x // page) for x in n]
    total = sum(pages) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    s["table"] = torch.zeros((B, max(pages)), dtype=torch.int32, device="cuda")
    for b in range(B):
        s["table"][b, :pages[b]] = order[sum(pages[:b]):sum(pages[:b + 1])]
    for name in ("k_cache", "v_cache"):
        s[name] = torch.randn((total, case["hkv"], page, D), generator=gen, device="cuda", dtype=dt)
    return s


def _prepare_shared(case, gen):
    """Sequences in groups; a group's whole prefix pages are the same for all of its sequences, the page that the
    prefix ends in is each one's own copy."""
    dt, B, page, D = DTYPES[case["dtype"]], case["B"], case["page"], case["D"]
    own_n, (first, prefix) = _lengths(case), _groups(case)
    total_len = [p + n for g, p in enumerate(prefix) for n in own_n[first[g]:first[g + 1]]]
    shared = [p // page for p in prefix]
    pages = [-(-n // page) for n in total_len]
    total = sum(shared) + sum(pages) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    k_cache, v_cache = (torch.randn((total, case["hkv"], page, D), generator=gen, device="cuda", dtype=dt) for _ in range(2))
    table = torch.zeros((B, max(pages)), dtype=torch.int32, device="cuda")
    at = 0
    for g, p in enumerate(prefix):
        common = order[at:at + shared[g]]
        at += shared[g]
        last = None
        for b in range(first[g], first[g + 1]):
            mine = order[at:at + pages[b] - shared[g]]
            at += pages[b] - shared[g]
            table[b, :pages[b]] = torch.cat([common, mine])
            if p % page:
                if last is not None:
                    for c in (k_cache, v_cache):
                        c[mine[:1].long(), :, :p % page] = c[last, :, :p % page]
                last = mine[:1].long()

    def rows(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dt)

    q = rows(B, case["K"], case["hq"], D)
    return {"case": case, "q": q, "k_cache": k_cache, "v_cache": v_cache, "table": table,
            "lens": torch.tensor(total_len, dtype=torch.int32, device="cuda"),
            "prefix": torch.tensor(prefix, dtype=torch.int32, device="cuda"),
            "cu_groups": torch.tensor(first, dtype=torch.int32, device="cuda"),
            "gate": rows(*q.shape) if case["gate"] else None, "groups": (first, prefix, max(own_n))}


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if op == "rope":
        return _run_rope(state)
    return _run_append(state) if op == "append" else _run_shared(state)


def _norm_rotate(x, w, cos, sin, pairs):
    """x [T, H, D] in 32 bits: head norm with weight w, then rotation by cos, sin [T, R / 2]."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    half = cos.shape[1]
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    if pairs == "halves":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _angles(pos, axis, inv_freq):
    """cos and sin [T, R / 2] in 32 bits, of angles in 64."""
    pos = pos.view(1, -1) if pos.dim() == 1 else pos
    each = pos[axis.long()] if axis is not None else pos[:1]
    angle = (each.double() * inv_freq.double().view(-1, 1)).t()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _run_rope(s):
    c = s["case"]
    if own:
        import gated_deltanet_linear_core_gb300 as gdn
        return gdn.gdn_rope(s["x"], s["inv_freq"], s["pos"], axes=s["axis"], norm_w=s["w"], norm_eps=EPS,
                            interleaved=c["pairs"] == "neighbours")
    cos, sin = _angles(s["pos"], s["axis"], s["inv_freq"])
    return _norm_rotate(s["x"], s["w"], cos, sin, c["pairs"]).to(s["x"].dtype)


def _run_append(s):
    c = s["case"]
    if own:
        import gated_deltanet_linear_core_gb300 as gdn
        q = gdn.gdn_rope_kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["inv_freq"],
                                   positions=s["pos"], axes=s["axis"], q_norm_w=s["qw"], k_norm_w=s["kw"], norm_eps=EPS,
                                   interleaved=c["pairs"] == "neighbours", cu_seqlens=s["cu"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    T, B, page = s["k"].shape[0], s["lens"].shape[0], c["page"]
    t = torch.arange(T, device="cuda")
    if s["cu"] is None:
        seq, end = t // (T // B), (t // (T // B) + 1) * (T // B)
    else:
        seq = torch.searchsorted(s["cu"], t, right=True) - 1
        end = s["cu"][seq + 1]
    place = s["lens"][seq] - (end - t)
    cos, sin = _angles(place if s["pos"] is None else s["pos"], s["axis"], s["inv_freq"])
    q = _norm_rotate(s["q"], s["qw"], cos, sin, c["pairs"]).to(s["q"].dtype)
    k = _norm_rotate(s["k"], s["kw"], cos, sin, c["pairs"]).to(s["k"].dtype)
    at = s["table"][seq, (place // page).long()].long()
    s["k_cache"][at, :, place % page] = k
    s["v_cache"][at, :, place % page] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _run_shared(s):
    if own:
        import gated_deltanet_linear_core_gb300 as gdn
        out, lse = gdn.gdn_attn_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["prefix"],
                                              cu_groups=s["cu_groups"], gate=s["gate"], return_lse=True)
        return {"out": out, "lse": lse}
    q, (first, prefix, most) = s["q"], s["groups"]
    B, K, hq, D = q.shape
    hkv, page = s["k_cache"].shape[1:3]
    G = hq // hkv
    x = q.float().view(B, K, hkv, G, D).permute(2, 0, 1, 3, 4)  # [hkv, B, K, G, D]

    def part(score, v):
        """Maxima, sums and unnormalised outputs of scores [.., rows, tokens] over v [.., tokens, D]."""
        top = score.amax(-1, keepdim=True).clamp(min=-3e38)
        score = torch.exp(score.sub_(top))
        return top, score.sum(-1, keepdim=True), torch.matmul(score, v)

    # the prefixes, each once for all rows of its group
    tops, sums, outs = [], [], []
    for g, p in enumerate(prefix):
        ids = s["table"][first[g], :-(-p // page)].long()

        def gathered(cache):  # [hkv, p, D]
            return cache[ids].transpose(0, 1).reshape(hkv, -1, D)[:, :p].float()

        rows = x[:, first[g]:first[g + 1]].reshape(hkv, -1, D) * D ** -0.5
        a, b, o = part(torch.matmul(rows, gathered(s["k_cache"]).transpose(1, 2)), gathered(s["v_cache"]))
        n = first[g + 1] - first[g]
        tops.append(a.view(hkv, n, K, G, 1))
        sums.append(b.view(hkv, n, K, G, 1))
        outs.append(o.view(hkv, n, K, G, D))
    top, total, out = torch.cat(tops, 1), torch.cat(sums, 1), torch.cat(outs, 1)
    # what each sequence has of its own
    counts = s["cu_groups"][1:] - s["cu_groups"][:-1]
    start = torch.repeat_interleave(s["prefix"], counts, output_size=B).view(B, 1).long()
    pos = start + torch.arange(most, device=q.device).view(1, most)
    left = s["lens"].view(B, 1, 1) - (K - 1 - torch.arange(K, device=q.device)).view(1, K, 1)
    hidden = (pos.view(B, 1, most) >= left).view(1, B, K, 1, most)
    pos = pos.clamp(max=s["table"].shape[1] * page - 1)
    page_of = torch.gather(s["table"], 1, pos // page).long()

    def rest(cache):  # [hkv, B, most, D]
        return cache[page_of, :, pos % page].permute(2, 0, 1, 3).float()

    score = torch.matmul(x.reshape(hkv, B, K * G, D) * D ** -0.5, rest(s["k_cache"]).transpose(2, 3))
    score = score.view(hkv, B, K, G, most).masked_fill(hidden, float("-inf"))
    a, b, o = part(score.view(hkv, B, K * G, most), rest(s["v_cache"]))
    a, b, o = a.view(hkv, B, K, G, 1), b.view(hkv, B, K, G, 1), o.view(hkv, B, K, G, D)
    most_of = torch.maximum(a, top)
    f, h = torch.exp(top - most_of), torch.exp(a - most_of)
    total = total * f + b * h
    out = ((out * f + o * h) / total).permute(1, 2, 0, 3, 4).reshape(B, K, hq, D)
    lse = (most_of + torch.log(total)).permute(1, 2, 0, 3, 4).reshape(B, K, hq)
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].float()))
    return {"out": out.to(q.dtype), "lse": lse}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "shared":
        return _exact_shared(s)
    if case["op"] == "rope":
        return _turned(s["x"], s["w"], s["pos"], s["axis"], s["inv_freq"], case["pairs"])
    lens = s["lens"].tolist()
    B, page, T = len(lens), case["page"], s["k"].shape[0]
    cu = s["cu"].tolist() if s["cu"] is not None else [b * (T // B) for b in range(B + 1)]
    place = torch.cat([torch.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b], device="cuda") for b in range(B)])
    pos = place if s["pos"] is None else s["pos"]
    k = _turned(s["k"], s["kw"], pos, s["axis"], s["inv_freq"], case["pairs"])
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for b in range(B):
        mine = slice(cu[b], cu[b + 1])
        ids = s["table"][b].long()[place[mine] // page]
        kc[ids, :, place[mine] % page] = k[mine]
        vc[ids, :, place[mine] % page] = s["v"][mine].double()
    return {"q": _turned(s["q"], s["qw"], pos, s["axis"], s["inv_freq"], case["pairs"]), "k_cache": kc, "v_cache": vc}


def _turned(x, w, pos, axis, inv_freq, pairs):
    """The rotation as a product of complex numbers."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    half = inv_freq.numel()
    out = x.clone()
    first = slice(0, half) if pairs == "halves" else slice(0, 2 * half, 2)
    second = slice(half, 2 * half) if pairs == "halves" else slice(1, 2 * half, 2)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous())
    for j in range(half):
        p = pos if pos.dim() == 1 else pos[int(axis[j])]
        angle = p.double() * inv_freq[j].double()
        z[..., j] *= torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_shared(s):
    """Sequence by sequence over its whole table row: that a prefix is shared changes no result."""
    q = s["q"].double()
    B, K, hq, D = q.shape
    hkv, page = s["k_cache"].shape[1:3]
    G = hq // hkv
    out, lse = torch.zeros_like(q), torch.zeros((B, K, hq), dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["lens"].tolist()):
        ids = s["table"][b, :-(-n // page)].long()
        for h in range(hkv):
            heads = slice(h * G, (h + 1) * G)
            k = s["k_cache"][ids, h].reshape(-1, D)[:n].double()
            v = s["v_cache"][ids, h].reshape(-1, D)[:n].double()
            a = (q[b, :, heads].reshape(K * G, D) @ k.t() / math.sqrt(D)).view(K, G, n)
            for i in range(K - 1):
                a[i, :, n - (K - 1 - i):] = -torch.inf
            lse[b, :, heads] = torch.logsumexp(a, -1)
            out[b, :, heads] = (torch.softmax(a, -1).view(K * G, n) @ v).view(K, G, D)
    if s["gate"] is not None:
        out *= torch.sigmoid(s["gate"].double())
    return {"out": out, "lse": lse}
