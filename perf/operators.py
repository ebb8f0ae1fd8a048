"""The operators of the attention half of a decoder layer, as cases that can be timed.

moe_linear (matrix product with bias, activation and residual in its epilogue), moe_qk_norm_rope (per-head norms of
queries and keys with the rotation, keys and values into the pages of the cache) and moe_attn_forward (attention over
the paged cache: a window of 1-8 new tokens per sequence, or ragged prompt chunks, both with an optional sliding
window and sink tokens).  `run` computes them with the library's calls where `own` is true, and in elementary torch
operations in 32 bits otherwise; `exact` gives the same outputs from the definitions in 64 bits.

Sizes follow the repository's workloads (hidden 2048; windows of 1-8 tokens; prompt chunks of 1024 to 32768 tokens)
with generic head counts.
"""
import math
import random

import torch

own = False

EPS = 1e-6
THETA = 1000000.0


# ---- cases ---------------------------------------------------------------------------------------------------------
def _linear(T, K, N, bias=False, act="none", resid=False):
    return {"op": "linear", "T": T, "K": K, "N": N, "bias": bias, "act": act, "resid": resid}


def _batch(op, heads, kv_heads, dim, page, seqs, q, ctx, lens, **more):
    """`seqs` sequences of at most q new tokens behind at most ctx cached ones; `lens` seeds the ragged lengths, and 0
    gives every sequence exactly q and ctx."""
    return {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "seqs": seqs, "q": q,
            "ctx": ctx, "lens": lens, **more}


def listed():
    return [
        # the query/key/value projection of a verify window: weights streamed once, launch latency counts
        dict(_linear(3, 2048, 2560, bias=True), name="linear window t3"),
        # output projection of a prompt chunk, added to the fp32 residual
        dict(_linear(1024, 2048, 2048, resid=True), name="linear chunk t1024 resid"),
        # a dense layer with an activation, odd token and feature counts
        dict(_linear(777, 1160, 1001, bias=True, act="silu"), name="linear odd silu"),
        # the projection of the largest prompt chunk
        dict(_linear(32768, 2048, 2560, bias=True), name="linear chunk t32768"),
        # one verify window of three tokens behind a long conversation: far positions, latency counts
        dict(_batch("norm", 16, 2, 128, 64, 1, 3, 262144, 0, rot=128, gain=True), name="norm window t3"),
        # the largest prompt chunk of one sequence
        dict(_batch("norm", 16, 2, 128, 64, 1, 32768, 0, 0, rot=128, gain=True), name="norm chunk t32768"),
        # one token of one short conversation
        dict(_batch("decode", 16, 2, 128, 64, 1, 1, 500, 0, window=0, sinks=0), name="decode b1 short"),
        # verify windows of three tokens, a few long conversations, narrow heads, small pages, window and sinks
        dict(_batch("decode", 32, 4, 64, 16, 7, 3, 32768, 5, window=4096, sinks=4), name="decode b7 window sinks"),
        # a full serving batch of ragged conversations, one token each
        dict(_batch("decode", 16, 2, 128, 64, 64, 1, 16384, 3, window=0, sinks=0), name="decode b64 ragged"),
        # one prompt chunk from its first token, causal
        dict(_batch("chunk", 16, 2, 128, 64, 1, 1024, 0, 0, window=0, sinks=0), name="chunk t1024"),
        # ragged prompts behind cached prefixes, odd lengths, odd head groups, narrow heads, small pages
        dict(_batch("chunk", 12, 4, 64, 16, 6, 700, 900, 11, window=333, sinks=5), name="chunk ragged window sinks"),
        # a long prompt with the whole chunk visible
        dict(_batch("chunk", 16, 2, 128, 64, 1, 8192, 0, 0, window=0, sinks=0), name="chunk t8192"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "norm", "decode", "chunk"])
    if op == "linear":
        K = 8 * rng.randint(16, 512)
        N = _log(rng, 64, 8192)
        T = _log(rng, 1, max(2, min(32768, (1 << 37) // (K * N))))
        return _linear(T, K, N, rng.random() < 0.5, rng.choice(["none", "silu", "gelu"]), rng.random() < 0.5)
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.randint(1, 8)
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randint(1, 1 << 20)
    if op == "norm":
        seqs = _log(rng, 1, 64)
        room = max(1, (32768 * 20 * 128) // (seqs * (heads + 2 * kv_heads) * dim))
        return _batch(op, heads, kv_heads, dim, page, seqs, _log(rng, 1, min(room, 16384)), _log(rng, 1, 262144), lens,
                      rot=rng.choice([dim, dim // 2, dim // 4]), gain=rng.random() < 0.7)
    window = rng.choice([0, _log(rng, 1, 8192)])
    sinks = rng.randint(0, 8) if window else 0
    if op == "decode":
        seqs = _log(rng, 1, 128)
        room = max(2, (1 << 28) // (seqs * kv_heads * dim))
        return _batch(op, heads, kv_heads, dim, page, seqs, rng.randint(1, 8), _log(rng, 1, min(room, 131072)), lens,
                      window=window, sinks=sinks)
    seqs = rng.randint(1, 6)
    q = _log(rng, 9, 2048)
    room = max(16, (1 << 27) // (seqs * heads * q))
    return _batch(op, heads, kv_heads, dim, page, seqs, q, _log(rng, 1, min(room, 16384)), lens, window=window,
                  sinks=sinks)


def _lengths(case):
    """(new tokens, all tokens) of each sequence, from the case alone."""
    n, q, ctx = case["seqs"], case["q"], case["ctx"]
    if not case["lens"]:
        return [q] * n, [q + ctx] * n
    r = random.Random(case["lens"])
    new = [q] * n if case["op"] == "decode" else [r.randint(1, q) for _ in range(n)]
    return new, [m + r.randint(0, ctx) for m in new]


def _visible(case):
    """Over all sequences: (query, key) pairs, and keys that some query sees."""
    w, s, pairs, keys = case["window"], case["sinks"], 0, 0
    for m, n in zip(*_lengths(case)):
        first = n - m
        if w:
            pairs += sum(min(i + 1, w) + min(s, max(0, i + 1 - w)) for i in range(first, n))
            gone = max(0, first - w + 1)
            keys += n - gone + min(s, gone)
        else:
            pairs += (first + 1 + n) * m // 2
            keys += n
    return pairs, keys


def work(case):
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": 2 * T * K + 2 * N * K + (8 if case["resid"] else 2) * T * N + (4 * N if case["bias"] else 0),
                "flops": 2 * T * K * N}
    T, D, H, V = sum(_lengths(case)[0]), case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "norm":
        return {"bytes": 4 * T * (H + 2 * V) * D + (8 * D if case["gain"] else 0), "flops": 8 * T * (H + V) * D}
    pairs, keys = _visible(case)
    return {"bytes": 4 * keys * V * D + 4 * T * H * D, "flops": 4 * pairs * H * D}


# ---- inputs --------------------------------------------------------------------------------------------------------
def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale

    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        # normalised activations, weights that keep their size, the stack's residual
        return {"x": normal(T, K).bfloat16(), "w": normal(N, K, scale=K ** -0.5).bfloat16(),
                "bias": normal(N, scale=0.1) if case["bias"] else None,
                "resid": normal(T, N, scale=2.0) if case["resid"] else None}
    D, H, V, ps = case["dim"], case["heads"], case["kv_heads"], case["page"]
    new, total = _lengths(case)
    T, B = sum(new), len(new)
    pages = [-(-n // ps) for n in total]
    # the norm writes the new tokens' pages only, so that no others are kept for it
    first = [(n - m) // ps if case["op"] == "norm" else 0 for m, n in zip(new, total)]
    used = sum(p - f for p, f in zip(pages, first))
    order = torch.randperm(used + 2, generator=g, device="cuda", dtype=torch.int64)[:used].to(torch.int32)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, first[b]:pages[b]] = order[at:at + pages[b] - first[b]]
        at += pages[b] - first[b]
    s = {"kv_len": torch.tensor(total, dtype=torch.int32, device="cuda"), "table": table,
         "k": normal(used + 2, V, ps, D).bfloat16(), "v": normal(used + 2, V, ps, D).bfloat16()}
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    s["q_start"] = None if len(set(new)) == 1 else torch.tensor(starts, dtype=torch.int32, device="cuda")
    if case["op"] == "norm":
        s["qkv"] = normal(T, (H + 2 * V) * D, scale=1.3).bfloat16()
        s["gq"] = 1.0 + normal(D, scale=0.2) if case["gain"] else None
        s["gk"] = 1.0 + normal(D, scale=0.2) if case["gain"] else None
    else:  # heads differ in how sharp they are
        sharp = 0.5 + 2.0 * torch.rand((1, H, 1), generator=g, device="cuda")
        s["q"] = (normal(T, H, D) * sharp).bfloat16()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "linear":
        s["out"] = torch.empty((case["T"], case["N"]), device="cuda",
                               dtype=torch.float32 if case["resid"] else torch.bfloat16)
    else:
        rows = s["qkv" if case["op"] == "norm" else "q"].shape[0]
        s["out"] = torch.empty((rows, case["heads"], case["dim"]), device="cuda", dtype=torch.bfloat16)
    if own:
        import bit_block_quantized_moe_b200 as M

        if case["op"] == "linear":
            nbytes = M.moe_linear_workspace_bytes(case["T"], case["K"], case["N"])
        else:
            s["dims"] = M.moe_attn_dims(case["heads"], case["kv_heads"], case["dim"], case["page"])
            nbytes = M.moe_attn_workspace_bytes(s["dims"], case["seqs"], s["out"].shape[0])
            if case["op"] == "norm":
                s["rope"] = M.moe_rope_init(THETA, case["rot"])
        s["ws"] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        import bit_block_quantized_moe_b200 as M

        if case["op"] == "linear":
            M.moe_linear(s["x"], s["w"], s["out"], s["ws"], bias=s["bias"], act=case["act"], resid=s["resid"])
            return s["out"]
        if case["op"] == "norm":
            M.moe_qk_norm_rope(s["dims"], s["qkv"], s["out"], s["k"], s["v"], s["kv_len"], s["table"], s["ws"],
                               rope=s["rope"], q_start=s["q_start"], q_gain=s["gq"], k_gain=s["gk"], eps=EPS)
            return {"q": s["out"], "k": s["k"], "v": s["v"]}
        M.moe_attn_forward(s["dims"], s["q"], s["out"], s["k"], s["v"], s["kv_len"], s["table"], s["ws"],
                           q_start=s["q_start"], window=case["window"], n_sinks=case["sinks"])
        return s["out"]
    if case["op"] == "linear":
        return _plain_linear(s)
    if case["op"] == "norm":
        return _plain_norm(s)
    return _plain_attention(s)


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"]
    if s["case"]["act"] == "silu":
        z = z / (1.0 + torch.exp(-z))
    elif s["case"]["act"] == "gelu":
        z = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if s["resid"] is not None:
        return s["resid"] + z
    return z.bfloat16()


def _rows(s, T):
    """Sequence and position of each of the T new tokens."""
    t = torch.arange(T, device="cuda")
    n = s["kv_len"].long()
    if s["q_start"] is None:
        m = T // n.numel()
        b = t // m
        return b, n[b] - m + t % m
    start = s["q_start"].long()
    b = (t[:, None] >= start[None, 1:]).sum(1)
    return b, n[b] - start[b + 1] + t


def _plain_norm(s):
    case = s["case"]
    D, H, V, ps, r = case["dim"], case["heads"], case["kv_heads"], case["page"], case["rot"]
    T = s["qkv"].shape[0]
    b, pos = _rows(s, T)
    # far positions: the angle in 64 bits
    freq = THETA ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
    angle = pos.double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def norm(h, gain):
        h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
        h = h if gain is None else h * gain
        x, y, rest = h[..., :r // 2], h[..., r // 2:r], h[..., r:]
        return torch.cat([x * cos - y * sin, y * cos + x * sin, rest], -1).bfloat16()

    h = s["qkv"].view(T, H + 2 * V, D)
    page, row = s["table"][b, pos // ps].long(), pos % ps
    s["k"][page, :, row] = norm(h[:, H:H + V].float(), s["gk"])
    s["v"][page, :, row] = h[:, H + V:]
    return {"q": norm(h[:, :H].float(), s["gq"]), "k": s["k"], "v": s["v"]}


def _plain_attention(s):
    case = s["case"]
    D, H, V, w = case["dim"], case["heads"], case["kv_heads"], case["window"]
    T, B = s["q"].shape[0], s["kv_len"].numel()
    b, pos = _rows(s, T)
    m = case["q"]
    # the sequences side by side: queries [B, V, m * H / V, D], keys and values [B, V, L, D]
    at = pos - (s["kv_len"].long() - m)[b]  # every sequence's last token in the last place
    q = torch.zeros((B, m, H, D), device="cuda")
    q[b, at] = s["q"].float()
    q = q.view(B, m, V, H // V, D).transpose(1, 2).reshape(B, V, -1, D)
    table = s["table"].clamp(min=0).long()
    k = s["k"][table].transpose(1, 2).reshape(B, V, -1, D).float()
    v = s["v"][table].transpose(1, 2).reshape(B, V, -1, D).float()
    scores = (q @ k.transpose(2, 3)).view(B, V, m, H // V, -1)
    scores *= D ** -0.5
    i = (s["kv_len"].long()[:, None] - m + torch.arange(m, device="cuda"))[:, :, None]
    j = torch.arange(k.shape[2], device="cuda")
    seen = j <= i
    if w:
        seen &= (i - j < w) | (j < case["sinks"])
    scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    # a padded query sees nothing: a finite largest score keeps it from NaN
    scores -= scores.amax(-1, keepdim=True).clamp(min=-1e30)
    scores.exp_()
    total = scores.sum(-1, keepdim=True).clamp(min=1e-30)
    out = (scores.view(B, V, -1, k.shape[2]) @ v).view(B, V, m, H // V, D) / total
    return out.permute(0, 2, 1, 3, 4).reshape(B, m, H, D)[b, at].bfloat16()


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "linear":
        out = torch.einsum("tk,nk->tn", s["x"].double(), s["w"].double())
        if s["bias"] is not None:
            out += s["bias"].double()
        if case["act"] == "silu":
            out *= torch.sigmoid(out)
        elif case["act"] == "gelu":
            out *= torch.special.ndtr(out)
        return out if s["resid"] is None else out + s["resid"].double()
    new, total = _lengths(case)
    D, H, V, ps = case["dim"], case["heads"], case["kv_heads"], case["page"]
    table = s["table"].tolist()
    row = 0
    if case["op"] == "norm":
        r = case["rot"]
        h = s["qkv"].double().view(-1, H + 2 * V, D)
        size = h.pow(2).sum(-1, keepdim=True).div(D).add(EPS).rsqrt()
        unit = torch.ones(D, dtype=torch.float64, device="cuda")
        gq = unit if s["gq"] is None else s["gq"].double()
        gk = unit if s["gk"] is None else s["gk"].double()
        q, k, v = h[:, :H] * size[:, :H] * gq, h[:, H:H + V] * size[:, H:H + V] * gk, h[:, H + V:]
        place = torch.cat([torch.arange(n - m, n, device="cuda") for m, n in zip(new, total)])
        wave = torch.exp(torch.arange(r // 2, device="cuda", dtype=torch.float64) * (-2.0 / r * math.log(THETA)))
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), place.double()[:, None] * wave)
        for x in (q, k):
            z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn[:, None]
            x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
        kc, vc = s["k"].double(), s["v"].double()
        for b, (m, n) in enumerate(zip(new, total)):
            p = n - m
            while p < n:  # up to the end of the page
                e = min(n, (p // ps + 1) * ps)
                i = row + p - (n - m)
                kc[table[b][p // ps], :, p % ps:p % ps + e - p] = k[i:i + e - p].transpose(0, 1)
                vc[table[b][p // ps], :, p % ps:p % ps + e - p] = v[i:i + e - p].transpose(0, 1)
                p = e
            row += m
        return {"q": q, "k": kc, "v": vc}
    out = torch.empty((sum(new), H, D), dtype=torch.float64, device="cuda")
    for b, (m, n) in enumerate(zip(new, total)):
        pages = torch.tensor(table[b][:-(-n // ps)], device="cuda")
        k = s["k"][pages].permute(1, 0, 2, 3).reshape(V, -1, D)[:, :n].double()
        v = s["v"][pages].permute(1, 0, 2, 3).reshape(V, -1, D)[:, :n].double()
        i = torch.arange(n - m, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None, :]
        hidden = j > i
        if case["window"]:
            hidden = hidden | ((j <= i - case["window"]) & (j >= case["sinks"]))
        for h in range(H):
            a = torch.einsum("md,nd->mn", s["q"][row:row + m, h].double(), k[h * V // H]) / math.sqrt(D)
            out[row:row + m, h] = torch.softmax(a.masked_fill(hidden, -math.inf), -1) @ v[h * V // H]
        row += m
    return out
