"""Cases and plain forms of the decoding operators: rotary positions, the paged
key-value cache, attention of one new token over it, and eviction by accumulated
attention weight.

Each operator is written twice: from elementary torch operations (`own` False), and
as the calls a program makes of this package (`own` True). `exact` computes the same
outputs from the definitions in 64 bits.

Shared layout. A cache of B sequences is a pool of pages [P, Hkv, page, C] for keys
and one for values; page_table[b, n] names the page that holds slots n*page ..
n*page+page-1 of sequence b, lens[b] counts its slots in use. The accumulated weight
(fp32) and the ordinal (the token's index in its sequence) of a slot are kept in
[P, Hkv, page] pools of their own. Query head h reads KV head h // (Hq / Hkv). Pages
that hold e4m3 values stand for value * scale[kv head].
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of 16 sequences: rotate the new queries and keys
        dict(name="rope_step_16", op="rope", B=16, M=1, Hq=32, Hkv=8, C=128, axes=1, pairs=64,
             interleaved=False, inverse=False, fused_qkv=True),
        # a 32K prompt, straight from a fused projection of queries, keys and values
        dict(name="rope_prompt_32k", op="rope", B=1, M=32768, Hq=32, Hkv=8, C=128, axes=1, pairs=64,
             interleaved=False, inverse=False, fused_qkv=True),
        # a video layer: 29 frames of 64 x 64 positions, axes time / height / width
        dict(name="rope_video_118k", op="rope", B=1, M=118784, Hq=24, Hkv=24, C=128, axes=3, pairs=64,
             interleaved=True, inverse=False, fused_qkv=False),
        # the gradient of a partial rotation of short, odd-length rows
        dict(name="rope_gradient_2x1003", op="rope", B=2, M=1003, Hq=12, Hkv=4, C=64, axes=2, pairs=16,
             interleaved=False, inverse=True, fused_qkv=False),
        # the same decoding step with the keys rotated on their way into the pages
        dict(name="append_step_16", op="append", B=16, T=1, Hq=32, Hkv=8, C=128, page=16, kv="bf16",
             rope=True, past=8192),
        # a finished 32K prompt goes into an 8-bit cache
        dict(name="append_prompt_32k", op="append", B=1, T=32768, Hq=32, Hkv=8, C=128, page=64, kv="e4m3",
             rope=False, past=0),
        # the shortest answer: one sequence, a short context
        dict(name="decode_1x777", op="decode", B=1, longest=777, ragged=False, Hq=32, Hkv=8, C=128,
             page=16, kv="bf16", weights=False),
        # one long sequence
        dict(name="decode_1x128k", op="decode", B=1, longest=131072, ragged=False, Hq=32, Hkv=8, C=128,
             page=64, kv="bf16", weights=False),
        # a serving batch of mixed lengths (one of them empty), 8-bit cache
        dict(name="decode_32_ragged", op="decode", B=32, longest=16384, ragged=True, Hq=32, Hkv=8, C=128,
             page=16, kv="e4m3", weights=False),
        # long contexts that also accumulate their weights, for eviction
        dict(name="decode_weights_8x32k", op="decode", B=8, longest=32768, ragged=False, Hq=32, Hkv=8,
             C=128, page=64, kv="bf16", weights=True),
        # online eviction: each sequence a page or so over its budget
        dict(name="evict_16x4k", op="evict", B=16, longest=4224, budget=4096, recent=256, sink=4,
             Hkv=8, C=128, page=16, kv="bf16"),
        # a long prompt cut to half
        dict(name="evict_1x128k", op="evict", B=1, longest=131072, budget=65536, recent=1024, sink=4,
             Hkv=8, C=128, page=64, kv="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "evict"])
    C = rng.choice([64, 128, 128])
    Hq, Hkv = rng.choice([(32, 8), (8, 8), (12, 4), (16, 1), (24, 24), (32, 1), (40, 8), (7, 7)])
    page, kv = rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "e4m3"])
    if op == "rope":
        tokens = _log_int(rng, 1, 118784)
        B = min(tokens, _log_int(rng, 1, 64))
        return dict(op=op, B=B, M=max(1, tokens // B), Hq=Hq, Hkv=Hkv, C=C, axes=rng.choice([1, 2, 3]),
                    pairs=rng.choice([C // 2, C // 4]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.3, fused_qkv=rng.random() < 0.5)
    if op == "append":
        tokens = _log_int(rng, 1, 32768)
        B = min(tokens, _log_int(rng, 1, 32))
        return dict(op=op, B=B, T=max(1, tokens // B), Hq=Hq, Hkv=Hkv, C=C, page=page, kv=kv,
                    rope=rng.random() < 0.5, past=_log_int(rng, 1, 32768 // B))
    if op == "decode":
        B = _log_int(rng, 1, 32)
        return dict(op=op, B=B, longest=_log_int(rng, 1, min(131072, 262144 // B) * 8 // max(8, Hkv)),
                    ragged=rng.random() < 0.6, Hq=Hq, Hkv=Hkv, C=C, page=page, kv=kv,
                    weights=rng.random() < 0.4)
    B = _log_int(rng, 1, 16)
    longest = _log_int(rng, 8, 131072 // B * 8 // max(8, Hkv))
    budget = max(1, int(longest * rng.uniform(0.2, 1.1)))
    recent = int(budget * rng.uniform(0.0, 0.6))
    return dict(op=op, B=B, longest=longest, budget=budget, recent=recent, sink=min(4, budget - recent),
                Hkv=Hkv, C=C, page=page, kv=kv)


def _sections(axes, pairs):
    """Pairs of each axis, e.g. 64 over (time, height, width) -> (16, 24, 24)."""
    if axes == 1:
        return (pairs,)
    if axes == 2:
        return (pairs // 2, pairs - pairs // 2)
    t = pairs // 4
    return (t, (pairs - t) // 2, pairs - t - (pairs - t) // 2)


def _lens(case, seed):
    rng = random.Random(seed * 7919 + 17)
    B = case["B"]
    if case["op"] == "decode" and case["ragged"]:
        n = [rng.randint(1, case["longest"]) for _ in range(B)]
        n[0] = case["longest"]
        if B > 2:
            n[B // 2] = 0
        return n
    if case["op"] == "evict":
        return [case["longest"] - (rng.randint(0, case["longest"] // 64) if b else 0) for b in range(B)]
    if case["op"] == "append":      # slots before the new tokens
        return [rng.randint(0, case["past"]) if case["past"] else 0 for _ in range(B)]
    return [case["longest"]] * B


def _new_tokens(case, seed):
    """Valid new tokens of each sequence of an append (the batch is padded to T)."""
    rng = random.Random(seed * 104729 + 3)
    T = case["T"]
    return [T if b == 0 or T == 1 else rng.randint(0, T) for b in range(case["B"])]


def work(case):
    B, C, Hkv = case["B"], case["C"], case["Hkv"]
    size = 2 if case.get("kv", "bf16") == "bf16" else 1
    if case["op"] == "rope":
        elems = B * case["M"] * (case["Hq"] + Hkv) * C
        return {"bytes": elems * 4 + B * case["M"] * case["axes"] * 4, "flops": elems * 3}
    if case["op"] == "append":
        tokens = sum(_new_tokens(case, 1))
        n = tokens * Hkv * C
        q = tokens * case["Hq"] * C * 4 if case["rope"] else 0
        return {"bytes": 2 * n * (2 + size) + q + tokens * Hkv * 8, "flops": 2 * n + q}
    keys = sum(_lens(case, 1))
    if case["op"] == "decode":
        return {"bytes": keys * Hkv * (2 * C * size + (8 if case["weights"] else 0)) +
                B * case["Hq"] * (4 * C + 4), "flops": 4 * keys * case["Hq"] * C}
    kept = sum(min(n, case["budget"]) for n in _lens(case, 1))
    moved = sum(min(n, case["budget"]) * max(0, n - case["budget"]) / max(1, n) for n in _lens(case, 1))
    return {"bytes": Hkv * (8 * (keys + kept) + moved * 4 * C * size), "flops": 0}


# ----------------------------------------------------------------- inputs
def _pages_of(case, lens, gen, spare=2):
    """A table of pages in random order; entries behind a sequence's last page are -1. The
    pool has room for every sequence at its longest, and `spare` last pages that belong to none."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    width = max(1, max(need))
    most = case["past"] + case["T"] if case["op"] == "append" else case["longest"]
    pool = len(lens) * -(-most // page) + spare
    order = torch.randperm(pool - spare, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


def _kv_pools(case, pool, gen):
    shape = (pool, case["Hkv"], case["page"], case["C"])
    k = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    # a few heavy keys, as attention sinks and topics leave them
    heavy = torch.rand(shape[:3] + (1,), generator=gen, device=DEV) < 1 / 256
    k = torch.where(heavy, k * 1.5, k)
    k[-1], v[-1] = 0, 0
    if case["kv"] == "bf16":
        return k, v, None, None
    ks = torch.rand(case["Hkv"], generator=gen, device=DEV) * 0.01 + 0.015
    vs = torch.rand(case["Hkv"], generator=gen, device=DEV) * 0.01 + 0.015
    return ((k / ks[:, None, None]).clamp(-448, 448).to(E4M3),
            (v / vs[:, None, None]).clamp(-448, 448).to(E4M3), ks, vs)


def _rotary(case, axes, pairs, interleaved):
    sections = _sections(axes, pairs)
    freq = torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / n) for n in sections])
    return dict(sections=sections, inv_freq=freq.to(DEV), interleaved=interleaved,
                axis=torch.cat([torch.full((n,), a) for a, n in enumerate(sections)]).to(DEV))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, C, Hkv = case["B"], case["C"], case["Hkv"]
    s = dict(case=dict(case))

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)

    if case["op"] == "rope":
        M, Hq = case["M"], case["Hq"]
        if case["fused_qkv"]:
            qkv = randn(B, M, Hq + 2 * Hkv, C)
            s["q"], s["k"] = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        else:
            s["q"], s["k"] = randn(B, Hq, M, C), randn(B, Hkv, M, C)
        t = torch.arange(M, device=DEV, dtype=torch.int32)
        if case["axes"] == 3:           # frames of 64 x 64 positions
            p = torch.stack([t // 4096, t // 64 % 64, t % 64], -1)
        elif case["axes"] == 2:
            p = torch.stack([t // 37, t % 37], -1)
        else:
            p = t[:, None]
        first = torch.randint(0, 200000, (B, 1, 1), generator=gen, device=DEV, dtype=torch.int32)
        s["pos"] = (p[None] + first).contiguous()
        s["rot"] = _rotary(case, case["axes"], case["pairs"], case["interleaved"])
        s["qo"] = torch.empty((B, Hq, M, C), dtype=torch.bfloat16, device=DEV)
        s["ko"] = torch.empty((B, Hkv, M, C), dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "append":
        T, Hq = case["T"], case["Hq"]
        past, new = _lens(case, seed), _new_tokens(case, seed)
        lens = [a + n for a, n in zip(past, new)]
        s["table"], pool = _pages_of(case, lens, gen)
        s["kp"], s["vp"], s["ks"], s["vs"] = _kv_pools(case, pool, gen)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["new"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        s["seen"] = s["lens"] + torch.randint(0, 1000, (B,), generator=gen, device=DEV, dtype=torch.int32)
        s["acc"] = torch.rand((pool, Hkv, case["page"]), generator=gen, device=DEV)
        s["ord"] = torch.zeros((pool, Hkv, case["page"]), dtype=torch.int32, device=DEV)
        s["acc"][-1] = 0
        qkv = randn(B, T, Hq + 2 * Hkv, C)
        s["q"] = qkv[:, :, :Hq].transpose(1, 2)
        s["k"] = qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        s["v"] = qkv[:, :, Hq + Hkv:].transpose(1, 2)
        t = torch.arange(T, device=DEV, dtype=torch.int32)
        s["pos"] = (s["seen"] - s["new"])[:, None, None] + t[None, :, None]
        s["rot"] = _rotary(case, 1, C // 2, False)
        s["qo"] = torch.zeros((B, Hq, T, C), dtype=torch.bfloat16, device=DEV)
    else:
        lens = _lens(case, seed)
        s["table"], pool = _pages_of(case, lens, gen)
        s["width"] = s["table"].shape[1] * case["page"]
        s["kp"], s["vp"], s["ks"], s["vs"] = _kv_pools(case, pool, gen)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        slots = (pool, Hkv, case["page"])
        s["acc"] = torch.exp(2 * torch.randn(slots, generator=gen, device=DEV))
        s["acc"][torch.rand(slots, generator=gen, device=DEV) < 0.125] = 0   # tokens nobody looked at
        s["acc"][-1] = 0
        s["acc_out"] = s["acc"].clone()
        if case["op"] == "decode":
            for x in (s["acc"], s["acc_out"]):      # what a few earlier steps left
                x *= case["Hq"] / Hkv / case["longest"]
            s["q"] = 2 * randn(B, case["Hq"], C)
            s["o"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((B, case["Hq"]), device=DEV)
        else:
            # ordinals rise with the slot but for tokens that earlier evictions moved
            j = torch.arange(s["width"], device=DEV)
            key = j + torch.rand((B, Hkv, s["width"]), generator=gen, device=DEV) * (s["width"] / 8)
            key = torch.where(j < s["lens"][:, None, None], key, math.inf)
            rank = (2 * key.argsort(-1).argsort(-1)).to(torch.int32)
            s["ord"] = torch.zeros(slots, dtype=torch.int32, device=DEV)
            at = _slot_index(s, s["width"])
            s["ord"].view(-1)[at.reshape(-1)] = rank.reshape(-1)
            s["ord"][-1] = 0
            s["ord_out"] = s["ord"].clone()
            s["seen"] = 2 * s["lens"]       # every second token was evicted before
    if own:     # what a program makes once and keeps: the plan, the cache's handle, the workspace
        import block_sparse_long_04_b200 as xa
        s["xa"] = xa
        if "rot" in s:
            s["rotary"] = xa.Rotary(s["rot"]["inv_freq"], s["rot"]["sections"], s["rot"]["interleaved"])
        if "kp" in s:
            s["cache"] = xa.PagedCache(s["kp"], s["vp"], s["table"], s["lens"], k_scale=s["ks"],
                                       v_scale=s["vs"], acc=s["acc"], ordinal=s.get("ord"))
        if case["op"] == "decode":
            n = xa.xattn_decode_workspace_size(s["cache"], case["Hq"], case["weights"])
        elif case["op"] == "evict":
            n = xa.xattn_cache_evict_workspace_size(s["cache"], case["budget"])
        else:
            n = 0
        s["ws"] = torch.empty(max(1, n), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------ plain forms
def _slot_index(s, width):
    """[B, Hkv, width] index of each slot in a flat [P * Hkv * page] pool; slots behind a
    sequence's end go to the pool's last slot, which belongs to no sequence."""
    pool, Hkv, page = s["acc"].shape
    j = torch.arange(width, device=DEV)
    row = s["table"].long().clamp(min=0)[:, j // page]                         # [B, width]
    at = (row[:, None] * Hkv + torch.arange(Hkv, device=DEV)[:, None]) * page + j % page
    return torch.where(j < s["lens"][:, None, None], at, pool * Hkv * page - 1)



def _rows(pages, scale, at):
    """fp32 rows [B, Hkv, width, C] of a pool at flat slot indices."""
    C, Hkv = pages.shape[-1], pages.shape[1]
    x = pages.view(torch.uint8 if pages.dtype == E4M3 else pages.dtype).view(-1, C)[at]
    x = (x.view(E4M3) if pages.dtype == E4M3 else x).float()
    return x if scale is None else x * scale.view(1, Hkv, 1, 1)


def _rotate(x, pos, rot, inverse, f=torch.float32):
    """x [B, H, M, C] rotated by its positions; angles in 64 bits, the product in `f`."""
    ang = pos.double()[..., rot["axis"]] * rot["inv_freq"]
    cos, sin = ang.cos().to(f)[:, None], ang.sin().to(f)[:, None]
    if inverse:
        sin = -sin
    x, P = x.to(f), rot["inv_freq"].numel()
    if rot["interleaved"]:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :P], x[..., P:2 * P]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * P:]], -1)


def _plain_rope(s):
    inv = s["case"]["inverse"]
    return {"q": _rotate(s["q"], s["pos"], s["rot"], inv).bfloat16(),
            "k": _rotate(s["k"], s["pos"], s["rot"], inv).bfloat16()}


def _plain_append(s):
    case, C = s["case"], s["case"]["C"]
    pool, Hkv, page = s["acc"].shape
    T = case["T"]
    q, k, v = s["q"], s["k"], s["v"].float()
    k = _rotate(k, s["pos"], s["rot"], False) if case["rope"] else k.float()
    t = torch.arange(T, device=DEV)
    valid = t < s["new"][:, None]                                              # [B, T]
    slot = torch.where(valid, s["lens"][:, None] - s["new"][:, None] + t, 0).long()
    row = s["table"].long().clamp(min=0).gather(1, slot // page)
    at = (row[:, None] * Hkv + torch.arange(Hkv, device=DEV)[:, None]) * page + (slot % page)[:, None]
    at = torch.where(valid[:, None], at, pool * Hkv * page - 1)                # [B, Hkv, T]
    for pages, x, scale in ((s["kp"], k, s["ks"]), (s["vp"], v, s["vs"])):
        x = torch.where(valid[:, None, :, None], x, 0.0)
        if scale is not None:
            x = (x / scale.view(1, Hkv, 1, 1)).clamp(-448, 448).to(E4M3).view(torch.uint8)
            pages.view(torch.uint8).view(-1, C)[at.reshape(-1)] = x.reshape(-1, C)
        else:
            pages.view(-1, C)[at.reshape(-1)] = x.bfloat16().reshape(-1, C)
    age = torch.where(valid, (s["seen"] - s["new"])[:, None] + t.int(), 0)
    s["acc"].view(-1)[at.reshape(-1)] = 0.0
    s["ord"].view(-1)[at.reshape(-1)] = age[:, None].expand(-1, Hkv, -1).reshape(-1)
    out = {"k_pages": s["kp"], "v_pages": s["vp"], "acc": s["acc"], "ordinal": s["ord"]}
    if case["rope"]:
        out["q"] = torch.where(valid[:, None, :, None], _rotate(q, s["pos"], s["rot"], False).bfloat16(), s["qo"])
    return out


def _plain_decode(s):
    case = s["case"]
    B, Hq, Hkv, C = case["B"], case["Hq"], case["Hkv"], case["C"]
    at = _slot_index(s, s["width"])
    seen = torch.arange(s["width"], device=DEV) < s["lens"][:, None, None, None]   # [B, 1, 1, W]
    x = torch.matmul(s["q"].float().view(B, Hkv, Hq // Hkv, C), _rows(s["kp"], s["ks"], at).transpose(-1, -2))
    x = torch.where(seen, x / math.sqrt(C), -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(x - torch.where(top.isinf(), 0.0, top)), 0.0)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p, _rows(s["vp"], s["vs"], at)).view(B, Hq, C)
    lse = (top + torch.log(total)).view(B, Hq)
    out = {"o": o.bfloat16(), "lse": lse}
    if case["weights"]:
        w = torch.where(seen[:, 0], s["acc"].view(-1)[at] + p.sum(2), 0.0)
        s["acc_out"].view(-1)[at.reshape(-1)] = w.reshape(-1)
        out["acc"] = s["acc_out"]
    return out


def _plain_evict(s):
    case, C, W = s["case"], s["case"]["C"], s["width"]
    at = _slot_index(s, W)
    j = torch.arange(W, device=DEV)
    lens = s["lens"][:, None, None].long()
    n = lens.clamp(max=case["budget"])
    valid = j < lens
    acc, age = s["acc"].view(-1)[at], s["ord"].view(-1)[at]
    safe = (age >= s["seen"][:, None, None] - case["recent"]) | (age < case["sink"])
    score = torch.where(valid, torch.where(safe, math.inf, acc), -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(score, dtype=torch.bool).scatter_(-1, order, (j < n).expand_as(order))
    before = kept.long().cumsum(-1) - kept.long()
    # the i-th evicted slot below n takes the i-th kept slot from the end
    moves = kept & (j >= n)
    source = torch.zeros((*kept.shape[:2], W + 1), dtype=torch.long, device=DEV)
    source.scatter_(-1, torch.where(moves, n - 1 - before, W), j.expand_as(before))
    hole = (j < n) & ~kept
    src = torch.where(hole, source.gather(-1, torch.where(hole, j - before, 0)), j)
    flat = at.gather(-1, src)
    to = torch.where(j < n, at, at.new_full((), s["acc"].numel() - 1)).reshape(-1)
    frm = torch.where(j < n, flat, s["acc"].numel() - 1).reshape(-1)
    for pages in (s["kp"], s["vp"]):
        rows = pages.view(torch.uint8 if pages.dtype == E4M3 else pages.dtype).view(-1, C)
        rows[to] = rows[frm]
    s["acc_out"].view(-1)[to] = s["acc"].view(-1)[frm]
    s["ord_out"].view(-1)[to] = s["ord"].view(-1)[frm]
    return {"k_pages": s["kp"], "v_pages": s["vp"], "acc": s["acc_out"], "ordinal": s["ord_out"]}


def _own(s):
    xa, case = s["xa"], s["case"]
    if case["op"] == "rope":
        xa.xattn_rope(s["q"], s["k"], s["pos"], s["rotary"], s["qo"], s["ko"], inverse=case["inverse"])
        return {"q": s["qo"], "k": s["ko"]}
    if case["op"] == "append":
        out = {"k_pages": s["kp"], "v_pages": s["vp"], "acc": s["acc"], "ordinal": s["ord"]}
        if case["rope"]:
            xa.xattn_rope_append(s["q"], s["k"], s["v"], s["pos"], s["rotary"], s["cache"], s["qo"],
                                 n_new=s["new"], seen=s["seen"])
            out["q"] = s["qo"]
        else:
            xa.xattn_cache_append(s["k"], s["v"], s["cache"], n_new=s["new"], seen=s["seen"])
        return out
    if case["op"] == "decode":
        scale = 1.0 / math.sqrt(case["C"])
        if case["weights"]:
            xa.xattn_decode_attn(s["q"], s["cache"], scale, s["o"], s["ws"], lse=s["lse"], weights=True,
                                 acc_out=s["acc_out"])
            return {"o": s["o"], "lse": s["lse"], "acc": s["acc_out"]}
        xa.xattn_decode_attn(s["q"], s["cache"], scale, s["o"], s["ws"], lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    xa.xattn_cache_evict(s["cache"], case["budget"], s["ws"], recent=case["recent"], sink=case["sink"],
                         seen=s["seen"], acc_out=s["acc_out"], ord_out=s["ord_out"])
    return {"k_pages": s["kp"], "v_pages": s["vp"], "acc": s["acc_out"], "ordinal": s["ord_out"]}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode,
            "evict": _plain_evict}[state["case"]["op"]](state)


# --------------------------------------------------- definitions in 64 bits
def _exact_rotation(x, pos, rot, inverse):
    """Each pair as a complex number times exp(i * angle)."""
    y = x.double().clone()
    P = rot["inv_freq"].numel()
    i = torch.arange(P, device=DEV)
    a, b = (2 * i, 2 * i + 1) if rot["interleaved"] else (i, i + P)
    for h in range(x.shape[1]):
        angle = pos[..., rot["axis"]].double() * rot["inv_freq"] * (-1.0 if inverse else 1.0)
        z = torch.complex(y[:, h][..., a], y[:, h][..., b]) * torch.polar(torch.ones_like(angle), angle)
        y[:, h][..., a] = z.real
        y[:, h][..., b] = z.imag
    return y


def exact(case, seed):
    if case["op"] == "evict":           # moves values, computes none
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"q": _exact_rotation(s["q"], s["pos"], s["rot"], case["inverse"]),
                "k": _exact_rotation(s["k"], s["pos"], s["rot"], case["inverse"])}
    page, Hkv = case["page"], case["Hkv"]
    table, lens = s["table"].tolist(), s["lens"].tolist()
    if case["op"] == "append":
        new = s["new"].tolist()
        kp, vp, acc = s["kp"].double(), s["vp"].double(), s["acc"].double()
        k = _exact_rotation(s["k"], s["pos"], s["rot"], False) if case["rope"] else s["k"].double()
        qo = s["qo"].double()
        for b in range(case["B"]):
            for first in range(lens[b] - new[b], lens[b]):
                if first != lens[b] - new[b] and first % page:
                    continue
                n = min(page - first % page, lens[b] - first)
                t = first - (lens[b] - new[b])
                pg, off = table[b][first // page], first % page
                for pool, x, sc in ((kp, k, s["ks"]), (vp, s["v"].double(), s["vs"])):
                    y = x[b, :, t:t + n]
                    pool[pg, :, off:off + n] = y if sc is None else (y / sc.double()[:, None, None]).clamp(-448, 448)
                acc[pg, :, off:off + n] = 0
        out = {"k_pages": kp, "v_pages": vp, "acc": acc, "ordinal": None}
        if case["rope"]:
            q = _exact_rotation(s["q"], s["pos"], s["rot"], False)
            for b in range(case["B"]):
                qo[b, :, :new[b]] = q[b, :, :new[b]]
            out["q"] = qo
        return out
    G = case["Hq"] // Hkv
    o = torch.zeros((case["B"], case["Hq"], case["C"]), dtype=torch.float64, device=DEV)
    lse = torch.full((case["B"], case["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    acc = s["acc_out"].double()
    for b in range(case["B"]):
        n = lens[b]
        if n == 0:
            continue
        pages = torch.tensor(table[b][:-(-n // page)], device=DEV)
        for h in range(Hkv):
            k = s["kp"].view(torch.uint8).view(*s["kp"].shape[:3], -1)[pages, h].view(s["kp"].dtype)
            v = s["vp"].view(torch.uint8).view(*s["vp"].shape[:3], -1)[pages, h].view(s["vp"].dtype)
            k, v = k.double().reshape(-1, case["C"])[:n], v.double().reshape(-1, case["C"])[:n]
            if s["ks"] is not None:
                k, v = k * s["ks"][h].double(), v * s["vs"][h].double()
            logits = s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(case["C"])
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(logits, -1)
            p = torch.softmax(logits, -1)
            o[b, h * G:(h + 1) * G] = p @ v
            if case["weights"]:
                w = torch.zeros(pages.numel() * page, dtype=torch.float64, device=DEV)
                w[:n] = p.sum(0)
                old = s["acc"][pages, h].double()
                live = (torch.arange(w.numel(), device=DEV) < n).view(-1, page)
                acc[pages, h] = torch.where(live, old + w.view(-1, page), acc[pages, h])
    return {"o": o, "lse": lse, "acc": acc} if case["weights"] else {"o": o, "lse": lse}
