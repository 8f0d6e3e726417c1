"""Measured operators of the streaming trunk: frames and tokens that arrive while a scene's earlier keys and
values stay in a paged cache.

  plan    block table, slot map and row offsets of a step, from the sequences' lengths
  append  the step's new K and V rows scattered into their pages
  attn    attention of the new rows (a single token, a frame, a ragged chunk) over the paged cache
  norm    a block's output added to the residual stream (post norm, layer scale, gate) and the next block's norm

With ``own`` false every operator runs in its plain form (elementary torch operations in 32 bits); with ``own`` true
through ``feed_forward_view_vggt_b200.attn``.
"""
import math
import random

import torch

own = False

D = 64  # head dimension of the framework


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Four scenes that each receive one new frame (5 + 37 x 37 tokens): the plan of a small streaming step.
        {"name": "plan_scenes", "op": "plan", "seqs": 4, "new": 1374, "new_min": 1374, "ctx_min": 1374, "ctx": 43968,
         "page": 128, "pad": 0, "lens": 1},
        # A full batch: 512 requests of very different lengths, small pages, rows padded behind the last request.
        {"name": "plan_batch", "op": "plan", "seqs": 512, "new": 1374, "new_min": 1, "ctx_min": 0, "ctx": 16000,
         "page": 16, "pad": 777, "lens": 2},
        # One new token for each of 64 sequences: the smallest append, all latency.
        {"name": "append_tokens", "op": "append", "seqs": 64, "new": 1, "new_min": 1, "ctx_min": 3, "ctx": 4000,
         "page": 16, "kv_heads": 16, "lens": 3},
        # One new frame for each of 16 scenes.
        {"name": "append_frames", "op": "append", "seqs": 16, "new": 1374, "new_min": 1374, "ctx_min": 1374,
         "ctx": 5496, "page": 128, "kv_heads": 16, "lens": 4},
        # A single token over the four-frame worked example: the smallest attention call.
        {"name": "attn_token", "op": "attn", "seqs": 1, "new": 1, "new_min": 1, "ctx_min": 5495, "ctx": 5495,
         "page": 64, "heads": 16, "kv_heads": 16, "unit": 1, "lens": 5},
        # Single tokens of 48 sequences of odd lengths, grouped heads, small pages: bound by the cache's bytes.
        {"name": "attn_tokens", "op": "attn", "seqs": 48, "new": 1, "new_min": 1, "ctx_min": 700, "ctx": 32000,
         "page": 16, "heads": 32, "kv_heads": 8, "unit": 1, "lens": 6},
        # Ragged chunks, causal by token, the first of a sequence among them.
        {"name": "attn_chunks", "op": "attn", "seqs": 7, "new": 613, "new_min": 1, "ctx_min": 0, "ctx": 9000,
         "page": 48, "heads": 12, "kv_heads": 4, "unit": 1, "lens": 11},
        # One new frame over 32 cached ones, causal by frame.
        {"name": "attn_frame_n32", "op": "attn", "seqs": 1, "new": 1374, "new_min": 1374, "ctx_min": 43968,
         "ctx": 43968, "page": 128, "heads": 16, "kv_heads": 16, "unit": 1374, "lens": 8},
        # One new frame over 100 cached ones: the headline scene, streamed.
        {"name": "attn_frame_n100", "op": "attn", "seqs": 1, "new": 1374, "new_min": 1374, "ctx_min": 137400,
         "ctx": 137400, "page": 128, "heads": 16, "kv_heads": 16, "unit": 1374, "lens": 9},
        # The special tokens of one frame: the smallest norm call.
        {"name": "norm_special", "op": "norm", "rows": 17, "cols": 1024, "res": "float32", "kind": "layer",
         "post": False, "gate_rows": 0, "scale": True},
        # An odd number of rows, grouped gates and a norm after the block as well, bf16 residual stream.
        {"name": "norm_gated", "op": "norm", "rows": 5497, "cols": 768, "res": "bfloat16", "kind": "rms",
         "post": True, "gate_rows": 1374, "scale": True},
        # A whole layer of the headline scene, fp32 residual stream with layer scale.
        {"name": "norm_n100", "op": "norm", "rows": 137400, "cols": 1024, "res": "float32", "kind": "layer",
         "post": False, "gate_rows": 0, "scale": True},
    ]


def log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "norm"])
    case = {"op": op, "lens": rng.randrange(1 << 30)}
    page = 8 * log_int(rng, 1, 32)
    if op == "plan":
        new = log_int(rng, 1, 1374)
        case |= {"seqs": log_int(rng, 1, 512), "new": new, "new_min": rng.choice([0, 1, new]), "ctx_min": 0,
                 "ctx": log_int(rng, 1, 16000), "page": page, "pad": rng.choice([0, log_int(rng, 1, 777)])}
    elif op == "append":
        seqs = log_int(rng, 1, 64)
        new = log_int(rng, 1, 20000 // seqs)
        case |= {"seqs": seqs, "new": new, "new_min": rng.choice([0, 1, new]), "ctx_min": 0,
                 "ctx": log_int(rng, 1, 4000), "page": page, "kv_heads": rng.randint(1, 16)}
    elif op == "attn":
        kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
        heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 8, 16) if kv_heads * g <= 32])
        if rng.random() < 0.5:  # single tokens
            seqs, new = log_int(rng, 1, 48), 1
            ctx = log_int(rng, 16, 32000)
        else:
            seqs = log_int(rng, 1, 6)
            new = log_int(rng, 2, 1400)
            ctx = log_int(rng, 16, min(60000, max(16, 1_500_000_000 // (seqs * new * heads))))
        case |= {"seqs": seqs, "new": new, "new_min": rng.choice([0, 1, new]), "ctx_min": rng.choice([0, ctx // 2, ctx]),
                 "ctx": ctx, "page": page, "heads": heads, "kv_heads": kv_heads,
                 "unit": rng.choice([0, 1, 1, log_int(rng, 2, 1400)])}
    else:
        cols = 64 * rng.randint(1, 32)
        case |= {"rows": log_int(rng, 1, 120_000_000 // cols if cols > 1000 else 120_000), "cols": cols,
                 "res": rng.choice(["float32", "bfloat16"]), "kind": rng.choice(["layer", "rms"]),
                 "post": rng.random() < 0.5, "gate_rows": rng.choice([0, 1, log_int(rng, 2, 1400)]),
                 "scale": rng.random() < 0.7}
    return case


def lengths(case):
    """(cached, new) tokens of every sequence; the case's own numbers give them."""
    rng = random.Random(case["lens"])
    spread = lambda lo, hi: lo if lo >= hi else log_int(rng, lo + 1, hi + 1) - 1  # noqa: E731
    cached = [spread(case["ctx_min"], case["ctx"]) for _ in range(case["seqs"])]
    new = [spread(case["new_min"], case["new"]) for _ in range(case["seqs"])]
    new[0] = max(new[0], 1)
    return cached, new


def pages_of(tokens, page):
    return -(-tokens // page)


def work(case):
    if case["op"] == "norm":
        n, width = case["rows"] * case["cols"], 4 if case["res"] == "float32" else 2
        gates = -(-case["rows"] // case["gate_rows"]) * case["cols"] * 2 if case["gate_rows"] else 0
        params = 4 * case["cols"] * (2 + bool(case["scale"]) + 2 * bool(case["post"]))
        return {"bytes": n * (2 * width + 4) + gates + params, "flops": n * (10 + 8 * bool(case["post"]))}
    cached, new = lengths(case)
    rows, page = sum(new), case["page"]
    if case["op"] == "plan":
        taken = sum(pages_of(c + n, page) - pages_of(c, page) for c, n in zip(cached, new))
        tails = sum(1 for c, n in zip(cached, new) if n and c % page)
        return {"bytes": 4 * (rows + case["pad"] + 2 * taken + tails + 4 * len(new)), "flops": 0}
    if case["op"] == "append":
        return {"bytes": rows * (4 * 2 * D * case["kv_heads"] + 4), "flops": 0}
    pairs = 0
    for c, n in zip(cached, new):
        kv, u = c + n, case["unit"]
        pairs += n * kv if u == 0 else sum(min(kv, ((c + i) // u + 1) * u) for i in range(n))
    keys = sum(c + n for c, n in zip(cached, new) if n)
    return {"bytes": 2 * rows * case["heads"] * D * 2 + 2 * keys * case["kv_heads"] * D * 2,
            "flops": 4 * D * case["heads"] * pairs}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        res = torch.float32 if case["res"] == "float32" else torch.bfloat16
        s = {"op": "norm", "kind": case["kind"], "gate_rows": case["gate_rows"], "post": case["post"], "eps": 1e-6,
             "x": (2.0 * normal(rows, cols) + 0.3).to(res), "y": normal(rows, cols).to(torch.bfloat16),
             "scale": 0.3 * normal(cols) if case["scale"] else None,
             "gate": normal(-(-rows // case["gate_rows"]), cols).to(torch.bfloat16) if case["gate_rows"] else None,
             "post_w": 1 + 0.2 * normal(cols) if case["post"] else None,
             "post_b": 0.1 * normal(cols) if case["post"] and case["kind"] == "layer" else None,
             "pre_w": 1 + 0.2 * normal(cols), "pre_b": 0.1 * normal(cols) if case["kind"] == "layer" else None}
        return s
    cached, new = lengths(case)
    page, seqs = case["page"], case["seqs"]
    width = max(pages_of(c + n, page) for c, n in zip(cached, new)) + 1
    have = torch.tensor([pages_of(c, page) for c in cached], device="cuda")
    need = torch.tensor([pages_of(c + n, page) for c, n in zip(cached, new)], device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    held = have if case["op"] == "plan" else need
    # the cache's pages in no order: those that the sequences hold, then the free ones
    n_pages = int(need.sum()) + 5
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    first = torch.cumsum(held, 0) - held
    table = torch.where(col < held[:, None], order[(first[:, None] + col).clamp(max=n_pages - 1)], -1).contiguous()
    s = {"op": case["op"], "page": page, "rows": sum(new) + case.get("pad", 0), "table": table}
    if case["op"] == "plan":
        free = order[int(held.sum()):].contiguous()
        return s | {"cached": i32(cached), "new": i32(new), "free": free, "n_free": i32([free.numel()])}
    starts = [sum(new[:b]) for b in range(seqs + 1)]
    kv = case["kv_heads"]
    pool = lambda: normal(n_pages, kv, page, D).to(torch.bfloat16)  # noqa: E731
    s |= {"k_pages": pool(), "v_pages": pool()}
    if case["op"] == "append":
        seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), torch.tensor(new, device="cuda"))
        pos = torch.arange(sum(new), device="cuda") - i32(starts)[seq] + i32(cached)[seq]
        s["slots"] = (table[seq, pos // page] * page + pos % page).to(torch.int32)
        # K and V as slices of one projection's rows
        both = normal(sum(new), 2, kv, D).to(torch.bfloat16)
        return s | {"k": both[:, 0], "v": both[:, 1]}
    return s | {"q": normal(sum(new), case["heads"], D).to(torch.bfloat16), "unit": case["unit"],
                "starts": i32(starts), "lens": i32([c + n for c, n in zip(cached, new)]),
                "longest": (max(new), max(c + n for c, n in zip(cached, new)))}


# -------------------------------------------------------------- the passes

def run(s):
    if own:
        return OWN[s["op"]](s)
    return PLAIN[s["op"]](s)


def own_plan(s):
    from feed_forward_view_vggt_b200 import attn
    cu_rows, kv_lens, slots, counts = attn.cache_plan(s["cached"], s["new"], s["free"], s["n_free"], s["table"],
                                                      page_size=s["page"], n_rows=s["rows"])
    return {"table": s["table"], "cu_rows": cu_rows, "kv_lens": kv_lens, "slots": slots, "counts": counts}


def own_append(s):
    from feed_forward_view_vggt_b200 import attn
    attn.cache_append(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def own_attn(s):
    from feed_forward_view_vggt_b200 import attn
    return attn.cached(s["q"], s["k_pages"], s["v_pages"], s["table"], s["starts"], s["lens"], causal_unit=s["unit"])


def own_norm(s):
    from feed_forward_view_vggt_b200 import attn
    x, h = attn.norm_residual(s["x"], s["y"], kind=s["kind"], eps=s["eps"], scale=s["scale"], gate=s["gate"],
                              rows_per_gate=s["gate_rows"], post_norm=s["post"], post_weight=s["post_w"],
                              post_bias=s["post_b"], weight=s["pre_w"], bias=s["pre_b"])
    return {"x": x, "h": h}


def plain_plan(s):
    page, rows, table = s["page"], s["rows"], s["table"]
    seqs, width = table.shape
    cached, new = s["cached"].long().clamp(min=0), s["new"].long().clamp(min=0)
    ends = torch.cumsum(new, 0)
    have = torch.div(cached + page - 1, page, rounding_mode="floor")
    want = torch.div(cached + new + page - 1, page, rounding_mode="floor")
    fits = (ends <= rows) & (want <= width)
    need = torch.where(fits, want - have, 0)
    upto = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (upto <= s["n_free"]))
    need = torch.where(granted, need, 0)
    before = upto - need
    col = torch.arange(width, device=table.device)
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    taken = (s["n_free"].long() - 1 - (before[:, None] + col - have[:, None])).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][taken], table)
    cu = torch.cat([ends.new_zeros(1), ends]).clamp(max=rows)
    kv = torch.where(granted, cached + new, cached)
    row = torch.arange(rows, device=table.device)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    of = seq.clamp(max=seqs - 1)
    pos = cached[of] + row - cu[of]
    at = table[of, torch.div(pos, page, rounding_mode="floor").clamp(max=width - 1)].long() * page + pos % page
    slots = torch.where((seq < seqs) & granted[of], at, -1)
    counts = torch.stack([s["n_free"][0].long() - need.sum(), (~granted).sum()])
    return {"table": table, "cu_rows": cu.int(), "kv_lens": kv.int(), "slots": slots.int(), "counts": counts.int()}


def plain_append(s):
    page = s["page"]
    at, off = s["slots"] // page, s["slots"] % page
    s["k_pages"][at, :, off] = s["k"]
    s["v_pages"][at, :, off] = s["v"]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def plain_attn(s):
    rows, heads, _ = s["q"].shape
    kv_heads, page, starts, lens = s["k_pages"].shape[1], s["page"], s["starts"].long(), s["lens"].long()
    group, seqs = heads // kv_heads, lens.numel()
    most_q, most_k = s["longest"]
    key = torch.arange(most_k, device="cuda")
    at = s["table"][:, key // page].long().clamp(min=0)
    k = s["k_pages"][at, :, key % page].float().permute(0, 2, 3, 1)  # [seqs, kv heads, d, keys]
    v = s["v_pages"][at, :, key % page].float().permute(0, 2, 1, 3)
    i = torch.arange(most_q, device="cuda")
    q = s["q"][(starts[:-1, None] + i).clamp(max=rows - 1)].float()  # [seqs, rows, heads, d]
    q = q.view(seqs, most_q, kv_heads, group, D).permute(0, 2, 1, 3, 4).reshape(seqs, kv_heads, most_q * group, D)
    n_new = starts[1:] - starts[:-1]
    pos = (lens - n_new)[:, None] + i
    unit = s["unit"]
    last = (torch.div(pos, unit, rounding_mode="floor") + 1) * unit if unit else torch.full_like(pos, most_k)
    seen = key < torch.minimum(last, lens[:, None])[:, :, None]  # [seqs, rows, keys]
    seen = seen.repeat_interleave(group, 1)[:, None]
    a = torch.matmul(q, k).mul_(D ** -0.5)
    a.masked_fill_(~seen, -math.inf)
    top = a.amax(-1, keepdim=True)
    a.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    o = torch.matmul(a, v) / a.sum(-1, keepdim=True).clamp(min=1e-37)
    o = o.view(seqs, kv_heads, most_q, group, D).permute(0, 2, 1, 3, 4).reshape(seqs, most_q, heads, D)
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    return o[seq, row - starts[seq]].to(s["q"].dtype)


def plain_norm_of(t, kind, eps, w, b):
    if kind == "layer":
        t = t - t.mean(-1, keepdim=True)
    t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + eps)
    t = t if w is None else t * w
    return t if b is None else t + b


def plain_norm(s):
    y = s["y"].float()
    if s["post"]:
        y = plain_norm_of(y, s["kind"], s["eps"], s["post_w"], s["post_b"])
    if s["scale"] is not None:
        y = y * s["scale"]
    if s["gate"] is not None:
        y = y * s["gate"].float()[torch.arange(y.shape[0], device="cuda") // s["gate_rows"]]
    x = s["x"].float() + y
    h = plain_norm_of(x, s["kind"], s["eps"], s["pre_w"], s["pre_b"])
    return {"x": x.to(s["x"].dtype), "h": h.to(torch.bfloat16)}


OWN = {"plan": own_plan, "append": own_append, "attn": own_attn, "norm": own_norm}
PLAIN = {"plan": plain_plan, "append": plain_append, "attn": plain_attn, "norm": plain_norm}


# ---------------------------------------------------------- 64-bit results

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits: one sequence and head, or one block of rows, at a time."""
    if case["op"] == "plan":  # whole numbers
        return None
    s = prepare(case, seed)
    if case["op"] == "append":  # the pools with every new row moved to its place, one sequence's page at a time
        pools = {"k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double()}
        cached, new = lengths(case)
        row, table = 0, s["table"].tolist()
        for b, (c, n) in enumerate(zip(cached, new)):
            while n:
                page, off = table[b][c // case["page"]], c % case["page"]
                step = min(n, case["page"] - off)
                for name in pools:
                    pools[name][page, :, off:off + step] = s[name[0]][row:row + step].double().transpose(0, 1)
                row, c, n = row + step, c + step, n - step
        return pools
    if case["op"] == "norm":
        x_out, h = torch.empty_like(s["x"], dtype=torch.float64), torch.empty_like(s["x"], dtype=torch.float64)

        def normed(t, w, b):
            centre = t.mean(1, keepdim=True) if s["kind"] == "layer" else 0.0
            z = (t - centre) / ((t - centre).pow(2).mean(1, keepdim=True) + s["eps"]).sqrt()
            z = z * w.double()
            return z + b.double() if b is not None else z

        for r in range(0, x_out.shape[0], 16384):
            rows = slice(r, min(r + 16384, x_out.shape[0]))
            add = s["y"][rows].double()
            if s["post"]:
                add = normed(add, s["post_w"], s["post_b"])
            if s["scale"] is not None:
                add = add * s["scale"].double()
            if s["gate"] is not None:
                add = add * s["gate"].double().repeat_interleave(s["gate_rows"], 0)[rows]
            x_out[rows] = s["x"][rows].double() + add
            h[rows] = normed(x_out[rows], s["pre_w"], s["pre_b"])
        return {"x": x_out, "h": h}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, lens, page = s["starts"].tolist(), s["lens"].tolist(), s["page"]
    group = case["heads"] // case["kv_heads"]
    for b, n_keys in enumerate(lens):
        rows = slice(starts[b], starts[b + 1])
        n = rows.stop - rows.start
        if not n:
            continue
        ids = s["table"][b, :pages_of(n_keys, page)].long()
        place = torch.arange(n_keys - n, n_keys, device="cuda")
        hidden = None
        if case["unit"]:
            hidden = (place // case["unit"])[:, None] < (torch.arange(n_keys, device="cuda") // case["unit"])[None]
        for h in range(case["kv_heads"]):
            k = s["k_pages"][ids, h].reshape(-1, D)[:n_keys].double()
            v = s["v_pages"][ids, h].reshape(-1, D)[:n_keys].double()
            for j in range(h * group, (h + 1) * group):
                logits = s["q"][rows, j].double() @ k.T / math.sqrt(D)
                if hidden is not None:
                    logits[hidden] = -math.inf
                out[rows, j] = torch.softmax(logits, 1) @ v
    return out
