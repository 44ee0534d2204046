"""A step of a serving batch beside the quantized projections: low-rank adapters of many requests, the paged 8-bit
cache and attention over it, and the verification of drafted tokens, each with its plain form, a 64-bit form and the
work it cannot avoid.

`own` selects what `run` calls: the library's kernels, or elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False
DEV = "cuda"
BLOCK = 16       # keys that share a scale, for each head
LIMIT = 57344.0  # the quantizer clamps its inputs here
GROW = 1.25      # a block's scale grows by this factor at least


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a small serving batch, 14B-shaped heads: each token goes into a block begun earlier
        {"name": "append8_decode", "op": "append", "seqs": 16, "n_lo": 1, "n_hi": 1, "old_lo": 1, "old_hi": 4000,
         "n_q": 40, "n_kv": 8, "hd": 128, "rot": 128, "page": 32, "f32": False},
        # one long prompt, 14B-shaped heads
        {"name": "append8_prefill", "op": "append", "seqs": 1, "n_lo": 8192, "n_hi": 8192, "old_lo": 0, "old_hi": 0,
         "n_q": 40, "n_kv": 8, "hd": 128, "rot": 128, "page": 32, "f32": False},
        # prompt chunks behind cached prefixes of odd lengths: 256-wide heads, a quarter rotated, projections in fp32
        {"name": "append8_ragged_f32", "op": "append", "seqs": 5, "n_lo": 33, "n_hi": 700, "old_lo": 1, "old_hi": 3000,
         "n_q": 24, "n_kv": 4, "hd": 256, "rot": 64, "page": 16, "f32": True},
        # one user, short context: latency
        {"name": "attn8_decode_one", "op": "attn", "seqs": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 517, "kv_hi": 517,
         "n_q": 40, "n_kv": 8, "hd": 128, "page": 32, "gate": False, "window": 0, "sinks": 0},
        # a serving batch with contexts of very different lengths
        {"name": "attn8_decode_batch", "op": "attn", "seqs": 64, "q_lo": 1, "q_hi": 1, "kv_lo": 100, "kv_hi": 16000,
         "n_q": 40, "n_kv": 8, "hd": 128, "page": 32, "gate": False, "window": 0, "sinks": 0},
        # a batch's drafted tokens over long streams: a window, and the first tokens stay visible
        {"name": "attn8_drafts_sinks", "op": "attn", "seqs": 16, "q_lo": 2, "q_hi": 6, "kv_lo": 9000, "kv_hi": 30000,
         "n_q": 24, "n_kv": 4, "hd": 256, "page": 16, "gate": True, "window": 4000, "sinks": 4},
        # prompt chunks of several users behind cached prefixes
        {"name": "attn8_prefill", "op": "attn", "seqs": 4, "q_lo": 300, "q_hi": 1500, "kv_lo": 1500, "kv_hi": 8000,
         "n_q": 40, "n_kv": 8, "hd": 128, "page": 32, "gate": False, "window": 0, "sinks": 0},
        # one user, drafts looked up in the prompt (no draft probabilities)
        {"name": "verify_one_lookup", "op": "verify", "seqs": 1, "n_lo": 5, "n_hi": 5, "vocab": 32000, "probs": False,
         "half": False},
        # a serving batch with a draft model's probabilities
        {"name": "verify_batch", "op": "verify", "seqs": 64, "n_lo": 1, "n_hi": 6, "vocab": 152001, "probs": True,
         "half": False},
        # one user's token beside the fused QKV projection, 14B-shaped
        {"name": "lora_decode_one", "op": "lora", "reqs": 1, "len_lo": 1, "len_hi": 1, "adapters": 8, "rank": 16,
         "K": 5120, "q_out": 5120, "kv_out": 1024, "f32": False},
        # a serving batch, most requests with an adapter of their own
        {"name": "lora_decode_batch", "op": "lora", "reqs": 64, "len_lo": 1, "len_hi": 1, "adapters": 48, "rank": 16,
         "K": 5120, "q_out": 5120, "kv_out": 1024, "f32": False},
        # prompts of several requests beside a down projection that leaves fp32
        {"name": "lora_prefill_f32", "op": "lora", "reqs": 5, "len_lo": 100, "len_hi": 1500, "adapters": 8, "rank": 64,
         "K": 13824, "q_out": 5120, "kv_out": 0, "f32": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "verify", "lora"])
    n_q, n_kv, hd, rot = rng.choice([(40, 8, 128, 128), (32, 8, 128, 128), (24, 4, 256, 64), (16, 2, 256, 64),
                                     (14, 2, 64, 64)])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        c = {"op": op, "n_q": n_q, "n_kv": n_kv, "hd": hd, "rot": rot, "page": page, "f32": rng.random() < 0.3}
        if rng.random() < 0.5:
            c["seqs"], c["n_lo"], c["n_hi"] = _log(rng, 1, 64), 1, rng.choice([1, 1, 6])
        else:
            c["seqs"] = _log(rng, 1, 4)
            c["n_hi"] = _log(rng, 20, 6000 // c["seqs"])
            c["n_lo"] = rng.randint(1, c["n_hi"])
        c["old_hi"] = _log(rng, 1, 4000)
        c["old_lo"] = rng.randint(0, c["old_hi"])
        return c
    if op == "attn":
        c = {"op": op, "n_q": n_q, "n_kv": n_kv, "hd": hd, "page": page, "gate": rng.random() < 0.4}
        kind = rng.choice(["decode", "decode", "few", "prefill"])
        if kind == "prefill":
            c["seqs"] = _log(rng, 1, 3)
            c["q_hi"] = _log(rng, 40, 1200)
            c["q_lo"] = rng.randint(1, c["q_hi"])
            c["kv_hi"] = c["q_hi"] + _log(rng, 1, 5000)
            c["kv_lo"] = rng.randint(c["q_hi"], c["kv_hi"])
        else:
            c["seqs"] = _log(rng, 1, 64)
            c["q_lo"], c["q_hi"] = (1, 1) if kind == "decode" else (1, rng.randint(2, 8))
            c["kv_hi"] = _log(rng, 8, 400000 // c["seqs"] if c["seqs"] > 4 else 100000)
            c["kv_lo"] = rng.randint(min(c["q_hi"], c["kv_hi"]), c["kv_hi"])
        c["window"] = _log(rng, 64, 4096) if rng.random() < 0.4 else 0
        c["sinks"] = rng.choice([0, 1, 4, 30, 128]) if c["window"] else 0
        return c
    if op == "verify":
        return {"op": op, "seqs": _log(rng, 1, 64), "n_lo": rng.randint(0, 3), "n_hi": rng.randint(3, 7),
                "vocab": _log(rng, 1000, 140000), "probs": rng.random() < 0.7, "half": rng.random() < 0.4}
    c = {"op": op, "adapters": _log(rng, 1, 48), "rank": rng.choice([8, 16, 32, 64]), "f32": rng.random() < 0.4,
         "K": 64 * rng.randint(8, 120), "q_out": rng.choice([rng.randint(500, 6000), 64 * rng.randint(8, 90)])}
    c["kv_out"] = rng.choice([0, 256, 1024])
    if rng.random() < 0.6:
        c["reqs"], c["len_lo"], c["len_hi"] = _log(rng, 1, 64), 1, rng.choice([1, 1, 5])
    else:
        c["reqs"] = _log(rng, 1, 6)
        c["len_hi"] = _log(rng, 30, 3500 // c["reqs"])
        c["len_lo"] = rng.randint(1, c["len_hi"])
    return c


def _rng(case):
    return random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))


def _lens(case):
    """From the case alone: (new tokens, keys) of an append's or an attention's sequences, numbers of drafts, or the
    requests' (tokens, adapter)."""
    r = _rng(case)
    if case["op"] == "append":
        n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["seqs"])]
        return n, [m + r.randint(case["old_lo"], case["old_hi"]) for m in n]
    if case["op"] == "attn":
        q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
        return q, [max(n, r.randint(case["kv_lo"], case["kv_hi"])) for n in q]
    if case["op"] == "verify":
        n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["seqs"])]
        return n if any(n) else [case["n_hi"]] * case["seqs"]
    return [(r.randint(case["len_lo"], case["len_hi"]),
             -1 if case["reqs"] > 3 and r.random() < 0.1 else r.randrange(case["adapters"]))
            for _ in range(case["reqs"])]


def _seen(n, s, w, sinks):
    """Keys that n queries at the end of s keys see in all, and how many of the keys any of them sees."""
    if not w:
        return n * s - n * (n - 1) // 2, s
    pairs = 0
    for p in range(s - n, s):
        lo = max(0, p - w + 1)
        pairs += p + 1 - lo + min(sinks, lo)
    lo = max(0, s - n - w + 1)
    return pairs, s - lo + min(sinks, lo)


def work(case):
    if case["op"] == "append":
        t, e = sum(_lens(case)[0]), 4 if case["f32"] else 2
        nq, nkv = case["n_q"] * case["hd"], case["n_kv"] * case["hd"]
        return {"bytes": t * (nq * (e + 2) + 2 * nkv * (e + 2 + 1) + 4 + 4 * case["rot"] + 8 * case["n_kv"] / BLOCK),
                "flops": t * (3 * (nq + nkv) * case["rot"] / case["hd"] + 2 * 4 * nkv)}
    if case["op"] == "attn":
        q, kv = _lens(case)
        nq, nkv, hd = case["n_q"], case["n_kv"], case["hd"]
        seen = [_seen(n, s, case["window"], case["sinks"]) for n, s in zip(q, kv)]
        keys, tok = sum(x[1] for x in seen), sum(q)
        return {"bytes": keys * nkv * 2 * (hd + 4 / BLOCK) + tok * nq * hd * 2 * (3 if case["gate"] else 2),
                "flops": 4.0 * hd * nq * sum(x[0] for x in seen)}
    if case["op"] == "verify":
        e, b, n = 2 if case["half"] else 4, case["seqs"], sum(_lens(case))
        rows = b * (2 if case["probs"] else 1)
        return {"bytes": rows * case["vocab"] * e + n * (2 * e + 8) + b * 4 * (case["n_hi"] + 3),
                "flops": 2.0 * rows * case["vocab"]}
    reqs = _lens(case)
    t = sum(n for n, _ in reqs)
    used = len({a for _, a in reqs if a >= 0})
    live = sum(n for n, a in reqs if a >= 0)
    parts, n_out = (3, case["q_out"] + 2 * case["kv_out"]) if case["kv_out"] else (1, case["q_out"])
    e, r = 4 if case["f32"] else 2, case["rank"]
    return {"bytes": live * case["K"] * 2 + 2 * t * n_out * e + used * r * (parts * case["K"] + n_out) * 2 + 4 * t,
            "flops": 2.0 * live * r * (parts * case["K"] + n_out)}


# ---- inputs --------------------------------------------------------------------------------

def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _sums(n):
    s = [0]
    for x in n:
        s.append(s[-1] + x)
    return s


def _paged(st, host, lens, page):
    """A page table of sequences of these many keys, pages in any order; returns the number of pages."""
    total = sum(-(-n // page) for n in lens)
    width = max(1, max(-(-n // page) for n in lens))
    order = list(range(total + 3))
    host.shuffle(order)
    table, used = [], 0
    for n in lens:
        p = -(-n // page)
        table.append(order[used:used + p] + [-1] * (width - p))
        used += p
    st["page_table"], st["kv_lens"] = _ints(table), _ints(lens)
    return total + 3


def _new_cache(pages, n_kv, page, hd, gen, mean):
    """A cache that earlier tokens filled: codes and a scale for each block of 16 and head."""
    kc = torch.empty(pages, n_kv, page, hd, dtype=torch.int8, device=DEV)
    ks = torch.empty(pages, n_kv, page // BLOCK, device=DEV)
    vc = torch.empty(pages, n_kv, page // 8, hd, 8, dtype=torch.int8, device=DEV)
    vs = torch.empty_like(ks)
    step = max(1, (1 << 26) // (n_kv * page * hd))

    def codes(x):
        x = x.unflatten(2, (-1, BLOCK))
        s = x.abs().amax((-1, -2)) / 127
        return (x / s[..., None, None]).round().clamp(-127, 127).to(torch.int8).flatten(2, 3), s

    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn(n, n_kv, page, hd, device=DEV, generator=gen)
        kc[at:at + n], ks[at:at + n] = codes(x + mean)
        c, vs[at:at + n] = codes(x.flip(2) * 0.7)
        vc[at:at + n] = c.unflatten(2, (-1, 8)).transpose(-1, -2)
    return kc, ks, vc, vs


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    host = random.Random(seed)
    st = {"case": case}
    if case["op"] == "append":
        n, lens = _lens(case)
        n_q, n_kv, hd, rot, page = (case[k] for k in ("n_q", "n_kv", "hd", "rot", "page"))
        dt = torch.float32 if case["f32"] else torch.bfloat16
        starts = _sums(n)
        t = starts[-1]
        loud = torch.rand(t, 1, 1, device=DEV, generator=gen) + 0.5  # some tokens exceed their block's scale
        for name, heads in (("q", n_q), ("k", n_kv), ("v", n_kv)):
            st[name] = (torch.randn(t, heads, hd, device=DEV, generator=gen) * loud).to(dt)
        pages = _paged(st, host, lens, page)
        st["q_start"], st["max_q"] = _ints(starts), max(n)
        st["positions"] = _ints([s - m + j for m, s in zip(n, lens) for j in range(m)])
        inv = 1e6 ** (-2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot)
        ang = torch.arange(16384, device=DEV, dtype=torch.float64)[:, None] * inv
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], -1).float()
        st["cache"] = _new_cache(pages, n_kv, page, hd, gen, 0.0)
        st["cache"][1].mul_(0.8)  # earlier tokens of the last blocks were fewer, so their scales smaller
        st["cache"][3].mul_(0.8)
        for name, heads in (("q_rot", n_q), ("k_held", n_kv), ("v_held", n_kv)):
            st[name] = torch.empty(t, heads, hd, dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "attn":
        n, lens = _lens(case)
        n_q, n_kv, hd, page = (case[k] for k in ("n_q", "n_kv", "hd", "page"))
        pages = _paged(st, host, lens, page)
        starts = _sums(n)
        st["q_start"], st["max_q"], st["max_kv"] = _ints(starts), max(n), max(lens)
        mean = torch.randn(n_kv, 1, hd, device=DEV, generator=gen)
        st["cache"] = _new_cache(pages, n_kv, page, hd, gen, mean)
        st["q"] = torch.randn(starts[-1], n_q, hd, device=DEV, generator=gen).bfloat16()
        st["gate"] = torch.randn(starts[-1], n_q, hd, device=DEV, generator=gen).bfloat16() if case["gate"] else None
        st["out"] = torch.empty_like(st["q"])
    elif case["op"] == "verify":
        n, b, v = _lens(case), case["seqs"], case["vocab"]
        starts = _sums(n)
        d = starts[-1]
        dt = torch.bfloat16 if case["half"] else torch.float32
        st["draft_start"], st["max_draft"] = _ints(starts), max(n)
        logits = torch.randn(d + b, v, device=DEV, generator=gen) * 3
        st["target"] = torch.softmax(logits, -1).to(dt)
        rows = torch.tensor([s + i + j for i, (s, m) in enumerate(zip(starts, n)) for j in range(m)], device=DEV)
        q = torch.softmax(logits[rows] + 0.4 * torch.randn(d, v, device=DEV, generator=gen), -1)
        st["draft"] = torch.multinomial(q, 1, generator=gen).flatten().to(torch.int32)
        st["draft_probs"] = q.to(dt) if case["probs"] else None
        st["u"] = torch.rand(d + b, device=DEV, generator=gen)
        if not case["probs"]:  # looked-up drafts are mostly the likely token
            top = logits[rows].argmax(-1).to(torch.int32)
            st["draft"] = torch.where(torch.rand(d, device=DEV, generator=gen) < 0.8, top, st["draft"])
        st["tokens"] = torch.empty(b, max(n) + 1, dtype=torch.int32, device=DEV)
        st["accepted"] = torch.empty(b, dtype=torch.int32, device=DEV)
    else:
        reqs = _lens(case)
        r, k, n_ad = case["rank"], case["K"], case["adapters"]
        outs = [case["q_out"], case["kv_out"], case["kv_out"]] if case["kv_out"] else [case["q_out"]]
        t = sum(n for n, _ in reqs)
        dt = torch.float32 if case["f32"] else torch.bfloat16
        st["x"] = torch.randn(t, k, device=DEV, generator=gen).bfloat16()
        st["a"] = (torch.randn(n_ad, len(outs) * r, k, device=DEV, generator=gen) / math.sqrt(k)).bfloat16()
        st["b"] = (torch.randn(n_ad, sum(outs), r, device=DEV, generator=gen) * 0.1).bfloat16()
        st["ids"] = _ints([a for n, a in reqs for _ in range(n)])
        st["scales"] = 0.5 + torch.rand(n_ad, device=DEV, generator=gen)
        st["base"] = [torch.randn(t, n, device=DEV, generator=gen).to(dt) for n in outs]  # the shared projection's
        st["y"] = [torch.empty_like(x) for x in st["base"]]
    return st


# ---- one pass ------------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return {"append": _own_append, "attn": _own_attn, "verify": _own_verify, "lora": _own_lora}[op](st)
    return {"append": _append, "attn": _attn, "verify": _verify, "lora": _lora}[op](st)


def _handle(st):
    import gemm_affine_u4_amd as qmm
    if "handle" not in st:  # a program keeps it, and the workspaces below, from the first step on
        st["handle"] = qmm.KV8Cache(*st["cache"])
    return qmm, st["handle"]


def _own_append(st):
    qmm, cache = _handle(st)
    qmm.qmm_kv8_append(cache, st["k"], st["v"], st["page_table"], st["kv_lens"], q_start=st["q_start"],
                       max_q=st["max_q"], positions=st["positions"], cos_sin=st["cos_sin"], q=st["q"],
                       q_out=st["q_rot"], k_held=st["k_held"], v_held=st["v_held"])
    return {"q": st["q_rot"], "k": st["k_held"], "v": st["v_held"], "k_scale": st["cache"][1],
            "v_scale": st["cache"][3]}


def _own_attn(st):
    qmm, cache = _handle(st)
    case = st["case"]
    if "workspace" not in st:
        need = qmm.qmm_kv8_attn_workspace_bytes(st["q"].shape[0], case["seqs"], st["max_q"], case["n_q"], case["n_kv"],
                                                case["hd"], st["page_table"].shape[1] * case["page"], case["window"],
                                                case["sinks"])
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    qmm.qmm_kv8_attn(st["q"], cache, st["page_table"], st["kv_lens"], st["out"], st["workspace"],
                     q_start=st["q_start"], max_q=st["max_q"], window=case["window"], sinks=case["sinks"],
                     gate=st["gate"])
    return {"out": st["out"]}


def _own_verify(st):
    import gemm_affine_u4_amd as qmm
    case = st["case"]
    if "workspace" not in st:
        need = qmm.qmm_spec_verify_workspace_bytes(case["seqs"], case["vocab"])
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    qmm.qmm_spec_verify(st["draft"], st["target"], st["u"], st["tokens"], st["accepted"], st["workspace"],
                        draft_start=st["draft_start"], draft_probs=st["draft_probs"])
    return {"tokens": st["tokens"], "accepted": st["accepted"]}


def _own_lora(st):
    import gemm_affine_u4_amd as qmm
    case = st["case"]
    if "workspace" not in st:
        need = qmm.qmm_lora_workspace_bytes(st["x"].shape[0], case["K"], case["rank"], len(st["y"]))
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    qmm.qmm_lora(st["x"], st["a"], st["b"], st["ids"], st["y"], st["workspace"], base=st["base"], scales=st["scales"])
    return {"y": st["y"]}


def _rotate(x, cos, sin):
    h = cos.shape[-1]
    a, b, rest = x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _append(st):
    page = st["case"]["page"]
    row = st["cos_sin"][st["positions"].long()].unsqueeze(1)
    cos, sin = row.chunk(2, -1)
    q, k, v = _rotate(st["q"].float(), cos, sin), _rotate(st["k"].float(), cos, sin), st["v"].float()
    start, lens = st["q_start"].long(), st["kv_lens"].long()
    t, b = k.shape[0], lens.shape[0]
    seq = torch.searchsorted(start, torch.arange(t, device=DEV), right=True) - 1
    at = torch.arange(t, device=DEV) - start[1:][seq] + lens[seq]  # key of each token in its sequence
    slot = st["page_table"].long()[seq, at // page] * page + at % page
    first = (lens - (start[1:] - start[:-1]))                      # key of a sequence's first new token
    per = page // BLOCK
    out = {"q": q.bfloat16()}
    for name, x, codes, scale in (("k", k, *st["cache"][:2]), ("v", v, *st["cache"][2:])):
        x = x.clamp(-LIMIT, LIMIT)
        flat = scale.transpose(1, 2).reshape(-1, scale.shape[1])   # [blocks, heads]
        blk = slot // BLOCK
        most = x.abs().amax(-1)
        need = torch.zeros_like(flat).scatter_reduce_(0, blk[:, None].expand_as(most), most, "amax") * (1.0 / 127.0)
        met = torch.zeros(flat.shape[0], 1, dtype=torch.bool, device=DEV).index_fill_(0, blk, True)
        begun = torch.zeros(flat.shape[0], 1, device=DEV).index_add_(0, blk, (at % BLOCK == 0).float()[:, None]) > 0
        new = torch.where(begun, need, torch.where(need <= flat, flat, torch.maximum(need, flat * GROW)))
        new = torch.where(met, new, flat)
        # a sequence's first block may hold earlier tokens: theirs are coded anew where the scale grew
        kb = first // BLOCK
        page_b = st["page_table"].long()[torch.arange(b, device=DEV), kb * BLOCK // page]
        blk_b = page_b * per + kb % per
        ratio = torch.where(flat[blk_b] < new[blk_b], flat[blk_b] / new[blk_b], torch.ones_like(new[blk_b]))
        place = ((kb % per) * BLOCK)[:, None] + torch.arange(BLOCK, device=DEV)
        head = torch.arange(x.shape[1], device=DEV)[None, :, None]
        keep = (torch.arange(BLOCK, device=DEV) < (first % BLOCK)[:, None])[:, None, :, None]
        where = (page_b[:, None, None], head, place[:, None])
        if name == "v":
            where = (where[0], head, place[:, None] // 8, slice(None), place[:, None] % 8)
        old = codes[where]
        codes[where] = torch.where(keep, (old.float() * ratio[..., None, None]).round().to(torch.int8), old)
        s = new[blk]
        inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
        c = (x * inv[..., None]).round().clamp(-127, 127)
        head = head[..., 0]
        if name == "v":
            codes[(slot // page)[:, None], head, ((slot % page) // 8)[:, None], :, (slot % 8)[:, None]] = c.to(torch.int8)
        else:
            codes[(slot // page)[:, None], head, (slot % page)[:, None]] = c.to(torch.int8)
        scale.copy_(new.unflatten(0, (-1, per)).transpose(1, 2))
        out[name] = (c * s[..., None]).bfloat16()
        out[name + "_scale"] = scale
    return out


def _attn(st):
    case = st["case"]
    n_kv, hd, w, sinks, page = (case[k] for k in ("n_kv", "hd", "window", "sinks", "page"))
    mq = st["max_q"]
    kc, ks, vc, vs = st["cache"]
    lens = st["kv_lens"].long()
    start, count = st["q_start"][:-1].long(), (st["q_start"][1:] - st["q_start"][:-1]).long()
    b = lens.shape[0]
    j = torch.arange(mq, device=DEV)
    # the keys that any query of a sequence sees: the window's, and the first ones
    wide = min(st["max_kv"], w + mq - 1) if w else st["max_kv"]
    low = (lens - count - w + 1).clamp(min=0) if w else torch.zeros_like(lens)
    t = low[:, None] + torch.arange(wide, device=DEV)
    there = t < lens[:, None]
    if sinks:
        more = torch.arange(min(sinks, st["max_kv"]), device=DEV).expand(b, -1)
        there = torch.cat([there, (more < low[:, None]) & (more < lens[:, None])], 1)
        t = torch.cat([t, more], 1)
    t = torch.where(there, t, torch.zeros_like(t))
    ids = st["page_table"].long().gather(1, t // page).clamp(min=0)[:, None]
    o = (t % page)[:, None]
    head = torch.arange(n_kv, device=DEV)[None, :, None]
    k = kc[ids, head, o].float() * ks[ids, head, o // BLOCK][..., None]           # [B, n_kv, L, hd]
    v = vc[ids, head, o // 8, :, o % 8].float() * vs[ids, head, o // BLOCK][..., None]
    live = j < count[:, None]
    rows = (start[:, None] + j).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().unflatten(2, (n_kv, -1)).permute(0, 2, 3, 1, 4)     # [B, n_kv, G, mq, hd]
    s = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (-1, mq)) * hd ** -0.5
    pos = ((lens - count)[:, None] + j)[..., None]
    seen = there[:, None] & (t[:, None] <= pos)
    if w:
        seen &= (t[:, None] > pos - w) | (t[:, None] < sinks)
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    p = (s - s.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    x = p.flatten(2, 3) @ v
    x = x / p.sum(-1).flatten(2, 3).clamp(min=1e-30).unsqueeze(-1)
    x = x.unflatten(2, (-1, mq)).permute(0, 3, 1, 2, 4).flatten(2, 3)[live]
    if st["gate"] is not None:
        x = x * torch.sigmoid(st["gate"].float())
    return {"out": x.bfloat16()}


def _verify(st):
    p, q, u, v = st["target"], st["draft_probs"], st["u"].double(), st["case"]["vocab"]
    start = st["draft_start"].long()
    n, b = start[1:] - start[:-1], st["case"]["seqs"]
    j = torch.arange(st["max_draft"], device=DEV)
    at = (start[:-1, None] + j).clamp(max=st["draft"].shape[0] - 1)
    rows = start[:-1] + torch.arange(b, device=DEV)
    d = st["draft"].long()[at]
    row = (rows[:, None] + j).clamp(max=p.shape[0] - 1)
    of_q = q[at, d].double() if q is not None else 1.0
    kept = (j < n[:, None]) & (u[row] * of_q < p[row, d].double())
    count = kept.long().cumprod(1).sum(1)
    refused = count < n
    w = p[rows + count].double()
    at = (start[:-1] + count).clamp(max=st["draft"].shape[0] - 1)
    if q is not None:
        rest = (w - q[at].double() * refused[:, None]).clamp(min=0)
    else:
        rest = w * ~(refused[:, None] & (torch.arange(v, device=DEV) == st["draft"].long()[at][:, None]))
    w = torch.where(rest.sum(-1, keepdim=True) > 0, rest, w)
    c = w.cumsum(-1)
    hit = (c > u[rows + n][:, None] * c[:, -1:]) & (w > 0)
    last = v - 1 - (w > 0).flip(-1).int().argmax(-1)
    new = torch.where(hit.any(-1), hit.int().argmax(-1), last).to(torch.int32)
    tokens = torch.full((b, st["max_draft"] + 1), -1, dtype=torch.int32, device=DEV)
    tokens[:, :-1] = torch.where(j < count[:, None], d.to(torch.int32), tokens[:, :-1])
    tokens.scatter_(1, count[:, None], new[:, None])
    return {"tokens": tokens, "accepted": count.to(torch.int32)}


def _lora(st):
    n_ad, r = st["a"].shape[0], st["case"]["rank"]
    ids = st["ids"].long()
    mine = (ids[:, None] == torch.arange(n_ad, device=DEV)).float() * st["scales"]  # [T, adapters]
    y, row = [], 0
    for i, base in enumerate(st["base"]):
        a, b = st["a"][:, i * r:(i + 1) * r].float(), st["b"][:, row:row + base.shape[1]].float()
        row += base.shape[1]
        h = (st["x"].float() @ a.flatten(0, 1).T).unflatten(1, (n_ad, r)) * mine[..., None]
        y.append((base.float() + h.flatten(1) @ b.transpose(1, 2).reshape(n_ad * r, -1)).to(base.dtype))
    return {"y": y}


# ---- the definitions in 64 bits ------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "verify": _exact_verify, "lora": _exact_lora}[case["op"]](st)


def _exact_append(st):
    case = st["case"]
    page, rot = case["page"], case["rot"]
    h = rot // 2
    angle = st["cos_sin"].double()[st["positions"].long()]

    def turned(x):
        y = x.double().clone()
        c, s = angle[:, None, :h], angle[:, None, h:]
        y[..., :h] = x[..., :h].double() * c - x[..., h:rot].double() * s
        y[..., h:rot] = x[..., h:rot].double() * c + x[..., :h].double() * s
        return y

    starts, lens, table = st["q_start"].tolist(), st["kv_lens"].tolist(), st["page_table"].tolist()
    out = {"q": turned(st["q"])}
    for name, x, scale in (("k", turned(st["k"]), st["cache"][1]), ("v", st["v"].double(), st["cache"][3])):
        x, scale = x.clamp(-LIMIT, LIMIT), scale.double()
        held = torch.empty_like(x)
        most = x.abs().amax(-1)                                   # [T, heads]
        spans, old = [], []
        for i, n in enumerate(lens):
            t = starts[i]
            key = n - (starts[i + 1] - t)
            while t < starts[i + 1]:
                stop = min(starts[i + 1], t + BLOCK - key % BLOCK)
                spans.append((t, stop, table[i][key // page], key % page // BLOCK))
                old.append(key % BLOCK != 0)
                key, t = key + stop - t, stop
        ids = torch.tensor([s[2] for s in spans], device=DEV)
        sub = torch.tensor([s[3] for s in spans], device=DEV)
        size = torch.tensor([s[1] - s[0] for s in spans], device=DEV)
        rows = torch.repeat_interleave(torch.arange(len(spans), device=DEV), size)
        need = torch.zeros(len(spans), x.shape[1], dtype=torch.float64, device=DEV)
        need = need.scatter_reduce(0, rows[:, None].expand_as(most), most, "amax") / 127
        before = scale[ids, :, sub]
        grown = torch.where(need > before, torch.maximum(need, before * GROW), before)
        s = torch.where(torch.tensor(old, device=DEV)[:, None], grown, need)
        scale[ids, :, sub] = s
        s = s[rows][..., None]
        held = torch.where(s > 0, (x / s).round().clamp(-127, 127) * s, torch.zeros_like(x))
        out[name], out[name + "_scale"] = held, scale
    return out


def _exact_attn(st):
    case = st["case"]
    hd, w, page = case["hd"], case["window"], case["page"]
    group = case["n_q"] // case["n_kv"]
    kc, ks, vc, vs = st["cache"]
    starts, lens, table = st["q_start"].tolist(), st["kv_lens"].tolist(), st["page_table"].tolist()
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    for i, n in enumerate(lens):
        ids = torch.tensor(table[i][:-(-n // page)], device=DEV)
        pos = torch.arange(n - (starts[i + 1] - starts[i]), n, device=DEV)[:, None]
        t = torch.arange(n, device=DEV)
        hidden = t > pos
        if w:
            hidden |= (t <= pos - w) & (t >= case["sinks"])
        for h in range(case["n_kv"]):
            step = ks[ids, h].double().flatten().repeat_interleave(BLOCK)[:n, None]
            kd = kc[ids, h].reshape(-1, hd)[:n].double() * step
            step = vs[ids, h].double().flatten().repeat_interleave(BLOCK)[:n, None]
            vd = vc[ids, h].transpose(-1, -2).reshape(-1, hd)[:n].double() * step
            x = st["q"][starts[i]:starts[i + 1], h * group:(h + 1) * group].double()
            s = torch.matmul(x.transpose(0, 1).reshape(-1, hd), kd.T.contiguous()).view(group, -1, n) / math.sqrt(hd)
            p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
            o = torch.matmul(p.view(-1, n), vd).view(group, -1, hd)
            out[starts[i]:starts[i + 1], h * group:(h + 1) * group] = o.transpose(0, 1)
    if st["gate"] is not None:
        out = out / (1 + torch.exp(-st["gate"].double()))
    return {"out": out}


def _exact_verify(st):
    p, q = st["target"], st["draft_probs"]
    starts, u, d = st["draft_start"].tolist(), st["u"].double().tolist(), st["draft"].tolist()
    tokens, accepted = [], []
    for b in range(len(starts) - 1):
        n, row = starts[b + 1] - starts[b], starts[b] + b
        got = []
        for j in range(n):
            at = starts[b] + j
            if u[row + j] * (float(q[at, d[at]]) if q is not None else 1.0) >= float(p[row + j, d[at]]):
                break
            got.append(d[at])
        j = len(got)
        w = p[row + j].double()
        if j < n:
            other = torch.zeros_like(w)
            if q is not None:
                other = q[starts[b] + j].double()
            else:
                other[d[starts[b] + j]] = 1.0
            left = torch.relu(w - other)
            w = left if float(left.sum()) > 0 else w
        c = torch.cumsum(w, 0)
        new = int(torch.searchsorted(c, u[row + n] * c[-1], right=True))
        new = min(new, int(w.nonzero().max()))
        tokens.append(got + [new] + [-1] * (st["max_draft"] - j))
        accepted.append(j)
    return {"tokens": _ints(tokens), "accepted": _ints(accepted)}


def _exact_lora(st):
    r, x, y, row = st["case"]["rank"], st["x"].double(), [], 0
    for i, base in enumerate(st["base"]):
        out = base.double()
        for a in sorted(set(st["ids"].tolist()) - {-1}):
            rows = (st["ids"] == a).nonzero().flatten()
            h = torch.matmul(x[rows], st["a"][a, i * r:(i + 1) * r].double().T.contiguous())
            b = st["b"][a, row:row + base.shape[1]].double().T.contiguous()
            out[rows] += float(st["scales"][a]) * torch.matmul(h, b)
        y.append(out)
        row += base.shape[1]
    return {"y": y}
