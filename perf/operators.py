"""The token mixers next to the quantized projections: appending to a 4-bit paged cache, attention over
that cache, and the gated delta rule, each with its plain form, a 64-bit form and the work it cannot avoid.

`own` selects what `run` calls: the library's kernels, or elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False
DEV = "cuda"
GROUP = 64      # dims that share a scale and a bias
LIMIT = 57344.0  # the quantizer clamps its inputs here (fp16 scales and biases)
CHUNK = 64


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a small serving batch: 14B-shaped heads
        {"name": "append_decode", "op": "append", "tokens": 16, "n_q": 40, "n_kv": 8, "hd": 128, "rot": 128,
         "page": 32, "f32": False},
        # one long prompt, 14B-shaped heads
        {"name": "append_prefill", "op": "append", "tokens": 8192, "n_q": 40, "n_kv": 8, "hd": 128, "rot": 128,
         "page": 32, "f32": False},
        # a prompt chunk of the hybrid model: 256-wide heads, a quarter rotated, projections left in fp32
        {"name": "append_partial_f32", "op": "append", "tokens": 1021, "n_q": 24, "n_kv": 4, "hd": 256, "rot": 64,
         "page": 16, "f32": True},
        # one user, short context: latency
        {"name": "attn_decode_one", "op": "attn", "seqs": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 517, "kv_hi": 517,
         "n_q": 40, "n_kv": 8, "hd": 128, "page": 32, "gate": False, "window": 0},
        # a serving batch with contexts of very different lengths
        {"name": "attn_decode_batch", "op": "attn", "seqs": 64, "q_lo": 1, "q_hi": 1, "kv_lo": 100, "kv_hi": 16000,
         "n_q": 40, "n_kv": 8, "hd": 128, "page": 32, "gate": False, "window": 0},
        # one user, a very long document, the hybrid model's gated attention
        {"name": "attn_decode_long", "op": "attn", "seqs": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 131071, "kv_hi": 131071,
         "n_q": 24, "n_kv": 4, "hd": 256, "page": 64, "gate": True, "window": 0},
        # one prompt from its start
        {"name": "attn_prefill", "op": "attn", "seqs": 1, "q_lo": 2048, "q_hi": 2048, "kv_lo": 2048, "kv_hi": 2048,
         "n_q": 40, "n_kv": 8, "hd": 128, "page": 32, "gate": False, "window": 0},
        # prompt chunks of several users behind cached prefixes
        {"name": "attn_prefill_ragged", "op": "attn", "seqs": 5, "q_lo": 100, "q_hi": 1500, "kv_lo": 1500,
         "kv_hi": 9000, "n_q": 24, "n_kv": 4, "hd": 256, "page": 16, "gate": True, "window": 0},
        # one user's decode step of a linear-attention layer
        {"name": "gdn_decode_one", "op": "gdn", "seqs": 1, "len_lo": 1, "len_hi": 1, "hk": 16, "hv": 32, "d": 128},
        # a serving batch's decode step
        {"name": "gdn_decode_batch", "op": "gdn", "seqs": 96, "len_lo": 1, "len_hi": 1, "hk": 16, "hv": 48, "d": 128},
        # one long prompt
        {"name": "gdn_prefill", "op": "gdn", "seqs": 1, "len_lo": 4096, "len_hi": 4096, "hk": 16, "hv": 32, "d": 128},
        # prompts of several users
        {"name": "gdn_prefill_ragged", "op": "gdn", "seqs": 6, "len_lo": 33, "len_hi": 2000, "hk": 16, "hv": 48,
         "d": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "gdn"])
    heads = rng.choice([(40, 8, 128, 128), (32, 8, 128, 128), (24, 4, 256, 64), (16, 2, 256, 64), (14, 2, 64, 64)])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        n_q, n_kv, hd, rot = heads
        return {"op": op, "tokens": _log(rng, 1, 8192), "n_q": n_q, "n_kv": n_kv, "hd": hd, "rot": rot, "page": page,
                "f32": rng.random() < 0.3}
    if op == "attn":
        n_q, n_kv, hd, _ = heads
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
            c["kv_hi"] = _log(rng, 8, 524288 // c["seqs"] if c["seqs"] > 4 else 131072)
            c["kv_lo"] = rng.randint(min(c["q_hi"], c["kv_hi"]), c["kv_hi"])
        c["window"] = _log(rng, 64, 4096) if rng.random() < 0.25 else 0
        return c
    hk = rng.choice([2, 4, 16])
    c = {"op": op, "hk": hk, "hv": hk * rng.choice([1, 2, 3]), "d": 128}
    kind = rng.choice(["decode", "few", "prefill", "prefill"])
    if kind == "prefill":
        c["seqs"] = _log(rng, 1, 4)
        c["len_hi"] = _log(rng, 20, 4096 if c["seqs"] == 1 else 1200)
        c["len_lo"] = rng.randint(1, c["len_hi"])
    else:
        c["seqs"] = _log(rng, 1, 96)
        c["len_lo"], c["len_hi"] = (1, 1) if kind == "decode" else (1, rng.randint(2, 8))
    return c


def _lens(case):
    """(query lengths, key lengths) of an attention case, or the lengths of a gated-delta case: from the case alone."""
    r = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))
    if case["op"] == "gdn":
        return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    kv = [max(n, r.randint(case["kv_lo"], case["kv_hi"])) for n in q]
    return q, kv


def work(case):
    if case["op"] == "append":
        t, e = case["tokens"], 4 if case["f32"] else 2
        nq, nkv, hd = case["n_q"] * case["hd"], case["n_kv"] * case["hd"], case["hd"]
        cached = 2 * nkv * (0.5 + 4 / GROUP)
        return {"bytes": t * (nq * (e + 2) + 2 * nkv * (e + 2) + cached + 8 + 4 * case["rot"]),
                "flops": t * (3 * (nq + nkv) * case["rot"] / hd + 2 * 6 * nkv)}
    if case["op"] == "attn":
        q, kv = _lens(case)
        nq, nkv, hd, w = case["n_q"], case["n_kv"], case["hd"], case["window"]
        pairs = keys = 0
        for n, s in zip(q, kv):
            for j in (range(n) if w else ()):
                p = s - n + j
                pairs += min(p + 1, w)
            if not w:
                pairs += n * s - n * (n - 1) // 2
            keys += min(s, w + n - 1) if w else s
        tok = sum(q)
        return {"bytes": keys * nkv * 2 * (hd / 2 + 4 * hd / GROUP) + tok * nq * hd * 2 * (3 if case["gate"] else 2),
                "flops": 4.0 * hd * nq * pairs}
    n, hv, hk, d = sum(_lens(case)), case["hv"], case["hk"], case["d"]
    return {"bytes": case["seqs"] * hv * d * d * 8.0 + n * (2 * hk * d * 2 + 2 * hv * d * 2 + hv * 8),
            "flops": 7.0 * n * hv * d * d}


# ---- the cache's layout --------------------------------------------------------------------

def _k_words(hd):
    """Logical word (8 dims) at each position of a stored key row."""
    if hd % 128:
        return list(range(hd // 8))
    return [16 * (p // 16) + 8 * ((p % 4) // 2) + 2 * ((p % 16) // 4) + p % 2 for p in range(hd // 8)]


def _quantize(x):
    """(codes int32, scale fp16, bias fp16) of the groups of 64 along the last axis of fp32 x."""
    x = x.clamp(-LIMIT, LIMIT).unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) * (1.0 / 15.0)).half()
    b = lo.half()
    sf = s.float()
    inv = torch.where(sf > 0, torch.reciprocal(sf), torch.zeros_like(sf))
    c = ((x - b.float()) * inv).round().clamp(0, 15).to(torch.int32)
    return c.flatten(-2), s.squeeze(-1), b.squeeze(-1)


def _meta(s, b):
    lo = s.view(torch.int16).to(torch.int32) & 0xFFFF
    return lo | (b.view(torch.int16).to(torch.int32) << 16)


def _pack(c, per):
    """Codes along the last axis, `per` to a value, the first in the lowest bits."""
    c = c.unflatten(-1, (-1, per))
    out = torch.zeros(c.shape[:-1], dtype=torch.int32, device=c.device)
    for i in range(per):
        out |= c[..., i] << (4 * i)
    return out


def _k_stored(x):
    """fp32 [.., hd] -> stored code words and meta words of a key row."""
    c, s, b = _quantize(x)
    w = _pack(c, 8)
    return w[..., torch.tensor(_k_words(x.shape[-1]), device=x.device)], _meta(s, b)


def _v_stored(x):
    """fp32 [.., hd] -> 16-bit units of 4 codes and meta words of a value row."""
    c, s, b = _quantize(x)
    return _pack(c, 4).to(torch.int16), _meta(s, b)


def _scales(meta):
    s = (meta & 0xFFFF).to(torch.int16).view(torch.float16).float()
    b = (meta >> 16).to(torch.int16).view(torch.float16).float()
    return s, b


def _values(codes, meta):
    """fp32 values s c + b of codes [.., hd] and meta words [.., hd / 64]."""
    s, b = _scales(meta)
    return (codes.unflatten(-1, (-1, GROUP)) * s.unsqueeze(-1) + b.unsqueeze(-1)).flatten(-2)


def _unpack(words, per):
    shift = torch.arange(0, 4 * per, 4, dtype=torch.int32, device=words.device)
    return ((words.unsqueeze(-1) >> shift) & 15).float().flatten(-2)


def _k_read(words, meta):
    hd = words.shape[-1] * 8
    back = torch.empty(hd // 8, dtype=torch.long, device=words.device)
    back[torch.tensor(_k_words(hd), device=words.device)] = torch.arange(hd // 8, device=words.device)
    return _values(_unpack(words[..., back], 8), meta)


def _v_read(units, meta):
    """units [.., page / 8, hd / 4, 8] -> values [.., page, hd]."""
    u = units.transpose(-1, -2).flatten(-3, -2).to(torch.int32)
    return _values(_unpack(u, 4), meta)


def _new_cache(pages, n_kv, page, hd, gen, mean):
    """A cache that earlier tokens filled."""
    kc = torch.empty(pages, n_kv, page, hd // 8, dtype=torch.int32, device=DEV)
    km = torch.empty(pages, n_kv, page, hd // GROUP, dtype=torch.int32, device=DEV)
    vc = torch.empty(pages, n_kv, page // 8, hd // 4, 8, dtype=torch.int16, device=DEV)
    vm = torch.empty_like(km)
    step = max(1, (1 << 26) // (n_kv * page * hd))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn(n, n_kv, page, hd, device=DEV, generator=gen)
        kc[at:at + n], km[at:at + n] = _k_stored(x + mean)
        u, vm[at:at + n] = _v_stored(x.flip(2) * 0.7)
        vc[at:at + n] = u.unflatten(2, (-1, 8)).transpose(-1, -2)
    return kc, km, vc, vm


# ---- inputs --------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    host = random.Random(seed)
    st = {"case": case}
    if case["op"] == "append":
        t, n_q, n_kv, hd, rot, page = (case[k] for k in ("tokens", "n_q", "n_kv", "hd", "rot", "page"))
        dt = torch.float32 if case["f32"] else torch.bfloat16
        for name, heads in (("q", n_q), ("k", n_kv), ("v", n_kv)):
            st[name] = torch.randn(t, heads, hd, device=DEV, generator=gen).to(dt)
        need = -(-t // page)
        pages = need + 7
        order = list(range(pages))
        host.shuffle(order)
        order = torch.tensor(order, device=DEV)
        at = torch.arange(t, device=DEV)
        slots = order[at // page] * page + at % page
        start = host.randint(0, 8000)
        if t <= 64:  # a decode batch: positions of their own, and a padded row where the batch has room
            st["positions"] = torch.randint(0, 16384, (t,), device=DEV, generator=gen, dtype=torch.int32)
            if t > 4:
                slots[host.randrange(t)] = -1
        else:
            st["positions"] = (start + at).to(torch.int32)
        st["slots"] = slots.to(torch.int32)
        inv = 1e6 ** (-2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot)
        ang = torch.arange(16384, device=DEV, dtype=torch.float64)[:, None] * inv
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], -1).float()
        st["cache"] = (torch.zeros(pages, n_kv, page, hd // 8, dtype=torch.int32, device=DEV),
                       torch.zeros(pages, n_kv, page, hd // GROUP, dtype=torch.int32, device=DEV),
                       torch.zeros(pages, n_kv, page // 8, hd // 4, 8, dtype=torch.int16, device=DEV),
                       torch.zeros(pages, n_kv, page, hd // GROUP, dtype=torch.int32, device=DEV))
        for name, heads in (("q_rot", n_q), ("k_held", n_kv), ("v_held", n_kv)):
            st[name] = torch.empty(t, heads, hd, dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "attn":
        q_len, kv_len = _lens(case)
        b, n_q, n_kv, hd, page = (case[k] for k in ("seqs", "n_q", "n_kv", "hd", "page"))
        width = max(-(-n // page) for n in kv_len)
        total = sum(-(-n // page) for n in kv_len)
        order = list(range(total + 3))
        host.shuffle(order)
        table, used = [], 0
        for n in kv_len:
            p = -(-n // page)
            table.append(order[used:used + p] + [-1] * (width - p))
            used += p
        st["page_table"] = torch.tensor(table, dtype=torch.int32, device=DEV)
        st["kv_lens"] = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
        starts = [0]
        for n in q_len:
            starts.append(starts[-1] + n)
        st["q_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        st["max_q"] = max(q_len)
        mean = torch.randn(n_kv, 1, hd, device=DEV, generator=gen)
        st["cache"] = _new_cache(total + 3, n_kv, page, hd, gen, mean)
        st["q"] = torch.randn(starts[-1], n_q, hd, device=DEV, generator=gen).bfloat16()
        st["gate"] = torch.randn(starts[-1], n_q, hd, device=DEV, generator=gen).bfloat16() if case["gate"] else None
        st["out"] = torch.empty_like(st["q"])
    else:
        lens = _lens(case)
        b, hk, hv, d = (case[k] for k in ("seqs", "hk", "hv", "d"))
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        t = starts[-1]
        st["seq_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        st["max_len"] = max(lens)
        for name, heads in (("q", hk), ("k", hk), ("v", hv)):
            x = torch.randn(t, heads, d, device=DEV, generator=gen)
            if name != "v":  # neighbouring tokens' keys are alike
                x = x + 0.7 * torch.randn(1, heads, d, device=DEV, generator=gen)
            st[name] = torch.nn.functional.silu(x).bfloat16()
        rate = torch.rand(hv, device=DEV, generator=gen) * 8 + 0.05
        st["g"] = -rate * torch.nn.functional.softplus(torch.randn(t, hv, device=DEV, generator=gen) - 4)
        st["beta"] = torch.sigmoid(torch.randn(t, hv, device=DEV, generator=gen))
        slots = list(range(b + 2))
        host.shuffle(slots)
        st["state_slots"] = torch.tensor(slots[:b], dtype=torch.int32, device=DEV)
        st["state_in"] = 0.3 * torch.randn(b + 2, hv, d, d, device=DEV, generator=gen)
        st["state"] = st["state_in"].clone()
        st["y"] = torch.empty(t, hv, d, dtype=torch.bfloat16, device=DEV)
    return st


# ---- one pass ------------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return {"append": _own_append, "attn": _own_attn, "gdn": _own_gdn}[op](st)
    return {"append": _append, "attn": _attn, "gdn": _gdn}[op](st)


def _own_append(st):
    import gemm_affine_u4_amd as qmm
    qmm.qmm_kv4_append(qmm.KV4Cache(*st["cache"]), st["k"], st["v"], st["slots"], positions=st["positions"],
                       cos_sin=st["cos_sin"], q=st["q"], q_out=st["q_rot"], k_held=st["k_held"], v_held=st["v_held"])
    return {"q": st["q_rot"], "k": st["k_held"], "v": st["v_held"]}


def _own_attn(st):
    import gemm_affine_u4_amd as qmm
    case = st["case"]
    if "workspace" not in st:  # a program keeps it from the first step on
        need = qmm.qmm_kv4_attn_workspace_bytes(st["q"].shape[0], case["seqs"], st["max_q"], case["n_q"], case["n_kv"],
                                                case["hd"], st["page_table"].shape[1] * case["page"])
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    qmm.qmm_kv4_attn(st["q"], qmm.KV4Cache(*st["cache"]), st["page_table"], st["kv_lens"], st["out"], st["workspace"],
                     q_start=st["q_start"], max_q=st["max_q"], window=case["window"], gate=st["gate"])
    return {"out": st["out"]}


def _own_gdn(st):
    import gemm_affine_u4_amd as qmm
    case = st["case"]
    if "workspace" not in st:
        need = qmm.qmm_gdn_workspace_bytes(st["q"].shape[0], case["seqs"], st["max_len"], case["hk"], case["hv"],
                                           case["d"], case["d"])
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    qmm.qmm_gdn(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state_in"], st["y"], st["workspace"],
                state_out=st["state"], seq_start=st["seq_start"], state_slots=st["state_slots"],
                max_len=st["max_len"], l2norm=True)
    return {"y": st["y"], "state": st["state"]}


def _rotate(x, cos, sin):
    h = cos.shape[-1]
    a, b, rest = x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _append(st):
    kc, km, vc, vm = st["cache"]
    page, rot = kc.shape[2], st["cos_sin"].shape[1]
    row = st["cos_sin"][st["positions"].long().clamp(0, st["cos_sin"].shape[0] - 1)].unsqueeze(1)
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    q = _rotate(st["q"].float(), cos, sin)
    k = _rotate(st["k"].float(), cos, sin)
    k_words, k_meta = _k_stored(k)
    v_units, v_meta = _v_stored(st["v"].float())
    slots = st["slots"].long()
    kept = (slots >= 0).nonzero().flatten()
    at = slots[kept]
    p, o = at // page, at % page
    kc[p, :, o], km[p, :, o] = k_words[kept], k_meta[kept]
    vc[p, :, o // 8, :, o % 8], vm[p, :, o] = v_units[kept], v_meta[kept]
    back = torch.empty(k_words.shape[-1], dtype=torch.long, device=DEV)
    back[torch.tensor(_k_words(k.shape[-1]), device=DEV)] = torch.arange(k_words.shape[-1], device=DEV)
    k_held = _values(_unpack(k_words[..., back], 8), k_meta)
    v_held = _values(_unpack(v_units.to(torch.int32), 4), v_meta)
    return {"q": q.bfloat16(), "k": k_held.bfloat16(), "v": v_held.bfloat16()}


def _attn(st):
    case = st["case"]
    n_q, n_kv, hd, w, mq = case["n_q"], case["n_kv"], case["hd"], case["window"], st["max_q"]
    kc, km, vc, vm = st["cache"]
    table = st["page_table"].long().clamp(min=0)
    b = table.shape[0]
    k = _k_read(kc[table], km[table]).transpose(1, 2).flatten(2, 3)  # [B, n_kv, L, hd]
    v = _v_read(vc[table], vm[table]).transpose(1, 2).flatten(2, 3)
    start, count = st["q_start"][:-1].long(), (st["q_start"][1:] - st["q_start"][:-1]).long()
    j = torch.arange(mq, device=DEV)
    live = j < count[:, None]
    rows = (start[:, None] + j).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().unflatten(2, (n_kv, -1)).permute(0, 2, 3, 1, 4)  # [B, n_kv, G, mq, hd]
    s = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (-1, mq)) * hd ** -0.5
    t = torch.arange(k.shape[2], device=DEV)
    pos = (st["kv_lens"].long() - count)[:, None] + j
    seen = (t <= pos[..., None]) & (t < st["kv_lens"].long()[:, None, None])
    if w:
        seen &= t > pos[..., None] - w
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    p = (s - s.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    o = p.flatten(2, 3) @ v
    o = o / p.sum(-1).flatten(2, 3).clamp(min=1e-30).unsqueeze(-1)
    o = o.unflatten(2, (-1, mq)).permute(0, 3, 1, 2, 4).flatten(2, 3)[live]
    if st["gate"] is not None:
        o = o * torch.sigmoid(st["gate"].float())
    return {"out": o.bfloat16()}


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _gdn(st):
    case = st["case"]
    hv, d = case["hv"], case["d"]
    start, count = st["seq_start"][:-1].long(), (st["seq_start"][1:] - st["seq_start"][:-1]).long()
    slots = st["state_slots"].long()
    state_all = st["state"]  # of the next step; this step's is kept, as a step that may be taken back needs it
    s = st["state_in"][slots]                                 # [B, hv, dv, dk]
    rep = hv // case["hk"]
    if st["max_len"] == 1:
        q = _unit(st["q"].float()).repeat_interleave(rep, 1) * d ** -0.5
        k = _unit(st["k"].float()).repeat_interleave(rep, 1)
        s = s * st["g"].exp()[..., None, None]
        delta = (st["v"].float() - (s @ k.unsqueeze(-1)).squeeze(-1)) * st["beta"].unsqueeze(-1)
        s = s + delta.unsqueeze(-1) * k.unsqueeze(-2)
        state_all[slots] = s
        return {"y": (s @ q.unsqueeze(-1)).squeeze(-1).bfloat16(), "state": state_all}
    n = -(-st["max_len"] // CHUNK) * CHUNK
    j = torch.arange(n, device=DEV)
    live = j < count[:, None]
    rows = (start[:, None] + j).clamp(max=st["q"].shape[0] - 1)

    def padded(x):  # [T, H, ..] -> [B, H, chunks, 64, ..], zeros behind a sequence
        x = x.float()[rows]
        x = torch.where(live.reshape(live.shape + (1,) * (x.dim() - 2)), x, torch.zeros((), device=DEV))
        return x.transpose(1, 2).unflatten(2, (-1, CHUNK))

    q = padded(_unit(st["q"].float()) * d ** -0.5).repeat_interleave(rep, 1)
    k = padded(_unit(st["k"].float())).repeat_interleave(rep, 1)
    v, g, beta = padded(st["v"]), padded(st["g"]).cumsum(-1), padded(st["beta"])
    fall = (g.unsqueeze(-1) - g.unsqueeze(-2)).tril().exp().tril()
    low = (beta.unsqueeze(-1) * (k @ k.transpose(-1, -2)) * fall).tril(-1)
    inv = torch.eye(CHUNK, device=DEV).expand_as(low).clone()
    for i in range(1, CHUNK):  # rows of the inverse of a unit lower triangle
        inv[..., i, :i] = -(low[..., i:i + 1, :i] @ inv[..., :i, :i]).squeeze(-2)
    u = inv @ (beta.unsqueeze(-1) * v)
    wk = inv @ ((beta * g.exp()).unsqueeze(-1) * k)
    qk = (q @ k.transpose(-1, -2)) * fall
    y = torch.empty_like(v)
    for c in range(n // CHUNK):
        gc = g[:, :, c]
        new = u[:, :, c] - wk[:, :, c] @ s.transpose(-1, -2)
        y[:, :, c] = (q[:, :, c] * gc.exp().unsqueeze(-1)) @ s.transpose(-1, -2) + qk[:, :, c] @ new
        last = gc[..., -1:]
        s = s * last.exp().unsqueeze(-1) + (new * (last - gc).exp().unsqueeze(-1)).transpose(-1, -2) @ k[:, :, c]
    state_all[slots] = s
    return {"y": y.flatten(2, 3).transpose(1, 2)[live].bfloat16(), "state": state_all}


# ---- the definitions in 64 bits ------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "gdn": _exact_gdn}[case["op"]](st)


def _exact_append(st):
    rot = st["cos_sin"].shape[1]
    h = rot // 2
    angle = st["cos_sin"].double()[st["positions"].long()]

    def turned(x):
        y = x.double().clone()
        c, s = angle[:, None, :h], angle[:, None, h:]
        y[..., :h] = x[..., :h].double() * c - x[..., h:rot].double() * s
        y[..., h:rot] = x[..., h:rot].double() * c + x[..., :h].double() * s
        return y

    def held(x):
        shape = x.shape
        x = x.clamp(-LIMIT, LIMIT).reshape(-1, GROUP)
        lo = x.min(1, keepdim=True).values
        step = ((x.max(1, keepdim=True).values - lo) / 15).half().double()
        base = lo.half().double()
        codes = torch.where(step > 0, (x - base) / step, torch.zeros_like(x)).round().clamp(0, 15)
        return (base + step * codes).reshape(shape)

    return {"q": turned(st["q"]), "k": held(turned(st["k"])), "v": held(st["v"].double())}


def _exact_attn(st):
    case = st["case"]
    hd, w = case["hd"], case["window"]
    group = case["n_q"] // case["n_kv"]
    kc, km, vc, vm = st["cache"]
    page = kc.shape[2]
    starts, lens, table = st["q_start"].tolist(), st["kv_lens"].tolist(), st["page_table"].tolist()
    where = {w_: i for i, w_ in enumerate(_k_words(hd))}
    nib = torch.arange(8, device=DEV)
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)

    def affine(codes, meta):  # [n, hd] whole numbers, [n, hd / 64] words
        halves = meta.contiguous().view(torch.float16).double().reshape(meta.shape[0], -1, 2)
        return codes.double() * halves[..., 0].repeat_interleave(GROUP, 1) + halves[..., 1].repeat_interleave(GROUP, 1)

    for i, n in enumerate(lens):
        if starts[i + 1] == starts[i]:
            continue
        ids = torch.tensor(table[i][:-(-n // page)], device=DEV)
        pos = torch.arange(n - (starts[i + 1] - starts[i]), n, device=DEV)
        for h in range(case["n_kv"]):
            words = kc[ids, h].reshape(-1, hd // 8)[:n].long()
            words = words[:, [where[x] for x in range(hd // 8)]]
            kd = affine(((words.unsqueeze(-1) >> (4 * nib)) & 15).reshape(n, hd), km[ids, h].reshape(-1, hd // GROUP)[:n])
            units = vc[ids, h].permute(0, 1, 3, 2).reshape(-1, hd // 4)[:n].long()
            vd = affine(((units.unsqueeze(-1) >> (4 * nib[:4])) & 15).reshape(n, hd), vm[ids, h].reshape(-1, hd // GROUP)[:n])
            t = torch.arange(n, device=DEV)
            hidden = t > pos[:, None]
            if w:
                hidden |= t <= pos[:, None] - w
            for a in range(h * group, (h + 1) * group):
                s = st["q"][starts[i]:starts[i + 1], a].double() @ kd.T / math.sqrt(hd)
                s[hidden] = -math.inf
                out[starts[i]:starts[i + 1], a] = torch.softmax(s, -1) @ vd
    if st["gate"] is not None:
        out = out / (1 + torch.exp(-st["gate"].double()))
    return {"out": out}


def _exact_gdn(st):
    case = st["case"]
    d, rep = case["d"], case["hv"] // case["hk"]
    starts, slots = st["seq_start"].tolist(), st["state_slots"].long()
    lens = [b - a for a, b in zip(starts, starts[1:])]
    order = sorted(range(len(lens)), key=lambda i: -lens[i])  # longest first: step t runs the first sequences only
    first = torch.tensor([starts[i] for i in order], device=DEV)
    where = slots[torch.tensor(order, device=DEV)]
    q, k = st["q"].double(), st["k"].double()
    q = q / (q.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt() / math.sqrt(d)
    k = k / (k.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
    v, fall, beta = st["v"].double(), st["g"].double().exp(), st["beta"].double()
    state = st["state_in"].double()
    s = state[where]
    y = torch.empty(v.shape, dtype=torch.float64, device=DEV)
    for t in range(max(lens)):
        n = sum(x > t for x in lens)
        at = first[:n] + t
        kt, qt = k[at].repeat_interleave(rep, 1), q[at].repeat_interleave(rep, 1)
        m = s[:n] * fall[at][..., None, None]
        wrong = v[at] - torch.matmul(m, kt.unsqueeze(-1)).squeeze(-1)
        m = m + (beta[at].unsqueeze(-1) * wrong).unsqueeze(-1) * kt.unsqueeze(-2)
        y[at] = torch.matmul(m, qt.unsqueeze(-1)).squeeze(-1)
        s[:n] = m
    state[where] = s
    return {"y": y, "state": state}
