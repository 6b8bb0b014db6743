"""Measured cases of the operators that let a latent cache serve long contexts:
a batch that shares a long prefix, the weight that attention gives each cached
token, and the eviction of the tokens that get little of it.

    shared   mla.decode_shared    attention over a group's shared prefix, read once for all its sequences, and each
                                  sequence's own cache
    mass     mla.attention_mass   the attention weight of every cached token, summed over query tokens and heads and
                                  added to a running sum
    evict    mla.evict            the tokens that stay (the first, the latest, the heaviest), the others' slots filled

With ``own`` false ``run`` computes them from elementary torch operations in
32 bits, with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False

D_LATENT, D_ROPE = 512, 64
D_QK = D_LATENT + D_ROPE
PAGE = 64
SCALE = 1.0 / math.sqrt(192.0)
#: queries are drawn this wide: scores then spread by about 2.6, as a trained model's heads with some heavy tokens do
Q_STD = 1.5
ROW = {"bf16": 1152, "fp8": 656, "fp8_tensor": 576}  # bytes of a cached token, its scales included

#: pairs of query rows and keys of the largest shared case
MOST_SHARED = 64 * 128 * (16384 + 1024)
#: cached tokens, and pairs of query rows and keys, of the largest mass cases
MOST_TOKENS = 64 * 16384
MOST_MASS = 64 * 128 * 16384
MOST_EVICT = 8 * 32768


def listed():
    return [
        # the smallest step: two samples of one short prompt, the heads of one rank of eight
        {"name": "shared_2_h16", "op": "shared", "batch": 2, "tokens": 1, "heads": 16, "groups": 1, "prefix": 200, "longest": 37,
         "causal": False, "format": "bf16"},
        # a batch behind one long system prompt, the heads of one rank of eight
        {"name": "shared_64_h16", "op": "shared", "batch": 64, "tokens": 1, "heads": 16, "groups": 1, "prefix": 8192, "longest": 1024,
         "causal": False, "format": "bf16"},
        # the same with all heads on one GPU and twice the prompt: the largest
        {"name": "shared_64_h128", "op": "shared", "batch": 64, "tokens": 1, "heads": 128, "groups": 1, "prefix": 16384, "longest": 1024,
         "causal": False, "format": "bf16"},
        # samples of three prompts of different lengths, groups of different sizes, four tokens a step, FP8 rows with scales
        {"name": "shared_48x4_h64_3_prompts_fp8", "op": "shared", "batch": 48, "tokens": 4, "heads": 64, "groups": 3, "prefix": 5000,
         "longest": 300, "causal": True, "format": "fp8"},
        # the smallest: one sequence
        {"name": "mass_1_h128", "op": "mass", "batch": 1, "tokens": 1, "heads": 128, "longest": 1000, "causal": False, "decay": 0.0,
         "format": "bf16"},
        # a decode step of a ragged batch, the running sums carried on
        {"name": "mass_64_h128", "op": "mass", "batch": 64, "tokens": 1, "heads": 128, "longest": 32768, "causal": False, "decay": 1.0,
         "format": "bf16"},
        # two tokens a step, FP8 rows with scales, older weights fading
        {"name": "mass_32x2_h64_fp8", "op": "mass", "batch": 32, "tokens": 2, "heads": 64, "longest": 8192, "causal": True, "decay": 0.9,
         "format": "fp8"},
        # the last 64 tokens of a prompt choose what of it is kept
        {"name": "mass_window_64_h128", "op": "mass", "batch": 1, "tokens": 64, "heads": 128, "longest": 12001, "causal": True, "decay": 0.0,
         "format": "bf16"},
        # the smallest: one sequence that has grown a little past what it may keep
        {"name": "evict_1_1100", "op": "evict", "batch": 1, "longest": 1100, "ragged": False, "keep": 1024, "sinks": 4, "recent": 64,
         "aged": True, "format": "bf16"},
        # prompts of a ragged batch cut down to what is kept
        {"name": "evict_prompts_8x32768", "op": "evict", "batch": 8, "longest": 32768, "ragged": True, "keep": 4096, "sinks": 4,
         "recent": 512, "aged": False, "format": "bf16"},
        # a full batch in the steady state: every 256 steps the newest push out the lightest, FP8 rows with scales
        {"name": "evict_64x4352_fp8", "op": "evict", "batch": 64, "longest": 4352, "ragged": False, "keep": 4096, "sinks": 4, "recent": 512,
         "aged": True, "format": "fp8"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "mass", "evict"])
    fmt = rng.choice(["bf16", "bf16", "fp8", "fp8_tensor"])
    if op == "evict":
        batch = _log(rng, 1, 64)
        longest = _log(rng, 16, min(32768, MOST_EVICT // batch))
        keep = _log(rng, 4, longest)
        sinks = min(rng.choice([0, 1, 4]), keep)
        return {"op": op, "batch": batch, "longest": longest, "ragged": rng.random() < 0.5, "keep": keep, "sinks": sinks,
                "recent": rng.randint(0, keep - sinks), "aged": rng.random() < 0.5, "format": fmt}
    heads = rng.choice([1, 8, 16, 20, 32, 64, 128])
    if op == "shared":
        tokens = rng.choice([1, 1, 1, 2, 4, 7])
        batch = _log(rng, 1, max(1, min(96, 64 * 128 // (heads * tokens))))
        rows = batch * tokens * heads
        prefix = _log(rng, 1, min(32768, max(64, MOST_SHARED // rows - 1024)))
        return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "groups": rng.randint(1, min(4, batch)), "prefix": prefix,
                "longest": _log(rng, 1, 1024), "causal": tokens > 1 and rng.random() < 0.7, "format": fmt}
    tokens = rng.choice([1, 1, 1, 2, 4, 16, 64])
    batch = _log(rng, 1, 64) if tokens < 16 else _log(rng, 1, 4)
    longest = _log(rng, 1, min(32768, MOST_TOKENS // batch, max(64, MOST_MASS // (batch * tokens * heads))))
    return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "longest": longest, "causal": tokens > 1 and rng.random() < 0.7,
            "decay": rng.choice([0.0, 1.0, 0.9]), "format": fmt}


# ---- sizes -----------------------------------------------------------------

def _lens(batch, longest):
    """Lengths of a batch: the longest first, the others spread between one and it."""
    return [longest] + [1 + int((longest - 1) * ((b * 0.6180339887498949) % 1.0)) for b in range(1, batch)]


def _groups(case):
    """The sequences at which the groups begin, and the end: groups of different sizes where there are several."""
    n, g = case["batch"], case["groups"]
    cuts = [0] + [max(i, min(n - (g - i), int(n * (i / g) ** 1.3))) for i in range(1, g)] + [n]
    for i in range(1, g):
        cuts[i] = max(cuts[i], cuts[i - 1] + 1)
    return cuts


def _evict_lens(case):
    if not case["ragged"]:
        return [case["longest"]] * case["batch"]
    return _lens(case["batch"], case["longest"])


def _visible(n, tokens, causal):
    """Keys of an own cache of n that all `tokens` queries see together."""
    return sum(min(max(n - tokens + t + 1, 0), n) for t in range(tokens)) if causal else n * tokens


def work(case):
    row = ROW[case["format"]]
    if case["op"] == "evict":
        keep, recent, sinks, nbytes = case["keep"], case["recent"], case["sinks"], 0.0
        for n in _evict_lens(case):
            nbytes += 4
            if n <= keep:
                continue
            # the expected number of rows that move: of the tokens behind the first `keep` slots the latest, and their
            # share of the others that stay (weights do not depend on the place)
            late = min(recent, n - keep)
            rest = max(1, n - sinks - recent)
            moved = late + (keep - sinks - recent) / rest * (n - keep - late)
            nbytes += 8 * n + moved * (2 * row + 8) + 8 * (n - keep)
        return {"bytes": nbytes, "flops": 0}
    tokens, heads = case["tokens"], case["heads"]
    lens = _lens(case["batch"], case["longest"])
    rows = case["batch"] * tokens * heads
    pairs = sum(_visible(n, tokens, case["causal"]) * heads for n in lens)
    keys = sum(lens)
    if case["op"] == "mass":
        sums = 4 * keys * (2 if case["decay"] else 1)
        return {"bytes": rows * (1152 + 4) + keys * row + sums + 4 * (keys // PAGE), "flops": 1152.0 * pairs}
    cuts = _groups(case)
    for g, p in enumerate(_lens(case["groups"], case["prefix"])):
        keys += p
        pairs += p * (cuts[g + 1] - cuts[g]) * tokens * heads
    return {"bytes": rows * (1152 + 1024 + 4) + keys * row + 4 * (keys // PAGE), "flops": 2176.0 * pairs}


# ---- inputs ----------------------------------------------------------------

def _cache(pages, fmt, gen):
    """A pool of pages with normalised latent rows and rotated keys -> (cache, scales or None)."""
    rows = torch.empty(pages, PAGE, D_QK, device="cuda")
    rows.normal_(generator=gen)
    if fmt == "bf16":
        return rows.to(torch.bfloat16), None
    if fmt == "fp8_tensor":
        scale = torch.tensor([1.0 / 64.0], device="cuda")
        return (rows / scale).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale
    tiles = rows[..., :D_LATENT].reshape(pages, PAGE, 4, 128)
    scales = (tiles.abs().amax(-1) / 448.0).contiguous()
    codes = (tiles / scales[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(pages, PAGE, D_LATENT)
    pe = rows[..., D_LATENT:].to(torch.bfloat16).view(torch.uint8)
    return torch.cat([codes, pe], -1), scales


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(n):
    return -(-n // PAGE)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "evict":
        lens, prefixes = _evict_lens(case), []
    else:
        lens = _lens(case["batch"], case["longest"])
        prefixes = _lens(case["groups"], case["prefix"]) if case["op"] == "shared" else []
    B, wide = case["batch"], _pages(max(lens))
    total = sum(_pages(n) for n in lens + prefixes)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    s["cache"], s["scales"] = _cache(total, case["format"], gen)
    s["lens"], s["seqlens"] = lens, _i32(lens)
    s["table"] = torch.zeros(B, wide, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        s["table"][b, :_pages(n)] = order[at:at + _pages(n)]
        at += _pages(n)
    if case["op"] == "evict":
        keep = case["keep"]
        s["mass"] = torch.empty(B, wide * PAGE, device="cuda").normal_(generator=gen).mul_(2.0).exp_()
        pos = torch.arange(wide * PAGE, device="cuda", dtype=torch.int32).repeat(B, 1)
        if case["aged"]:
            # earlier evictions have left older tokens, in no order, in the first `keep` slots; newer ones follow
            kept = min(keep, wide * PAGE)
            for b in range(B):
                pos[b, :kept] = torch.randperm(4 * kept, generator=gen, device="cuda")[:kept].to(torch.int32)
                pos[b, kept:] += 3 * kept
        s["positions"] = pos
        return s
    q = torch.empty(B, case["tokens"], case["heads"], D_QK, device="cuda").normal_(generator=gen).mul_(Q_STD)
    s["q"] = q.to(torch.bfloat16)
    if case["op"] == "shared":
        s["prefixes"], s["prefix_lens"] = prefixes, _i32(prefixes)
        s["cuts"] = _groups(case)
        s["offsets"] = _i32(s["cuts"])
        s["prefix_table"] = torch.zeros(len(prefixes), _pages(max(prefixes)), dtype=torch.int32, device="cuda")
        for g, n in enumerate(prefixes):
            s["prefix_table"][g, :_pages(n)] = order[at:at + _pages(n)]
            at += _pages(n)
        return s
    # the sums that earlier steps have left, and this step's log-sum-exp, as the decode has given it
    s["mass"] = torch.empty(B, wide * PAGE, device="cuda").normal_(generator=gen).exp_()
    s["lse"] = torch.empty(B, case["heads"], case["tokens"], device="cuda")
    for b, n in enumerate(lens):
        k = _rows(s, s["table"][b], n, torch.float32)
        x = _scores(s["q"][b].float(), k, n, case["causal"])
        s["lse"][b] = torch.logsumexp(x, -1).t()
        del x
    return s


# ---- plain forms -----------------------------------------------------------

def _rows(s, pages, n, dtype):
    """The first n cached rows behind a row of a page table, decoded -> [n, 576]."""
    pages = pages[:_pages(n)].long()
    raw, fmt = s["cache"][pages], s["case"]["format"]
    if fmt == "bf16":
        return raw.reshape(-1, D_QK)[:n].to(dtype)
    if fmt == "fp8_tensor":
        return raw.view(torch.float8_e4m3fn).reshape(-1, D_QK)[:n].to(dtype) * s["scales"].to(dtype)
    codes = raw[..., :D_LATENT].contiguous().view(torch.float8_e4m3fn).to(dtype).reshape(-1, 4, 128)
    latent = (codes * s["scales"][pages].to(dtype).reshape(-1, 4, 1)).reshape(-1, D_LATENT)
    pe = raw[..., D_LATENT:].contiguous().view(torch.bfloat16).to(dtype).reshape(-1, D_ROPE)
    return torch.cat([latent, pe], -1)[:n]


def _scores(q, k, n, causal):
    """q [T, H, 576], k [n, 576] -> scaled scores [T, H, n], -inf where a token does not see a key."""
    T = q.shape[0]
    x = torch.matmul(q, k.t()) * SCALE
    if causal and T > 1:
        last = n - T + torch.arange(T, device=q.device)
        x.masked_fill_(torch.arange(n, device=q.device)[None, None, :] > last[:, None, None], -math.inf)
    return x


def _part(x, v):
    """Scores [..., n] and values [n, 512] -> (maximum, sum, weighted sum); a maximum of 0 for a row without keys."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    return m, p.sum(-1, keepdim=True), torch.matmul(p, v)


def _plain_shared(s):
    case = s["case"]
    T, H = case["tokens"], case["heads"]
    out = torch.empty(case["batch"], T, H, D_LATENT, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(case["batch"], H, T, device="cuda")
    for g, n in enumerate(s["prefixes"]):
        b0, b1 = s["cuts"][g], s["cuts"][g + 1]
        k = _rows(s, s["prefix_table"][g], n, torch.float32)
        x = torch.matmul(s["q"][b0:b1].float(), k.t()) * SCALE
        m1, l1, o1 = _part(x, k[:, :D_LATENT])
        del x
        for b in range(b0, b1):
            k = _rows(s, s["table"][b], s["lens"][b], torch.float32)
            m2, l2, o2 = _part(_scores(s["q"][b].float(), k, s["lens"][b], case["causal"]), k[:, :D_LATENT])
            m = torch.maximum(m1[b - b0], m2)
            w1, w2 = torch.exp(m1[b - b0] - m), torch.exp(m2 - m)
            total = w1 * l1[b - b0] + w2 * l2
            out[b] = ((w1 * o1[b - b0] + w2 * o2) / total).to(torch.bfloat16)
            lse[b] = (m + torch.log(total))[..., 0].t()
    return out, lse


def _plain_mass(s):
    case = s["case"]
    mass = s["mass"].clone()
    for b, n in enumerate(s["lens"]):
        k = _rows(s, s["table"][b], n, torch.float32)
        x = _scores(s["q"][b].float(), k, n, case["causal"])
        w = torch.exp(x - s["lse"][b].t()[..., None])
        w = torch.where(x == -math.inf, torch.zeros_like(w), w).sum((0, 1))
        mass[b, :n] = case["decay"] * mass[b, :n] + w if case["decay"] else w
    return mass


def _evict_plan(mass, pos, n, case):
    """Slots that empty and fill: (holes, movers), both ascending, of one sequence of n > keep tokens."""
    keep = case["keep"]
    mass, pos = mass[:n], pos[:n]
    forced = (pos < case["sinks"]) | (pos > pos.amax() - case["recent"])
    order = torch.argsort(mass, descending=True, stable=True)
    order = order[torch.argsort(forced[order].to(torch.int8), descending=True, stable=True)]
    stays = torch.zeros(n, dtype=torch.bool, device=mass.device)
    stays[order[:keep]] = True
    return torch.nonzero(~stays[:keep])[:, 0], torch.nonzero(stays[keep:])[:, 0] + keep


def _evict_out(s, lens, mass, pos):
    c, fmt = s["cache"], s["case"]["format"]
    if fmt == "bf16":
        held = [c]
    elif fmt == "fp8_tensor":
        held = [c.view(torch.float8_e4m3fn)]
    else:
        held = [c[..., :D_LATENT].view(torch.float8_e4m3fn), c[..., D_LATENT:].view(torch.bfloat16), s["scales"]]
    return [lens, mass, pos] + held


def _plain_evict(s):
    case, keep = s["case"], s["case"]["keep"]
    mass, pos = s["mass"].clone(), s["positions"].clone()
    for b, n in enumerate(s["lens"]):
        if n <= keep:
            continue
        holes, movers = _evict_plan(mass[b], pos[b], n, case)
        src, dst = s["table"][b][movers // PAGE].long(), s["table"][b][holes // PAGE].long()
        s["cache"][dst, holes % PAGE] = s["cache"][src, movers % PAGE]
        if case["format"] == "fp8":
            s["scales"][dst, holes % PAGE] = s["scales"][src, movers % PAGE]
        mass[b, holes], pos[b, holes] = mass[b, movers], pos[b, movers]
        mass[b, keep:n], pos[b, keep:n] = 0.0, -1
    return _evict_out(s, s["seqlens"].clamp(max=keep), mass, pos)


def run(s):
    case = s["case"]
    if not own:
        return {"shared": _plain_shared, "mass": _plain_mass, "evict": _plain_evict}[case["op"]](s)
    import mla_decode_attention_05_gb300 as mla
    if case["op"] == "shared":
        return mla.decode_shared(s["q"], s["cache"], s["prefix_table"], s["prefix_lens"], s["table"], s["seqlens"],
                                 softmax_scale=SCALE, group_offsets=s["offsets"], causal=case["causal"], kv_scales=s["scales"])
    if case["op"] == "mass":
        # (the sums are carried on in a copy, so that a pass can be made again)
        mass = s["mass"].clone()
        return mla.attention_mass(s["q"], s["cache"], s["table"], s["seqlens"], s["lse"], mass, softmax_scale=SCALE,
                                  causal=case["causal"], decay=case["decay"], kv_scales=s["scales"])
    # (sums and positions in copies too; the rows that move stay where they were as well, so a pass can be made again)
    mass, pos = s["mass"].clone(), s["positions"].clone()
    lens = mla.evict(s["cache"], s["table"], s["seqlens"], mass, pos, keep=case["keep"], sinks=case["sinks"], recent=case["recent"],
                     kv_scales=s["scales"])
    return _evict_out(s, lens, mass, pos)


# ---- from the definitions, in 64 bits --------------------------------------

def _keys64(s, pages, n):
    """Row by row of the page table, in 64 bits."""
    slots = pages.long()[torch.arange(n, device="cuda") // PAGE] * PAGE + torch.arange(n, device="cuda") % PAGE
    raw = s["cache"].reshape(-1, s["cache"].shape[-1])[slots]
    fmt = s["case"]["format"]
    if fmt == "bf16":
        return raw.double()
    if fmt == "fp8_tensor":
        return raw.view(torch.float8_e4m3fn).double() * float(s["scales"][0])
    k = torch.empty(n, D_QK, dtype=torch.float64, device="cuda")
    per = s["scales"].reshape(-1, 4)[slots].double()
    for t in range(4):
        k[:, 128 * t:128 * t + 128] = raw[:, 128 * t:128 * t + 128].contiguous().view(torch.float8_e4m3fn).double() * per[:, t:t + 1]
    k[:, D_LATENT:] = raw[:, D_LATENT:].contiguous().view(torch.bfloat16).double()
    return k


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s)
    T, H = case["tokens"], case["heads"]
    if case["op"] == "mass":
        mass = s["mass"].double()
        for b, n in enumerate(s["lens"]):
            k = _keys64(s, s["table"][b], n)
            total = torch.zeros(n, dtype=torch.float64, device="cuda")
            for t in range(T):
                sees = max(0, n - T + t + 1) if case["causal"] else n
                x = k[:sees] @ s["q"][b, t].double().t() * SCALE
                total[:sees] += (x - s["lse"][b, :, t].double()).exp().sum(1)
            mass[b, :n] = total + (case["decay"] * mass[b, :n] if case["decay"] else 0.0)
        return mass
    out = torch.empty(case["batch"], T, H, D_LATENT, dtype=torch.float64, device="cuda")
    lse = torch.empty(case["batch"], H, T, dtype=torch.float64, device="cuda")
    for g, n in enumerate(s["prefixes"]):
        prefix = _keys64(s, s["prefix_table"][g], n)
        for b in range(s["cuts"][g], s["cuts"][g + 1]):
            k = torch.cat([prefix, _keys64(s, s["table"][b], s["lens"][b])])
            for t in range(T):
                sees = n + (max(0, s["lens"][b] - T + t + 1) if case["causal"] else s["lens"][b])
                x = s["q"][b, t].double() @ k[:sees].t() * SCALE
                lse[b, :, t] = torch.logsumexp(x, -1)
                out[b, t] = torch.softmax(x, -1) @ k[:sees, :D_LATENT]
    return out, lse


def _exact_evict(s):
    """The rule token by token, on the host."""
    case, keep = s["case"], s["case"]["keep"]
    if sum(s["lens"]) > 400_000:
        return None
    mass, pos, table = s["mass"].cpu(), s["positions"].cpu(), s["table"].cpu().tolist()
    src, dst = [], []
    for b, n in enumerate(s["lens"]):
        if n <= keep:
            continue
        m, p = mass[b, :n].tolist(), pos[b, :n].tolist()
        newest = max(p)
        place = lambda i: table[b][i // PAGE] * PAGE + i % PAGE  # noqa: E731
        rank = sorted(range(n), key=lambda i: (not (p[i] < case["sinks"] or p[i] > newest - case["recent"]), -m[i], i))
        stays = set(rank[:keep])
        holes = [i for i in range(keep) if i not in stays]
        movers = [i for i in range(keep, n) if i in stays]
        for h, i in zip(holes, movers):
            m[h], p[h] = m[i], p[i]
            src.append(place(i))
            dst.append(place(h))
        mass[b, :n] = torch.tensor(m[:keep] + [0.0] * (n - keep))
        pos[b, :n] = torch.tensor(p[:keep] + [-1] * (n - keep), dtype=torch.int32)
    if src:
        src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
        for held in (s["cache"], s["scales"]) if case["format"] == "fp8" else (s["cache"],):
            flat = held.view(-1, held.shape[-1])
            flat[dst] = flat[src].clone()
    return _evict_out(s, torch.tensor([min(n, keep) for n in s["lens"]], dtype=torch.int32), mass, pos)
