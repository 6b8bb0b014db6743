"""Measured cases of the operators around the latent attention decode: what
fills the cache (insert with rotation), what reads it for a prompt (expansion
of cached rows to per-head keys and values, and the causal attention over
them) and what follows the decode (projection of its 512-value output rows).

    insert   mla.kv_insert_rope   append rotated keys to the paged cache, rotate the queries
    expand   mla.kv_expand        cached latent rows -> keys and values of every head
    prefill  mla.prefill          attention of a prompt's or a chunk's queries over them
    value    mla.value_project    the decode's latent output rows -> values of every head

With ``own`` false ``run`` computes them from elementary torch operations in
32 bits (64 where a rounding border needs them), with ``own`` true it calls
the library.
"""
import math
import random

import torch

own = False

D_LATENT, D_ROPE, D_NOPE, D_V = 512, 64, 128, 128
D_HEAD = D_NOPE + D_ROPE
PAGE = 64
SCALE = 1.0 / math.sqrt(D_HEAD)
MAX_POS = 32768
EPS = 1e-6
#: 1 / scale of a cache with one scale: normalised rows stay below 448 * 8
K_SCALE_INV = 0.75

#: pairs of queries and keys of the largest prefill case (heads * longest queries * longest keys of every sequence)
MOST_PAIRS = 32 * 8192 * 8192
MOST_ROWS = 16384 * 128   # expand: cached rows * heads
MOST_QROWS = 8191 * 64    # insert and value: tokens * heads


def listed():
    return [
        # one decode step of a batch: new rows of 64 sequences, rotated queries of the absorbed width
        {"name": "insert_step_64_h128", "op": "insert", "tokens": 64, "heads": 128, "width": 576, "format": "bf16", "interleaved": True},
        # a whole prompt into an FP8 cache, an odd token count, queries of the expanded width
        {"name": "insert_prompt_8191_h64_fp8", "op": "insert", "tokens": 8191, "heads": 64, "width": 192, "format": "fp8", "interleaved": True},
        # a single token: latency; the other pairing of the rotation and the one-scale cache
        {"name": "insert_single_h128_fp8t", "op": "insert", "tokens": 1, "heads": 128, "width": 576, "format": "fp8_tensor", "interleaved": False},
        # a long context of one sequence, all heads on one GPU
        {"name": "expand_16384_h128", "op": "expand", "batch": 1, "longest": 16384, "heads": 128, "format": "bf16"},
        # ragged contexts of a batch, the heads of one rank of a larger group, FP8 rows with scales
        {"name": "expand_ragged_16x2000_h8_fp8", "op": "expand", "batch": 16, "longest": 2000, "heads": 8, "format": "fp8"},
        # one short prompt: the weights outweigh the rows
        {"name": "expand_short_100_h64_fp8t", "op": "expand", "batch": 1, "longest": 100, "heads": 64, "format": "fp8_tensor"},
        # one long prompt
        {"name": "prefill_8192_h32", "op": "prefill", "batch": 1, "queries": 8192, "context": 0, "heads": 32, "causal": True},
        # a batch of ragged prompts
        {"name": "prefill_ragged_8x1500_h128", "op": "prefill", "batch": 8, "queries": 1500, "context": 0, "heads": 128, "causal": True},
        # a chunk of new tokens on a long cached context, few heads
        {"name": "prefill_chunk_200_on_12000_h8", "op": "prefill", "batch": 1, "queries": 200, "context": 12000, "heads": 8, "causal": True},
        # the smallest call: a short prompt's queries over all of a short context
        {"name": "prefill_short_77_h8", "op": "prefill", "batch": 2, "queries": 77, "context": 30, "heads": 8, "causal": False},
        # one decode step of a batch
        {"name": "value_64_h128", "op": "value", "tokens": 64, "heads": 128},
        # many query tokens at once (a large batch with several tokens each), an odd count
        {"name": "value_4095_h64", "op": "value", "tokens": 4095, "heads": 64},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["insert", "expand", "prefill", "prefill", "value"])
    heads = rng.choice([1, 4, 8, 20, 32, 64, 128])
    if op == "insert":
        tokens = min(_log(rng, 1, 8191), MOST_QROWS // heads)
        return {"op": op, "tokens": tokens, "heads": heads, "width": rng.choice([192, 576]),
                "format": rng.choice(["bf16", "fp8", "fp8_tensor"]), "interleaved": rng.random() < 0.5}
    if op == "expand":
        batch = _log(rng, 1, 32)
        longest = _log(rng, 1, min(16384, MOST_ROWS // (heads * batch)))
        return {"op": op, "batch": batch, "longest": longest, "heads": heads, "format": rng.choice(["bf16", "fp8", "fp8_tensor"])}
    if op == "prefill":
        batch = _log(rng, 1, 16)
        queries = _log(rng, 1, 4096)
        context = rng.choice([0, _log(rng, 1, 8192)])
        while batch > 1 and batch * heads * queries * (queries + context) > MOST_PAIRS:
            batch = (batch + 1) // 2
        while heads > 1 and batch * heads * queries * (queries + context) > MOST_PAIRS:
            heads = heads // 2
        return {"op": op, "batch": batch, "queries": queries, "context": context, "heads": heads, "causal": rng.random() < 0.7}
    return {"op": op, "tokens": min(_log(rng, 1, 4095), MOST_QROWS // heads), "heads": heads}


def _lens(batch, longest):
    """Lengths of a batch: the longest first, the others spread between one and it."""
    return [longest] + [1 + int((longest - 1) * ((b * 0.6180339887498949) % 1.0)) for b in range(1, batch)]


def _prefill_lens(case):
    """Queries and keys of each sequence: every sequence has up to `context` keys before its queries."""
    nq = _lens(case["batch"], case["queries"])
    ctx = _lens(case["batch"], case["context"]) if case["context"] else [0] * case["batch"]
    return nq, [q + c for q, c in zip(nq, ctx)]


def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return c


ROW = {"bf16": 1152, "fp8": 640, "fp8_tensor": 576}


def work(case):
    h = case["heads"]
    if case["op"] == "insert":
        n = case["tokens"]
        row = ROW[case["format"]] + (16 if case["format"] == "fp8" else 0)
        # latent and key in, slot and position, one row of the angle table, the cache row, the queries in and out
        return {"bytes": n * (1152 + 16 + 256 + row + h * 4 * D_ROPE) + 1024, "flops": n * (4 * D_LATENT + 3 * D_ROPE + 3 * D_ROPE * h)}
    if case["op"] == "expand":
        n = sum(_lens(case["batch"], case["longest"]))
        row = ROW[case["format"]] + (16 if case["format"] == "fp8" else 0)
        return {"bytes": n * (row + 512 * h + 128) + h * 256 * 512 * 2, "flops": 2 * n * h * 256 * 512}
    if case["op"] == "prefill":
        nq, nk = _prefill_lens(case)
        pairs = sum(q * k - (q * (q - 1) // 2 if case["causal"] else 0) for q, k in zip(nq, nk))
        return {"bytes": sum(nq) * h * (D_HEAD + D_V) * 2 + sum(nq) * h * 4 + sum(nk) * (h * (D_NOPE + D_V) + D_ROPE) * 2,
                "flops": 2 * pairs * h * (D_HEAD + D_V)}
    n = case["tokens"]
    return {"bytes": n * h * (D_LATENT + D_V) * 2 + h * D_V * D_LATENT * 2, "flops": 2 * n * h * D_V * D_LATENT}


def _normal(g, shape, std):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _angles():
    """cos and sin of every position, fp32 [MAX_POS, 64] (cosines first), from angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, D_ROPE, 2, dtype=torch.float64, device="cuda") / D_ROPE)
    a = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = case["heads"]
    s = dict(case)
    if case["op"] == "insert":
        n = case["tokens"]
        pages = n // 48 + 2
        # rows of the fused projection, of a size of their own each, as a layer gives them
        qkv = _normal(g, (n, 2112), 1.0) * torch.exp2(torch.rand((n, 1), generator=g, device="cuda") * 6 - 4).to(torch.bfloat16)
        slots = torch.randperm(pages * PAGE - 1, generator=g, device="cuda")[:n].contiguous()
        slots[8::9] = -1  # a padded batch
        s.update(kv_c=qkv[:, 1536:2048], k_pe=qkv[:, 2048:], w=(1 + 0.25 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16),
                 slots=slots, positions=torch.randint(0, MAX_POS, (n,), generator=g, device="cuda"), cos_sin=_angles(),
                 q=_normal(g, (n, h, case["width"]), 1.0), q_out=torch.zeros((n, h, D_ROPE), dtype=torch.bfloat16, device="cuda"),
                 cache=torch.zeros((pages, PAGE, 576), dtype=torch.bfloat16, device="cuda") if case["format"] == "bf16"
                 else torch.zeros((pages, PAGE, ROW[case["format"]]), dtype=torch.uint8, device="cuda"),
                 scales=torch.zeros((pages, PAGE, 4), device="cuda") if case["format"] == "fp8" else None,
                 ksi=torch.tensor([K_SCALE_INV], device="cuda") if case["format"] == "fp8_tensor" else None)
    elif case["op"] == "expand":
        lens = _lens(case["batch"], case["longest"])
        per = [-(-n // PAGE) for n in lens]
        pages = sum(per) + 3
        ids = torch.randperm(pages, generator=g, device="cuda").int()
        table = torch.full((len(lens), max(per)), -1, dtype=torch.int32, device="cuda")
        at = _cu(per)
        for b, n in enumerate(per):
            table[b, :n] = ids[at[b]:at[b] + n]
        x = torch.randn((pages, PAGE, 576), generator=g, device="cuda")
        scales = None
        if case["format"] == "bf16":
            cache = x.to(torch.bfloat16)
        elif case["format"] == "fp8":
            scales = x[..., :512].reshape(pages, PAGE, 4, 128).abs().amax(-1) / 448
            codes = (x[..., :512].reshape(pages, PAGE, 4, 128) / scales[..., None]).to(torch.float8_e4m3fn).reshape(pages, PAGE, 512)
            cache = torch.cat([codes.view(torch.uint8), x[..., 512:].to(torch.bfloat16).view(torch.uint8)], 2)
        else:
            scales = torch.full((1,), 1 / K_SCALE_INV, device="cuda")
            cache = (x * K_SCALE_INV).to(torch.float8_e4m3fn).view(torch.uint8)
        s.update(cache=cache, scales=scales, table=table, cu=torch.tensor(_cu(lens), dtype=torch.int32, device="cuda"), total=sum(lens),
                 w_uk=_normal(g, (h, D_NOPE, 512), 1 / math.sqrt(512)), w_uv=_normal(g, (h, D_V, 512), 1 / math.sqrt(512)))
    elif case["op"] == "prefill":
        nq, nk = _prefill_lens(case)
        kv = _normal(g, (sum(nk), h, D_NOPE + D_V), 1.0)
        s.update(q=_normal(g, (sum(nq), h, D_HEAD), 1.5), k_nope=kv[..., :D_NOPE], v=kv[..., D_NOPE:], k_pe=_normal(g, (sum(nk), D_ROPE), 1.0),
                 cu_q=torch.tensor(_cu(nq), dtype=torch.int32, device="cuda"), cu_k=torch.tensor(_cu(nk), dtype=torch.int32, device="cuda"),
                 most_q=max(nq), most_k=max(nk))
    else:
        s.update(attn=_normal(g, (case["tokens"], h, 512), 0.5), w_uv=_normal(g, (h, D_V, 512), 1 / math.sqrt(512)))
    return s


def run(s):
    return {"insert": _insert, "expand": _expand, "prefill": _prefill, "value": _value}[s["op"]](s)


def _cache_parts(s):
    """The cache by what its bytes hold: bf16 rows; e4m3 codes, bf16 keys and scales; or e4m3 codes."""
    c = s["cache"]
    if s["format"] == "bf16":
        return [c]
    if s["format"] == "fp8":
        return [c[..., :512].view(torch.float8_e4m3fn), c[..., 512:].view(torch.bfloat16), s["scales"]]
    return [c.view(torch.float8_e4m3fn)]


def _rotate(x, cs, interleaved):
    """Rotates the 32 pairs of the last axis of x (fp32) by the angles of cs."""
    c, sn = cs[..., :32], cs[..., 32:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * c - b * sn, a * sn + b * c], -1)


def _insert(s):
    if own:
        import mla_decode_attention_05_gb300 as mla
        mla.kv_insert_rope(s["kv_c"], s["k_pe"], s["w"], s["slots"], s["cache"], eps=EPS, positions=s["positions"], cos_sin=s["cos_sin"],
                           interleaved=s["interleaved"], q_pe=s["q"][..., -D_ROPE:], q_out=s["q_out"], kv_scales=s["scales"],
                           k_scale_inv=s["ksi"], fp8_per_tensor=s["format"] == "fp8_tensor")
        return _cache_parts(s) + [s["q_out"]]
    cs = s["cos_sin"][s["positions"]]
    x = s["kv_c"].float()
    # the rounding of a normalised value to the row's 16 bits, and of the row's largest to its scale, lies next to a border: the sum in 64 bits
    mean = (x.double().square().sum(1, keepdim=True) / 512).float() + EPS
    n = ((x * s["w"].float()) * (1.0 / mean.sqrt())).to(torch.bfloat16)
    pe = _rotate(s["k_pe"].float(), cs, s["interleaved"]).to(torch.bfloat16)
    s["q_out"].copy_(_rotate(s["q"][..., -D_ROPE:].float(), cs[:, None], s["interleaved"]))
    if s["format"] == "bf16":
        row = torch.cat([n, pe], 1)
    elif s["format"] == "fp8":
        t = n.float().view(-1, 4, 128)
        sc = (t.abs().amax(2) / 448).clamp_min(2.0 ** -126)
        codes = (t * (1.0 / sc)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 512)
        row = torch.cat([codes, pe.view(torch.uint8)], 1)
    else:
        row = (torch.cat([n, pe], 1).float() * s["ksi"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    # a token without a slot writes back what the pool's last slot (never given out) holds
    flat = s["cache"].view(-1, s["cache"].shape[2])
    skip = (s["slots"] < 0)[:, None]
    at = torch.where(skip[:, 0], flat.shape[0] - 1, s["slots"])
    flat[at] = torch.where(skip, flat[-1], row)
    if s["format"] == "fp8":
        fs = s["scales"].view(-1, 4)
        fs[at] = torch.where(skip, fs[-1], sc)
    return _cache_parts(s) + [s["q_out"]]


def _expand(s):
    if own:
        import mla_decode_attention_05_gb300 as mla
        return mla.kv_expand(s["cache"], s["table"], s["cu"], s["w_uk"], s["w_uv"], total=s["total"], kv_scales=s["scales"])
    cu = s["cu"].long()
    r = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu[1:], r, right=True)
    pos = r - cu[b]
    slot = s["table"][b, pos // PAGE].long() * PAGE + pos % PAGE
    rows = s["cache"].view(-1, s["cache"].shape[2])[slot]
    if s["format"] == "bf16":
        lat, pe = rows[:, :512].float(), rows[:, 512:]
    elif s["format"] == "fp8":
        sc = s["scales"].view(-1, 4)[slot]
        lat = (rows[:, :512].view(torch.float8_e4m3fn).float().view(-1, 4, 128) * sc[..., None]).view(-1, 512)
        pe = rows[:, 512:].contiguous().view(torch.bfloat16)
    else:
        x = rows.view(torch.float8_e4m3fn).float() * s["scales"]
        lat, pe = x[:, :512], x[:, 512:].to(torch.bfloat16)
    w = torch.cat([s["w_uk"], s["w_uv"]], 1).float().view(-1, 512)
    return (lat @ w.T).to(torch.bfloat16).view(s["total"], -1, 256), pe.contiguous()


def _prefill(s):
    if own:
        import mla_decode_attention_05_gb300 as mla
        return mla.prefill(s["q"], s["k_nope"], s["k_pe"], s["v"], s["cu_q"], s["cu_k"], softmax_scale=SCALE, causal=s["causal"])
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cq.diff(), ck.diff()
    iq, ik = torch.arange(s["most_q"], device="cuda"), torch.arange(s["most_k"], device="cuda")
    # every sequence padded to the longest: rows [batch, length]
    rq = (cq[:-1, None] + iq).clamp_max(s["q"].shape[0] - 1)
    rk = (ck[:-1, None] + ik).clamp_max(s["v"].shape[0] - 1)
    k = torch.cat([s["k_nope"], s["k_pe"][:, None].expand(-1, s["heads"], -1)], 2)[rk].float()
    sc = torch.einsum("bqhd,bkhd->bhqk", s["q"][rq].float(), k).mul_(SCALE)
    most = lk[:, None] - lq[:, None] + iq + 1 if s["causal"] else lk[:, None].expand(-1, s["most_q"])
    seen = ik < torch.minimum(most, lk[:, None])[:, :, None]
    sc.masked_fill_(~seen[:, None], -math.inf)
    m = sc.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = sc.sub_(m).exp_()
    z = p.sum(3)
    o = torch.einsum("bhqk,bkhd->bqhd", p, s["v"][rk].float()) / torch.where(z > 0, z, 1.0).transpose(1, 2)[..., None]
    lse = m[..., 0] + z.log()
    # back to packed rows
    r = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cq[1:], r, right=True)
    return o[b, r - cq[b]].to(torch.bfloat16), lse[b, :, r - cq[b]].T.contiguous()


def _value(s):
    if own:
        import mla_decode_attention_05_gb300 as mla
        return mla.value_project(s["attn"], s["w_uv"])
    return torch.einsum("nhl,hvl->nhv", s["attn"].float(), s["w_uv"].float()).to(torch.bfloat16)


def exact(case, seed):
    """The outputs in 64 bits.  The scales of an FP8 row have no such value
    here: they follow the largest of the row's 16-bit values, and which way
    that one was rounded."""
    s = prepare(case, seed)
    h, d = case["heads"], torch.float64
    if case["op"] == "insert":
        def turned(x, axis_heads):
            theta = torch.outer(s["positions"].to(d), torch.pow(torch.tensor(10000.0, dtype=d, device="cuda"), -torch.arange(32, dtype=d, device="cuda") / 32))
            z = torch.polar(torch.ones_like(theta), theta)
            z = z[:, None] if axis_heads else z
            if case["interleaved"]:
                return torch.view_as_real(torch.view_as_complex(x.to(d).unflatten(-1, (32, 2)).contiguous()) * z).flatten(-2)
            y = torch.complex(x[..., :32].to(d), x[..., 32:].to(d)) * z
            return torch.cat([y.real, y.imag], -1)

        x = s["kv_c"].to(d)
        n = x * s["w"].to(d) / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
        pe = turned(s["k_pe"], False)
        live = s["slots"] >= 0
        slots = s["slots"][live]

        def laid(rows):
            c = torch.zeros((s["cache"].shape[0] * PAGE, rows.shape[1]), dtype=d, device="cuda")
            c[slots] = rows[live]
            return c.view(-1, PAGE, rows.shape[1])

        if case["format"] == "bf16":
            parts = [laid(torch.cat([n, pe], 1))]
        elif case["format"] == "fp8":
            top = n.unflatten(1, (4, 128)).abs().max(2, keepdim=True).values
            parts = [laid((n.unflatten(1, (4, 128)) * 448 / top).flatten(1)), laid(pe), None]
        else:
            parts = [laid(torch.cat([n, pe], 1) * K_SCALE_INV)]
        return parts + [turned(s["q"][..., -D_ROPE:], True)]
    if case["op"] == "expand":
        lens = _lens(case["batch"], case["longest"])
        c = s["cache"]
        if case["format"] == "bf16":
            x = c.to(d)
        elif case["format"] == "fp8":
            lat = c[..., :512].view(torch.float8_e4m3fn).to(d).unflatten(2, (4, 128)) * s["scales"].to(d)[..., None]
            x = torch.cat([lat.flatten(2), c[..., 512:].view(torch.bfloat16).to(d)], 2)
        else:
            x = c.view(torch.float8_e4m3fn).to(d) * s["scales"].to(d)
        x = torch.cat([x[s["table"][b, :-(-n // PAGE)].long()].flatten(0, 1)[:n] for b, n in enumerate(lens)])
        kv = torch.empty((len(x), h, 256), dtype=d, device="cuda")
        for i in range(h):
            kv[:, i, :D_NOPE] = x[:, :512] @ s["w_uk"][i].to(d).T
            kv[:, i, D_NOPE:] = x[:, :512] @ s["w_uv"][i].to(d).T
        return kv, x[:, 512:].contiguous()
    if case["op"] == "prefill":
        nq, nk = _prefill_lens(case)
        cq, ck = _cu(nq), _cu(nk)
        out = torch.zeros((cq[-1], h, D_V), dtype=d, device="cuda")
        lse = torch.full((h, cq[-1]), -math.inf, dtype=d, device="cuda")
        for b in range(len(nq)):
            rows, keys = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
            hidden = torch.ones((nq[b], nk[b]), dtype=torch.bool, device="cuda").triu(nk[b] - nq[b] + 1) if case["causal"] else None
            for i in range(h):
                t = (s["q"][rows, i, :D_NOPE].to(d) @ s["k_nope"][keys, i].to(d).T + s["q"][rows, i, D_NOPE:].to(d) @ s["k_pe"][keys].to(d).T) * SCALE
                if hidden is not None:
                    t[hidden] = -math.inf
                lse[i, rows] = torch.logsumexp(t, 1)
                out[rows, i] = torch.softmax(t, 1) @ s["v"][keys, i].to(d)
        return out, lse
    return torch.stack([s["attn"][:, i].to(d) @ s["w_uv"][i].to(d).T for i in range(h)], 1)
