"""Cases of the serving-step operators: rotate-and-append, decode attention with lengths on the device, packed prompt attention.

``listed()`` names the measured cases, ``draw(rng)`` gives more of the same ranges, ``prepare`` makes what a serving program has
in hand before the call, ``run`` is one call: the plain form in elementary torch operations, or, where ``own`` is true, the
framework's entry point.  ``work`` counts the bytes and operations a pass cannot do without, ``exact`` evaluates the definition in
64 bits.

Lengths are part of a case (drawn from its ``lens`` number), every value is made from the seed.
"""

import math
import random

import torch

own = False

BLOCK = 64  # tokens of a cache block


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One new token for each of 4 sequences: the rotation and append of a small decode step (latency).
        dict(name="append decode 4", op="append", fp8=False, heads=32, kv_heads=8, dq=128, dv=128, batch=4, new_lo=1, new_hi=1,
             past_lo=100, past_hi=4000, rot=128, rot_start=0, interleaved=False, lens=1),
        # One new token for each of 256 sequences into an E4M3 cache: a full decode step.
        dict(name="append decode 256 fp8", op="append", fp8=True, heads=64, kv_heads=8, dq=128, dv=128, batch=256, new_lo=1, new_hi=1,
             past_lo=500, past_hi=8000, rot=128, rot_start=0, interleaved=False, lens=2),
        # A prefill chunk of 16384 tokens behind a long prefix (the long128k head counts): the largest append.
        dict(name="append chunk 16384", op="append", fp8=False, heads=64, kv_heads=8, dq=128, dv=128, batch=1, new_lo=16384, new_hi=16384,
             past_lo=98304, past_hi=98304, rot=128, rot_start=0, interleaved=False, lens=3),
        # Ragged prompts with the mla24k head shape: only the last 64 of 192 query/key dims rotate, neighbouring dims as pairs.
        dict(name="append ragged mla", op="append", fp8=False, heads=128, kv_heads=128, dq=192, dv=128, batch=7, new_lo=1, new_hi=700,
             past_lo=0, past_hi=900, rot=64, rot_start=128, interleaved=True, lens=4),
        # One sequence of about a thousand keys: the smallest decode call (latency).
        dict(name="decode 1x1000", op="decode", fp8=False, heads=32, kv_heads=8, dq=128, dv=128, batch=1, ctx_lo=1000, ctx_hi=1000, empty=0, lens=5),
        # One sequence at the end of a 128K context: the whole card on one row of the batch.
        dict(name="decode 1x131071", op="decode", fp8=False, heads=64, kv_heads=8, dq=128, dv=128, batch=1, ctx_lo=131071, ctx_hi=131071, empty=0, lens=6),
        # The decode rows of the mixed workload: 256 sequences, 1024 to 32768 keys.
        dict(name="decode 256 mixed", op="decode", fp8=False, heads=32, kv_heads=8, dq=128, dv=128, batch=256, ctx_lo=1024, ctx_hi=32768, empty=0, lens=7),
        # A padded batch over an E4M3 cache: ragged short and middling contexts, 16 empty rows.
        dict(name="decode 200 fp8 ragged", op="decode", fp8=True, heads=64, kv_heads=8, dq=128, dv=128, batch=200, ctx_lo=1, ctx_hi=9000, empty=16, lens=8),
        # One short prompt (latency).
        dict(name="prompt 1x77", op="prompt", heads=32, kv_heads=8, dq=128, dv=128, batch=1, len_lo=77, len_hi=77, lens=9),
        # Packed prompts of very different lengths.
        dict(name="prompt 24 ragged", op="prompt", heads=32, kv_heads=8, dq=128, dv=128, batch=24, len_lo=5, len_hi=2500, lens=10),
        # One long prompt: bound by the tensor cores.
        dict(name="prompt 1x16384", op="prompt", heads=32, kv_heads=8, dq=128, dv=128, batch=1, len_lo=16384, len_hi=16384, lens=11),
        # Prompts with the mla24k head shape: 128 heads of their own keys, 192 query/key dims.
        dict(name="prompt 3 mla", op="prompt", heads=128, kv_heads=128, dq=192, dv=128, batch=3, len_lo=300, len_hi=1900, lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    """Head counts and dims: grouped heads of every group size to 16, one kv head, no grouping."""
    kv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    group = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16])
    while kv * group > 128:
        group = max(1, group // 2)
    dq, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128), (64, 128), (128, 64), (192, 64)])
    return dict(heads=kv * group, kv_heads=kv, dq=dq, dv=dv)


def draw(rng):
    op = rng.choice(["append", "decode", "prompt"])
    h = _heads(rng)
    lens = rng.randrange(1 << 30)
    if op == "append":
        batch = _log(rng, 1, 256)
        new_hi = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, 8192 // batch))
        start = rng.choice([0, h["dq"] // 2]) if rng.random() < 0.4 else 0
        rot = h["dq"] - start if rng.random() < 0.7 else (h["dq"] - start) // 2
        return dict(op="append", fp8=rng.random() < 0.5, **h, batch=batch, new_lo=1, new_hi=new_hi, past_lo=0, past_hi=_log(rng, 1, 4000),
                    rot=rot, rot_start=start, interleaved=rng.random() < 0.5, lens=lens)
    if op == "decode":
        batch = _log(rng, 1, 300)
        most = min(131072, 2_000_000_000 // (batch * h["kv_heads"] * (h["dq"] + h["dv"])))
        hi = _log(rng, 1, max(1, most))
        return dict(op="decode", fp8=rng.random() < 0.5, **h, batch=batch, ctx_lo=max(1, hi // rng.choice([1, 4, 30, hi])), ctx_hi=hi,
                    empty=rng.choice([0, 0, batch // 10]), lens=lens)
    batch = _log(rng, 1, 64)
    most = int(min(8192, math.sqrt(4_000_000_000 / (batch * h["heads"]))))
    hi = _log(rng, 1, most)
    return dict(op="prompt", **h, batch=batch, len_lo=max(1, hi // rng.choice([1, 4, 30, hi])), len_hi=hi, lens=lens)


def _lens(case):
    """The case's lengths: (new tokens, cached tokens before them) of an append, contexts of a decode, prompt lengths."""
    r, n = random.Random(case["lens"]), case["batch"]
    if case["op"] == "append":
        return [_log(r, case["new_lo"], case["new_hi"]) for _ in range(n)], [r.randint(case["past_lo"], case["past_hi"]) for _ in range(n)]
    if case["op"] == "decode":
        ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
        for i in r.sample(range(n), min(case["empty"], n - 1)):
            ctx[i] = 0
        return ctx
    return [_log(r, case["len_lo"], case["len_hi"]) for _ in range(n)]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 12345)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _table(ctx, g):
    """A block table over a shuffled pool that just holds the sequences (unused entries name block 0), and the pool's size."""
    pages = [-(-n // BLOCK) for n in ctx]
    pool, width = max(1, sum(pages)), max(1, max(pages))
    p = torch.tensor(pages, device="cuda")
    order = torch.randperm(pool, generator=g, device="cuda")
    at = torch.cumsum(p, 0)[:, None] - p[:, None] + torch.arange(width, device="cuda")[None, :]
    used = torch.arange(width, device="cuda")[None, :] < p[:, None]
    return torch.where(used, order[at.clamp(max=pool - 1)], 0).to(torch.int32), pool


def _qkv(g, tokens, case):
    """q, k, v as views of one fused projection output."""
    h, kv, dq, dv = case["heads"], case["kv_heads"], case["dq"], case["dv"]
    x = _randn(g, tokens, h * dq + kv * (dq + dv))
    q, k, v = x.split([h * dq, kv * dq, kv * dv], dim=1)
    return q.unflatten(1, (h, dq)), k.unflatten(1, (kv, dq)), v.unflatten(1, (kv, dv))


def _pool(g, blocks, kv, d, fp8):
    """A cache pool of N(0, 1) values, or of E4M3 codes and the scale of each kv head."""
    if not fp8:
        return _randn(g, blocks, BLOCK, kv, d), None
    scale = 0.01 + 0.02 * torch.rand(kv, generator=g, device="cuda")
    x = _randn(g, blocks, BLOCK, kv, d).div_(scale.to(torch.bfloat16)[:, None]).clamp_(-448, 448)
    return x.to(torch.float8_e4m3fn).view(torch.uint8), scale


def _cos_sin(rows, rot):
    """cos and sin of position times frequency, angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    ang = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32)


def prepare(case, seed):
    g = _gen(seed)
    h, kv, dq, dv = case["heads"], case["kv_heads"], case["dq"], case["dv"]
    s = dict(case=case, scale=dq ** -0.5)
    if case["op"] == "append":
        new, past = _lens(case)
        ctx, cu = [a + b for a, b in zip(new, past)], _starts(new)
        s["table"], pool = _table(ctx, g)
        s["q"], s["k"], s["v"] = _qkv(g, cu[-1], case)
        s["kc"], s["ks"] = _pool(g, pool, kv, dq, case["fp8"])
        s["vc"], s["vs"] = _pool(g, pool, kv, dv, case["fp8"])
        s["cu"], s["ctx"] = _i32(cu), _i32(ctx)
        s["cos_sin"] = _cos_sin(-(-max(ctx) // 1024) * 1024, case["rot"])
        s["q_out"] = torch.zeros((cu[-1], h, dq), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "decode":
        ctx = _lens(case)
        s["table"], pool = _table(ctx, g)
        s["q"] = _randn(g, len(ctx), h, dq)
        s["kc"], s["ks"] = _pool(g, pool, kv, dq, case["fp8"])
        s["vc"], s["vs"] = _pool(g, pool, kv, dv, case["fp8"])
        s["ctx"], s["longest"] = _i32(ctx), max(ctx)
        s["out"] = torch.zeros((len(ctx), h, dv), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros((h, len(ctx)), dtype=torch.float32, device="cuda")
    else:
        lens = _lens(case)
        cu = _starts(lens)
        s["q"], s["k"], s["v"] = _qkv(g, cu[-1], case)
        s["cu"], s["longest"] = _i32(cu), max(lens)
        s["out"] = torch.zeros((cu[-1], h, dv), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros((h, cu[-1]), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"append": _append, "decode": _decode, "prompt": _prompt}[s["case"]["op"]](s)


def _append(s):
    c = s["case"]
    if own:
        from chunked_prefill_causal_gb300 import vpp

        if c["fp8"]:
            vpp.vpp_rope_append_fp8(s["q"], s["k"], s["v"], s["cos_sin"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["ctx"],
                                    q_out=s["q_out"], rot_start=c["rot_start"], interleaved=c["interleaved"])
        else:
            vpp.vpp_rope_append(s["q"], s["k"], s["v"], s["cos_sin"], s["kc"], s["vc"], s["table"], s["cu"], s["ctx"],
                                q_out=s["q_out"], rot_start=c["rot_start"], interleaved=c["interleaved"])
    else:
        t = torch.arange(s["q"].shape[0], device="cuda")
        seq = torch.searchsorted(s["cu"][1:], t, right=True)
        pos = s["ctx"][seq] - (s["cu"][seq + 1] - t)
        slot = s["table"][seq, pos // BLOCK].long() * BLOCK + pos % BLOCK
        cos, sin = s["cos_sin"][pos][:, None, :].chunk(2, dim=-1)
        s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, c))
        k, v = _rotate(s["k"].float(), cos, sin, c), s["v"].float()
        if c["fp8"]:
            k = (k / s["ks"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            v = (v / s["vs"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["kc"].flatten(0, 1)[slot] = k.to(s["kc"].dtype)
        s["vc"].flatten(0, 1)[slot] = v.to(s["vc"].dtype)
    held = torch.float8_e4m3fn if c["fp8"] else torch.bfloat16
    return {"q": s["q_out"], "k_cache": s["kc"].view(held), "v_cache": s["vc"].view(held)}


def _rotate(x, cos, sin, c):
    head, mid, tail = x.split([c["rot_start"], c["rot"], x.shape[-1] - c["rot_start"] - c["rot"]], dim=-1)
    if c["interleaved"]:
        a, b = mid[..., 0::2], mid[..., 1::2]
        mid = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = mid.chunk(2, dim=-1)
        mid = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, mid, tail], -1)


def _decode(s):
    c = s["case"]
    if own:
        from chunked_prefill_causal_gb300 import vpp

        if c["fp8"]:
            vpp.vpp_decode_attn_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["ctx"], out=s["out"], lse=s["lse"])
        else:
            vpp.vpp_decode_attn(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    used = s["table"][:, : max(1, -(-s["longest"] // BLOCK))]
    q = s["q"].float().unflatten(1, (c["kv_heads"], -1))
    p = q @ _pages(s["kc"], s["ks"], used).permute(0, 2, 3, 1)  # [batch, kv head, group, key]
    hidden = torch.arange(p.shape[-1], device="cuda")[None, :] >= s["ctx"][:, None]
    p.mul_(s["scale"]).masked_fill_(hidden[:, None, None, :], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top.clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ _pages(s["vc"], s["vs"], used).permute(0, 2, 1, 3)) / total.clamp(min=1e-30)
    s["out"].copy_(o.flatten(1, 2))
    s["lse"].copy_((top + total.log()).flatten(1).t())
    return {"out": s["out"], "lse": s["lse"]}


def _pages(cache, scale, used):
    """The tokens of the named blocks, in 32 bits: [batch, key, kv head, d]."""
    x = cache[used].flatten(1, 2)
    return x.float() if scale is None else x.view(torch.float8_e4m3fn).float().mul_(scale[:, None])


def _prompt(s):
    c = s["case"]
    if own:
        from chunked_prefill_causal_gb300 import vpp

        vpp.vpp_prompt_attn(s["q"], s["k"], s["v"], s["cu"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    tokens, longest = s["q"].shape[0], s["longest"]
    start, length = s["cu"][:-1], s["cu"].diff()
    i = torch.arange(longest, device="cuda")
    at = (start[:, None] + i).clamp(max=tokens - 1)  # the prompts padded to the longest: [batch, token]
    q = s["q"][at].float().unflatten(2, (c["kv_heads"], -1)).permute(0, 2, 3, 1, 4)  # [batch, kv head, group, token, d]
    k = s["k"][at].float().permute(0, 2, 3, 1)[:, :, None]
    p = q @ k
    hidden = (i[None, :] > i[:, None])[None] | (i >= length[:, None])[:, None, :]
    p.mul_(s["scale"]).masked_fill_(hidden[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ s["v"][at].float().permute(0, 2, 1, 3)[:, :, None]) / total
    t = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(s["cu"][1:], t, right=True)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, t - start[seq]])
    s["lse"].copy_((top + total.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)[seq, t - start[seq]].t())
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    h, kv, dq, dv = case["heads"], case["kv_heads"], case["dq"], case["dv"]
    if case["op"] == "append":
        new, past = _lens(case)
        t, width = sum(new), 1 if case["fp8"] else 2
        pages = sum(-(-(a + b) // BLOCK) - b // BLOCK for a, b in zip(new, past))
        moved = t * ((2 * h * dq + kv * (dq + dv)) * 2 + kv * (dq + dv) * width + case["rot"] * 4)
        return dict(bytes=moved + 4 * (pages + 2 * len(new)), flops=3 * t * (h + kv) * case["rot"])
    if case["op"] == "decode":
        ctx = _lens(case)
        n, width = len(ctx), 1 if case["fp8"] else 2
        moved = sum(ctx) * kv * (dq + dv) * width + n * h * ((dq + dv) * 2 + 4) + 4 * sum(-(-x // BLOCK) for x in ctx) + 4 * n
        return dict(bytes=moved, flops=2 * h * (dq + dv) * sum(ctx))
    lens = _lens(case)
    t = sum(lens)
    return dict(bytes=t * ((h + kv) * (dq + dv) * 2 + 4 * h) + 4 * len(lens), flops=h * (dq + dv) * sum(n * (n + 1) for n in lens))


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "prompt": _exact_prompt}[case["op"]](case, s)


def _turn(x, angles, case):
    """Rotates the pairs of a [token, head, d] tensor in 64 bits as complex numbers."""
    r0, r = case["rot_start"], case["rot"]
    i = torch.arange(r // 2, device="cuda")
    a, b = (r0 + 2 * i, r0 + 2 * i + 1) if case["interleaved"] else (r0 + i, r0 + r // 2 + i)
    y = x.double()
    z = torch.complex(y[:, :, a], y[:, :, b]) * angles[:, None, :]
    y[:, :, a], y[:, :, b] = z.real, z.imag
    return y


def _exact_append(case, s):
    new, past = _lens(case)
    turns = torch.complex(*s["cos_sin"].double().chunk(2, dim=1))
    stored = (lambda c: c.view(torch.float8_e4m3fn).double()) if case["fp8"] else (lambda c: c.double())
    kc, vc, q = stored(s["kc"]), stored(s["vc"]), torch.empty_like(s["q"], dtype=torch.float64, memory_format=torch.contiguous_format)
    first = 0
    for b, (n, p) in enumerate(zip(new, past)):
        rows, pos = slice(first, first + n), torch.arange(p, p + n, device="cuda")
        k, v = _turn(s["k"][rows], turns[pos], case), s["v"][rows].double()
        if case["fp8"]:
            k = (k / s["ks"].double()[None, :, None]).clamp(-448, 448)
            v = (v / s["vs"].double()[None, :, None]).clamp(-448, 448)
        block = s["table"][b].long()[pos // BLOCK]
        kc[block, pos % BLOCK], vc[block, pos % BLOCK] = k, v
        q[rows] = _turn(s["q"][rows], turns[pos], case)
        first += n
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _exact_decode(case, s):
    h, kv = case["heads"], case["kv_heads"]
    out = torch.zeros((case["batch"], h, case["dv"]), dtype=torch.float64, device="cuda")
    lse = torch.full((h, case["batch"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        blocks = s["table"][b, : -(-n // BLOCK)].long()
        k, v = s["kc"][blocks].flatten(0, 1)[:n], s["vc"][blocks].flatten(0, 1)[:n]
        if case["fp8"]:
            k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        k, v = k.double(), v.double()
        if case["fp8"]:
            k, v = k * s["ks"].double()[:, None], v * s["vs"].double()[:, None]
        e = torch.einsum("kgd,nkd->kgn", s["q"][b].double().view(kv, h // kv, -1), k) / math.sqrt(case["dq"])
        norm = torch.logsumexp(e, -1)
        out[b] = torch.einsum("kgn,nkd->kgd", (e - norm[..., None]).exp(), v).reshape(h, -1)
        lse[:, b] = norm.reshape(h)
    return {"out": out, "lse": lse}


def _exact_prompt(case, s):
    h, kv = case["heads"], case["kv_heads"]
    tokens = s["q"].shape[0]
    out = torch.zeros((tokens, h, case["dv"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((h, tokens), dtype=torch.float64, device="cuda")
    first = 0
    for n in _lens(case):
        rows = slice(first, first + n)
        above = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
        for j in range(kv):  # one kv head at a time: n x n scores in 64 bits
            mine = slice(j * (h // kv), (j + 1) * (h // kv))
            e = torch.einsum("igd,nd->gin", s["q"][rows, mine].double(), s["k"][rows, j].double()) / math.sqrt(case["dq"])
            e.masked_fill_(above, -math.inf)
            norm = torch.logsumexp(e, -1)
            out[rows, mine] = torch.einsum("gin,nd->igd", e.sub_(norm[..., None]).exp_(), s["v"][rows, j].double())
            lse[mine, rows] = norm
        first += n
    return {"out": out, "lse": lse}
