"""The prompt and cache-eviction operators beside the decode step, as a serving program calls them.

Rotary positions fused with the append, attention over packed prompts and over a chunk of new tokens of a paged cache,
attention with the weights accumulated per cached position (one new token, or the last tokens of a prompt), and eviction
of the least attended positions.  Each case is one call on seeded inputs; `run` has the plain form in elementary torch
operations and the call of the package.  Cache tensors are fp16 [num_blocks, num_kv_heads, block_size, 128], scattered
block tables, scores float32 [num_seqs, num_kv_heads, capacity].
"""
import math

import torch

own = False

D = 128
DEV = "cuda"
F16, F32, F64 = torch.float16, torch.float32, torch.float64


def listed():
    return [
        # the smallest call: one decode step of a small batch, whole heads rotated, half layout
        dict(name="rope_append_step", op="rope_append", tokens=16, hq=32, hkv=8, rotary=128, interleaved=False,
             block=16, fused=False, far=4096, method="none"),
        # a prompt chunk straight out of a fused q/k/v projection (strided rows), part of the head rotated, pairs interleaved
        dict(name="rope_append_prompt", op="rope_append", tokens=8192, hq=32, hkv=8, rotary=64, interleaved=True,
             block=16, fused=True, far=8192, method="none"),
        # rotation alone (before an 8-bit append), far positions of a scaled long context, an odd number of tokens
        dict(name="rope_far", op="rope", tokens=4099, hq=32, hkv=32, rotary=128, interleaved=False,
             block=0, fused=True, far=1000000, method="ramp"),
        # sixteen user prompts of very different lengths packed into one call
        dict(name="prompts_ragged", op="prefill", seqs=16, longest=1000, shortest=17, hq=32, hkv=8, fused=True),
        # one long document
        dict(name="prompt_long", op="prefill", seqs=1, longest=16384, shortest=16384, hq=32, hkv=8, fused=False),
        # chunked prefill: four requests each add a chunk behind what their cache holds
        dict(name="chunk_2k", op="chunk", seqs=4, chunk=2048, context=8192, hq=32, hkv=8, block=16),
        # a follow-up question of some tens of tokens behind a very long document: few rows, a long axis
        dict(name="chunk_few_rows", op="chunk", seqs=2, chunk=37, context=32768, hq=32, hkv=8, block=64),
        # decode steps that keep the attention each position received (the decode workloads' sizes)
        dict(name="step_weights", op="step_weights", seqs=64, context=2049, ragged=False, hq=32, hkv=8, block=16),
        dict(name="step_weights_long", op="step_weights", seqs=4, context=32768, ragged=True, hq=32, hkv=8, block=32),
        # the weights that a prompt's last tokens give to its cached positions, before the first eviction
        dict(name="prompt_weights", op="prompt_weights", seqs=2, chunk=256, context=16384, hq=32, hkv=8, block=16),
        # long documents cut to a budget, into blocks of their own (the old ones are shared with other requests)
        dict(name="evict_fork", op="evict", seqs=4, context=32768, budget=4096, recent=512, sinks=4, hkv=8, block=16, in_place=False),
        # a batch of chats cut back in place
        dict(name="evict_in_place", op="evict", seqs=16, context=3900, budget=1024, recent=256, sinks=0, hkv=8, block=16, in_place=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_append", "rope", "prefill", "prefill", "chunk", "chunk", "step_weights", "step_weights",
                     "prompt_weights", "evict", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    block = rng.choice([16, 32, 48, 64, 128, 256])
    if op in ("rope_append", "rope"):
        return dict(op=op, tokens=_log(rng, 1, 8192), hq=hq, hkv=hkv, rotary=rng.choice([16, 32, 64, 96, 128]),
                    interleaved=rng.random() < 0.5, block=block if op == "rope_append" else 0, fused=rng.random() < 0.5,
                    far=_log(rng, 4096, 1000000), method=rng.choice(["none", "linear", "base", "bands", "ramp"]))
    if op == "prefill":
        longest = _log(rng, 1, 8192)
        most = 16384 * 16384 * 32 // (longest * longest * hq)  # no more work than the long document's
        return dict(op=op, seqs=_log(rng, 1, max(1, min(16, most))), longest=longest, shortest=_log(rng, 1, longest), hq=hq, hkv=hkv,
                    fused=rng.random() < 0.5)
    if op == "chunk":
        context = _log(rng, 64, 32768)
        chunk = _log(rng, 1, min(context, 2048))
        most = 16384 * 8192 * 32 // (chunk * context * hq)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(4, most))), chunk=chunk, context=context, hq=hq, hkv=hkv, block=block)
    if op == "step_weights":
        context = _log(rng, 16, 32768)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(64, 131072 // context))), context=context, ragged=rng.random() < 0.7,
                    hq=hq, hkv=hkv, block=block)
    if op == "prompt_weights":
        context = _log(rng, 64, 16384)
        return dict(op=op, seqs=_log(rng, 1, 4), chunk=_log(rng, 1, min(context, 512)), context=context, hq=hq, hkv=hkv,
                    block=block)
    context = _log(rng, 64, 32768)
    budget = _log(rng, 16, context)
    recent = rng.randint(0, budget // 2)
    return dict(op=op, seqs=_log(rng, 1, max(1, min(16, 131072 // context))), context=context, budget=budget, recent=recent,
                sinks=rng.randint(0, min(8, budget - recent)), hkv=hkv, block=block, in_place=rng.random() < 0.5)


# ---------------------------------------------------------------- sizes and inputs

def _lens(case):
    """The lengths of a case's requests, spread between its shortest and its longest."""
    n = case["seqs"]
    if case["op"] == "prefill":
        lo, hi = case["shortest"], case["longest"]
    elif case["op"] == "step_weights":
        lo, hi = (case["context"] // 4 + 1 if case["ragged"] else case["context"]), case["context"]
    elif case["op"] == "evict":
        lo, hi = case["context"] // 2 + 1, case["context"]
    else:
        lo, hi = case["context"] // 2 + 1, case["context"]
    lo = min(lo, hi)
    return [hi - (hi - lo) * ((5 * i) % n) // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _chunks(case, lens):
    return [max(1, min(c, case["chunk"] - (3 * i) % max(1, case["chunk"] // 4 + 1))) for i, c in enumerate(lens)]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32).to(F16)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tables(g, lens, block, spare=0, times=1):
    """`times` block tables per request over one pool in random order, and the pool's size."""
    need = [-(-n // block) for n in lens]
    width, total = max(1, max(need)), times * sum(need) + spare
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    tables, at = [], 0
    for _ in range(times):
        t = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
        for b, n in enumerate(need):
            t[b, :n] = perm[at:at + n]
            at += n
        tables.append(t)
    return tables, total


def _rope_spec(case):
    d, base = case["rotary"], 10000.0
    if case["method"] == "none":
        return dict(rotary_dim=d, base=base)
    return dict(rotary_dim=d, base=base, method=case["method"], factor=8.0, original_context=4096)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case), "op": op, "scale": D ** -0.5}
    if op in ("rope", "rope_append"):
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        if case["fused"]:
            qkv = _randn(g, t, hq + 2 * hkv, D)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = _randn(g, t, hq, D), _randn(g, t, hkv, D), _randn(g, t, hkv, D)
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV, dtype=torch.int32)
        s["q_out"] = torch.empty((t, hq, D), dtype=F16, device=DEV)
        if op == "rope":
            s["k_out"] = torch.empty((t, hkv, D), dtype=F16, device=DEV)
        else:
            nb = -(-t // case["block"]) + 3
            s["k_cache"], s["v_cache"] = _randn(g, nb, hkv, case["block"], D), _randn(g, nb, hkv, case["block"], D)
            s["slots"] = torch.randperm(nb * case["block"], generator=g, device=DEV)[:t].contiguous()
            if t > 8:
                s["slots"][t // 2] = -1  # a padding token
        return s
    lens = _lens(case)
    s["lens"] = lens
    if op == "prefill":
        t, hq, hkv = sum(lens), case["hq"], case["hkv"]
        if case["fused"]:
            qkv = _randn(g, t, hq + 2 * hkv, D)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = _randn(g, t, hq, D), _randn(g, t, hkv, D), _randn(g, t, hkv, D)
        s["start"] = _int([sum(lens[:i]) for i in range(len(lens) + 1)])
        s["out"] = torch.empty((t, hq, D), dtype=F16, device=DEV)
        return s
    hkv, block = case["hkv"], case["block"]
    fork = op == "evict" and not case["in_place"]
    tables, nb = _tables(g, lens, block, spare=2, times=2 if fork else 1)
    s["tables"], s["ctx"] = tables[0], _int(lens)
    s["k_cache"], s["v_cache"] = _randn(g, nb, hkv, block, D), _randn(g, nb, hkv, block, D)
    s["cap"] = cap = tables[0].shape[1] * block
    if op == "evict":
        # accumulated weights: a few heavy positions, a long light tail, some never attended (ties at zero)
        x = torch.randn((len(lens), hkv, cap), generator=g, device=DEV, dtype=F32)
        s["scores"] = torch.where(x > -1.5, torch.exp(2.0 * x), torch.zeros_like(x))
        s["new_tables"] = tables[1] if fork else tables[0]
        s["new_scores"] = torch.empty_like(s["scores"])
        s["new_ctx"] = torch.empty_like(s["ctx"])
        s["kept"] = torch.empty((len(lens), hkv, case["budget"]), dtype=torch.int32, device=DEV)
        return s
    hq = case["hq"]
    if op in ("step_weights", "prompt_weights"):
        s["scores"] = torch.rand((len(lens), hkv, cap), generator=g, device=DEV, dtype=F32) * 4.0
    if op == "step_weights":
        s["q"] = _randn(g, len(lens), hq, D)
        s["out"] = torch.empty_like(s["q"])
        return s
    s["chunks"] = chunks = _chunks(case, lens)
    s["start"] = _int([sum(chunks[:i]) for i in range(len(chunks) + 1)])
    s["q"] = _randn(g, sum(chunks), hq, D)
    s["lse"] = torch.empty((sum(chunks), hq), dtype=F32, device=DEV)
    if op == "prompt_weights":
        _chunk(s, None, s["lse"])  # as the attention over the chunk left it
    else:
        s["out"] = torch.empty_like(s["q"])
    return s


# ---------------------------------------------------------------- the plain forms

def _frequencies(case):
    """Rotations per position in radians, float64 [rotary / 2], and the factor on cos and sin."""
    d, base, s, ctx = case["rotary"], 10000.0, 8.0, 4096
    i = torch.arange(0, d, 2, dtype=F64, device=DEV)
    f = base ** (-i / d)
    m = case["method"]
    if m == "linear":
        return f / s, 1.0
    if m == "base":
        return (base * s ** (d / (d - 2))) ** (-i / d), 1.0
    if m == "bands":  # wavelengths over ctx / 1 are stretched, under ctx / 4 kept, between them blended
        turns = ctx * f / (2 * math.pi)
        keep = torch.clamp((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return keep * f + (1 - keep) * f / s, 1.0
    if m == "ramp":  # blended over the index between 32 turns and 1 turn over the original context
        at = lambda turns: d * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), d - 1)
        keep = 1 - torch.clamp((i / 2 - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return keep * f + (1 - keep) * f / s, 0.1 * math.log(s) + 1.0
    return f, 1.0


def _rotate(x, positions, freq, magnitude, case):
    r = case["rotary"]
    angle = positions.to(F64)[:, None] * freq
    cos, sin = (torch.cos(angle) * magnitude).to(F32)[:, None], (torch.sin(angle) * magnitude).to(F32)[:, None]
    y = x.to(F32).clone()
    if case["interleaved"]:
        a, b = y[..., 0:r:2].clone(), y[..., 1:r:2].clone()
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., :r // 2].clone(), y[..., r // 2:r].clone()
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    return y.to(F16)


def _attend(q, k, v, scale):
    """q [n, Hq, D] are the last n of the positions of k, v [m, Hkv, D]; out [n, Hq, D] and the log of the sums, in 32 bits."""
    n, hq, _ = q.shape
    m, hkv, _ = k.shape
    kt, vt = k.to(F32).permute(1, 2, 0), None if v is None else v.to(F32).permute(1, 0, 2)
    out, lse = [], []
    rows = max(1, min(n, (1 << 27) // (hq * m)))
    for i in range(0, n, rows):
        x = q[i:i + rows].to(F32)
        c, e = x.shape[0], m - n + min(n, i + rows)  # keys up to e are visible to some row
        x = x.view(c, hkv, hq // hkv, D).permute(1, 2, 0, 3).reshape(hkv, -1, D)
        p = torch.matmul(x, kt[:, :, :e]).mul_(scale).view(hkv, hq // hkv, c, e)
        p.masked_fill_(torch.arange(e, device=DEV) > m - n + torch.arange(i, i + c, device=DEV)[:, None], -math.inf)
        top = p.amax(-1, keepdim=True)
        p.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        lse.append((top + total.log()).view(hq, c).t())
        if vt is not None:
            o = torch.matmul(p.view(hkv, -1, e), vt[:, :e]).view(hkv, hq // hkv, c, D) / total
            out.append(o.permute(2, 0, 1, 3).reshape(c, hq, D).to(F16))
    return torch.cat(out) if out else None, torch.cat(lse)


def _rows(cache, table, n):
    """The first n positions of one request's cache as [n, Hkv, D]."""
    block = cache.shape[2]
    return cache[table[:-(-n // block)].long()].permute(0, 2, 1, 3).reshape(-1, cache.shape[1], D)[:n]


def _chunk(s, out, lse):
    at = 0
    for b, (n, c) in enumerate(zip(s["lens"], s["chunks"])):
        v = None if out is None else _rows(s["v_cache"], s["tables"][b], n)
        o, z = _attend(s["q"][at:at + c], _rows(s["k_cache"], s["tables"][b], n), v, s["scale"])
        lse[at:at + c] = z
        if out is not None:
            out[at:at + c] = o
        at += c


def _plain(s):
    op, case = s["op"], s["case"]
    if op in ("rope", "rope_append"):
        freq, magnitude = _frequencies(case)
        s["q_out"].copy_(_rotate(s["q"], s["positions"], freq, magnitude, case))
        k = _rotate(s["k"], s["positions"], freq, magnitude, case)
        if op == "rope":
            s["k_out"].copy_(k)
            return s["q_out"], s["k_out"]
        live = s["slots"] >= 0
        block, slot = case["block"], s["slots"][live]
        s["k_cache"][slot // block, :, slot % block] = k[live]
        s["v_cache"][slot // block, :, slot % block] = s["v"][live]
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "prefill":
        at = 0
        for n in s["lens"]:
            s["out"][at:at + n] = _attend(s["q"][at:at + n], s["k"][at:at + n], s["v"][at:at + n], s["scale"])[0]
            at += n
        return s["out"]
    if op == "chunk":
        _chunk(s, s["out"], s["lse"])
        return s["out"], s["lse"]
    if op in ("step_weights", "prompt_weights"):
        at = 0
        for b, n in enumerate(s["lens"]):
            c = 1 if op == "step_weights" else s["chunks"][b]
            q, k = s["q"][at:at + c], _rows(s["k_cache"], s["tables"][b], n)
            hkv = k.shape[1]
            if op == "step_weights":
                o, lse = _attend(q, k, _rows(s["v_cache"], s["tables"][b], n), s["scale"])
                s["out"][at:at + c] = o
            else:
                lse = s["lse"][at:at + c]
            x = q.to(F32).view(c, hkv, -1, D).permute(1, 2, 0, 3).reshape(hkv, -1, D)
            p = torch.matmul(x, k.to(F32).permute(1, 2, 0)).mul_(s["scale"]).view(hkv, -1, c, n)
            p = (p - lse.view(c, hkv, -1).permute(1, 2, 0)[..., None]).exp_()
            p.masked_fill_(torch.arange(n, device=DEV) > n - c + torch.arange(c, device=DEV)[:, None], 0.0)
            s["scores"][b, :, :n] += p.sum((1, 2))
            at += c
        return (s["out"], s["scores"]) if op == "step_weights" else s["scores"]
    # evict
    budget, recent, sinks, block = case["budget"], case["recent"], case["sinks"], case["block"]
    s["new_scores"].zero_()
    s["kept"].fill_(-1)
    for b, n in enumerate(s["lens"]):
        m = min(n, budget)
        key = s["scores"][b, :, :n].clone()
        key[:, max(0, n - recent):] = math.inf  # always kept
        key[:, :min(sinks, n)] = math.inf
        keep = key.sort(dim=-1, descending=True, stable=True)[1][:, :m].sort(dim=-1)[0]
        s["kept"][b, :, :m] = keep
        s["new_scores"][b, :, :m] = s["scores"][b].gather(1, keep)
        head = torch.arange(keep.shape[0], device=DEV)[:, None]
        src, dst = s["tables"][b].long()[keep // block], s["new_tables"][b].long()[torch.arange(m, device=DEV) // block]
        for cache in (s["k_cache"], s["v_cache"]):
            rows = cache[src, head, keep % block]
            cache[dst[None], head, (torch.arange(m, device=DEV) % block)[None]] = rows
    torch.clamp(s["ctx"], max=budget, out=s["new_ctx"])
    return s["k_cache"], s["v_cache"], s["new_scores"], s["kept"], s["new_ctx"]


# ---------------------------------------------------------------- the package's calls

def _own(s):
    import paged_kv_cache_278_gb300 as pkv
    op, case = s["op"], s["case"]
    if op in ("rope", "rope_append"):
        if "freq" not in s:  # once per model
            spec = _rope_spec(case)
            s["freq"] = pkv.rope_frequencies(device=DEV, **spec)
            s["magnitude"] = pkv.rope_magnitude(spec["factor"]) if case["method"] == "ramp" else 1.0
        more = dict(interleaved=case["interleaved"], magnitude=s["magnitude"])
        if op == "rope":
            pkv.rope(s["q_out"], s["k_out"], s["q"], s["k"], s["positions"], s["freq"], **more)
            return s["q_out"], s["k_out"]
        pkv.rope_append(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], s["freq"],
                        **more)
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "prefill":
        if "ws" not in s:
            s["ws"] = pkv.make_prefill_workspace(len(s["lens"]), s["q"].shape[0], case["hq"], case["hkv"], max(s["lens"]), DEV)
        pkv.prefill_attention(s["out"], s["q"], s["k"], s["v"], s["start"], max(s["lens"]), s["scale"], workspace=s["ws"])
        return s["out"]
    if op == "chunk":
        if "ws" not in s:
            s["ws"] = pkv.make_prefill_workspace(len(s["lens"]), s["q"].shape[0], case["hq"], case["hkv"], s["cap"], DEV)
        pkv.prefill_attention_paged(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["ctx"], s["start"],
                                    max(s["chunks"]), s["scale"], lse=s["lse"], workspace=s["ws"])
        return s["out"], s["lse"]
    if op == "step_weights":
        if "ws" not in s:
            s["ws"] = pkv.make_weights_workspace(len(s["lens"]), case["hq"], s["cap"], DEV)
        pkv.decode_attention_weights(s["out"], s["scores"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["ctx"],
                                     s["scale"], workspace=s["ws"])
        return s["out"], s["scores"]
    if op == "prompt_weights":
        pkv.prefill_attention_weights(s["scores"], s["q"], s["lse"], s["k_cache"], s["tables"], s["ctx"], s["start"],
                                      max(s["chunks"]), s["scale"])
        return s["scores"]
    pkv.evict(s["k_cache"], s["v_cache"], s["kept"], s["new_scores"], s["new_ctx"], s["scores"], s["tables"], s["ctx"],
              case["budget"], recent=case["recent"], sinks=case["sinks"], new_tables=None if case["in_place"] else s["new_tables"])
    return s["k_cache"], s["v_cache"], s["new_scores"], s["kept"], s["new_ctx"]


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------- what each pass cannot do without

def work(case):
    op = case["op"]
    row = D * 2
    if op in ("rope", "rope_append"):
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        heads = hq + hkv + (hkv if op == "rope_append" else 0)
        return {"bytes": 2 * t * heads * row + t * 4 + (t * 8 if op == "rope_append" else 0), "flops": 3 * t * (hq + hkv) * case["rotary"]}
    lens = _lens(case)
    hkv = case["hkv"]
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        cap = -(-max(lens) // case["block"]) * case["block"]
        b = sum(lens) * hkv * 4 + kept * hkv * 4 * row + len(lens) * hkv * (cap + case["budget"]) * 4
        return {"bytes": b, "flops": sum(lens) * hkv}
    hq = case["hq"]
    if op == "prefill":
        t = sum(lens)
        return {"bytes": (2 * hq + 2 * hkv) * t * row, "flops": sum(2 * n * (n + 1) for n in lens) * hq * D}
    if op == "step_weights":
        t = sum(lens)
        return {"bytes": t * hkv * 2 * row + 2 * len(lens) * hq * row + 2 * t * hkv * 4, "flops": 4 * t * hq * D}
    chunks = _chunks(case, lens)
    pairs = sum(c * (n - c) + c * (c + 1) // 2 for n, c in zip(lens, chunks))
    kv, q = sum(lens) * hkv * row, sum(chunks) * hq * row
    if op == "chunk":
        return {"bytes": 2 * kv + 2 * q + sum(chunks) * hq * 4, "flops": 4 * pairs * hq * D}
    return {"bytes": kv + q + sum(chunks) * hq * 4 + 2 * sum(lens) * hkv * 4, "flops": 2 * pairs * hq * D}


# ---------------------------------------------------------------- the definitions in 64 bits

def _positions_of(tables, b, n, block):
    p = torch.arange(n, device=DEV)
    return tables[b].long()[p // block], p % block


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rope", "rope_append"):
        freq, magnitude = _frequencies(case)
        r = case["rotary"]
        turn = torch.polar(torch.full((case["tokens"], r // 2), magnitude, dtype=F64, device=DEV), s["positions"].to(F64)[:, None] * freq)

        def spin(x):
            x = x.to(F64)
            part = x[..., :r]
            pairs = part.unflatten(-1, (r // 2, 2)) if case["interleaved"] else part.unflatten(-1, (2, r // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
            z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
            return torch.cat([z, x[..., r:]], -1)
        q, k = spin(s["q"]), spin(s["k"])
        if op == "rope":
            return q, k
        kc, vc = s["k_cache"].to(F64), s["v_cache"].to(F64)
        flat = [c.transpose(1, 2).reshape(-1, case["hkv"], D).clone() for c in (kc, vc)]
        live = (s["slots"] >= 0).nonzero()[:, 0]
        for c, x in zip(flat, (k, s["v"].to(F64))):
            c.index_copy_(0, s["slots"][live], x[live])
        return (q, *(c.view(-1, case["block"], case["hkv"], D).transpose(1, 2) for c in flat))
    lens = s["lens"]
    if op == "evict":
        budget, block, hkv = case["budget"], case["block"], case["hkv"]
        new = [s["k_cache"].to(F64), s["v_cache"].to(F64)]
        scores = torch.zeros(s["scores"].shape, dtype=F64, device=DEV)
        kept = torch.full_like(s["kept"], -1)
        for b, n in enumerate(lens):
            m, fixed = min(n, budget), torch.zeros(n, dtype=torch.bool, device=DEV)
            fixed[:min(n, case["sinks"])] = True
            fixed[max(0, n - case["recent"]):] = True
            free = m - int(fixed.sum())
            blk, off = _positions_of(s["tables"], b, n, block)
            to, at = _positions_of(s["new_tables"], b, m, block)
            for h in range(hkv):
                keep = fixed.clone()
                if n <= budget:
                    keep[:] = True
                elif free > 0:  # all above the free-th largest, then the lowest positions at it
                    x = torch.where(fixed, torch.full_like(s["scores"][b, h, :n], -math.inf), s["scores"][b, h, :n])
                    border = torch.topk(x, free)[0][-1]
                    ties = (x == border) & ~fixed
                    keep |= (x > border) & ~fixed
                    keep |= ties & (torch.cumsum(ties, 0) <= m - int(keep.sum()))
                p = keep.nonzero()[:, 0]
                kept[b, h, :m] = p
                scores[b, h, :m] = s["scores"][b, h, p].to(F64)
                for c, x in zip((s["k_cache"], s["v_cache"]), new):
                    x[to, h, at] = c[blk[p], h, off[p]].to(F64)
        return (*new, scores, None, None)
    scale, hq, hkv = s["scale"], case["hq"], case["hkv"]
    out, lses, at = torch.zeros(s["q"].shape, dtype=F64, device=DEV), torch.zeros(s["q"].shape[:2], dtype=F64, device=DEV), 0
    scores = s["scores"].to(F64) if "scores" in s else None
    for b, n in enumerate(lens):
        c = n if op == "prefill" else 1 if op == "step_weights" else s["chunks"][b]
        if op == "prefill":
            k, v = (s[x][at:at + n].to(F64) for x in "kv")
        else:
            blk, off = _positions_of(s["tables"], b, n, case["block"])
            k, v = (s[x][blk, :, off].to(F64) for x in ("k_cache", "v_cache"))
        for h in range(hq):
            kh, vh = k[:, h * hkv // hq], v[:, h * hkv // hq]
            for i in range(0, c, 2048):
                j = min(c, i + 2048)
                e = n - c + j
                z = s["q"][at + i:at + j, h].to(F64) @ kh[:e].t() * scale
                z += torch.full((j - i, e), -math.inf, dtype=F64, device=DEV).triu(n - c + i + 1)
                lse = torch.logsumexp(z, -1)
                w = torch.exp(z - (s["lse"][at + i:at + j, h].to(F64) if op == "prompt_weights" else lse)[:, None])
                if scores is not None:
                    scores[b, h * hkv // hq, :e] += w.sum(0)
                if op != "prompt_weights":
                    out[at + i:at + j, h] = w @ vh[:e]
                lses[at + i:at + j, h] = lse
        at += c
    if op == "prefill":
        return out
    if op == "chunk":
        return out, lses
    return (out, scores) if op == "step_weights" else scores
