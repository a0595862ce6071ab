"""The operators around a tree of drafted tokens and an 8-bit cache, as a serving program calls them.

Per-head norms of q and k with the rotary rotation (positions of one axis or several) in the same pass, alone, fused with
the append, and fused with the quantising append of the fp8 cache; cached blocks read back from fp8 into an fp16 cache;
attention of a tree of drafted tokens over the paged cache; and the accepted path of such a tree moved together.  Each case
is one call on seeded inputs; `run` has the plain form in elementary torch operations and the call of the package.  fp16
caches are [num_blocks, num_kv_heads, block_size, 128], fp8 caches E4M3 codes of that shape with a float32 scale per row,
block tables scattered.
"""
import math

import torch

own = False

D = 128
DEV = "cuda"
F8, F16, F32, F64, I32 = torch.float8_e4m3fn, torch.float16, torch.float32, torch.float64, torch.int32
EPS = 1e-6


def listed():
    return [
        # the smallest call: one decode step of a small batch
        dict(name="norm_append_step", op="norm_append", tokens=16, hq=32, hkv=8, rotary=128, axes=1, interleaved=False,
             block=16, fused=False),
        # a prompt with pictures straight out of a fused q/k/v projection: time, height and width turn a section of the pairs each
        dict(name="norm_append_video", op="norm_append", tokens=8192, hq=32, hkv=8, rotary=128, axes=3, interleaved=False,
             block=16, fused=True),
        # norms and rotation alone, half of the head rotated in neighbouring pairs, an odd number of tokens
        dict(name="norm_only", op="norm", tokens=4099, hq=32, hkv=8, rotary=64, axes=1, interleaved=True, block=0, fused=True),
        # a decode step of a large batch into the 8-bit cache
        dict(name="norm_fp8_step", op="norm_fp8", tokens=64, hq=32, hkv=8, rotary=128, axes=1, interleaved=False, block=16, fused=True),
        # a prompt into the 8-bit cache
        dict(name="norm_fp8_prompt", op="norm_fp8", tokens=8192, hq=32, hkv=8, rotary=128, axes=1, interleaved=False, block=64,
             fused=True),
        # one short request brought back to fp16 blocks before its drafted tokens are checked
        dict(name="read_one", op="read", seqs=1, context=600, hkv=8, block=16),
        # long documents brought back
        dict(name="read_long", op="read", seqs=4, context=32768, hkv=8, block=64),
        # one chat, a handful of drafted tokens: latency
        dict(name="tree_one", op="tree", seqs=1, nodes=8, context=300, hq=32, hkv=8, block=16),
        # a batch of chats (the decode workload's contexts), a small tree each
        dict(name="tree_batch", op="tree", seqs=64, nodes=16, context=2049, hq=32, hkv=8, block=16),
        # long documents, a large tree each
        dict(name="tree_long", op="tree", seqs=4, nodes=61, context=32768, hq=32, hkv=8, block=64),
        # what was accepted of one chat's tree
        dict(name="keep_one", op="keep", seqs=1, nodes=8, path=4, context=300, hkv=8, block=16),
        # a batch of large trees, long accepted paths
        dict(name="keep_batch", op="keep", seqs=256, nodes=61, path=12, context=600, hkv=8, block=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_append", "norm", "norm_fp8", "norm_fp8", "read", "tree", "tree", "tree", "tree", "keep"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4])
    block = rng.choice([16, 32, 48, 64, 128, 256])
    if op in ("norm_append", "norm", "norm_fp8"):
        return dict(op=op, tokens=_log(rng, 1, 8192), hq=hq, hkv=hkv, rotary=rng.choice([16, 32, 64, 96, 128]),
                    axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.5, block=0 if op == "norm" else block,
                    fused=rng.random() < 0.5)
    if op == "read":
        context = _log(rng, 16, 32768)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(64, 131072 // context))), context=context, hkv=hkv, block=block)
    if op == "tree":
        nodes = _log(rng, 1, 256)
        context = _log(rng, nodes, 32768)
        most = min(64, 131072 // context, 4 * 61 * 32768 * 32 // (nodes * context * hq))  # no more than the long documents
        return dict(op=op, seqs=_log(rng, 1, max(1, most)), nodes=nodes, context=context, hq=hq, hkv=hkv, block=block)
    nodes = _log(rng, 1, 256)
    return dict(op=op, seqs=_log(rng, 1, 256), nodes=nodes, path=_log(rng, 1, min(nodes, 16)), context=_log(rng, nodes, 1000),
                hkv=hkv, block=block)


# ---------------------------------------------------------------- sizes and inputs

def _lens(case):
    """The lengths of a case's requests, spread between a half of its context and all of it, each with its tree's nodes."""
    n, hi = case["seqs"], case["context"]
    lo = max(hi // 2 + 1, min(hi, max(_nodes(case)) if "nodes" in case else 1))
    return [hi - (hi - lo) * ((5 * i) % n) // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _nodes(case):
    m = case["nodes"]
    return [max(1, m - (3 * i) % max(1, m // 4 + 1)) for i in range(case["seqs"])]


def _paths(case):
    return [min(n, (7 * i + 3) % case["path"] + 1) for i, n in enumerate(_nodes(case))]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32).to(F16)


def _int(values):
    return torch.tensor(values, dtype=I32, device=DEV)


def _start(counts):
    return _int([sum(counts[:i]) for i in range(len(counts) + 1)])


def _tables(g, lens, block, spare=2):
    """A block table per request over one pool in random order, and the pool's size."""
    need = [-(-n // block) for n in lens]
    width, total = max(1, max(need)), sum(need) + spare
    perm = torch.randperm(total, generator=g, device=DEV).to(I32)
    t = torch.full((len(lens), width), -1, dtype=I32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, total


def _sections(case):
    """The axis that turns each pair: one section of the pairs for each."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    return [i * axes // pairs for i in range(pairs)]


def _codes(g, *shape):
    return (torch.randn(shape, generator=g, device=DEV, dtype=F32) * 120.0).clamp_(-448.0, 448.0).to(F8).view(torch.uint8)


def _ancestors(g, counts):
    """Random trees, [B, N, N]: whether node j is i itself or above it.  The first nodes hang from the last cached token."""
    b, n = len(counts), max(counts)
    parent = (torch.rand((b, n), generator=g, device=DEV) * torch.arange(n, device=DEV)).long()  # any earlier node
    reach = torch.eye(n, dtype=F32, device=DEV).expand(b, n, n).clone()
    root = torch.rand((b, n), generator=g, device=DEV) < 2.0 / n
    root[:, 0] = True
    reach.scatter_add_(2, parent[..., None], (~root).to(F32)[..., None])
    steps = 1
    while steps < n:  # the closure, twice as far each time
        reach = (torch.matmul(reach, reach) > 0).to(F32)
        steps *= 2
    return reach > 0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case), "op": op, "scale": D ** -0.5}
    if op in ("norm", "norm_append", "norm_fp8"):
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        # what a projection leaves: heads of different sizes
        size = torch.exp(0.5 * torch.randn((1, hq + 2 * hkv, 1), generator=g, device=DEV, dtype=F32))
        qkv = (torch.randn((t, hq + 2 * hkv, D), generator=g, device=DEV, dtype=F32) * size).to(F16)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        if not case["fused"]:
            s["q"], s["k"], s["v"] = (s[x].contiguous() for x in "qkv")
        s["q_weight"], s["k_weight"] = (1.0 + 0.25 * torch.randn(D, generator=g, device=DEV, dtype=F32) for _ in range(2))
        shape = (t,) if case["axes"] == 1 else (t, case["axes"])
        s["positions"] = torch.randint(0, 32768, shape, generator=g, device=DEV, dtype=I32)
        s["axes"] = None if case["axes"] == 1 else _int(_sections(case))
        s["q_out"] = torch.empty((t, hq, D), dtype=F16, device=DEV)
        if op == "norm":
            s["k_out"] = torch.empty((t, hkv, D), dtype=F16, device=DEV)
            return s
        nb, block = -(-t // case["block"]) + 3, case["block"]
        s["slots"] = torch.randperm(nb * block, generator=g, device=DEV)[:t].contiguous()
        if t > 8:
            s["slots"][t // 2] = -1  # a padding token
        if op == "norm_append":
            s["k_cache"], s["v_cache"] = _randn(g, nb, hkv, block, D), _randn(g, nb, hkv, block, D)
        else:
            s["k_codes"], s["v_codes"] = _codes(g, nb, hkv, block, D), _codes(g, nb, hkv, block, D)
            s["k_scale"], s["v_scale"] = (torch.rand((nb, hkv, block), generator=g, device=DEV) * 0.01 for _ in range(2))
        return s
    lens, hkv, block = _lens(case), case["hkv"], case["block"]
    s["lens"] = lens
    s["tables"], nb = _tables(g, lens, block)
    if op == "read":
        live = sum(-(-n // block) for n in lens)
        s["src"] = s["tables"][s["tables"] >= 0].contiguous()
        s["dst"] = torch.randperm(live + 2, generator=g, device=DEV)[:live].to(I32)
        s["k_codes"], s["v_codes"] = _codes(g, nb, hkv, block, D), _codes(g, nb, hkv, block, D)
        s["k_scale"], s["v_scale"] = (torch.rand((nb, hkv, block), generator=g, device=DEV) * 0.01 + 1e-4 for _ in range(2))
        s["k_cache"], s["v_cache"] = (torch.zeros((live + 2, hkv, block, D), dtype=F16, device=DEV) for _ in range(2))
        return s
    s["ctx"], counts = _int(lens), _nodes(case)
    s["counts"], s["start"] = counts, _start(counts)
    s["k_cache"], s["v_cache"] = _randn(g, nb, hkv, block, D), _randn(g, nb, hkv, block, D)
    if op == "tree":
        above = _ancestors(g, counts)
        n = above.shape[1]
        words = -(-n // 32)
        bits = torch.zeros((len(counts), n, words * 32), dtype=torch.int64, device=DEV)
        bits[..., :n] = above
        packed = (bits.view(len(counts), n, words, 32) << torch.arange(32, device=DEV)).sum(-1)
        packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(I32)
        s["mask"] = torch.cat([packed[b, :c] for b, c in enumerate(counts)]).contiguous()
        s["q"] = _randn(g, sum(counts), case["hq"], D)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=F32, device=DEV)
        return s
    paths = _paths(case)
    order = torch.rand((len(counts), case["nodes"]), generator=g, device=DEV)
    order.masked_fill_(torch.arange(case["nodes"], device=DEV) >= _int(counts)[:, None], 2.0)
    chosen = order.argsort(-1)[:, :case["path"]]  # nodes in random order
    chosen = chosen.masked_fill(torch.arange(case["path"], device=DEV) >= _int(paths)[:, None], 1 << 20).sort(-1)[0]
    s["path"] = torch.where(chosen < 1 << 20, chosen, -1).to(I32).contiguous()
    s["path_lens"] = _int(paths)
    s["new_ctx"] = torch.empty_like(s["ctx"])
    return s


# ---------------------------------------------------------------- the plain forms

def _frequencies(rotary):
    return 10000.0 ** (-torch.arange(0, rotary, 2, dtype=F64, device=DEV) / rotary)


def _norm_rotate(x, weight, s):
    """The rows normalised to a mean square of one, weighted and rotated, in 32 bits (the angles in 64)."""
    case, r = s["case"], s["case"]["rotary"]
    y = x.to(F32)
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight
    p = s["positions"].to(F64)
    p = p[:, None] if s["axes"] is None else p[:, s["axes"].long()]  # the position that turns each pair
    angle = p * _frequencies(r)
    cos, sin = torch.cos(angle).to(F32)[:, None], torch.sin(angle).to(F32)[:, None]
    if case["interleaved"]:
        a, b = y[..., 0:r:2].clone(), y[..., 1:r:2].clone()
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., :r // 2].clone(), y[..., r // 2:r].clone()
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    return y


def _quantise(x):
    scale = x.abs().amax(-1) / 448.0
    codes = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    return codes.clamp_(-448.0, 448.0).to(F8).view(torch.uint8), scale


def _locate(s, positions):
    """Blocks and offsets of positions [B, n] of each request."""
    block = s["case"]["block"]
    return s["tables"].long().gather(1, positions // block).clamp_(min=0), positions % block


def _tree(s):
    case, lens, counts = s["case"], s["lens"], s["counts"]
    hkv, group, b, n, m = case["hkv"], case["hq"] // case["hkv"], len(lens), max(counts), max(lens)
    at = torch.arange(m, device=DEV)
    blk, off = _locate(s, at.expand(b, m))
    k, v = (s[x][blk, :, off].to(F32).transpose(1, 2) for x in ("k_cache", "v_cache"))  # [B, Hkv, m, D]
    node = torch.arange(n, device=DEV)
    row = (s["start"][:-1, None] + node).clamp_(max=sum(counts) - 1).long()  # [B, n]; rows past a request's last: unused
    q = s["q"].to(F32)[row].view(b, n, hkv, group, D).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * n, D)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, group, n, m)
    base = s["ctx"] - (s["start"][1:] - s["start"][:-1])
    bits = (s["mask"][:, :, None] >> torch.arange(32, device=DEV, dtype=I32)) & 1  # [T, W, 32]
    index = at - base[:, None]  # [B, m]: the node at a position
    seen = bits.flatten(1)[row].gather(2, index.clamp(0, bits.shape[1] * 32 - 1)[:, None].expand(b, n, m).long()) == 1
    seen = (index < 0)[:, None] | (seen & (at < s["ctx"][:, None])[:, None])
    p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, hkv, group * n, m), v).view(b, hkv, group, n, D) / total
    lse = (top + total.log())[..., 0]
    live = torch.cat([i * n + node[:c] for i, c in enumerate(counts)])
    s["out"].copy_(out.permute(0, 3, 1, 2, 4).reshape(b * n, case["hq"], D)[live])
    s["lse"].copy_(lse.permute(0, 3, 1, 2).reshape(b * n, case["hq"])[live])
    return s["out"], s["lse"]


def _plain(s):
    op, case = s["op"], s["case"]
    if op in ("norm", "norm_append", "norm_fp8"):
        s["q_out"].copy_(_norm_rotate(s["q"], s["q_weight"], s))
        k = _norm_rotate(s["k"], s["k_weight"], s)
        if op == "norm":
            s["k_out"].copy_(k)
            return s["q_out"], s["k_out"]
        live = s["slots"] >= 0
        slot = s["slots"][live]
        blk, off = slot // case["block"], slot % case["block"]
        if op == "norm_append":
            s["k_cache"][blk, :, off] = k[live].to(F16)
            s["v_cache"][blk, :, off] = s["v"][live]
            return s["q_out"], s["k_cache"], s["v_cache"]
        for name, x in (("k", k), ("v", s["v"].to(F32))):
            s[name + "_codes"][blk, :, off], s[name + "_scale"][blk, :, off] = _quantise(x[live])
        return s["q_out"], s["k_codes"].view(F8), s["k_scale"], s["v_codes"].view(F8), s["v_scale"]
    if op == "read":
        src, dst = s["src"].long(), s["dst"].long()
        for x in "kv":
            s[x + "_cache"][dst] = (s[x + "_codes"][src].view(F8).to(F32) * s[x + "_scale"][src][..., None]).to(F16)
        return s["k_cache"], s["v_cache"]
    if op == "tree":
        return _tree(s)
    base = s["ctx"] - (s["start"][1:] - s["start"][:-1])
    i = torch.arange(case["path"], device=DEV)
    kept = i < s["path_lens"][:, None]
    to = torch.minimum(base[:, None] + i, s["ctx"][:, None] - 1).long()  # past the path: the row onto itself
    src, src_off = _locate(s, torch.where(kept, base[:, None] + s["path"], to).long())
    dst, dst_off = _locate(s, to)
    for x in ("k_cache", "v_cache"):
        s[x][dst, :, dst_off] = s[x][src, :, src_off]
    torch.add(base, s["path_lens"], out=s["new_ctx"])
    return s["k_cache"], s["v_cache"], s["new_ctx"]


# ---------------------------------------------------------------- the package's calls

def _own(s):
    import paged_kv_cache_278_gb300 as pkv
    op, case = s["op"], s["case"]
    if op in ("norm", "norm_append", "norm_fp8"):
        if "freq" not in s:  # once per model
            s["freq"] = pkv.rope_frequencies(case["rotary"], device=DEV)
        more = dict(axes=s["axes"], interleaved=case["interleaved"])
        last = (s["positions"], s["freq"], s["q_weight"], s["k_weight"], EPS)
        if op == "norm":
            pkv.norm_rope(s["q_out"], s["k_out"], s["q"], s["k"], *last, **more)
            return s["q_out"], s["k_out"]
        if op == "norm_append":
            pkv.norm_rope_append(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], *last, **more)
            return s["q_out"], s["k_cache"], s["v_cache"]
        pkv.norm_rope_append_fp8kv(s["q_out"], s["q"], s["k"], s["v"], s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"],
                                   s["slots"], *last, **more)
        return s["q_out"], s["k_codes"].view(F8), s["k_scale"], s["v_codes"].view(F8), s["v_scale"]
    if op == "read":
        pkv.read_blocks_fp8kv(s["k_cache"], s["v_cache"], s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"], s["src"], s["dst"])
        return s["k_cache"], s["v_cache"]
    if op == "tree":
        if "ws" not in s:
            s["ws"] = pkv.make_tree_workspace(len(s["counts"]), s["q"].shape[0], max(s["counts"]), case["hq"], case["hkv"],
                                              s["tables"].shape[1] * case["block"], DEV)
        pkv.decode_attention_tree(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["ctx"], s["start"], s["mask"],
                                  max(s["counts"]), s["scale"], lse=s["lse"], workspace=s["ws"])
        return s["out"], s["lse"]
    pkv.keep_path(s["k_cache"], s["v_cache"], s["tables"], s["ctx"], s["start"], s["path"], s["path_lens"], new_lens=s["new_ctx"])
    return s["k_cache"], s["v_cache"], s["new_ctx"]


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------- what each pass cannot do without

def work(case):
    op, row = case["op"], D * 2
    if op in ("norm", "norm_append", "norm_fp8"):
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        read = t * (hq + hkv + (hkv if op != "norm" else 0)) * row + t * 4 * case["axes"] + (t * 8 if op != "norm" else 0)
        write = t * hq * row + t * hkv * (row if op == "norm" else 2 * row if op == "norm_append" else 2 * (D + 4))
        return {"bytes": read + write, "flops": t * (hq + hkv) * (4 * D + 3 * case["rotary"])}
    lens, hkv, block = _lens(case), case["hkv"], case["block"]
    if op == "read":
        rows = 2 * sum(-(-n // block) for n in lens) * block * hkv
        return {"bytes": rows * (D + 4 + row), "flops": rows * D}
    if op == "tree":
        counts, hq = _nodes(case), case["hq"]
        pairs = sum(c * n for c, n in zip(counts, lens))
        t = sum(counts)
        return {"bytes": 2 * sum(lens) * hkv * row + 2 * t * hq * row + t * hq * 4 + t * -(-max(counts) // 32) * 4,
                "flops": 4 * pairs * hq * D}
    rows = 2 * sum(_paths(case)) * hkv
    return {"bytes": 2 * rows * row + case["seqs"] * (case["path"] + 4) * 4, "flops": rows}


# ---------------------------------------------------------------- the definitions in 64 bits

def _spin(x, weight, s):
    """x [T, H, D] in 64 bits: over the root of its mean square, weighted, its pairs turned as complex numbers."""
    case, r = s["case"], s["case"]["rotary"]
    x = x.to(F64)
    x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS) * weight.to(F64)
    i = torch.arange(r // 2, device=DEV)
    place = s["positions"].to(F64).view(case["tokens"], case["axes"])[:, i * case["axes"] // (r // 2)]
    turn = torch.polar(torch.ones_like(place), place * torch.exp(-math.log(10000.0) * 2.0 / r * i.to(F64)))
    part = x[..., :r]
    pairs = part.unflatten(-1, (r // 2, 2)) if case["interleaved"] else part.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., r:]], -1)


def _written(cache, rows, s):
    """cache [NB, Hkv, bs, ...] in 64 bits with the live tokens' rows [T, Hkv, ...] in their slots."""
    x = cache.to(F64).transpose(1, 2)
    flat = x.reshape(-1, *x.shape[2:]).clone()
    live = (s["slots"] >= 0).nonzero()[:, 0]
    flat.index_copy_(0, s["slots"][live], rows[live])
    return flat.view(x.shape).transpose(1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_append", "norm_fp8"):
        q, k, v = _spin(s["q"], s["q_weight"], s), _spin(s["k"], s["k_weight"], s), s["v"].to(F64)
        if op == "norm":
            return q, k
        if op == "norm_append":
            return q, _written(s["k_cache"], k, s), _written(s["v_cache"], v, s)
        out = [q]
        for name, x in (("k", k), ("v", v)):
            scale = x.abs().amax(-1) / 448.0
            out += [_written(s[name + "_codes"].view(F8), x / scale[..., None], s), _written(s[name + "_scale"], scale, s)]
        return tuple(out)
    if op == "read":
        out = []
        for x in "kv":
            new = s[x + "_cache"].to(F64)
            new.index_copy_(0, s["dst"].long(), (s[x + "_codes"].view(F8).to(F64) * s[x + "_scale"].to(F64)[..., None])[s["src"].long()])
            out.append(new)
        return tuple(out)
    lens, counts, block, hkv = s["lens"], s["counts"], case["block"], case["hkv"]
    if op == "keep":
        new = [s["k_cache"].to(F64), s["v_cache"].to(F64)]
        tables, paths = s["tables"].tolist(), s["path"].tolist()
        for b, (n, c, m) in enumerate(zip(lens, counts, _paths(case))):
            for i in range(m):
                x, y = n - c + paths[b][i], n - c + i
                for cache, to in zip((s["k_cache"], s["v_cache"]), new):
                    to[tables[b][y // block], :, y % block] = cache[tables[b][x // block], :, x % block].to(F64)
        return (*new, None)
    hq, at = case["hq"], 0
    out = torch.zeros(s["q"].shape, dtype=F64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=F64, device=DEV)
    for b, (n, c) in enumerate(zip(lens, counts)):
        p = torch.arange(n, device=DEV)
        blk = s["tables"][b].long()[p // block]
        words = s["mask"][at:at + c].long() & 0xffffffff
        node = torch.arange(c, device=DEV)
        hidden = torch.zeros((c, n), dtype=F64, device=DEV)
        hidden[:, n - c:] = torch.where((words[:, node // 32] >> (node % 32)) % 2 == 1, 0.0, -math.inf)
        for h in range(hkv):
            k, v = (s[x][blk, h, p % block].to(F64) for x in ("k_cache", "v_cache"))
            for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                z = s["q"][at:at + c, j].to(F64) @ k.t() * s["scale"] + hidden
                lse[at:at + c, j] = torch.logsumexp(z, -1)
                out[at:at + c, j] = torch.softmax(z, -1) @ v
        at += c
    return out, lse
