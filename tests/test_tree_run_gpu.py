"""The tree operators together, as a speculative serving loop uses them: prompts normalised, rotated and appended, then
steps that draft a tree, check it and keep a path of it.  Every stage is held to its float64 definition on the tensors
that the stage before it left, and the caches to those of a run that never drafted."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import paged_kv_cache_278_gb300 as pkv
import tree_ref
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu
SCALE, EPS, BS, HQ, HKV = 128 ** -0.5, 1e-6, 16, 8, 2


def host(x):
    return x.float().cpu().numpy().astype(np.float64)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Model:
    """What one layer makes of token `t` of request `r` (any draft of the same token makes the same)."""

    def __init__(self, seed):
        self.seed = seed
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.qw, self.kw = (1 + 0.2 * torch.randn(128, generator=g, device="cuda") for _ in range(2))
        self.freq = pkv.rope_frequencies(128)
        self.axes = pkv.rope_axes([16, 24, 24])

    def qkv(self, tokens):
        out = []
        for r, t in tokens:
            g = torch.Generator(device="cuda").manual_seed(1000 * self.seed + 100000 * r + t)
            out.append(torch.randn((HQ + 2 * HKV, 128), generator=g, device="cuda"))
        return torch.stack(out).half()


def positions_of(pos):
    """Three axes that differ: what a picture's patches would have."""
    pos = np.asarray(pos)
    return i32(np.stack([pos, pos // 7, pos % 7], 1))


def slots_of(table, r, at):
    return pkv.slot_mapping(table[r:r + 1].expand(len(at), -1).contiguous(), torch.tensor(at, dtype=torch.int32), BS)


@pytest.mark.parametrize("quantised", [False, True])
def test_draft_check_keep(quantised):
    model, rng = Model(3), np.random.default_rng(4)
    prompts, steps, nodes = [70, 9], 3, 12
    b, width = len(prompts), -(-(max(prompts) + steps * nodes + nodes) // BS)
    nb = b * width + 2
    pool = pkv.BlockPool(nb, seed=2)
    table = torch.full((b, width), -1, dtype=torch.int32)
    for r in range(b):
        pool.reserve(table[r], 0, width * BS, BS)
    dev_table = table.cuda()
    kc, vc = (torch.zeros((nb, HKV, BS, 128), dtype=torch.float16, device="cuda") for _ in range(2))

    def write(tokens, pos, slots, caches=None):
        qkv = model.qkv(tokens)
        q = torch.empty((len(tokens), HQ, 128), dtype=torch.float16, device="cuda")
        rows = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        pkv.norm_rope_append(q, *rows, *(caches or (kc, vc)), slots.cuda(), positions_of(pos), model.freq, model.qw, model.kw, EPS, axes=model.axes)
        f64, _ = ref.frequencies(128)
        want, size = tree_ref.norm_rotate(host(rows[0]), host(model.qw), EPS, positions_of(pos).cpu().numpy(), model.axes.cpu().numpy(), f64)
        assert (np.abs(host(q) - want) <= 2.0 ** -11 * np.abs(want) * (1 + 1e-5) + 1.35e-6 * size + 2.0 ** -25).all()
        return q

    # the prompts, by way of the fp8 cache in the quantised run: written as codes, brought back as blocks
    ctx = list(prompts)
    tokens = [(r, t) for r in range(b) for t in range(prompts[r])]
    slots = torch.cat([slots_of(table, r, list(range(prompts[r]))) for r in range(b)])
    pos = [t for _, t in tokens]
    if quantised:
        fp8 = pkv.empty_fp8kv_cache(nb, HKV, BS, "cuda")
        qkv = model.qkv(tokens)
        q = torch.empty((len(tokens), HQ, 128), dtype=torch.float16, device="cuda")
        pkv.norm_rope_append_fp8kv(q, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], *fp8, slots.cuda(), positions_of(pos), model.freq,
                                   model.qw, model.kw, EPS, axes=model.axes)
        used = torch.cat([table[r, :-(-prompts[r] // BS)] for r in range(b)]).cuda()
        pkv.read_blocks_fp8kv(kc, vc, *fp8, used, used)
    else:
        write(tokens, pos, slots)
    straight = [kc.clone(), vc.clone()]  # the caches of a run that appends accepted tokens one after another
    lens = i32(ctx)
    accepted_tokens = [list(range(n)) for n in prompts]
    ws = pkv.make_tree_workspace(b, b * nodes, nodes, HQ, HKV, width * BS, "cuda")
    for step in range(steps):
        counts = [nodes, nodes - 5] if step % 2 else [3, nodes]
        parents = [[-1 if i == 0 or rng.random() < 0.2 else int(rng.integers(0, i)) for i in range(c)] for c in counts]
        start = np.concatenate([[0], np.cumsum(counts)])
        mask = torch.empty((sum(counts), 1), dtype=torch.int32, device="cuda")
        depths = torch.empty(sum(counts), dtype=torch.int32, device="cuda")
        pkv.tree_masks(mask, depths, i32(sum(parents, [])), i32(start), nodes)
        # node i of request r drafts some token; its position follows from its depth
        drafted = [[int(rng.integers(500, 60000)) for _ in range(c)] for c in counts]
        depth = depths.cpu().numpy()
        pos = [ctx[r] + depth[start[r] + i] for r in range(b) for i in range(counts[r])]
        at = [list(range(ctx[r], ctx[r] + counts[r])) for r in range(b)]
        q = write([(r, t) for r in range(b) for t in drafted[r]], pos, torch.cat([slots_of(table, r, at[r]) for r in range(b)]))
        lens += i32(counts)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        pkv.decode_attention_tree(out, q, kc, vc, dev_table, lens, i32(start), mask, nodes, SCALE, lse=lse, workspace=ws)
        for r in range(b):
            n, rows = ctx[r] + counts[r], slice(start[r], start[r + 1])
            k, v = (tree_ref.rows_of(host(c), table[r].numpy(), n) for c in (kc, vc))
            want, z, _ = tree_ref.attend(host(q[rows]), k, v, tree_ref.ancestors(parents[r]))
            # weights rounded to fp16, outputs too, scores off by some 1e-5: 2^-10 of values up to |v| < 8
            assert np.abs(host(out[rows]) - want).max() <= 8 * 2.0 ** -10 and np.abs(host(lse[rows]) - z).max() <= 1e-4
        # accept the path to some node
        paths = []
        for r in range(b):
            node, path = int(rng.integers(0, counts[r])), []
            while node >= 0:
                path.insert(0, node)
                node = parents[r][node]
            paths.append(path)
        longest = max(len(p) for p in paths)
        path = i32([p + [-1] * (longest - len(p)) for p in paths])
        pkv.keep_path(kc, vc, dev_table, lens, i32(start), path, i32([len(p) for p in paths]), new_lens=lens)
        new = [(r, drafted[r][i]) for r in range(b) for i in paths[r]]
        new_pos = [ctx[r] + i for r in range(b) for i in range(len(paths[r]))]
        write(new, new_pos, torch.cat([slots_of(table, r, list(range(ctx[r], ctx[r] + len(paths[r])))) for r in range(b)]), straight)
        for r in range(b):
            accepted_tokens[r] += [drafted[r][i] for i in paths[r]]
            ctx[r] += len(paths[r])
        assert lens.tolist() == ctx == [len(t) for t in accepted_tokens]
        for got, want in zip((kc, vc), straight):
            for r in range(b):
                assert np.array_equal(tree_ref.rows_of(host(got), table[r].numpy(), ctx[r]), tree_ref.rows_of(host(want), table[r].numpy(), ctx[r]))
    # and a plain decode step behind it all, on both caches
    q = torch.randn((b, HQ, 128), device="cuda").half()
    outs = [torch.empty_like(q) for _ in range(2)]
    dws = pkv.make_workspace(b, HQ, width * BS, "cuda")
    for out, caches in zip(outs, ((kc, vc), straight)):
        pkv.decode_attention(out, q, *caches, dev_table, lens, SCALE, workspace=dws)
    assert torch.equal(*outs)
    assert_no_device_error()


def test_captured_step():
    """Masks, append, attention and the accepted path of one step in one graph, replayed with other trees and lengths."""
    model = Model(5)
    b, nodes, width = 2, 8, 6
    nb = b * width
    table = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(b, width)
    g = torch.Generator(device="cuda").manual_seed(6)
    kc, vc = (torch.randn((nb, HKV, BS, 128), generator=g, device="cuda").half() for _ in range(2))
    qkv = torch.randn((b * nodes, HQ + 2 * HKV, 128), generator=g, device="cuda").half()
    parents, start = i32([-1] * (b * nodes)), i32([0, nodes, 2 * nodes])
    mask, depths = torch.zeros((b * nodes, 1), dtype=torch.int32, device="cuda"), torch.zeros(b * nodes, dtype=torch.int32, device="cuda")
    slots, pos, lens = torch.zeros(b * nodes, dtype=torch.int64, device="cuda"), i32([0] * (b * nodes)), i32([nodes, nodes])
    path, path_lens = i32([[0, 0, 0]] * b), i32([0, 0])
    q, out = (torch.empty((b * nodes, HQ, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    new = torch.empty_like(lens)
    dev_table = table.cuda()

    def step(caches, out, new, stream=None):
        pkv.tree_masks(mask, depths, parents, start, nodes, stream=stream)
        pkv.norm_rope_append(q, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], *caches, slots, pos, model.freq, model.qw, model.kw, EPS,
                             stream=stream)
        pkv.decode_attention_tree(out, q, *caches, dev_table, lens, start, mask, nodes, SCALE, stream=stream)
        pkv.keep_path(*caches, dev_table, lens, start, path, path_lens, new_lens=new, stream=stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step((kc, vc), out, new)
    rng = np.random.default_rng(8)
    for ctx in ([20, 8], [90, 33], [64, 16]):
        parents.copy_(i32([int(rng.integers(-1, i)) if i else -1 for _ in range(b) for i in range(nodes)]))
        lens.copy_(i32(ctx))
        slots.copy_(torch.cat([slots_of(table, r, list(range(n - nodes, n))) for r, n in enumerate(ctx)]))
        pos.copy_(i32(rng.integers(0, 5000, b * nodes)))
        path.copy_(i32([[0, 2, 5], [1, 3, 7]]))
        path_lens.copy_(i32([3, 2]))
        eager = [kc.clone(), vc.clone()]
        graph.replay()
        torch.cuda.synchronize()
        out2, new2 = torch.empty_like(out), torch.empty_like(new)
        s.wait_stream(torch.cuda.current_stream())
        step(eager, out2, new2, stream=s)
        s.synchronize()
        assert torch.equal(out, out2) and torch.equal(new, new2) and new.tolist() == [ctx[0] - nodes + 3, ctx[1] - nodes + 2]
        assert torch.equal(kc, eager[0]) and torch.equal(vc, eager[1])
    assert_no_device_error()
