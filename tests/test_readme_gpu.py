"""The README's example of a speculative step, run as it stands, over several layers and two steps."""
import os
import re
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import paged_kv_cache_278_gb300 as pkv
import tree_ref
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu
B, HQ, HKV, D, BS, MAX_BLOCKS = 2, 8, 2, 128, 16, 8


def example():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        section = f.read().split("### Trees of drafted tokens")[1]
    return re.search(r"```python\n(.*?)```", section, re.S).group(1)


def host(x):
    return x.double().cpu().numpy()


def test_trees_of_drafted_tokens():
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda").half()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = []

    class Layer:
        def __init__(self):
            self.k_cache, self.v_cache = rand(B * MAX_BLOCKS, HKV, BS, D), rand(B * MAX_BLOCKS, HKV, BS, D)
            self.q_weight, self.k_weight = (1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2))

        def project(self, x):
            self.q, self.k, self.v = rand(x.shape[0], HQ, D), rand(x.shape[0], HKV, D), rand(x.shape[0], HKV, D)
            return self.q, self.k, self.v

        def finish(self, x, out):
            outs.append(out.clone())
            self.before = self.k_cache.clone(), self.v_cache.clone()  # with the whole tree
            return x

    layers = [Layer() for _ in range(3)]
    tables = torch.randperm(B * MAX_BLOCKS, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, MAX_BLOCKS).cuda()
    ctx = i32([37, 15])
    trees = [[-1, 0, 0, 1, 1, -1], [-1, 0, 1]]
    start = [0, 6, 9]
    for step, (path, lens) in enumerate((([[0, 2, 7], [0, 1, 2]], [2, 3]), ([[0, 1, 4], [7, 7, 7]], [3, 0]))):
        old = ctx.tolist()
        slots = torch.cat([pkv.slot_mapping(tables[b:b + 1].cpu().expand(len(t), -1).contiguous(), torch.arange(old[b], old[b] + len(t), dtype=torch.int32), BS)
                           for b, t in enumerate(trees)]).cuda()
        outs.clear()
        names = SimpleNamespace(path=i32(path), lens=i32(lens))
        space = dict(pkv=pkv, torch=torch, T=9, longest=6, dev="cuda", parents=i32(trees[0] + trees[1]), query_start=i32(start), counts=i32([6, 3]), B=B, Hq=HQ,
                     Hkv=HKV, D=D, max_blocks=MAX_BLOCKS, bs=BS, layers=layers, x=rand(9, 64), ctx=ctx, tables=tables, slots=slots,
                     freq=pkv.rope_frequencies(D), out=torch.empty((9, HQ, D), dtype=torch.float16, device="cuda"),
                     accept=lambda x: (names.path, names.lens))
        exec(example(), space)
        assert ctx.tolist() == [n + m for n, m in zip(old, lens)]
        assert space["positions"].tolist() == [old[0] + d for d in (0, 1, 1, 2, 2, 0)] + [old[1] + d for d in (0, 1, 2)]
        for layer, out in zip(layers, outs):
            k_full, v_full = (host(x) for x in layer.before)
            for b, parents in enumerate(trees):
                n = old[b] + len(parents)
                table = tables[b].cpu().numpy()
                k, v = (tree_ref.rows_of(x, table, n) for x in (k_full, v_full))
                assert np.array_equal(v[old[b]:], host(layer.v)[start[b]:start[b + 1]])  # where the example says
                want, _, p = tree_ref.attend(host(layer.q)[start[b]:start[b + 1]], k, v, tree_ref.ancestors(parents))
                size = np.einsum("chn,nhd->chd", p, np.abs(np.repeat(v, HQ // HKV, 1)))
                # a score of up to 50 in 136 steps of 2^-23, a weight in fp16 at worst, the output's rounding
                assert (np.abs(host(out)[start[b]:start[b + 1]] - want) <= size * (2 * 50 * 136 * 2.0 ** -23 + 2.0 ** -11) + 2.0 ** -11 * np.abs(want) + 2.0 ** -25).all()
                # kept: the context as it was, and the accepted nodes behind it
                rows = list(range(old[b])) + [old[b] + i for i in path[b][:lens[b]]]
                for cache, full in ((layer.k_cache, k), (layer.v_cache, v)):
                    assert np.array_equal(tree_ref.rows_of(host(cache), table, old[b] + lens[b]), full[rows])
    assert_no_device_error()
