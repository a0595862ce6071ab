"""The operators together, as a serving loop uses them: prompts rotated and appended, attended in chunks with
their weights accumulated, decode steps that keep accumulating, an eviction in place, and steps behind it.
Every stage is held to its float64 definition on the tensors that the stage before it left."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import paged_kv_cache_278_gb300 as pkv
from gpu_util import ATTN_TOL, assert_no_device_error

pytestmark = pytest.mark.gpu
SCALE, BS, HQ, HKV = 128 ** -0.5, 16, 8, 2


def host(x):
    return x.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("chunk", [64, 200])
def test_prompt_steps_eviction_steps(chunk):
    prompts, budget, recent, steps = [200, 77], 96, 24, 3
    b, width = len(prompts), -(-(max(prompts) + 2 * steps) // BS)
    nb = b * width + 3
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    kc, vc = torch.zeros((nb, HKV, BS, 128), dtype=torch.float16, device="cuda"), torch.zeros((nb, HKV, BS, 128), dtype=torch.float16, device="cuda")
    pool = pkv.BlockPool(nb, seed=1)
    table = torch.full((b, width), -1, dtype=torch.int32)
    scores = torch.zeros((b, HKV, width * BS), device="cuda")
    want = np.zeros(scores.shape)
    freq = pkv.rope_frequencies(128)
    f64, _ = ref.frequencies(128)
    ctx, seen = [0] * b, [0] * b  # cached positions, tokens so far (the next token's position)
    weights_ws = pkv.make_weights_workspace(b, HQ, width * BS, "cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def append(qkv, counts):
        """Rotate and append counts[r] new tokens of each request; returns the rotated q."""
        slots, pos = [], []
        for r, n in enumerate(counts):
            if n == 0:
                continue
            pool.reserve(table[r], ctx[r], ctx[r] + n, BS)
            at = torch.arange(ctx[r], ctx[r] + n, dtype=torch.int32)
            slots.append(pkv.slot_mapping(table[r:r + 1].expand(n, -1).contiguous(), at, BS))
            pos.append(torch.arange(seen[r], seen[r] + n, dtype=torch.int32))
            ctx[r] += n
            seen[r] += n
        slots, pos = torch.cat(slots).cuda(), torch.cat(pos).cuda()
        q = torch.empty((qkv.shape[0], HQ, 128), dtype=torch.float16, device="cuda")
        pkv.rope_append(q, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], kc, vc, slots, pos, freq)
        rows = host(kc).transpose(0, 2, 1, 3).reshape(-1, HKV, 128)[slots.cpu().numpy()]
        for got, x in ((host(q), qkv[:, :HQ]), (rows, qkv[:, HQ:HQ + HKV])):
            y, size = ref.rotate(host(x), pos.cpu().numpy(), f64)
            assert (np.abs(got - y) <= 2.0 ** -11 * np.abs(y) + 5e-7 * size + 2.0 ** -25).all()
        return q

    def rows_of(r):
        return (ref.rows_of(c.cpu().numpy(), table[r].numpy(), ctx[r]) for c in (kc, vc))

    def expect(q, out, counts):
        at = 0
        for r, n in enumerate(counts):
            if n:
                k, v = rows_of(r)
                p, _ = ref.weights(host(q[at:at + n]), k, SCALE)
                o = np.einsum("chn,nhd->chd", p, np.repeat(v, HQ // HKV, axis=1))
                assert np.abs(host(out[at:at + n]) - o).max() <= ATTN_TOL
                want[r, :, :ctx[r]] += p.reshape(n, HKV, -1, ctx[r]).sum((0, 2))
            at += n
        # weights are within 1e-3 of themselves (the score's bound, 136 x 2^-23 x |q| |k| scale, twice, at |q| |k| scale < 25)
        assert (np.abs(scores.cpu().numpy() - want) <= 1e-3 * want + 1e-9).all()

    def decode_steps():
        for _ in range(steps):
            q = append(randn(b, HQ + 2 * HKV, 128), [1] * b)
            out = torch.empty_like(q)
            pkv.decode_attention_weights(out, scores, q, kc, vc, table.cuda(), i32(ctx), SCALE, weights_ws)
            expect(q, out, [1] * b)

    left = list(prompts)
    while any(left):
        counts = [min(chunk, n) for n in left]
        left = [n - c for n, c in zip(left, counts)]
        q = append(randn(sum(counts), HQ + 2 * HKV, 128), counts)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        start = i32(np.concatenate([[0], np.cumsum(counts)]))
        args = (table.cuda(), i32(ctx), start, max(counts), SCALE)
        ws = pkv.make_prefill_workspace(b, q.shape[0], HQ, HKV, width * BS, "cuda")
        pkv.prefill_attention_paged(out, q, kc, vc, *args, lse=lse, workspace=ws)
        pkv.prefill_attention_weights(scores, q, lse, kc, *args)
        expect(q, out, counts)
    decode_steps()

    before = [x.cpu().numpy().copy() for x in (kc, vc, scores)]
    lens = i32(ctx)
    kept = torch.empty((b, HKV, budget), dtype=torch.int32, device="cuda")
    pkv.evict(kc, vc, kept, scores, lens, scores, table.cuda(), lens, budget, recent=recent, sinks=2)  # all in place
    old = table.numpy()
    k2, v2, kept2, s2, l2 = ref.evict(*before, old, old, np.array(ctx, np.int32), budget, recent, 2)
    assert np.array_equal(kept.cpu().numpy(), kept2) and np.array_equal(lens.cpu().numpy(), l2)
    assert np.array_equal(scores.cpu().numpy(), s2)
    for r in range(b):  # the blocks past the budget go back to the pool; their rows are nobody's
        keep = -(-int(l2[r]) // BS)
        for c, c2 in ((kc, k2), (vc, v2)):
            assert np.array_equal(ref.rows_of(c.cpu().numpy(), old[r], int(l2[r])), ref.rows_of(c2, old[r], int(l2[r])))
        gone = [int(x) for x in old[r, keep:] if x >= 0]
        pool.free(gone)
        table[r, keep:] = -1
    free = pool.num_free()
    moved = np.zeros_like(want)
    for r in range(b):
        for h in range(HKV):
            m = int(l2[r])
            moved[r, h, :m] = want[r, h, kept2[r, h, :m]]
    want[:] = moved
    ctx[:] = [int(n) for n in l2]
    decode_steps()  # positions go on from the tokens seen, not from the shortened caches
    assert seen == [p + 2 * steps for p in prompts] and pool.num_free() <= free
    assert_no_device_error()
