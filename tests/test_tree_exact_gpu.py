"""How exact tree attention is where one key or one infinity decides, whichever kernel and cut of the keys a call gets: a short
table, whole items, split items."""
import numpy as np
import pytest
import torch

import paged_kv_cache_278_gb300 as pkv
import tree_ref
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu
SCALE = tree_ref.SCALE
GROUP, BS = 4, 16


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def attend(q, k, v, seen, copies=1, width=None):
    """Tree attention of the same request (q [c, Hq, 128] behind the first n - c of k, v [n, Hkv, 128]) `copies` times over, in
    blocks of its own each, tables `width` positions wide: out, lse of every copy."""
    n, c, hkv = k.shape[0], q.shape[0], k.shape[1]
    blocks = -(-n // BS)
    wide = max(blocks, -(-(width or 0) // BS))
    g = torch.Generator().manual_seed(3)
    table = torch.full((copies, wide), -7, dtype=torch.int32)
    table[:, :blocks] = torch.randperm(copies * blocks, generator=g).to(torch.int32).view(copies, blocks)
    kc, vc = (torch.full((copies * blocks, hkv, BS, 128), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    for b in range(copies):
        slots = pkv.slot_mapping(table[b:b + 1, :blocks].expand(n, -1).contiguous(), torch.arange(n, dtype=torch.int32), BS).cuda()
        pkv.append(kc, vc, slots, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
    mask = torch.from_numpy(tree_ref.pack_masks(seen, -(-c // 32))).cuda().repeat(copies, 1)
    qs = torch.from_numpy(q).cuda().repeat(copies, 1, 1)
    out = torch.full(qs.shape, 7.0, dtype=torch.float16, device="cuda")
    z = torch.full(qs.shape[:2], 7.0, device="cuda")
    ws = pkv.make_tree_workspace(copies, copies * c, c, q.shape[1], hkv, wide * BS, "cuda")
    pkv.decode_attention_tree(out, qs, kc, vc, table.cuda(), i32([n] * copies), i32(np.arange(copies + 1) * c), mask, c, SCALE, lse=z, workspace=ws)
    assert_no_device_error()
    return out.view(copies, c, -1, 128).double().cpu().numpy(), z.view(copies, c, -1).double().cpu().numpy()


def tree(c, seed=1):
    rng = np.random.default_rng(seed)
    return tree_ref.ancestors([int(rng.integers(-1, i)) if i else -1 for i in range(c)])


# (positions, nodes, kv heads, copies, table, how exact a weight is): few rows over short tables, the longest among them, take two fp16
# parts; whole items of a call of many, short contexts behind a wide table and split items one
SHORT = [(300, 8, 1, 1, None, 2.0 ** -21), (1000, 5, 1, 1, 1024, 2.0 ** -21), (41, 33, 2, 1, None, 2.0 ** -21)]
LONG = [(700, 16, 8, 40, 1100, 2.0 ** -11), (300, 8, 1, 1, 20000, 2.0 ** -11), (5000, 16, 1, 1, None, 2.0 ** -11),
        (20000, 33, 2, 1, None, 2.0 ** -11)]


@pytest.mark.parametrize("n,c,hkv,copies,width,part", SHORT + LONG)
def test_weights_in_the_product(n, c, hkv, copies, width, part):
    """How far a weight is off in the product with V, where little else is.

    24 keys have scores between -2 and 2, the others some 40 less (their weights, e^-36 at most, are 0 in the product: n e^-36 max|v|
    of the output).  A score is one exact product, so that it is off by a few steps of 2^-23 of its size, 4 at most with the scale; a
    weight besides by 8 steps for exponential, scaling and rescaling, the float32 sums by one per addition that changes them: 24
    keys in two parts, 24 in the row's sum.  The output's rounding is half a step of fp16."""
    rng = np.random.default_rng(n)
    q, k = np.zeros((c, GROUP * hkv, 128), np.float16), np.zeros((n, hkv, 128), np.float16)
    q[..., 0] = 16.0
    live = np.concatenate([rng.choice(n - c, 20, replace=False) if n - c >= 20 else np.arange(n - c), n - c + rng.permutation(c)[:4]])
    k[..., 0] = -40.0 / (16.0 * SCALE)
    k[live, :, 0] = rng.uniform(-2.0, 2.0, (len(live), hkv)) / (16.0 * SCALE)
    v = rng.standard_normal((n, hkv, 128)).astype(np.float16)
    seen = tree(c)
    out, z = attend(q, k, v, seen, copies, width)
    want, lse, p = tree_ref.attend(q.astype(np.float64), k.astype(np.float64), v.astype(np.float64), seen)
    whole = np.concatenate([np.ones((c, n - c), bool), seen], 1)
    near = whole[:, live].any(1)  # rows that see one of the live keys: the others see keys of one score
    size = np.einsum("chn,nhd->chd", p, np.abs(np.repeat(v.astype(np.float64), GROUP, 1)))
    tol = size * (part + (4 * 4 + 8 + 3 * 24) * 2.0 ** -23) + n * np.exp(-36.0) * 8 + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
    assert near.sum() >= min(c, 4)
    for b in range(copies):
        err = np.abs(out[b] - want)[near]
        assert (err <= tol[near]).all(), (b, err.max(), (err / tol[near]).max())
        assert (np.abs(z[b] - lse)[near] <= 64 * 2.0 ** -23 * (1 + np.abs(lse[near]))).all()


def case_of_infinity(kind, n, c, hkv, far):
    """One key 140 nats above all others, or half of the keys at minus infinity, and an infinity or a NaN in V of a key `far` away
    from what decides the row: (q, k, v, the key, and the key that decides or None)."""
    rng = np.random.default_rng(n + c)
    q, k = np.zeros((c, GROUP * hkv, 128), np.float16), np.zeros((n, hkv, 128), np.float16)
    v = rng.standard_normal((n, hkv, 128)).astype(np.float16)
    q[..., 0] = 16.0
    at, decides = (n - c // 2 - 1, (n - c) // 8) if far == "node" else ((n - c) // 8, (n - c) // 8 * 7)
    if kind == "minus infinity":
        k[:(n - c) // 2, :, 0] = -np.inf
        v[at, 0, 5] = np.inf
        return q, k, v, at, None
    k[decides, :, 0] = 140.0 / (16.0 * SCALE)
    v[at, 0, 5] = np.nan if kind == "nan" else -np.inf
    return q, k, v, at, decides


@pytest.mark.parametrize("n,c,hkv,copies,width,part", SHORT + LONG)
@pytest.mark.parametrize("kind,far", [("infinity", "node"), ("infinity", "context"), ("nan", "node"), ("nan", "context"), ("minus infinity", "context")])
def test_an_infinity_far_below_the_largest_score(n, c, hkv, copies, width, part, kind, far):
    """An infinity or a NaN in V of a key that a row sees is in that row's output, however small its weight is and wherever the
    keys are cut; the rest of the output is what the largest score says.  (A weight is off by 2^-11 of itself, an output by as
    much; all other weights together are below n e^-140.)"""
    q, k, v, at, decides = case_of_infinity(kind, n, c, hkv, far)
    seen = tree(c)
    out, _ = attend(q, k, v, seen, copies, width)
    sees = seen[:, at - (n - c)] if far == "node" else np.ones(c, bool)
    assert sees.any()
    for b in range(copies):
        got = out[b].reshape(c, hkv, GROUP, 128)
        assert not np.isfinite(got[sees, 0, :, 5]).any(), (b, got[sees, 0, :, 5])
        rest = np.ones(got.shape, bool)
        rest[sees, 0, :, 5] = False
        assert np.isfinite(got[rest]).all()
        if decides is not None:
            want = np.broadcast_to(v[decides].astype(np.float64)[None, :, None], got.shape)
            assert (np.abs(got - want)[rest] <= (2.0 ** -9 * np.abs(want) + 2.0 ** -24)[rest]).all()


@pytest.mark.parametrize("nats", [12.0, 18.0, 19.5])
@pytest.mark.parametrize("n,c,hkv,copies,width,part", SHORT + LONG + [(700, 90, 1, 1, None, 2.0 ** -11), (9000, 61, 1, 1, None, 2.0 ** -11)])
def test_a_long_tail_below_one_key(n, c, hkv, copies, width, part, nats):
    """One key far above all others, whose values are all positive: what the tail gives is there.

    A weight of w relative to the row's largest is held at 2^7 w: what it is off by is `part` of it, or 2^-25 where fp16 is subnormal, so at
    most 2^-32 / w of itself.  The output is off by no more than the weights are, whatever the number of keys, but for the float32
    sums: a step of 2^-23 per matrix instruction of 16 keys, of two parts, and tile of 128, and a few for the scores, one product each."""
    at = (n - c) // 3
    rng = np.random.default_rng(5)
    q, k = np.zeros((c, GROUP * hkv, 128), np.float16), np.zeros((n, hkv, 128), np.float16)
    q[..., 0], k[at, :, 0] = 16.0, nats / (16.0 * SCALE)
    v = rng.uniform(16.0, 64.0, (n, hkv, 128)).astype(np.float16)
    v[at] = 0
    seen = tree(c)
    out, z = attend(q, k, v, seen, copies, width)
    want, lse, _ = tree_ref.attend(q.astype(np.float64), k.astype(np.float64), v.astype(np.float64), seen)
    w = np.exp(-SCALE * 16.0 * float(k[at, 0, 0]))
    tol = want * (max(part, 2.0 ** -32 / w) + 2.0 ** -11 + (64 + n / 8 + n / 128) * 2.0 ** -23) + 2.0 ** -25
    for b in range(copies):
        err = np.abs(out[b] - want)
        assert (err <= tol).all(), (b, err.max(), want.max(), (err / tol).max())
        assert (np.abs(z[b] - lse) <= 64 * 2.0 ** -23 * (1 + np.abs(lse))).all()
