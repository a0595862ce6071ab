"""Prompt and chunk attention on the GPU against causal float64 attention."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import paged_kv_cache_278_gb300 as pkv
import workloads
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def check(out, lse, want_rows):
    """want_rows: (row slice, q, k, v) per request.  A score's error is at most 136 x 2^-23 of scale |q| |k| (8
    matrix instructions of 17 addends, each cut to 24 bits, on values no larger); a weight's twice that relative
    to itself, 8 steps of 2^-23 for its exponential, scaling and the sums, and half a step of fp16 (2^-11; 2^-25 of the
    largest weight when it is subnormal).  The output adds its own half step."""
    for rows, q, k, v in want_rows:
        if q.shape[0] == 0:
            continue
        p, z = ref.weights(q, k, SCALE)
        rep = q.shape[1] // k.shape[1]
        vv = np.repeat(v, rep, axis=1)
        o = np.einsum("chn,nhd->chd", p, vv)
        size = SCALE * np.sqrt((q.astype(np.float64) ** 2).sum(-1)).max() * np.sqrt((k ** 2).sum(-1)).max()
        dot = 136 * size * 2.0 ** -23
        tol = (np.einsum("chn,nhd->chd", p, np.abs(vv)) * (2.0 ** -11 + 2 * dot + 8 * 2.0 ** -23)
               + k.shape[0] * 2.0 ** -25 * np.abs(v).max() + 2.0 ** -11 * np.abs(o) + 2.0 ** -25)
        err = np.abs(out[rows].astype(np.float64) - o)
        assert (err <= tol).all(), (rows, err.max(), np.argwhere(~(err <= tol))[:4])
        if lse is not None:
            assert (np.abs(lse[rows] - z) <= dot + 8 * 2.0 ** -23 * (1 + np.abs(z))).all()


def packed(lens, hq, hkv, seed, fused=True, before=0, behind=0, sharpen=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = before + sum(lens) + behind
    if fused:
        x = torch.randn((t, hq + 2 * hkv, 128), generator=g, device="cuda").half()
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = (torch.randn((t, h, 128), generator=g, device="cuda").half() for h in (hq, hkv, hkv))
    if sharpen != 1.0:  # later keys larger: the running maximum keeps rising
        k *= torch.linspace(0.2, sharpen, t, device="cuda").half()[:, None, None]
    start = before + np.concatenate([[0], np.cumsum(lens)])
    return q, k, v, start


def run_packed(lens, hq, hkv, seed, lse=True, **more):
    q, k, v, start = packed(lens, hq, hkv, seed, **more)
    t = q.shape[0]
    out = torch.full((t, hq, 128), 7.0, dtype=torch.float16, device="cuda")
    z = torch.full((t, hq), 7.0, device="cuda") if lse else None
    longest = max(1, max(lens))
    ws = pkv.make_prefill_workspace(len(lens), t, hq, hkv, longest, "cuda")
    pkv.prefill_attention(out, q, k, v, torch.tensor(start, dtype=torch.int32, device="cuda"), longest, SCALE, lse=z, workspace=ws)
    assert_no_device_error()
    o, zz = out.float().cpu().numpy(), z.cpu().numpy() if lse else None
    h = [x.float().cpu().numpy() for x in (q, k, v)]
    check(o, zz, [(slice(a, b), *(x[a:b].astype(np.float64) for x in h)) for a, b in zip(start, start[1:])])
    outside = np.r_[0:start[0], start[-1]:t]
    assert (o[outside] == 7).all() and (zz is None or (zz[outside] == 7).all())
    return out, z, (q, k, v, start, ws)


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("hkv", [1, 3])
def test_packed_ragged(group, hkv):
    run_packed([1, 2, 16, 127, 0, 128, 129, 33, 300, 257, 64], group * hkv, hkv, group, fused=group != 2, before=3, behind=5)


@pytest.mark.parametrize("lens,hq,hkv", [([1], 8, 1), ([1], 1, 1), ([1500], 4, 2), ([700, 1100], 16, 2), ([0, 0, 5], 2, 2)])
def test_packed_sizes(lens, hq, hkv):
    run_packed(lens, hq, hkv, 31 + len(lens))


def test_many_sequences():
    """More work items than SMs, more sequences than a warp has lanes."""
    run_packed([(37 * i) % 150 for i in range(70)], 8, 4, 5, lse=False)


def test_rising_scores():
    run_packed([900, 40], 4, 1, 6, sharpen=12.0)


def test_other_sequences_do_not_leak():
    q, k, v, start = packed([100, 60, 200], 4, 1, 7, fused=False)
    clean = torch.empty_like(q)
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    pkv.prefill_attention(clean, q, k, v, st, 200, SCALE)
    k[100:160] = float("nan")
    v[100:160] = float("inf")
    out = torch.empty_like(q)
    pkv.prefill_attention(out, q, k, v, st, 200, SCALE)
    assert torch.equal(out[:100], clean[:100]) and torch.equal(out[160:], clean[160:])
    assert_no_device_error()


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 1)])
@pytest.mark.parametrize("paged", [False, True])
def test_infinities_in_later_values(hq, hkv, paged):
    """An infinity or NaN in a token's V reaches the rows at and after that token, in its dim and kv head, and no others:
    everything else is bit for bit what it is with zeros there."""
    n = 420
    g = torch.Generator(device="cuda").manual_seed(hq)
    q, k, v = (torch.randn((n, h, 128), generator=g, device="cuda").half() for h in (hq, hkv, hkv))
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    spots = [(3, 0, 5, float("inf")), (130, hkv - 1, 127, float("nan")), (131, 0, 64, float("-inf")), (300, 0, 5, float("-inf")),
             (419, 0, 9, float("inf"))]
    zeros, values = v.clone(), v.clone()
    for t, h, d, x in spots:
        zeros[t, h, d] = 0
        values[t, h, d] = x

    def run(x):
        out = torch.empty_like(q)
        if not paged:
            return pkv.prefill_attention(out, q, k, x, start, n, SCALE)
        bs, nb = 32, -(-n // 32)
        table = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(1, -1)
        kc, vc = (torch.full((nb, hkv, bs, 128), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
        slots = pkv.slot_mapping(table.expand(n, -1).contiguous(), torch.arange(n, dtype=torch.int32), bs).cuda()
        pkv.append(kc, vc, slots, k, x)
        return pkv.prefill_attention_paged(out, q, kc, vc, table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), start, n, SCALE)
    clean, got = run(zeros).view(n, hkv, -1, 128), run(values).view(n, hkv, -1, 128)
    expect = clean.float()
    for t, h, d, x in spots:
        expect[t:, h, :, d] += x  # inf - inf is NaN here too
    assert torch.equal(torch.isnan(got), torch.isnan(expect))
    same = ~torch.isnan(expect)
    assert torch.equal(got.float()[same], expect[same])
    assert_no_device_error()


def run_paged(ctxs, chunks, group, hkv, bs, seed, peaky=0.0, poison=False):
    case = workloads.random_case(seed, ctxs, group * hkv, hkv, block_size=bs, peaky_fraction=peaky, peaky_factor=6.0)
    if poison:  # whatever lies behind a context in its last block, and in blocks of nobody
        for b, n in enumerate(ctxs):
            if n % bs:
                blk = int(case.block_tables[b, n // bs])
                case.k_cache[blk, :, n % bs:] = float("nan")
                case.v_cache[blk, :, n % bs:] = float("inf")
    start = np.concatenate([[0], np.cumsum(chunks)])
    rng = np.random.default_rng(seed)
    q = rng.standard_normal((start[-1], group * hkv, 128)).astype(np.float16)
    dev = case.to("cuda")
    qd = torch.from_numpy(q).cuda()
    out, z = torch.full_like(qd, float("nan")), torch.full(qd.shape[:2], float("nan"), device="cuda")
    cap = case.max_blocks_per_seq * bs
    ws = pkv.make_prefill_workspace(len(ctxs), q.shape[0], group * hkv, hkv, cap, "cuda")
    if ws is not None:
        ws.fill_(255)  # no initial contents are needed
    args = (qd, dev.k_cache, dev.v_cache, dev.block_tables, dev.context_lens, torch.tensor(start, dtype=torch.int32, device="cuda"),
            max(1, max(chunks)), SCALE)
    pkv.prefill_attention_paged(out, *args, lse=z, workspace=ws)
    assert_no_device_error()
    rows = []
    for b, n in enumerate(ctxs):
        if chunks[b]:
            table = case.block_tables.numpy()[b]
            rows.append((slice(start[b], start[b + 1]), q[start[b]:start[b + 1]], ref.rows_of(case.k_cache.numpy(), table, n),
                         ref.rows_of(case.v_cache.numpy(), table, n)))
    check(out.float().cpu().numpy(), z.cpu().numpy(), rows)
    return out, z, args, ws


def test_long_prompt():
    """Rows of a long prompt at and around tile borders, and of short ones packed beside it."""
    lens = [300, 16384, 5]
    q, k, v, start = packed(lens, 8, 2, 90)
    out, z = torch.full((q.shape[0], 8, 128), float("nan"), dtype=torch.float16, device="cuda"), torch.zeros((q.shape[0], 8), device="cuda")
    pkv.prefill_attention(out, q, k, v, torch.tensor(start, dtype=torch.int32, device="cuda"), max(lens), SCALE, lse=z,
                          workspace=pkv.make_prefill_workspace(3, q.shape[0], 8, 2, max(lens), "cuda"))
    assert_no_device_error()
    assert torch.isfinite(out).all()
    o, zz, h = out.float().cpu().numpy(), z.cpu().numpy(), [x.float().cpu().numpy() for x in (q, k, v)]
    rows = [(b, t) for b, some in ((0, (0, 299)), (1, (0, 31, 32, 127, 128, 4095, 8191, 8192, 12345, 16351, 16352, 16383)), (2, (4,)))
            for t in some]
    check(o, zz, [(slice(start[b] + t, start[b] + t + 1), h[0][start[b] + t:start[b] + t + 1],
                   *(x[start[b]:start[b] + t + 1].astype(np.float64) for x in h[1:])) for b, t in rows])


def test_many_decode_rows_beside_a_chunk():
    """One call with hundreds of requests of one new token each and one chunk of many, as continuous batching makes it."""
    ctxs = [(53 * i) % 190 + 1 for i in range(420)]
    chunks = [1] * 420
    ctxs[200], chunks[200] = 1700, 900
    chunks[17] = 0
    run_paged(ctxs, chunks, 4, 2, 16, 91)


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [16, 48, 64, 256])
def test_paged_ragged(group, bs):
    run_paged([1, 17, 128, 129, 500, 1000, 300, 4, 260], [1, 5, 128, 1, 33, 200, 300, 0, 64], group, 2, bs, 40 + bs + group, poison=True)


@pytest.mark.parametrize("ctxs,chunks,group,hkv,bs", [([5000, 2049], [37, 1], 4, 1, 16), ([3000], [70], 8, 1, 32),
                                                      ([4097], [1], 1, 2, 128), ([2500, 600, 40], [16, 600, 0], 2, 1, 96)])
def test_paged_split_keys(ctxs, chunks, group, hkv, bs):
    _, _, _, ws = run_paged(ctxs, chunks, group, hkv, bs, 77, peaky=0.02)
    assert ws is not None  # the plan splits these


# The plan, which knows no lengths, allows splits; the launch takes one (short contexts behind a wide table, or more
# tiles than the rows' number needs), or three.
@pytest.mark.parametrize("ctxs,chunks,group,hkv,bs,planned", [
    ([5000, 200, 129], [0, 37, 2], 4, 2, 16, True), ([1100] * 17, [130] * 17, 2, 4, 32, False),  # under three splits' keys: none
    ([3200] * 17, [130] * 17, 2, 4, 32, True), ([3100, 3073, 3090, 3099, 3076], [257] * 5, 1, 8, 64, True)])
def test_paged_splits_by_the_actual_lengths(ctxs, chunks, group, hkv, bs, planned):
    out, z, args, ws = run_paged(ctxs, chunks, group, hkv, bs, 81)
    again, z2 = torch.empty_like(out), torch.empty_like(z)
    pkv.prefill_attention_paged(again, *args, lse=z2, workspace=ws)
    assert (ws is not None) == planned and torch.equal(again, out) and torch.equal(z2, z)


def test_paged_long_chunk_past_the_multi_call():
    run_paged([1400], [1300], 4, 2, 16, 78)


def test_paged_equals_the_multi_call():
    ctxs, chunks = [700, 90, 333], [40, 8, 333]
    out, _, args, _ = run_paged(ctxs, chunks, 4, 2, 16, 79)
    other = torch.empty_like(out)
    ws = pkv.make_multi_workspace(3, sum(chunks), 333, 8, 2, 704, "cuda")
    pkv.decode_attention_multi(other, *args, workspace=ws)
    assert (out.float() - other.float()).abs().max() <= 4e-3  # twice the decode tests' bound


def one_key_above(n, hkv, nats, at, seed):
    """Keys of which the one at position `at` scores `nats` above all others for every row; its V is zero, the others' are
    all positive, so that the output is what the tail gives: (q [n, 4 hkv, 128], k, v [n, hkv, 128])."""
    rng = np.random.default_rng(seed)
    q, k = np.zeros((n, 4 * hkv, 128), np.float16), np.zeros((n, hkv, 128), np.float16)
    q[..., 0], k[at, :, 0] = 16.0, nats / (16.0 * SCALE)
    v = rng.uniform(16.0, 64.0, (n, hkv, 128)).astype(np.float16)
    v[at] = 0
    return q, k, v


def check_tail(out, lse, q, k, v, at):
    """A weight of w relative to the row's largest is held in fp16 at 2^7 w or more: half a step is 2^-11 of it, or 2^-25 where that
    is subnormal, so at most 2^-32 / w of itself.  All values and weights of the tail are positive: the output is off by no more
    than the weights are, whatever the number of keys, but for the float32 sums: a step of 2^-23 per matrix instruction of 16 keys
    and tile of 128.  The scores are one product each, a few steps of 2^-23 times their size."""
    c, n = q.shape[0], k.shape[0]
    p, z = ref.weights(q, k, SCALE)
    o = np.einsum("chn,nhd->chd", p, np.repeat(v.astype(np.float64), 4, axis=1))
    w = np.exp(-SCALE * 16.0 * float(k[at, 0, 0]))
    sees = (np.arange(n - c, n) >= at)[:, None, None]
    off = np.where(sees, max(2.0 ** -11, 2.0 ** -32 / w), 2.0 ** -11)
    tol = o * (off + 2.0 ** -11 + (64 + n / 16 + n / 128) * 2.0 ** -23) + 2.0 ** -25
    err = np.abs(out.astype(np.float64) - o)
    assert (err <= tol).all(), (err.max(), o.max(), np.argwhere(~(err <= tol))[:4])
    assert (np.abs(lse - z) <= 64 * 2.0 ** -23 * (1 + np.abs(z))).all()


@pytest.mark.parametrize("nats", [12.0, 18.0, 19.5])
@pytest.mark.parametrize("n,c,at", [(700, 700, 0), (700, 200, 130), (5000, 37, 0), (5000, 129, 4899), (20000, 3, 7)])
def test_a_long_tail_below_one_key(nats, n, c, at):
    """One key far above a long tail (an attention sink): what the tail's values give is there, in whole and split rows."""
    q, k, v = one_key_above(n, 1, nats, at, 5)
    q = q[n - c:]
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    bs, nb = 16, -(-n // 16)
    table = torch.randperm(nb, generator=torch.Generator().manual_seed(2)).to(torch.int32).view(1, -1)
    kc, vc = (torch.zeros((nb, 1, bs, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    slots = pkv.slot_mapping(table.expand(n, -1).contiguous(), torch.arange(n, dtype=torch.int32), bs).cuda()
    pkv.append(kc, vc, slots, t(k), t(v))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, z = torch.full((c, 4, 128), float("nan"), dtype=torch.float16, device="cuda"), torch.full((c, 4), float("nan"), device="cuda")
    ws = pkv.make_prefill_workspace(1, c, 4, 1, nb * bs, "cuda")
    pkv.prefill_attention_paged(out, t(q), kc, vc, table.cuda(), i32(n), i32(0, c), c, SCALE, lse=z, workspace=ws)
    check_tail(out.float().cpu().numpy(), z.cpu().numpy(), q, k, v, at)
    if c == n:
        o2, z2 = torch.empty_like(out), torch.empty_like(z)
        pkv.prefill_attention(o2, t(q), t(k), t(v), i32(0, n), n, SCALE, lse=z2,
                              workspace=pkv.make_prefill_workspace(1, n, 4, 1, n, "cuda"))
        check_tail(o2.float().cpu().numpy(), z2.cpu().numpy(), q, k, v, at)
    assert_no_device_error()


@pytest.mark.parametrize("n,c", [(6, 6), (300, 300), (2500, 5)])
def test_scores_of_minus_infinity(n, c):
    """A key whose scores are minus infinity takes no part, and a row that sees no other has no softmax: NaN, and a log-sum-exp of
    minus infinity, whether its keys are split or not."""
    g = torch.Generator(device="cuda").manual_seed(n)
    q = torch.rand((c, 4, 128), generator=g, device="cuda").half() + 0.5
    k, v = (torch.randn((n, 1, 128), generator=g, device="cuda").half() for _ in range(2))
    gone = n - c + 1  # all that the first row of the chunk sees, and one key more
    k[:gone] = float("-inf")
    k[gone + 2] = float("-inf")
    bs, nb = 16, -(-n // 16)
    kc, vc = (torch.zeros((nb, 1, bs, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    pkv.append(kc, vc, torch.arange(n, device="cuda"), k, v)
    table = torch.arange(nb, dtype=torch.int32, device="cuda").view(1, -1)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = pkv.make_prefill_workspace(1, c, 4, 1, nb * bs, "cuda")
    assert (ws is not None) == (n == 2500)
    out, z = torch.zeros_like(q), torch.zeros((c, 4), device="cuda")
    pkv.prefill_attention_paged(out, q, kc, vc, table, i32(n), i32(0, c), c, SCALE, lse=z, workspace=ws)
    assert torch.isnan(out[0]).all() and (z[0] == float("-inf")).all()
    rows = [i for i in range(gone, n) if i != gone + 2]
    qn, kn, vn = (x.float().cpu().numpy().astype(np.float64) for x in (q, k, v))
    for t in range(1, c):
        seen = [i for i in rows if i <= n - c + t]
        s = np.einsum("hd,nd->hn", qn[t], kn[seen, 0]) * SCALE
        p = np.exp(s - s.max(-1, keepdims=True))
        want = (p / p.sum(-1, keepdims=True)) @ vn[seen, 0]
        assert np.abs(out[t].float().cpu().numpy() - want).max() <= 2e-3
    if n == c:
        o2, z2 = torch.zeros_like(out), torch.zeros_like(z)
        pkv.prefill_attention(o2, q, k, v, i32(0, n), n, SCALE, lse=z2)
        assert torch.isnan(o2[0]).all() and torch.equal(o2[1:], out[1:]) and torch.equal(z2, z)
    assert_no_device_error()


def test_bad_requests_are_skipped_and_recorded():
    out, z, args, ws = run_paged([300, 200, 100], [20, 30, 40], 4, 2, 16, 80)
    q, kc, vc, bt, cl, qs, n, scale = args

    def call(**change):
        a = dict(bt=bt, cl=cl, qs=qs, n=n)
        a.update(change)
        o = torch.full_like(out, 5.0)
        pkv.prefill_attention_paged(o, q, kc, vc, a["bt"], a["cl"], a["qs"], a["n"], scale, workspace=ws)
        return o
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for change, gone in ((dict(cl=i32(300, 29, 100)), slice(20, 50)), (dict(cl=i32(300, 10 ** 6, 100)), slice(20, 50)),
                         (dict(n=30), slice(50, 90)), (dict(qs=i32(0, 20, 50, 91)), slice(50, 90))):
        o = call(**change)
        assert pkv.device_error() == pkv.PKV_DEV_BAD_CONTEXT, change
        keep = torch.ones(90, dtype=torch.bool, device="cuda")
        keep[gone] = False
        assert (o[gone] == 5).all() and torch.equal(o[keep], out[keep]), change
    bad = bt.clone()
    bad[1, 3] = -7
    o = call(bt=bad)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_BLOCK_ID
    assert torch.equal(o[:20], out[:20]) and torch.equal(o[50:], out[50:])
    if ws is not None:
        with pytest.raises(pkv.PkvError):
            pkv.prefill_attention_paged(torch.empty_like(out), *args, workspace=ws[:ws.numel() - 256])


def test_graph_replay_and_stream():
    out, z, args, ws = run_paged([900, 77], [100, 77], 4, 2, 16, 81)
    o = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.prefill_attention_paged(o, *args, workspace=ws)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o.zero_()
    s.wait_stream(torch.cuda.current_stream())
    pkv.prefill_attention_paged(o, *args, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o, out)
