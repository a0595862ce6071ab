"""Accumulated attention weights on the GPU against their float64 definition."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import paged_kv_cache_278_gb300 as pkv
import workloads
from gpu_util import ATTN_TOL, assert_no_device_error, max_err

pytestmark = pytest.mark.gpu


def score_tolerance(total, q, k, scale, prior):
    """A dot product of 128 terms in float32 is off by at most 136 x 2^-23 of the sum of its terms'
    sizes (8 matrix instructions of 17 addends, each cut to 24 bits); a weight exp(s - lse) by that
    twice (s and lse) and 4 steps of 2^-23 for the exponentials; the sum over the heads and the
    addition round once each."""
    hkv = k.shape[1]
    size = scale * np.abs(q).astype(np.float64).sum(-1).max() * np.abs(k).max()  # crude: sum |q_i| max |k|
    size = min(size, scale * float(np.sqrt((q.astype(np.float64) ** 2).sum(-1).max()) * np.sqrt((k ** 2).sum(-1).max())))
    return total * (2 * 136 * size + 8) * 2.0 ** -23 + np.abs(prior + total) * 2.0 ** -23 + hkv * 2.0 ** -126


def reference(case, prior):
    h = case.to("cpu")
    out = np.zeros(h.q.shape)
    add, tol = np.zeros(prior.shape), np.zeros(prior.shape)
    for b, n in enumerate(h.context_lens.tolist()):
        if n == 0:
            continue
        k = ref.rows_of(h.k_cache.numpy(), h.block_tables.numpy()[b], n)
        v = ref.rows_of(h.v_cache.numpy(), h.block_tables.numpy()[b], n)
        q = h.q[b:b + 1].numpy()
        p, _ = ref.weights(q, k, case.scale)
        out[b] = np.einsum("hn,nhd->hd", p[0], np.repeat(v, q.shape[1] // k.shape[1], axis=1))
        w = p[0].reshape(k.shape[1], -1, n).sum(1)
        add[b, :, :n] = w
        tol[b, :, :n] = score_tolerance(w, q, k, case.scale, prior[b, :, :n].astype(np.float64))
    return out, add, tol


def run(case, extra=0, seed=0, ws=None, stream=None):
    rng = np.random.default_rng(seed)
    cap = case.max_blocks_per_seq * case.block_size
    prior = rng.exponential(1.0, (case.num_seqs, case.num_kv_heads, cap + extra)).astype(np.float32)
    want, add, tol = reference(case, prior)
    dev = case.to("cuda")
    scores = torch.from_numpy(prior.copy()).cuda()
    out = torch.full_like(dev.q, float("nan"))
    if ws is None:
        ws = pkv.make_weights_workspace(case.num_seqs, case.num_q_heads, cap, "cuda")
    pkv.decode_attention_weights(out, scores, dev.q, dev.k_cache, dev.v_cache, dev.block_tables, dev.context_lens,
                                 case.scale, ws, stream=stream)
    assert max_err(out, want) <= ATTN_TOL
    got = scores.cpu().numpy().astype(np.float64)
    err = np.abs(got - (prior + add))
    assert (err <= tol).all(), (err.max(), np.argwhere(err > tol)[:3])
    assert_no_device_error()  # untouched entries have a tolerance of zero: they must be as they were
    return out, scores, ws, prior


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [16, 48, 256])
def test_ragged(group, bs):
    case = workloads.random_case(900 + group + bs, [0, 1, 15, 16, 17, 1023, 1024, 1025, 2500, 70], 2 * group, 2, block_size=bs)
    run(case, extra=group, seed=bs)


def test_long_and_peaky():
    case = workloads.random_case(910, [9000, 333], 8, 1, block_size=32, peaky_fraction=0.01, peaky_factor=8.0)
    run(case)


def test_contexts_of_many_partitions():
    run(workloads.random_case(926, [32768, 20001, 1024], 8, 2, block_size=32))


@pytest.mark.parametrize("group", [1, 8])
def test_more_partitions_than_pieces_and_threads(group):
    """264 partitions: more than the 32 pieces of one head's row, and than a CTA has threads."""
    run(workloads.random_case(927, [270000, 40000], group, 1, block_size=256))


def test_steps_accumulate_and_leave_the_workspace_clean():
    case = workloads.random_case(911, [1500, 40, 0], 8, 2, block_size=16)
    _, first, ws, prior = run(case, seed=1)
    counters = ws.clone()
    _, again, _, _ = run(case, seed=1, ws=ws)
    assert torch.equal(first, again)
    assert torch.equal(counters, ws)
    # three steps on one scores tensor add up to three times one step's weights
    dev = case.to("cuda")
    scores = torch.zeros_like(first)
    out = torch.empty_like(dev.q)
    for _ in range(3):
        pkv.decode_attention_weights(out, scores, dev.q, dev.k_cache, dev.v_cache, dev.block_tables, dev.context_lens,
                                     case.scale, ws)
    one = torch.zeros_like(first)
    pkv.decode_attention_weights(out, one, dev.q, dev.k_cache, dev.v_cache, dev.block_tables, dev.context_lens, case.scale, ws)
    assert torch.allclose(scores, 3 * one, rtol=3 * 2.0 ** -23, atol=0)
    # a position's weights over all keys sum to one per q head: 4 heads per kv head (float64 sum of float32 values)
    sums = one.double().sum(-1).cpu().numpy()
    assert np.abs(sums[:2] - 4).max() < 4 * 1e-4 and (sums[2] == 0).all()


def test_one_workspace_for_calls_of_other_sizes():
    """A batch that shrinks and grows again, tables that get narrower and wider, other head counts: one workspace, as large
    as the largest call needs and filled with anything."""
    long, less = [2100, 1025, 1100, 40, 1500, 1030], [1300, 1025, 1100, 40, 1290]
    wide = workloads.random_case(920, [6000, 1040], 8, 2, block_size=16)
    cases = [workloads.random_case(921, long, 8, 2, block_size=16), workloads.random_case(922, long[:5], 8, 2, block_size=16), wide,
             workloads.random_case(923, less, 8, 2, block_size=16), workloads.random_case(924, less, 4, 1, block_size=48),
             workloads.random_case(925, long, 2, 2, block_size=32)]
    sizes = [pkv.make_weights_workspace(c.num_seqs, c.num_q_heads, c.max_blocks_per_seq * c.block_size, "cuda").numel() for c in cases]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 0, 2, 0, 3, 4, 5, 1, 0, 2):
        run(cases[i], seed=i, ws=ws)
    ws.fill_(255)
    for i in (0, 3, 2):
        run(cases[i], seed=i, ws=ws)


def test_stale_rows_past_the_context():
    """Positions past a context hold whatever they held, infinities and NaN included."""
    case = workloads.random_case(912, [21, 1030], 4, 1, block_size=32)
    for b, n in enumerate(case.context_lens.tolist()):
        blk = int(case.block_tables[b, n // 32])
        case.k_cache[blk, :, n % 32:] = float("nan")
        case.v_cache[blk, :, n % 32:] = float("inf")
    run(case)


def test_bad_indices_are_recorded():
    case = workloads.random_case(913, [300, 200], 4, 1, block_size=16)
    dev = case.to("cuda")
    cap = case.max_blocks_per_seq * 16
    ws = pkv.make_weights_workspace(2, 4, cap, "cuda")
    out = torch.empty_like(dev.q)

    def call(bt, cl):
        scores = torch.zeros((2, 1, cap), device="cuda")
        pkv.decode_attention_weights(out, scores, dev.q, dev.k_cache, dev.v_cache, bt, cl, case.scale, ws)
        return scores
    good = call(dev.block_tables, dev.context_lens)
    bad = dev.block_tables.clone()
    bad[0, 2] = case.num_blocks
    s = call(bad, dev.context_lens)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_BLOCK_ID
    assert torch.equal(s[1], good[1])
    s = call(dev.block_tables, torch.tensor([cap + 1, -5], dtype=torch.int32, device="cuda"))
    assert pkv.device_error() == pkv.PKV_DEV_BAD_CONTEXT
    assert not out[1].any() and not s[1].any()
    assert pkv.device_error() == pkv.PKV_DEV_OK


def test_graph_and_other_stream():
    case = workloads.random_case(914, [1100, 64], 8, 2, block_size=16)
    dev = case.to("cuda")
    cap = case.max_blocks_per_seq * 16
    ws = pkv.make_weights_workspace(2, 8, cap, "cuda")
    scores, out = torch.zeros((2, 2, cap), device="cuda"), torch.empty_like(dev.q)
    args = (dev.q, dev.k_cache, dev.v_cache, dev.block_tables, dev.context_lens, case.scale, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.decode_attention_weights(out, scores, *args)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    scores2, out2 = torch.zeros_like(scores), torch.empty_like(out)
    pkv.decode_attention_weights(out2, scores2, *args, stream=s)
    pkv.decode_attention_weights(out2, scores2, *args, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(scores, scores2) and torch.equal(out, out2)


# ---------------------------------------------------------------- a chunk's rows

def run_chunk(ctxs, chunks, group, hkv, bs, seed, poison=False, last=None):
    case = workloads.random_case(seed, ctxs, group * hkv, hkv, block_size=bs)
    if poison:
        for b, n in enumerate(ctxs):
            if n % bs:
                case.k_cache[int(case.block_tables[b, n // bs]), :, n % bs:] = float("nan")
    rng = np.random.default_rng(seed)
    start = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    q = rng.standard_normal((start[-1], group * hkv, 128)).astype(np.float16)
    cap = case.max_blocks_per_seq * bs
    prior = rng.exponential(1.0, (len(ctxs), hkv, cap + 3)).astype(np.float32)
    lse = np.zeros(q.shape[:2])
    add, tol = np.zeros(prior.shape), np.zeros(prior.shape)
    for b, n in enumerate(ctxs):
        if chunks[b] == 0:
            continue
        rows = slice(start[b], start[b + 1])
        k = ref.rows_of(case.k_cache.numpy(), case.block_tables.numpy()[b], n)
        p, z = ref.weights(q[rows], k, case.scale)
        lse[rows] = z
        w = p.reshape(chunks[b], hkv, group, n).sum((0, 2))
        add[b, :, :n] = w
        # lse arrives rounded to float32: 2^-24 of it, twice 2^-23 with its conversion to log2 units; the sum over the
        # rows adds 2^-23 for each of the levels a value passes (128 columns / 4 in turn, then the row tiles)
        size = 4 * float(np.abs(z).max()) * 2.0 ** -23 + (32 + chunks[b] * group / 128) * 2.0 ** -23
        tol[b, :, :n] = score_tolerance(w, q[rows], k, case.scale, prior[b, :, :n].astype(np.float64)) + w * size
    dev = case.to("cuda")
    scores = torch.from_numpy(prior.copy()).cuda()
    qd, zd = torch.from_numpy(q).cuda(), torch.from_numpy(lse.astype(np.float32)).cuda()
    args = (qd, zd, dev.k_cache, dev.block_tables, dev.context_lens, torch.from_numpy(start).cuda(), max(1, max(chunks)), case.scale)
    pkv.prefill_attention_weights(scores, *args)
    got = scores.cpu().numpy().astype(np.float64)
    err = np.abs(got - (prior + add))
    assert (err <= tol).all(), (err.max(), np.argwhere(err > tol)[:3])
    assert_no_device_error()
    return scores, prior, args, dev


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [16, 48, 256])
def test_chunk_ragged(group, bs):
    run_chunk([1, 17, 128, 129, 500, 1000, 300, 4, 260], [1, 5, 128, 1, 33, 200, 300, 0, 64], group, 2, bs, 50 + bs + group, poison=True)


@pytest.mark.parametrize("ctxs,chunks,group,hkv,bs", [([5000], [600], 4, 1, 16), ([1300, 64], [1300, 64], 2, 3, 64), ([700] * 40, [1] * 40, 8, 1, 16)])
def test_chunk_sizes(ctxs, chunks, group, hkv, bs):
    run_chunk(ctxs, chunks, group, hkv, bs, 60)


def test_chunk_behind_long_contexts():
    run_chunk([16384, 8193], [64, 33], 4, 1, 16, 62)


def test_chunk_follows_the_attention():
    """With the log-sum-exps of prefill_attention_paged every row's weights sum to one; one row per request
    adds what decode_attention_weights adds."""
    scores, prior, args, dev = run_chunk([900, 333], [100, 333], 4, 2, 16, 61)
    q, _, kc, bt, cl, qs, n, scale = args
    lse, out = torch.empty(q.shape[:2], device="cuda"), torch.empty_like(q)
    ws = pkv.make_prefill_workspace(2, q.shape[0], 8, 2, bt.shape[1] * 16, "cuda")
    pkv.prefill_attention_paged(out, q, kc, dev.v_cache, bt, cl, qs, n, scale, lse=lse, workspace=ws)
    s = torch.zeros_like(scores)
    pkv.prefill_attention_weights(s, q, lse, kc, bt, cl, qs, n, scale)
    sums = s.double().sum(-1).cpu().numpy()
    assert np.abs(sums - 4 * np.array([[100], [333]])).max() <= 4 * 333 * 2e-4  # each weight within 2 x 1e-4 (see run_chunk)
    one = torch.zeros_like(scores)
    last = torch.tensor([99, 432], device="cuda")
    pkv.prefill_attention_weights(one, q[last], lse[last], kc, bt, cl, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), 1, scale)
    step = torch.zeros_like(scores)
    w = pkv.make_weights_workspace(2, 8, bt.shape[1] * 16, "cuda")
    pkv.decode_attention_weights(torch.empty_like(q[last]), step, q[last], kc, dev.v_cache, bt, cl, scale, w)
    assert torch.allclose(one, step, rtol=1e-3, atol=1e-9)
    # a request cut by a bad range keeps its scores, the other's are the same
    bad = torch.zeros_like(scores)
    pkv.prefill_attention_weights(bad, q, lse, kc, bt, torch.tensor([99, 333], dtype=torch.int32, device="cuda"), qs, n, scale)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_CONTEXT
    assert not bad[0].any() and torch.equal(bad[1], s[1])
