"""Eviction on the GPU: the kept positions, rows and scores must equal the plain definition's bit for bit."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import paged_kv_cache_278_gb300 as pkv
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu


def tables(lens, bs, width, first, rng, total):
    ids = rng.permutation(total) + first
    t, at = np.full((len(lens), width), -1, np.int32), 0
    for b, n in enumerate(lens):
        m = -(-n // bs)
        t[b, :m] = ids[at:at + m]
        at += m
    return t


def state(lens, hkv, bs, seed, kind="heavy", spare_capacity=0):
    rng = np.random.default_rng(seed)
    width = max(1, max(-(-n // bs) for n in lens))
    need = sum(-(-n // bs) for n in lens)
    old = tables(lens, bs, width, 0, rng, need)
    k, v = (rng.standard_normal((2 * need + 2, hkv, bs, 128)).astype(np.float16) for _ in range(2))
    shape = (len(lens), hkv, width * bs + spare_capacity)
    s = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        s = rng.integers(0, 3, shape).astype(np.float32)
    elif kind == "zeros":
        s[:] = 0.0
        s[rng.random(shape) < 0.5] = -0.0
    elif kind == "wild":
        s = rng.standard_normal(shape).astype(np.float32)
        for x in (np.nan, np.inf, -np.inf, 1e-42, -1e-42, -0.0, 0.0):
            s[rng.random(shape) < 0.08] = x
    elif kind == "nan":
        s[:] = np.nan
    fresh = tables(lens, bs, width, need, rng, need)
    return k, v, s, old, fresh, np.array(lens, np.int32)


def bits(x):
    return x.view({2: np.uint16, 4: np.uint32}[x.dtype.itemsize])


def check(k, v, s, old, new, lens, budget, recent, sinks, in_place=False, alias=False, stream=None):
    want = ref.evict(k, v, s, old, new, lens, budget, recent, sinks)
    d = [torch.from_numpy(x.copy()).cuda() for x in (k, v, s, old, new, lens)]
    kept = torch.full((len(lens), s.shape[1], budget), -7, dtype=torch.int32, device="cuda")
    ns = d[2] if alias else torch.full_like(d[2], 9.0)
    nl = d[5] if alias else torch.full_like(d[5], -7)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    pkv.evict(d[0], d[1], kept, ns, nl, d[2], d[3], d[5], budget, recent=recent, sinks=sinks,
              new_tables=None if in_place else d[4], stream=stream)
    torch.cuda.synchronize()
    got = [x.cpu().numpy() for x in (d[0], d[1], kept, ns, nl)]
    assert np.array_equal(got[2], want[2])
    assert np.array_equal(got[4], want[4])
    assert np.array_equal(bits(got[3]), bits(want[3]))
    assert np.array_equal(bits(got[0]), bits(want[0])) and np.array_equal(bits(got[1]), bits(want[1]))
    assert_no_device_error()


LENS = [0, 1, 31, 64, 65, 100, 333, 1000]


@pytest.mark.parametrize("budget,recent,sinks", [(64, 16, 4), (1, 0, 0), (1, 1, 0), (100, 100, 0), (33, 0, 33), (64, 0, 0),
                                                 (999, 500, 7), (2000, 5, 5)])
@pytest.mark.parametrize("kind", ["heavy", "ties"])
def test_fresh_blocks(budget, recent, sinks, kind):
    k, v, s, old, fresh, lens = state(LENS, 2, 16, budget, kind)
    check(k, v, s, old, fresh, lens, budget, recent, sinks)


@pytest.mark.parametrize("bs,hkv", [(16, 1), (48, 2), (256, 3)])
@pytest.mark.parametrize("alias", [False, True])
def test_in_place(bs, hkv, alias):
    k, v, s, old, _, lens = state(LENS + [2100], hkv, bs, bs)
    check(k, v, s, old, old, lens, 200, 30, 2, in_place=True, alias=alias)


@pytest.mark.parametrize("kind", ["zeros", "wild", "nan"])
def test_unusual_scores(kind):
    k, v, s, old, _, lens = state([500, 77, 1500], 2, 32, 5, kind, spare_capacity=13)
    check(k, v, s, old, old, lens, 70, 8, 1, in_place=True)
    check(k, v, s, old, old, lens, 1400, 0, 0, in_place=True, alias=True)


def test_some_blocks_shared():
    """The first blocks go to fresh ones, the others stay: both kinds in one table."""
    k, v, s, old, fresh, lens = state([400, 650], 2, 16, 8)
    mixed = old.copy()
    mixed[:, :5] = fresh[:, :5]
    mixed[1, 7] = fresh[1, 7]
    check(k, v, s, old, mixed, lens, 250, 20, 4)


def test_narrower_new_table():
    k, v, s, old, fresh, lens = state([400, 650, 20], 2, 16, 9)
    check(k, v, s, old, np.ascontiguousarray(fresh[:, :7]), lens, 100, 20, 4)


@pytest.mark.parametrize("n,budget", [(4097, 4096), (8192, 500), (16384, 5000), (32768, 32767), (40001, 20000), (70000, 130),
                                      (140001, 60000)])
def test_long_rows(n, budget):
    """Two to eight CTAs to a row, 4 to 64 scores a thread."""
    k, v, s, old, _, lens = state([n, 1025], 1, 256, n, "ties" if n == 40001 else "wild" if n == 70000 else "heavy")
    check(k, v, s, old, old, lens, budget, 100, 4, in_place=True, alias=True)


def test_many_rows_take_whole_row_slices():
    k, v, s, old, _, lens = state([40 + 3 * i for i in range(40)], 8, 16, 77)
    check(k, v, s, old, old, lens, 50, 10, 0, in_place=True, stream=torch.cuda.Stream())


def test_bad_indices_are_recorded():
    k, v, s, old, fresh, lens = state([100, 100], 1, 16, 2)
    t = lambda x: torch.from_numpy(x.copy()).cuda()  # noqa: E731
    kept = torch.empty((2, 1, 50), dtype=torch.int32, device="cuda")

    def run(tab, new, ln, budget=50):
        nl, kp = torch.empty(2, dtype=torch.int32, device="cuda"), kept[..., :budget].contiguous()
        kd, vd = t(k), t(v)
        pkv.evict(kd, vd, kp, torch.empty_like(t(s)), nl, t(s), t(tab), t(ln), budget, recent=5, new_tables=t(new))
        return kd, nl
    bad = old.copy()
    bad[0, 0], bad[0, 3] = -1, 10 ** 6
    kd, _ = run(bad, fresh, lens)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_BLOCK_ID
    want = ref.evict(k, v, s, old, fresh, lens, 50, 5, 0)[0]
    rows = np.setdiff1d(np.arange(k.shape[0]), fresh[0][fresh[0] >= 0])  # the other request's are right
    assert np.array_equal(bits(kd.cpu().numpy()[rows]), bits(want[rows]))
    _, nl = run(old, fresh, np.array([5000, -3], np.int32))
    assert pkv.device_error() == pkv.PKV_DEV_BAD_CONTEXT
    assert nl.tolist() == [50, 0]
    run(old, fresh[:, :1].copy(), lens)  # 50 positions do not fit one block of 16
    assert pkv.device_error() == pkv.PKV_DEV_BAD_CONTEXT
    assert pkv.device_error() == pkv.PKV_DEV_OK


@pytest.mark.parametrize("alias", [False, True])
def test_short_new_table(alias):
    """A new table too short for what is kept: recorded, and everything the call writes describes the rows that were moved."""
    k, v, s, old, fresh, lens = state([100, 30, 70], 2, 16, 12)
    want = ref.evict(k, v, s, old, np.pad(fresh, ((0, 0), (0, 1)), constant_values=0), lens, 50, 5, 2)
    d = [torch.from_numpy(x.copy()).cuda() for x in (k, v, s, old, np.ascontiguousarray(fresh[:, :2]), lens)]
    kept = torch.full((3, 2, 50), -7, dtype=torch.int32, device="cuda")
    ns, nl = (d[2], d[5]) if alias else (torch.full_like(d[2], 9.0), torch.full_like(d[5], -7))
    pkv.evict(d[0], d[1], kept, ns, nl, d[2], d[3], d[5], 50, recent=5, sinks=2, new_tables=d[4])
    assert pkv.device_error() == pkv.PKV_DEV_BAD_CONTEXT
    assert nl.tolist() == [32, 30, 32]  # two blocks of 16
    kept, ns = kept.cpu().numpy(), ns.cpu().numpy()
    for b, n in enumerate([32, 30, 32]):
        assert np.array_equal(kept[b, :, :n], want[2][b, :, :n]) and (kept[b, :, n:] == -1).all()
        assert np.array_equal(bits(ns[b, :, :n].copy()), bits(want[3][b, :, :n].copy())) and (ns[b, :, n:] == 0).all()
        for h in range(2):
            for c, x in ((d[0], k), (d[1], v)):
                got = ref.rows_of(c.cpu().numpy(), fresh[b], n)[:, h]
                assert np.array_equal(got, ref.rows_of(x, old[b], int(lens[b]))[kept[b, h, :n], h])
    assert pkv.device_error() == pkv.PKV_DEV_OK


def test_largest_budget():
    """A budget near the end of 32 bits: everything is kept, and -1 behind it to the last entry."""
    k, v, s, old, fresh, lens = state([40], 1, 16, 13)
    d = [torch.from_numpy(x.copy()).cuda() for x in (k, v, s, old, fresh, lens)]
    budget = 2 ** 31 - 1
    kept = torch.zeros((1, 1, budget), dtype=torch.int32, device="cuda")  # 8.6 GB
    ns, nl = torch.empty_like(d[2]), torch.empty_like(d[5])
    pkv.evict(d[0], d[1], kept, ns, nl, d[2], d[3], d[5], budget, recent=2 ** 30, sinks=2 ** 30 - 1, new_tables=d[4])
    assert nl.tolist() == [40] and kept[0, 0, :40].tolist() == list(range(40))
    for part in kept[0, 0, 40:].split(1 << 28):
        assert int(part.max()) == -1 == int(part.min())
    assert np.array_equal(ref.rows_of(d[0].cpu().numpy(), fresh[0], 40), ref.rows_of(k, old[0], 40))
    assert_no_device_error()


def test_graph_replay_follows_the_inputs():
    k, v, s, old, fresh, lens = state([300, 200], 2, 16, 4)
    d = [torch.from_numpy(x.copy()).cuda() for x in (k, v, s, old, fresh, lens)]
    kept = torch.empty((2, 2, 64), dtype=torch.int32, device="cuda")
    ns, nl = torch.empty_like(d[2]), torch.empty_like(d[5])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.evict(d[0], d[1], kept, ns, nl, d[2], d[3], d[5], 64, recent=8, new_tables=d[4])
    s2, l2 = s[:, :, ::-1].copy(), np.array([250, 40], np.int32)
    d[2].copy_(torch.from_numpy(s2))
    d[5].copy_(torch.from_numpy(l2))
    graph.replay()
    torch.cuda.synchronize()
    want = ref.evict(k, v, s2, old, fresh, l2, 64, 8, 0)
    assert np.array_equal(kept.cpu().numpy(), want[2]) and np.array_equal(nl.cpu().numpy(), want[4])
    assert np.array_equal(bits(d[0].cpu().numpy()), bits(want[0]))
