"""Attention of drafted trees over the paged cache, their masks and accepted paths, on the GPU against float64."""
import numpy as np
import pytest
import torch

import paged_kv_cache_278_gb300 as pkv
import tree_ref
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu
SCALE = tree_ref.SCALE


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def host(x):
    return x.float().cpu().numpy().astype(np.float64)


def random_parents(rng, n):
    return [int(rng.integers(-1, i)) if i and rng.random() > 0.1 else -1 for i in range(n)]


class Call:
    """One call's tensors: contexts `lens` (trees included), `counts` nodes each."""

    def __init__(self, lens, counts, hq, hkv, bs, seed=0, masks=None, words=None, before=0, behind=0, fused=False):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.counts, self.hq, self.hkv, self.bs = lens, counts, hq, hkv, bs
        need = [-(-n // bs) for n in lens]
        self.width, nb = max(1, max(need)), sum(need) + 3
        perm = rng.permutation(nb)
        self.table = np.full((len(lens), self.width), -7, np.int32)  # entries past a request's blocks are never read
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.kc, self.vc = (torch.randn((nb, hkv, bs, 128), generator=g, device="cuda").half() for _ in range(2))
        t = before + sum(counts) + behind
        self.start = before + np.concatenate([[0], np.cumsum(counts)])
        self.longest = max(1, max(counts))
        words = words or -(-self.longest // 32)
        self.seen = masks or [tree_ref.ancestors(random_parents(rng, n)) for n in counts]
        self.mask = rng.integers(-2 ** 31, 2 ** 31, (t, words)).astype(np.int32)  # garbage past each tree's nodes
        for b, n in enumerate(counts):
            if n:
                own = tree_ref.pack_masks(self.seen[b], words).view(np.uint32)
                live = tree_ref.pack_masks(np.ones((n, n), bool), words).view(np.uint32)
                rows = slice(self.start[b], self.start[b + 1])
                self.mask[rows] = ((self.mask[rows].view(np.uint32) & ~live) | own).view(np.int32)
        x = torch.randn((t, hq + 5, 128), generator=g, device="cuda").half()
        self.q = x[:, 2:2 + hq] if fused else x[:, :hq].contiguous()
        self.ws = pkv.make_tree_workspace(len(lens), t, self.longest, hq, hkv, self.width * bs, "cuda")

    def run(self, lse=True, stream=None, out=None):
        t = self.q.shape[0]
        out = torch.full((t, self.hq, 128), 7.0, dtype=torch.float16, device="cuda") if out is None else out
        z = torch.full((t, self.hq), 7.0, device="cuda") if lse else None
        pkv.decode_attention_tree(out, self.q, self.kc, self.vc, i32(self.table), i32(self.lens), i32(self.start), i32(self.mask),
                                  self.longest, SCALE, lse=z, workspace=self.ws, stream=stream)
        return out, z

    def check(self, out, z, requests=None):
        """A score's error is at most 136 x 2^-23 of scale |q| |k| (8 matrix instructions of 17 addends, each cut to 24
        bits, on values no larger); a weight's twice that relative to itself, 8 steps of 2^-23 for its exponential, scaling
        and the sums, and half a step of fp16 (2^-11; 2^-25 of the largest weight when it is subnormal).  The output
        adds its own half step."""
        kc, vc, q = host(self.kc), host(self.vc), host(self.q)
        o, zz = host(out), None if z is None else z.double().cpu().numpy()
        inside = np.zeros(q.shape[0], bool)
        for b, (n, c) in enumerate(zip(self.lens, self.counts)):
            rows = slice(self.start[b], self.start[b + 1])
            inside[rows] = True
            if c == 0 or (requests is not None and b not in requests):
                continue
            k, v = (tree_ref.rows_of(x, self.table[b], n) for x in (kc, vc))
            want, lse, p = tree_ref.attend(q[rows], k, v, self.seen[b])
            rep = self.hq // self.hkv
            vv = np.abs(np.nan_to_num(np.repeat(v, rep, 1)))
            size = SCALE * np.sqrt((q[rows] ** 2).sum(-1)).max() * np.sqrt((np.nan_to_num(k) ** 2).sum(-1)).max()
            dot = 136 * size * 2.0 ** -23
            tol = (np.einsum("chn,nhd->chd", p, vv) * (2.0 ** -11 + 2 * dot + 8 * 2.0 ** -23) + n * 2.0 ** -25 * vv.max()
                   + 2.0 ** -11 * np.abs(want) + 2.0 ** -25)
            err = np.abs(o[rows] - want)
            assert (err <= tol).all(), (b, np.nanmax(err), np.argwhere(~(err <= tol))[:4])
            if zz is not None:
                blind = np.isneginf(lse)
                assert np.array_equal(np.isneginf(zz[rows]), blind)
                lse, got = lse[~blind], zz[rows][~blind]
                assert (np.abs(got - lse) <= dot + 8 * 2.0 ** -23 * (1 + np.abs(lse))).all()
        assert (o[~inside] == 7).all() and (zz is None or (zz[~inside] == 7).all())


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("hkv,bs", [(1, 16), (3, 48), (2, 256)])
def test_ragged(group, hkv, bs):
    """Trees of 1 to 150 nodes, contexts that are the tree alone, end in the middle of tiles and blocks, rows of no request."""
    c = Call([1, 5, 40, 129, 0, 300, 257, 700, 128, 131], [1, 5, 1, 2, 0, 61, 64, 150, 128, 3], group * hkv, hkv, bs, group, before=3, behind=4,
             fused=group != 2)
    c.check(*c.run())
    assert_no_device_error()


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("lens,counts,hkv,bs", [([1], [1], 1, 16), ([16, 17, 300, 0, 33], [1, 16, 8, 0, 33], 2, 16), ([480, 129, 5], [61, 3, 1], 1, 48),
                                                ([256, 500], [20, 31], 3, 256), ([512], [130], 1, 128)])
def test_short_contexts(group, lens, counts, hkv, bs):
    """Few rows over tables of up to 512 positions: one warp has no chunk or several, rows end inside a tile, trees start
    inside a chunk."""
    c = Call(lens, counts, group * hkv, hkv, bs, group + len(lens), before=2, behind=3, fused=group != 2)
    assert c.ws is None
    out, z = c.run()
    c.check(out, z)
    assert torch.equal(c.run()[0], out)
    assert_no_device_error()


def test_short_contexts_any_mask():
    rng = np.random.default_rng(7)
    lens, counts = [40, 40, 300, 33, 8], [40, 17, 40, 33, 8]
    masks = [rng.random((n, n)) < 0.3 for n in counts]
    masks[0][5] = masks[0][39] = False
    masks[1][3] = False
    masks[3][:] = False
    masks[4][:] = True
    c = Call(lens, counts, 8, 2, 16, 4, masks=masks, words=4)
    out, z = c.run()
    c.check(out, z)
    assert (out[5] == 0).all() and torch.isneginf(z[5]).all()
    assert (out[c.start[3]:c.start[4]] == 0).all()
    c.check(out, c.run(lse=False)[1])
    assert_no_device_error()


@pytest.mark.parametrize("lens,counts,hq,hkv,bs", [([4000], [8], 8, 2, 16), ([9000], [37], 4, 1, 64), ([3000, 20, 5000], [61, 20, 7], 32, 8, 16),
                                                    ([2500, 2500], [300, 200], 16, 2, 32), ([1030] * 70, [3] * 70, 8, 1, 16),
                                                    ([700] * 40, [1] * 40, 8, 8, 16)])
def test_long_contexts(lens, counts, hq, hkv, bs):
    """Items cut over several CTAs and joined, and more items than CTAs."""
    c = Call(lens, counts, hq, hkv, bs, len(lens))
    out, z = c.run()
    c.check(out, z, requests=range(0, len(lens), max(1, len(lens) // 6)))
    again, z2 = c.run()
    assert torch.equal(out, again) and torch.equal(z, z2)  # no order of arrival enters a result
    assert_no_device_error()


@pytest.mark.parametrize("seqs", [127, 128, 300])
def test_hundreds_of_requests(seqs):
    """More requests than are read at once, most of them without a tree, some with long contexts cut over CTAs."""
    counts = [(7 * i) % 5 if i % 3 else 0 for i in range(seqs)]
    lens = [c + (13 * i) % 90 + (2000 if i % 50 == 1 else 0) for i, c in enumerate(counts)]
    c = Call(lens, counts, 4, 2, 16, seqs, before=1, behind=2)
    out, z = c.run()
    c.check(out, z)
    assert torch.equal(c.run()[0], out)
    assert_no_device_error()


def test_out_may_be_q():
    for lens, counts in (([300, 40], [8, 5]), ([3000, 700], [50, 70])):
        c = Call(lens, counts, 8, 2, 16, 3)
        want = c.run()[0]
        q = c.q.clone()
        c.run(out=c.q)
        assert torch.equal(c.q, want)
        c.q.copy_(q)
    assert_no_device_error()


def test_a_line_is_the_causal_step():
    """A tree without branches is a chunk: the same values as the causal call to its own tolerance."""
    lens, counts = [500, 90, 1500], [16, 5, 33]
    c = Call(lens, counts, 8, 2, 16, 9, masks=[np.tril(np.ones((n, n), bool)) for n in counts])
    out, z = c.run()
    c.check(out, z)
    other, z2 = torch.empty_like(out), torch.empty_like(z)
    ws = pkv.make_prefill_workspace(3, c.q.shape[0], 8, 2, c.width * 16, "cuda")
    pkv.prefill_attention_paged(other, c.q, c.kc, c.vc, i32(c.table), i32(lens), i32(c.start), 33, SCALE, lse=z2, workspace=ws)
    # two results, each within the tolerance above: some 2^-10 of values up to 4
    assert (out.float() - other.float()).abs().max() <= 4 * 2.0 ** -9 and (z - z2).abs().max() <= 1e-3


def test_any_mask():
    """Masks that are no trees: rows without their own bit, rows that see nothing of the tree, later nodes, all of it, and
    without a context before the tree rows that see nothing at all."""
    rng = np.random.default_rng(3)
    lens, counts = [40, 40, 700, 33, 8], [40, 17, 70, 33, 8]
    masks = [rng.random((n, n)) < 0.3 for n in counts]
    masks[0][5] = masks[0][39] = False
    masks[1][3] = False
    masks[3][:] = False
    masks[4][:] = True
    c = Call(lens, counts, 8, 2, 16, 4, masks=masks, words=4)
    out, z = c.run()
    c.check(out, z)
    assert (out[5] == 0).all() and torch.isneginf(z[5]).all()
    assert (out[c.start[3]:c.start[4]] == 0).all()
    assert_no_device_error()


def test_a_long_blind_row():
    """A tree of 1024 nodes without a context: rows that see nothing in any of several CTAs' parts."""
    rng = np.random.default_rng(5)
    seen = rng.random((1024, 1024)) < 0.05
    seen[::7] = False
    seen[1::7, :900] = False  # nothing in the first parts
    c = Call([1024], [1024], 2, 1, 16, 6, masks=[seen])
    out, z = c.run()
    c.check(out, z)
    assert (out[::7] == 0).all() and torch.isneginf(z[::7]).all()
    assert_no_device_error()


@pytest.mark.parametrize("hq,hkv,long", [(2, 2, False), (8, 1, False), (8, 1, True)])
def test_infinities_in_what_a_row_does_not_see(hq, hkv, long):
    """NaN and infinities in a node's K and V and past the context reach the rows that see the node and no others; those
    rows get V's whole."""
    n, c = (3000 if long else 200), 40
    rng = np.random.default_rng(2)
    call = Call([n], [c], hq, hkv, 16, 8, masks=[tree_ref.ancestors(random_parents(rng, c))])
    call.seen[0][:, [4, 11, 39]] = False  # K: nobody sees them
    call.seen[0][[6, 30], 20] = True
    call.seen[0][7, 20] = False
    own = tree_ref.pack_masks(call.seen[0], call.mask.shape[1])
    call.mask[:] = own
    slot = lambda node: (int(call.table[0, (n - c + node) // 16]), (n - c + node) % 16)  # noqa: E731
    call.vc[slot(20)[0], 0, slot(20)[1], 5] = 0
    clean, z = call.run()
    call.check(clean, z)
    for node, x in ((4, float("nan")), (11, float("inf")), (39, float("-inf"))):
        b, o = slot(node)
        call.kc[b, :, o] = x
        call.vc[b, :, o] = float("nan")
    last = n % 16
    if last:
        call.kc[int(call.table[0, n // 16]), :, last:] = float("nan")
        call.vc[int(call.table[0, n // 16]), :, last:] = float("inf")
    b, o = slot(20)
    call.vc[b, 0, o, 5] = float("-inf")
    out, z2 = call.run()
    expect = clean.float().view(c, hkv, -1, 128).clone()
    rows = torch.tensor(call.seen[0][:, 20], device="cuda")
    expect[rows, 0, :, 5] = float("-inf")
    assert torch.equal(out.float().view(expect.shape), expect) and torch.equal(z, z2)
    assert_no_device_error()


def test_bad_requests_are_skipped():
    c = Call([50, 60, 70], [4, 5, 6], 4, 2, 16, 1)
    good, z = c.run()
    for lens in ([50, 4, 70], [50, 10 ** 6, 70]):
        c.lens = lens
        out, _ = c.run()
        assert pkv.device_error() == pkv.PKV_DEV_BAD_CONTEXT
        assert (out[4:9] == 7).all() and torch.equal(out[:4], good[:4]) and torch.equal(out[9:], good[9:])
    c.lens = [50, 60, 70]
    c.longest = 5  # the last tree is longer than the call says
    out, _ = c.run()
    assert pkv.device_error() == pkv.PKV_DEV_BAD_CONTEXT
    assert (out[9:] == 7).all() and torch.equal(out[:9], good[:9])
    c.longest = 6
    c.table[1, 0] = 10 ** 6
    c.run()
    assert pkv.device_error() == pkv.PKV_DEV_BAD_BLOCK_ID


def test_nothing_to_do():
    c = Call([20, 30], [0, 0], 4, 2, 16, 1, behind=3)
    out, z = c.run()
    assert (out == 7).all() and (z == 7).all()
    assert_no_device_error()


def test_graph_streams_and_shared_workspace():
    """A captured call replayed on new contexts, and eager calls of other sizes between the replays on the same workspace."""
    c = Call([3000, 900], [20, 9], 8, 2, 16, 12)
    other = Call([2000], [30], 8, 1, 16, 13)
    ws = torch.empty(max(c.ws.numel(), other.ws.numel()), dtype=torch.uint8, device="cuda")
    want_other = other.run()[0]
    c.ws = other.ws = ws
    lens, table, start, mask = i32(c.lens), i32(c.table), i32(c.start), i32(c.mask)
    out = torch.empty((c.q.shape[0], 8, 128), dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pkv.decode_attention_tree(out, c.q, c.kc, c.vc, table, lens, start, mask, c.longest, SCALE, workspace=ws)
    for new in ([3000, 900], [500, 899], [2047, 10]):
        lens.copy_(i32(new))
        ws.fill_(0xff)  # NaN everywhere: nothing of the workspace is read before it is written
        graph.replay()
        got = out.clone()
        assert torch.equal(other.run()[0], want_other)
        c.lens = new
        assert torch.equal(c.run(lse=False)[0], got)
    c.check(got, None)
    c.lens = [3000, 900]
    want = c.run()[0]
    torch.cuda.synchronize()
    mine = torch.empty_like(want)
    c.run(stream=s, out=mine)
    s.synchronize()
    assert torch.equal(mine, want)
    assert_no_device_error()


@pytest.mark.parametrize("counts,extra", [([1], 0), ([5, 0, 64, 33], 1), ([300, 1024, 2], 0)])
def test_masks(counts, extra):
    rng = np.random.default_rng(len(counts))
    parents = [random_parents(rng, n) for n in counts]
    parents[-1] = list(range(-1, counts[-1] - 1))  # a line, the deepest
    start = 2 + np.concatenate([[0], np.cumsum(counts)])
    t, words = start[-1] + 3, -(-max(counts) // 32) + extra
    flat = np.full(t, 99, np.int32)
    for b, p in enumerate(parents):
        flat[start[b]:start[b + 1]] = p
    mask, depths = torch.full((t, words), 7, dtype=torch.int32, device="cuda"), torch.full((t,), 7, dtype=torch.int32, device="cuda")
    pkv.tree_masks(mask, depths, i32(flat), i32(start), max(counts))
    assert_no_device_error()
    want, want_depth = np.full((t, words), 7, np.int32), np.full(t, 7, np.int32)
    for b, p in enumerate(parents):
        if p:
            seen = tree_ref.ancestors(p)
            want[start[b]:start[b + 1]] = tree_ref.pack_masks(seen, words)
            want_depth[start[b]:start[b + 1]] = seen.sum(1) - 1
    assert np.array_equal(mask.cpu().numpy(), want) and np.array_equal(depths.cpu().numpy(), want_depth)
    again = torch.full_like(mask, 7)
    pkv.tree_masks(again, None, i32(flat), i32(start), max(counts))
    assert torch.equal(again, mask)


def test_masks_of_bad_parents():
    """A parent at or behind its node is taken for the context, and recorded."""
    mask = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    pkv.tree_masks(mask, None, i32([-1, 1, 3, 0]), i32([0, 4]), 4)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_PATH
    assert mask.view(-1).tolist() == [1, 2, 4, 9]


def keep(c, paths, in_place=False, max_path=None):
    """(what the call leaves, what it should leave) for accepted nodes `paths`."""
    kc, vc = c.kc.clone(), c.vc.clone()
    most = max_path or max(1, max(len(p) for p in paths))
    path = np.full((len(paths), most), -5, np.int32)  # entries past a path's length are not read
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    lens = i32(c.lens)
    new = lens if in_place else torch.full_like(lens, -1)
    pkv.keep_path(kc, vc, i32(c.table), lens, i32(c.start), i32(path), i32([len(p) for p in paths]), new_lens=new)
    want = [c.kc.clone(), c.vc.clone()]
    for b, p in enumerate(paths):
        base = c.lens[b] - c.counts[b]
        for i, node in enumerate(p):
            x, y = base + node, base + i
            for old, to in zip((c.kc, c.vc), want):
                to[int(c.table[b, y // c.bs]), :, y % c.bs] = old[int(c.table[b, x // c.bs]), :, x % c.bs]
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    assert new.tolist() == [n - m + len(p) for n, m, p in zip(c.lens, c.counts, paths)]


@pytest.mark.parametrize("hkv,bs,in_place", [(1, 16, False), (8, 16, True), (3, 48, False), (40, 32, True)])
def test_keep_path(hkv, bs, in_place):
    rng = np.random.default_rng(hkv)
    lens, counts = [40, 1, 333, 64, 90, 500, 30], [16, 1, 61, 64, 8, 300, 0]
    c = Call(lens, counts, hkv, hkv, bs, 5)
    paths = [sorted(rng.choice(n, size=min(n, 1 + 5 * b), replace=False).tolist()) if n else [] for b, n in enumerate(counts)]
    paths[0] = [0, 1, 2, 15]        # rows that stay and one that moves
    paths[3] = list(range(64))      # all of it
    paths[4] = []                   # nothing accepted
    paths[5] = list(range(100, 300, 2))  # longer than what is in flight at once, sources and targets overlap
    keep(c, paths, in_place)
    assert_no_device_error()


def test_keep_path_layer_by_layer():
    """Without new_lens the lengths stay, for the next layer's call."""
    c = Call([40, 50], [8, 9], 2, 2, 16, 5)
    kc, vc, lens = c.kc.clone(), c.vc.clone(), i32([40, 50])
    args = i32(c.table), lens, i32(c.start), i32([[1, 5], [3, -1]]), i32([2, 1])
    pkv.keep_path(kc, vc, *args)
    assert lens.tolist() == [40, 50]
    k2, v2 = c.kc.clone(), c.vc.clone()
    pkv.keep_path(k2, v2, *args, new_lens=lens)
    assert lens.tolist() == [34, 42] and torch.equal(kc, k2) and torch.equal(vc, v2)
    assert_no_device_error()


@pytest.mark.parametrize("path,n,code", [([3, 2], 2, "BAD_PATH"), ([1, 1], 2, "BAD_PATH"), ([-1, 2], 2, "BAD_PATH"), ([0, 8], 2, "BAD_PATH"),
                                         ([0, 1], 3, "BAD_PATH"), ([0, 1], -1, "BAD_PATH")])
def test_bad_paths_change_nothing(path, n, code):
    c = Call([40, 50], [8, 9], 2, 2, 16, 5)
    kc, vc, new = c.kc.clone(), c.vc.clone(), i32([-1, -1])
    pkv.keep_path(kc, vc, i32(c.table), i32(c.lens), i32(c.start), i32([path, [2, 4]]), i32([n, 2]), new_lens=new)
    assert pkv.device_error() == getattr(pkv, "PKV_DEV_" + code)
    assert new.tolist() == [40, 43]
    for got, old in ((kc, c.kc), (vc, c.vc)):
        own = torch.tensor(c.table[0, :3], device="cuda").long()
        assert torch.equal(got[own], old[own]) and not torch.equal(got, old)


def test_bad_contexts_and_blocks():
    c = Call([40, 50], [8, 9], 2, 2, 16, 5)
    kc, vc, new = c.kc.clone(), c.vc.clone(), i32([-1, -1])
    args = i32(c.start), i32([[2, 4], [2, 4]]), i32([2, 2])
    pkv.keep_path(kc, vc, i32(c.table), i32([5, 10 ** 6]), *args, new_lens=new)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_CONTEXT
    assert new.tolist() == [5, 10 ** 6] and torch.equal(kc, c.kc) and torch.equal(vc, c.vc)
    c.table[0, 2] = -1  # positions 32 .. 39: the tree's
    pkv.keep_path(kc, vc, i32(c.table), i32(c.lens), *args, new_lens=new)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_BLOCK_ID
    assert new.tolist() == [34, 43]
