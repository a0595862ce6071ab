"""Norms per head with the rotation on the GPU against float64: layouts, head sizes, several axes, strides, in place, the
fused appends (fp16 and fp8), and the fp8 cache read back."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import paged_kv_cache_278_gb300 as pkv
import tree_ref
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu
EPS = 1e-6
F8 = torch.float8_e4m3fn


def error(size, normed):
    """float32 error of a rotated row's elements.  Rotation: 5e-7 of |y_a| + |y_b| (angle pi 2^-25, cos and sin two
    steps of 2^-24, each product and the sum 2^-24).  Norm: a sum of 16-element chains of eight, four shuffles and an fma, at
    most 16 roundings of 2^-24 on positive terms and half of that on its root, rsqrt 2 steps of 2^-23, two products:
    (8 + 4 + 2) x 2^-24 = 8.4e-7."""
    return (1.35e-6 if normed else 5e-7) * size


def close(got, want, size, normed=True):
    """fp16 rounds by half a step: 2^-11 of the value, 2^-25 under the normal range."""
    got = got.float().cpu().numpy().astype(np.float64)
    tol = 2.0 ** -11 * np.abs(want) * (1 + 1e-5) + error(size, normed) + 2.0 ** -25
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def make(t, hq, hkv, d, seed, fused=False, axes=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((t, hq + 2 * hkv, d), generator=g, device="cuda") * torch.exp(torch.randn((t, hq + 2 * hkv, 1), generator=g, device="cuda"))).half()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw, kw = (1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    pos = torch.randint(-3000, 70000, (t, axes), generator=g, device="cuda", dtype=torch.int32)
    return q, k, v, qw, kw, pos


def host(x):
    return x.cpu().numpy().astype(np.float64)


def want_of(x, w, pos, axes, rotary, magnitude=1.0, interleaved=False):
    ax = np.zeros(rotary // 2, int) if axes is None else axes.cpu().numpy()
    return tree_ref.norm_rotate(host(x), None if w is None else host(w), EPS, pos.cpu().numpy().reshape(x.shape[0], -1), ax,
                                ref.frequencies(rotary)[0], magnitude, interleaved)


@pytest.mark.parametrize("t,hq,hkv,d,rotary,interleaved,fused,sections", [
    (1, 1, 1, 128, 128, False, False, None), (1, 8, 1, 128, 16, True, True, None), (17, 32, 8, 128, 128, False, True, [16, 24, 24]),
    (305, 4, 4, 128, 64, True, False, [8, 24]), (5, 3, 1, 96, 48, False, False, None), (7, 2, 2, 256, 256, False, True, [32, 32, 32, 32]),
    (400, 40, 8, 128, 96, False, True, None), (33, 130, 2, 128, 128, True, False, [20, 22, 22]), (2, 5, 1, 16, 16, True, False, None),
    (9, 6, 2, 64, 32, False, True, None), (3, 4, 2, 32, 32, False, False, [10, 6]), (6, 2, 1, 144, 80, False, True, None),
    (310, 3, 3, 240, 240, True, True, None)])
def test_norm_rope(t, hq, hkv, d, rotary, interleaved, fused, sections):
    q, k, _, qw, kw, pos = make(t, hq, hkv, d, t + d, fused, 1 if sections is None else len(sections))
    axes = None if sections is None else pkv.rope_axes(sections)
    if sections is None:
        pos = pos[:, 0].contiguous()
    freq = pkv.rope_frequencies(rotary)
    qo, ko = torch.full((t, hq, d), float("nan"), dtype=torch.float16, device="cuda"), torch.zeros((t, hkv, d), dtype=torch.float16, device="cuda")
    pkv.norm_rope(qo, ko, q, k, pos, freq, qw, kw, EPS, axes=axes, interleaved=interleaved)
    for out, x, w in ((qo, q, qw), (ko, k, kw)):
        close(out, *want_of(x, w, pos, axes, rotary, interleaved=interleaved))
    # in place, inside the projection's rows: same bits, and nothing else of the rows changes
    whole = q._base.clone() if fused else None
    pkv.norm_rope(q, k, q, k, pos, freq, qw, kw, EPS, axes=axes, interleaved=interleaved)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    if fused:
        assert torch.equal(q._base[:, hq + hkv:], whole[:, hq + hkv:])
    assert_no_device_error()


def test_scrambled_axes_and_magnitude():
    """Any assignment of pairs to axes; equal positions on all axes are one axis."""
    q, k, _, qw, kw, pos = make(20, 4, 2, 128, 4, axes=3)
    axes = torch.randint(0, 3, (64,), dtype=torch.int32, device="cuda")
    freq = pkv.rope_frequencies(128)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.norm_rope(qo, ko, q, k, pos, freq, qw, kw, EPS, axes=axes, magnitude=1.25)
    close(qo, *want_of(q, qw, pos, axes, 128, magnitude=1.25))
    close(ko, *want_of(k, kw, pos, axes, 128, magnitude=1.25))
    same = pos[:, :1].expand(-1, 3).contiguous()
    a, b = torch.empty_like(q), torch.empty_like(q)
    pkv.norm_rope(a, ko, q, k, same, freq, qw, kw, EPS, axes=axes)
    pkv.norm_rope(b, ko, q, k, pos[:, 0].contiguous(), freq, qw, kw, EPS)
    assert torch.equal(a, b)
    assert_no_device_error()


@pytest.mark.parametrize("which", ["q", "k", "none"])
def test_without_weights(which):
    """Rows without a weight are rotated as rope rotates them, bit for bit."""
    q, k, _, qw, kw, pos = make(11, 6, 2, 128, 8)
    pos, freq = pos[:, 0].contiguous(), pkv.rope_frequencies(64)
    qo, ko, qr, kr = (torch.empty_like(x) for x in (q, k, q, k))
    pkv.rope(qr, kr, q, k, pos, freq)
    pkv.norm_rope(qo, ko, q, k, pos, freq, qw if which == "q" else None, kw if which == "k" else None, EPS)
    if which == "q":
        close(qo, *want_of(q, qw, pos, None, 64))
    else:
        close(qo, *want_of(q, None, pos, None, 64), normed=False)
        assert torch.equal(qo, qr)
    if which == "k":
        close(ko, *want_of(k, kw, pos, None, 64))
    else:
        assert torch.equal(ko, kr)


def test_extreme_rows():
    """Rows of zeros stay zero (eps > 0), rows of fp16's largest values and of its smallest subnormals keep their norm; an
    infinity makes its row NaN where the formula does, and no other row."""
    d = 128
    x = torch.randn((6, 2, d), device="cuda").half()
    x[0] = 0
    x[1] = 65504
    x[2] = 2.0 ** -24
    x[4, 0, 3] = float("inf")
    w = torch.ones(d, device="cuda")
    pos, freq = torch.arange(6, dtype=torch.int32, device="cuda"), pkv.rope_frequencies(d)
    qo, ko = torch.empty_like(x), torch.empty_like(x)
    for eps in (1e-6, 1e-12):
        pkv.norm_rope(qo, ko, x, x, pos, freq, w, w, eps)
        assert torch.equal(qo.nan_to_num(7.0), ko.nan_to_num(7.0)) and (qo[0] == 0).all()  # (NaN is not equal to itself)
        keep = [1, 2, 3, 5]
        want = tree_ref.norm_rotate(host(x[keep]), host(w), eps, host(pos[keep])[:, None].astype(int), np.zeros(64, int), ref.frequencies(d)[0])
        close(qo[keep], *want)
        assert torch.isfinite(qo[4, 1]).all() and torch.isnan(qo[4, 0, 3]) and torch.isnan(qo[4, 0, 67])
    assert_no_device_error()


@pytest.mark.parametrize("t,hq,hkv,bs,rotary,interleaved,axes", [(1, 8, 8, 16, 128, False, 1), (40, 16, 2, 48, 64, True, 2), (333, 32, 8, 16, 128, False, 3)])
def test_append(t, hq, hkv, bs, rotary, interleaved, axes):
    q, k, v, qw, kw, pos = make(t, hq, hkv, 128, t, True, axes)
    ax = torch.randint(0, axes, (rotary // 2,), dtype=torch.int32, device="cuda")
    nb = -(-t // bs) + 2
    g = torch.Generator(device="cuda").manual_seed(t)
    kc, vc = (torch.randn((nb, hkv, bs, 128), generator=g, device="cuda").half() for _ in range(2))
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:t].contiguous()
    if t > 3:
        slots[2] = -1
    freq = pkv.rope_frequencies(rotary)
    more = dict(axes=ax, interleaved=interleaved)
    qo, ko = torch.empty((t, hq, 128), dtype=torch.float16, device="cuda"), torch.empty((t, hkv, 128), dtype=torch.float16, device="cuda")
    pkv.norm_rope(qo, ko, q, k, pos, freq, qw, kw, EPS, **more)
    want_k, want_v = kc.clone(), vc.clone()
    pkv.append(want_k, want_v, slots, ko, v.contiguous())
    qa = torch.full_like(qo, float("nan"))
    pkv.norm_rope_append(qa, q, k, v, kc, vc, slots, pos, freq, qw, kw, EPS, **more)
    assert torch.equal(qa, qo) and torch.equal(kc, want_k) and torch.equal(vc, want_v)
    assert_no_device_error()
    # a slot past the pool: skipped and recorded, the others written
    slots[0] = nb * bs
    kc2, vc2 = kc.clone(), vc.clone()
    pkv.norm_rope_append(q, q, k, v, kc2, vc2, slots, pos, freq, qw, kw, EPS, **more)  # q in place
    assert torch.equal(q, qo) and torch.equal(kc2, kc) and torch.equal(vc2, vc)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_SLOT


@pytest.mark.parametrize("t,hq,hkv,bs,rotary,interleaved,normed", [(1, 8, 8, 16, 128, False, True), (40, 16, 2, 48, 64, True, True),
                                                                    (333, 32, 8, 16, 96, False, False), (310, 1, 1, 256, 16, False, True)])
def test_append_fp8kv(t, hq, hkv, bs, rotary, interleaved, normed):
    """K rows: codes within half an E4M3 step of the float64 row (2^-4 of the value, 2^-10 scales under the normal range)
    and its scale; V rows as append_fp8kv leaves them; untouched slots as they were."""
    q, k, v, qw, kw, pos = make(t, hq, hkv, 128, t, True)
    pos, freq = pos[:, 0].contiguous(), pkv.rope_frequencies(rotary)
    if t > 30:
        k[7], v[8] = 0, 0  # zero rows: scale 0, codes 0
    if not normed:
        qw = kw = None
    nb = -(-t // bs) + 2
    cache = pkv.empty_fp8kv_cache(nb, hkv, bs, "cuda")
    for x in cache:
        x.fill_(3)
    other = [x.clone() for x in cache]
    slots = torch.randperm(nb * bs, device="cuda")[:t].contiguous()
    if t > 3:
        slots[2] = -1
    qo = torch.empty((t, hq, 128), dtype=torch.float16, device="cuda")
    pkv.norm_rope_append_fp8kv(qo, q, k, v, *cache, slots, pos, freq, qw, kw, EPS, interleaved=interleaved)
    qr, kr = torch.empty_like(qo), torch.empty((t, hkv, 128), dtype=torch.float16, device="cuda")
    pkv.norm_rope(qr, kr, q, k, pos, freq, qw, kw, EPS, interleaved=interleaved)
    assert torch.equal(qo, qr)
    pkv.append_fp8kv(*other, slots, kr, v.contiguous())
    assert torch.equal(cache[2], other[2]) and torch.equal(cache[3], other[3])
    flat = lambda x: x.transpose(1, 2).reshape(nb * bs, hkv, *x.shape[3:])  # noqa: E731
    live = slots >= 0
    at = slots[live]
    codes, scale = flat(cache[0])[at].view(F8).double().cpu().numpy(), host(flat(cache[1])[at])
    z, size = want_of(k, kw, pos, None, rotary, interleaved=interleaved)
    z, size = z[live.cpu().numpy()], size[live.cpu().numpy()]
    err = error(size, normed)
    most = np.abs(z).max(-1)
    assert (np.abs(scale - most / 448) <= err.max(-1) / 448 + 2.0 ** -23 * scale).all()
    assert (np.abs(codes * scale[..., None] - z) <= 2.0 ** -4 * np.abs(z) * (1 + 1e-5) + 2.0 ** -10 * scale[..., None] * 1.001 + 2 * err).all()
    if normed and t > 30:
        assert (flat(cache[0])[slots[7]] == 0).all() and (flat(cache[1])[slots[7]] == 0).all()
    rest = torch.ones(nb * bs, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (flat(cache[0])[rest] == 3).all() and (flat(cache[1])[rest] == 3).all()
    assert_no_device_error()


@pytest.mark.parametrize("weight", [1e-30, 1e30, 3e36])
@pytest.mark.parametrize("t", [3, 400])
def test_fp8_scales_of_any_size(weight, t):
    """Rows whose scale is far from one: the codes are still those of the quotient."""
    hkv, bs = 2, 16
    q, k, v, qw, kw, pos = make(t, 2, hkv, 128, 17)
    kw = kw * weight
    pos, freq, slots = pos[:, 0].contiguous(), pkv.rope_frequencies(128), torch.arange(t, device="cuda")
    cache = pkv.empty_fp8kv_cache(-(-t // bs), hkv, bs, "cuda")
    pkv.norm_rope_append_fp8kv(torch.empty_like(q), q, k, v, *cache, slots, pos, freq, qw, kw, EPS)
    flat = lambda x: x.transpose(1, 2).reshape(-1, hkv, *x.shape[3:])[:t]  # noqa: E731
    codes, scale = flat(cache[0]).view(F8).double().cpu().numpy(), host(flat(cache[1]))
    z, size = want_of(k, kw, pos, None, 128)
    err = error(size, True)
    assert (np.abs(scale - np.abs(z).max(-1) / 448) <= err.max(-1) / 448 + 2.0 ** -23 * scale).all()
    assert (np.abs(codes * scale[..., None] - z) <= 2.0 ** -4 * np.abs(z) * (1 + 1e-5) + 2.0 ** -10 * scale[..., None] * 1.001 + 2 * err).all()
    assert_no_device_error()


def test_fp8_codes_are_the_append_s():
    """K rows that are neither normalised nor turned (position 0) have append_fp8kv's codes and scales, bit for bit: rows of
    all sizes, infinities and NaN among them."""
    t, hkv, bs = 700, 2, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    k = (torch.randn((t, hkv, 128), generator=g, device="cuda") * torch.exp(4 * torch.randn((t, hkv, 1), generator=g, device="cuda"))).half()
    k[5] = 0
    k[6, 0] = 2.0 ** -24
    k[7, 1, 3] = float("inf")
    k[8, 0, 9] = float("nan")
    k[9] = -k[9].abs()
    k[10, :, 1:] = 0
    q, slots = torch.zeros((t, 2, 128), dtype=torch.float16, device="cuda"), torch.arange(t, device="cuda")
    a, b = pkv.empty_fp8kv_cache(-(-t // bs), hkv, bs, "cuda"), pkv.empty_fp8kv_cache(-(-t // bs), hkv, bs, "cuda")
    pkv.append_fp8kv(*b, slots, k, k)
    for n in (t, 20):  # both kernels
        for x in a:
            x.zero_()
        pos = torch.zeros(n, dtype=torch.int32, device="cuda")
        # 16 dims are turned by nothing, which makes NaN of what an infinity is paired with (inf x 0): of rows with an infinity or a
        # NaN (some of the largest ones too) only V's codes are compared
        pkv.norm_rope_append_fp8kv(torch.empty_like(q[:n]), q[:n], k[:n], k[:n], *a, slots[:n], pos, pkv.rope_frequencies(16), None, None, EPS)
        flat = lambda x: x.transpose(1, 2).reshape(-1, hkv, *x.shape[3:])[:n]  # noqa: E731
        rows = torch.isfinite(k[:n]).flatten(1).all(1)
        assert rows.sum() > n // 2
        got, want = flat(a[0])[rows], flat(b[0])[rows]
        # The 16 dims that are turned by nothing keep their value, but not the sign of a zero: -0 x 1 - y x 0 is +0 for y < 0.
        assert torch.equal(got[..., 16:], want[..., 16:]) and torch.equal(got[..., :16].view(F8).float(), want[..., :16].view(F8).float())
        assert torch.equal(flat(a[1])[rows], flat(b[1])[rows])
        assert torch.equal(flat(a[2]), flat(b[2])) and torch.equal(flat(a[3]).nan_to_num(7.0), flat(b[3]).nan_to_num(7.0))
    assert_no_device_error()


def test_bad_axis_is_recorded():
    q, k, _, qw, kw, pos = make(4, 2, 1, 128, 5, axes=2)
    axes = torch.zeros(64, dtype=torch.int32, device="cuda")
    freq = pkv.rope_frequencies(128)
    a, b, ko = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)
    pkv.norm_rope(a, ko, q, k, pos, freq, qw, kw, EPS, axes=axes)
    assert_no_device_error()
    axes[3], axes[40] = 2, -1
    pkv.norm_rope(b, ko, q, k, pos, freq, qw, kw, EPS, axes=axes)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_AXIS
    assert torch.equal(a, b)


def test_graph_and_stream():
    q, k, v, qw, kw, pos = make(9, 8, 2, 128, 1)
    kc, vc = (torch.zeros((4, 2, 16, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    slots, pos, freq = torch.arange(9, device="cuda"), pos[:, 0].contiguous(), pkv.rope_frequencies(128)
    qo = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pkv.norm_rope_append(qo, q, k, v, kc, vc, slots, pos, freq, qw, kw, EPS)
    pos += 100  # replays read the positions of their time
    graph.replay()
    torch.cuda.synchronize()
    want, kc2, vc2 = torch.empty_like(q), torch.zeros_like(kc), torch.zeros_like(vc)
    pkv.norm_rope_append(want, q, k, v, kc2, vc2, slots, pos, freq, qw, kw, EPS, stream=s)
    s.synchronize()
    assert torch.equal(qo, want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_empty_call():
    z = torch.empty((0, 4, 128), dtype=torch.float16, device="cuda")
    w = torch.ones(128, device="cuda")
    pkv.norm_rope(z, z, z, z, torch.empty(0, dtype=torch.int32, device="cuda"), pkv.rope_frequencies(128), w, w, EPS)
    assert_no_device_error()


@pytest.mark.parametrize("n,hkv,bs", [(1, 1, 16), (3, 2, 48), (37, 8, 16), (5, 3, 256), (700, 1, 16)])
def test_read_blocks(n, hkv, bs):
    """Every code times its row's scale in float32, rounded once: equal to torch's own product bit for bit."""
    src_nb, nb = n + 3, n + 2
    g = torch.Generator(device="cuda").manual_seed(n)
    codes = [torch.randint(0, 256, (src_nb, hkv, bs, 128), generator=g, device="cuda").to(torch.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 0x7f) == 0x7f] = 0x38  # no NaN codes
    scale = [torch.rand((src_nb, hkv, bs), generator=g, device="cuda") * 0.02 for _ in range(2)]
    cache = [torch.full((nb, hkv, bs, 128), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    src = torch.randint(0, src_nb, (n,), generator=g, device="cuda", dtype=torch.int32)  # a block may be read twice
    dst = torch.randperm(nb, generator=g, device="cuda")[:n].to(torch.int32)
    want = [c.clone() for c in cache]
    for w, c, s in zip(want, codes, scale):
        w[dst.long()] = (c.view(F8).float() * s[..., None]).half()[src.long()]
    pkv.read_blocks_fp8kv(*cache, codes[0], scale[0], codes[1], scale[1], src, dst)
    assert torch.equal(cache[0], want[0]) and torch.equal(cache[1], want[1])
    assert_no_device_error()
    # ids outside their cache: skipped and recorded
    bad_src, bad_dst = src.clone(), dst.clone()
    bad_src[0] = src_nb
    bad_dst[n - 1] = -1
    again = [torch.zeros_like(c) for c in cache]
    pkv.read_blocks_fp8kv(*again, codes[0], scale[0], codes[1], scale[1], bad_src, bad_dst)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_BLOCK_ID
    for a, w in zip(again, want):
        inner = dst[1:n - 1].long()
        assert torch.equal(a[inner], w[inner])
        rest = torch.ones(nb, dtype=torch.bool, device="cuda")
        rest[inner] = False
        assert (a[rest] == 0).all()


def test_written_and_read_back():
    """A prompt quantised as it is written and read back: within the two roundings of the fp16 append's rows."""
    t, hkv, bs = 50, 2, 16
    q, k, v, qw, kw, pos = make(t, 8, hkv, 128, 2, True)
    pos, freq = pos[:, 0].contiguous(), pkv.rope_frequencies(128)
    nb = 5
    slots = torch.arange(t, device="cuda")
    fp8 = pkv.empty_fp8kv_cache(nb, hkv, bs, "cuda")
    kc, vc, kb, vb = (torch.zeros((nb, hkv, bs, 128), dtype=torch.float16, device="cuda") for _ in range(4))
    qo = torch.empty((t, 8, 128), dtype=torch.float16, device="cuda")
    pkv.norm_rope_append_fp8kv(qo, q, k, v, *fp8, slots, pos, freq, qw, kw, EPS)
    pkv.norm_rope_append(qo, q, k, v, kc, vc, slots, pos, freq, qw, kw, EPS)
    ids = torch.arange(4, dtype=torch.int32, device="cuda")
    pkv.read_blocks_fp8kv(kb, vb, *fp8, ids, ids)
    for a, b in ((kb, kc), (vb, vc)):
        a, b = host(a), host(b)
        most = np.abs(b).max(-1, keepdims=True)
        assert (np.abs(a - b) <= (2.0 ** -4 + 2.0 ** -10) * np.abs(b) + (2.0 ** -10 / 448 + 2.0 ** -20) * most + 2.0 ** -24).all()
    assert_no_device_error()
