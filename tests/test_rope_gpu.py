"""Rotary positions on the GPU against the float64 rotation: layouts, partial heads, strides, in place,
far and negative positions, the fused append."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import paged_kv_cache_278_gb300 as pkv
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu


def close(got, want, size):
    """fp16 rounds by half a step (2^-11 of the value, 2^-25 under the normal range).  In float32 the
    angle is off by at most pi 2^-25 (the phase's 24 bits) and cos, sin by 2 steps of 2^-24 near 1:
    3e-7 together; each of the two products and their sum rounds by 2^-24.  So 5e-7 of |x_a| + |x_b|."""
    got = got.float().cpu().numpy().astype(np.float64)
    tol = 2.0 ** -11 * np.abs(want) + 5e-7 * size + 2.0 ** -25
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def make(t, hq, hkv, d, seed, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        x = torch.randn((t, hq + 2 * hkv, d), generator=g, device="cuda").half()
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return tuple(torch.randn((t, h, d), generator=g, device="cuda").half() for h in (hq, hkv, hkv))


def host(x):
    return x.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("t,hq,hkv,d,rotary,interleaved,fused", [
    (1, 1, 1, 128, 128, False, False), (1, 8, 1, 128, 16, True, True), (17, 32, 8, 128, 128, False, True),
    (305, 4, 4, 128, 64, True, False), (5, 3, 1, 96, 48, False, False), (7, 2, 2, 256, 256, False, True),
    (400, 40, 8, 128, 96, False, True), (33, 130, 2, 128, 128, True, False), (2, 5, 1, 16, 16, True, False)])
def test_rope(t, hq, hkv, d, rotary, interleaved, fused):
    q, k, _ = make(t, hq, hkv, d, t + d, fused)
    pos = torch.randint(-70000, 1 << 20, (t,), dtype=torch.int32, device="cuda")
    freq = pkv.rope_frequencies(rotary)
    f64, m = ref.frequencies(rotary)
    qo, ko = torch.full((t, hq, d), float("nan"), dtype=torch.float16, device="cuda"), torch.zeros((t, hkv, d), dtype=torch.float16, device="cuda")
    pkv.rope(qo, ko, q, k, pos, freq, interleaved=interleaved)
    for out, x in ((qo, q), (ko, k)):
        want, size = ref.rotate(host(x), pos.cpu().numpy(), f64, m, interleaved)
        close(out, want, size)
        assert torch.equal(out[..., rotary:], x[..., rotary:])
    # in place, inside the projection's rows: same bits, and nothing else of the rows changes
    whole = q._base.clone() if fused else None
    pkv.rope(q, k, q, k, pos, freq, interleaved=interleaved)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    if fused:
        assert torch.equal(q._base[:, hq + hkv:], whole[:, hq + hkv:])
    assert_no_device_error()


def test_extreme_positions_and_identity():
    q, k, _ = make(4, 2, 1, 128, 3)
    pos = torch.tensor([0, 2 ** 31 - 1, -(2 ** 31), 1], dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.rope(qo, ko, q, k, pos, pkv.rope_frequencies(128))
    assert torch.equal(qo[0], q[0]) and torch.equal(ko[0], k[0])
    want, size = ref.rotate(host(q), pos.cpu().numpy(), ref.frequencies(128)[0])
    # at 2^31 the fixed-point frequency's 2^-54 relative rounding (float64's) is 2^31 x 2^-54 x 1 rad = 1.2e-7 more
    close(qo, want, size * 1.5)


@pytest.mark.parametrize("spec", [dict(method="linear", factor=4.0), dict(method="base", factor=8.0),
                                  dict(method="bands", factor=8.0, original_context=8192),
                                  dict(method="bands", factor=2.0, original_context=512, slow_turns=0.5, fast_turns=9.0),
                                  dict(method="ramp", factor=16.0, original_context=4096), dict(method="ramp", factor=1.0, original_context=64)])
def test_scaled_frequencies(spec):
    q, k, _ = make(64, 4, 2, 128, 9)
    pos = torch.randint(0, 200000, (64,), dtype=torch.int32, device="cuda")
    f64, m = ref.frequencies(128, base=500000.0, **spec)
    magnitude = pkv.rope_magnitude(spec["factor"]) if spec["method"] == "ramp" else 1.0
    assert magnitude == pytest.approx(m, rel=1e-15)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.rope(qo, ko, q, k, pos, pkv.rope_frequencies(128, base=500000.0, **spec), magnitude=magnitude)
    want, size = ref.rotate(host(q), pos.cpu().numpy(), f64, m)
    close(qo, want, size)


@pytest.mark.parametrize("t,hq,hkv,bs,rotary,interleaved", [(1, 8, 8, 16, 128, False), (40, 16, 2, 48, 64, True),
                                                            (333, 32, 8, 16, 128, True)])
def test_rope_append(t, hq, hkv, bs, rotary, interleaved):
    q, k, v = make(t, hq, hkv, 128, t, fused=True)
    nb = -(-t // bs) + 2
    g = torch.Generator(device="cuda").manual_seed(t)
    kc, vc = (torch.randn((nb, hkv, bs, 128), generator=g, device="cuda").half() for _ in range(2))
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:t].contiguous()
    if t > 3:
        slots[2] = -1
    pos = torch.randint(0, 9000, (t,), dtype=torch.int32, device="cuda")
    freq = pkv.rope_frequencies(rotary)
    qo, ko = torch.empty((t, hq, 128), dtype=torch.float16, device="cuda"), torch.empty((t, hkv, 128), dtype=torch.float16, device="cuda")
    pkv.rope(qo, ko, q, k, pos, freq, interleaved=interleaved)
    want_k, want_v = kc.clone(), vc.clone()
    pkv.append(want_k, want_v, slots, ko, v.contiguous())
    qa = torch.full_like(qo, float("nan"))
    pkv.rope_append(qa, q, k, v, kc, vc, slots, pos, freq, interleaved=interleaved)
    assert torch.equal(qa, qo) and torch.equal(kc, want_k) and torch.equal(vc, want_v)
    assert_no_device_error()
    # a slot past the pool: skipped and recorded, the others written
    slots[0] = nb * bs
    kc2, vc2 = kc.clone(), vc.clone()
    pkv.rope_append(q, q, k, v, kc2, vc2, slots, pos, freq, interleaved=interleaved)  # q in place
    assert torch.equal(q, qo) and torch.equal(kc2, kc) and torch.equal(vc2, vc)
    assert pkv.device_error() == pkv.PKV_DEV_BAD_SLOT


def test_graph_and_stream():
    q, k, v = make(9, 8, 2, 128, 1)
    kc, vc = (torch.zeros((4, 2, 16, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    slots = torch.arange(9, device="cuda")
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    freq = pkv.rope_frequencies(128)
    qo = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pkv.rope_append(qo, q, k, v, kc, vc, slots, pos, freq)
    pos += 100  # replays read the positions of their time
    graph.replay()
    torch.cuda.synchronize()
    want = torch.empty_like(q)
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    pkv.rope_append(want, q, k, v, kc2, vc2, slots, pos, freq, stream=s)
    s.synchronize()
    assert torch.equal(qo, want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_empty_call():
    z = torch.empty((0, 4, 128), dtype=torch.float16, device="cuda")
    pkv.rope(z, z, z, z, torch.empty(0, dtype=torch.int32, device="cuda"), pkv.rope_frequencies(128))
    assert_no_device_error()
