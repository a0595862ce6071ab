"""The operators' refusals and host-side results on the CPU (no kernel runs)."""
import ctypes

import numpy as np
import pytest

import operators_ref as ref
from paged_kv_cache_278_gb300 import _lib
from paged_kv_cache_278_gb300.build import build
import paged_kv_cache_278_gb300 as pkv

P, BAD, NULL = ctypes.c_void_p(4096), ctypes.c_void_p(4098), None  # never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE = (_lib.PKV_OK, _lib.PKV_ERR_INVALID_ARG, _lib.PKV_ERR_UNSUPPORTED,
                                       _lib.PKV_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def call(lib, name, good, **change):
    args = dict(good)
    assert set(change) <= set(args)
    args.update(change)
    return getattr(lib, name)(*args.values())


@pytest.mark.parametrize("spec", [dict(), dict(method="linear", factor=2.5), dict(method="base", factor=8.0),
                                  dict(method="bands", factor=8.0, original_context=8192),
                                  dict(method="ramp", factor=40.0, original_context=4096)])
@pytest.mark.parametrize("d", [16, 64, 96, 128])
def test_rope_frequencies(lib, spec, d):
    got = pkv.rope_frequencies(d, base=10000.0, device="cpu", **spec).numpy().astype(np.float64) * 2.0 ** -64 * 2 * np.pi
    want, m = ref.frequencies(d, 10000.0, **spec)
    # float64 throughout: a few steps of 2^-53 each, and half a unit of the fixed point
    assert np.abs(got - want).max() <= 1e-14 and np.all(np.abs(got - want) <= 1e-13 * want + 2.0 ** -61)
    if spec.get("method") == "ramp":
        assert pkv.rope_magnitude(spec["factor"]) == pytest.approx(m, rel=1e-15)


@pytest.mark.parametrize("spec", [dict(rotary_dim=0), dict(rotary_dim=7), dict(base=1.0), dict(base=float("inf")),
                                  dict(base=float("nan")), dict(method="linear", factor=0.5), dict(method="base", factor=2.0, rotary_dim=2),
                                  dict(method="bands", factor=2.0), dict(method="ramp", factor=2.0, original_context=4096, slow_turns=40.0),
                                  dict(method="ramp", factor=float("nan"), original_context=4096)])
def test_rope_frequency_refusals(lib, spec):
    spec = dict(dict(rotary_dim=128), **spec)
    with pytest.raises(pkv.PkvError):
        pkv.rope_frequencies(device="cpu", **spec)
    with pytest.raises(ValueError):
        pkv.rope_frequencies(128, method="other", device="cpu")
    assert lib.pkv_rope_frequencies(None, None, None) == INVALID


ROPE = dict(q_out=P, qos=512, k_out=P, kos=128, q=P, qs=512, k=P, ks=128, positions=P, frequencies=P, tokens=0, hq=4, hkv=1,
            d=128, rotary=128, interleaved=0, magnitude=1.0, stream=NULL)
APPEND = dict(q_out=P, qos=512, q=P, qs=512, k=P, ks=128, v=P, vs=128, kc=P, vc=P, slots=P, positions=P, frequencies=P, tokens=0,
              hq=4, hkv=1, d=128, rotary=128, bs=16, nb=4, interleaved=0, magnitude=1.0, stream=NULL)


@pytest.mark.parametrize("name,good", [("pkv_rope", ROPE), ("pkv_rope_append", APPEND)])
def test_rope_refusals(lib, name, good):
    assert call(lib, name, good) == OK  # no tokens: nothing to do
    for change in (dict(tokens=-1), dict(hq=-1), dict(d=0), dict(rotary=0), dict(rotary=144), dict(magnitude=float("nan"))):
        assert call(lib, name, good, **change) == INVALID, change
    for change in (dict(d=264), dict(d=120, rotary=112), dict(rotary=24), dict(d=272, rotary=16)):
        assert call(lib, name, good, **change) == UNSUPPORTED, change
    one = dict(good, tokens=2)
    for key in ("q_out", "q", "k", "positions", "frequencies"):
        assert call(lib, name, one, **{key: NULL}) == INVALID, key
        assert call(lib, name, one, **{key: BAD}) == INVALID, key
    for change in (dict(qs=511), dict(qs=504), dict(ks=120), dict(qos=0)):
        assert call(lib, name, one, **change) == INVALID, change
    if name == "pkv_rope_append":
        for change in (dict(kc=NULL), dict(vc=BAD), dict(bs=0), dict(nb=0), dict(hkv=0)):
            assert call(lib, name, good, **change) == INVALID, change
        for change in (dict(v=NULL), dict(slots=NULL), dict(slots=BAD), dict(vs=64)):
            assert call(lib, name, one, **change) == INVALID, change
    else:
        assert call(lib, name, one, k_out=NULL) == INVALID
        assert call(lib, name, dict(good, hq=0, hkv=0)) == INVALID


WEIGHTS = dict(out=P, scores=P, capacity=64, q=P, kc=P, vc=P, bt=P, cl=P, seqs=0, width=4, hq=8, hkv=2, d=128, bs=16, nb=9, scale=1.0,
               ws=NULL, ws_bytes=0, stream=NULL)


def test_weights_refusals(lib):
    f = "pkv_decode_attention_weights"
    assert call(lib, f, WEIGHTS) == OK
    for change in (dict(out=NULL), dict(scores=NULL), dict(scores=BAD), dict(q=NULL), dict(kc=BAD), dict(capacity=63), dict(hq=7),
                   dict(seqs=-1), dict(width=0)):
        assert call(lib, f, WEIGHTS, **change) == INVALID, change
    for change in (dict(hq=6), dict(hq=32), dict(d=64), dict(bs=8, capacity=64), dict(bs=272, capacity=4096)):
        assert call(lib, f, WEIGHTS, **change) == UNSUPPORTED, change
    need = lib.pkv_weights_workspace_size(1, 8, 128, 64)
    assert need >= 64 * 8 * 4
    for change in (dict(ws=NULL), dict(ws=P, ws_bytes=need - 1), dict(ws=ctypes.c_void_p(4096 + 128), ws_bytes=need)):
        assert call(lib, f, dict(WEIGHTS, seqs=1), **change) == WORKSPACE, change
    assert call(lib, f, dict(WEIGHTS, seqs=1, nb=2 ** 26)) == UNSUPPORTED  # row coordinates past 31 bits
    for bad in ((0, 8, 128, 64), (1, 0, 128, 64), (1, 8, 64, 64), (1, 8, 128, 0)):
        assert lib.pkv_weights_workspace_size(*bad) == 0


EVICT = dict(kc=P, vc=P, kept=P, new_scores=P, new_lens=P, scores=P, bt=P, nt=P, cl=P, seqs=0, width=4, new_width=4, capacity=64,
             hkv=2, d=128, bs=16, nb=9, budget=16, recent=4, sinks=2, stream=NULL)


def test_evict_refusals(lib):
    assert call(lib, "pkv_evict", EVICT) == OK
    for change in (dict(seqs=-1), dict(width=0), dict(new_width=0), dict(capacity=63), dict(budget=0), dict(recent=-1),
                   dict(sinks=-1), dict(recent=17), dict(recent=10, sinks=7), dict(nb=0), dict(hkv=0), dict(bs=0)):
        assert call(lib, "pkv_evict", EVICT, **change) == INVALID, change
    for change in (dict(d=64), dict(width=262144 // 16 + 1, capacity=1 << 20), dict(hkv=70000)):
        assert call(lib, "pkv_evict", EVICT, **change) == UNSUPPORTED, change
    one = dict(EVICT, seqs=1)
    for key in ("kc", "vc", "kept", "new_scores", "new_lens", "scores", "bt", "nt", "cl"):
        assert call(lib, "pkv_evict", one, **{key: NULL}) == INVALID, key
        assert call(lib, "pkv_evict", one, **{key: BAD}) == INVALID, key


PACKED = dict(out=P, lse=NULL, q=P, qs=1024, k=P, ks=256, v=P, vs=256, start=P, seqs=0, total=64, longest=64, hq=8, hkv=2, d=128,
              scale=1.0, ws=NULL, ws_bytes=0, stream=NULL)
PAGED = dict(out=P, lse=NULL, q=P, qs=1024, kc=P, vc=P, bt=P, cl=P, start=P, seqs=0, total=64, longest=64, width=4, hq=8, hkv=2, d=128,
             bs=16, nb=9, scale=1.0, ws=NULL, ws_bytes=0, stream=NULL)
CHUNK = dict(scores=P, capacity=64, q=P, qs=1024, lse=P, kc=P, bt=P, cl=P, start=P, seqs=0, total=64, longest=64, width=4, hq=8, hkv=2,
             d=128, bs=16, nb=9, scale=1.0, stream=NULL)


@pytest.mark.parametrize("name,good", [("pkv_prefill_attention", PACKED), ("pkv_prefill_attention_paged", PAGED),
                                       ("pkv_prefill_attention_weights", CHUNK)])
def test_prompt_refusals(lib, name, good):
    for empty in (dict(), dict(seqs=1, total=0), dict(seqs=1, longest=0)):
        assert call(lib, name, good, **empty) == OK, empty
    for change in (dict(seqs=-1), dict(total=-1), dict(longest=-1), dict(hq=7), dict(hkv=0), dict(scale=0.0), dict(scale=-1.0),
                   dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(lib, name, good, **change) == INVALID, change
    for change in (dict(hq=6), dict(hq=32), dict(d=64), dict(seqs=70000)):
        assert call(lib, name, good, **change) == UNSUPPORTED, change
    one = dict(good, seqs=1)
    keys = [k for k in ("out", "q", "k", "v", "kc", "vc", "bt", "cl", "start", "scores") if k in good]
    for key in keys:
        assert call(lib, name, one, **{key: NULL}) == INVALID, key
        assert call(lib, name, one, **{key: BAD}) == INVALID, key
    if "out" in good:
        assert call(lib, name, one, out=ctypes.c_void_p(4096 + 8)) == INVALID  # 16-byte stores
    for key in ("qs", "ks", "vs"):
        if key in good:
            for stride in (good[key] - 8, good[key] + 4):
                assert call(lib, name, one, **{key: stride}) == INVALID, key
    assert call(lib, name, one, lse=BAD) == INVALID
    if name == "pkv_prefill_attention_weights":
        assert call(lib, name, one, lse=NULL) == INVALID
        assert call(lib, name, one, capacity=63) == INVALID
    if "nb" in good:
        assert call(lib, name, one, nb=2 ** 26) == UNSUPPORTED


def test_prefill_workspace(lib):
    f = lib.pkv_prefill_workspace_size
    assert f(1, 16384, 32, 8, 128, 16384) == 0       # enough rows: no split
    assert f(64, 64, 32, 8, 128, 32768) == 0         # enough requests
    few = f(1, 16, 32, 8, 128, 32768)
    assert few > 0 and few % 256 == 0 and few >= 16 * 32 * 2 * (128 * 4 + 8)
    assert f(1, 16, 32, 8, 128, 600) == 0            # a short axis
    for bad in ((0, 16, 32, 8, 128, 4096), (1, 0, 32, 8, 128, 4096), (1, 16, 24, 8, 128, 4096), (1, 16, 32, 8, 64, 4096),
                (1, 16, 32, 8, 128, 0)):
        assert f(*bad) == 0


def test_prefill_workspace_bound(lib):
    """What the header promises to a program that allocates once: never more than 81 MB, whatever the call's sizes."""
    most = 0
    for hkv in (1, 2, 3, 8, 31, 50, 101, 102):
        for group in (1, 2, 4, 8):
            for seqs in (1, 2, 7, 20, 101, 5000):
                for rows in [2 ** i + d for i in range(15) for d in (-1, 0, 1)]:
                    for context in (1, 300, 4096, 40000, 1 << 20, 1 << 30):
                        if rows > 0:
                            most = max(most, lib.pkv_prefill_workspace_size(seqs, rows, hkv * group, hkv, 128, context))
    # 608 / items splits at most of the 256 rows of each item: 155,648 partial rows of 128 + 2 floats, and alignment
    assert 0 < most <= 608 * 256 * 130 * 4 + 3 * 256 < 81 * 10 ** 6


def test_long_tables_are_refused(lib):
    wide = dict(width=(1 << 30) // 16 + 1, seqs=1, nb=1000)
    assert call(lib, "pkv_prefill_attention_paged", dict(PAGED, **wide)) == UNSUPPORTED
    assert call(lib, "pkv_prefill_attention_weights", dict(CHUNK, **wide), capacity=1 << 31) == UNSUPPORTED
