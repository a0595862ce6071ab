"""What the tree, norm and read-back calls refuse, and the sizes they ask for, on the CPU (no kernel runs)."""
import ctypes

import pytest

from paged_kv_cache_278_gb300 import _lib
from paged_kv_cache_278_gb300.build import build

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


NORM = dict(q_out=P, qos=512, k_out=P, kos=128, q=P, qs=512, k=P, ks=128, positions=P, axes=P, n_axes=3, frequencies=P, qw=P, kw=P, eps=1e-6,
            tokens=0, hq=4, hkv=1, d=128, rotary=128, interleaved=0, magnitude=1.0, stream=NULL)
APPEND = dict(q_out=P, qos=512, q=P, qs=512, k=P, ks=128, v=P, vs=128, kc=P, vc=P, slots=P, positions=P, axes=P, n_axes=3, frequencies=P,
              qw=P, kw=P, eps=1e-6, tokens=0, hq=4, hkv=1, d=128, rotary=128, bs=16, nb=4, interleaved=0, magnitude=1.0, stream=NULL)
FP8 = dict(q_out=P, qos=512, q=P, qs=512, k=P, ks=128, v=P, vs=128, kc=P, kscale=P, vc=P, vscale=P, slots=P, positions=P, axes=P, n_axes=3,
           frequencies=P, qw=P, kw=P, eps=1e-6, tokens=0, hq=4, hkv=1, d=128, rotary=128, bs=16, nb=4, interleaved=0, magnitude=1.0, stream=NULL)


@pytest.mark.parametrize("name,good", [("pkv_norm_rope", NORM), ("pkv_norm_rope_append", APPEND), ("pkv_norm_rope_append_fp8kv", FP8)])
def test_norm_refusals(lib, name, good):
    assert call(lib, name, good) == OK  # no tokens: nothing to do
    assert call(lib, name, good, qw=NULL, kw=NULL) == OK and call(lib, name, good, axes=NULL, n_axes=1) == OK
    for change in (dict(tokens=-1), dict(hq=-1), dict(d=0), dict(rotary=0), dict(rotary=144), dict(magnitude=float("nan")), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(eps=float("inf")), dict(n_axes=0), dict(axes=NULL), dict(qw=BAD),
                   dict(kw=ctypes.c_void_p(4096 + 8)), dict(axes=BAD)):
        assert call(lib, name, good, **change) == INVALID, change
    for change in (dict(d=264), dict(d=120, rotary=112), dict(rotary=24), dict(d=272, rotary=16), dict(n_axes=5), dict(hq=70000)):
        assert call(lib, name, good, **change) == UNSUPPORTED, change
    one = dict(good, tokens=2)
    for key in ("q_out", "q", "k", "positions", "frequencies"):
        assert call(lib, name, one, **{key: NULL}) == INVALID, key
        assert call(lib, name, one, **{key: BAD}) == INVALID, key
    for change in (dict(qs=511), dict(qs=504), dict(ks=120), dict(qos=0)):
        assert call(lib, name, one, **change) == INVALID, change
    if name == "pkv_norm_rope":
        assert call(lib, name, one, k_out=NULL) == INVALID and call(lib, name, one, k_out=BAD) == INVALID
        assert call(lib, name, one, kos=64) == INVALID
        assert call(lib, name, dict(good, hq=0, hkv=0)) == INVALID
        return
    for change in (dict(kc=NULL), dict(vc=BAD), dict(bs=0), dict(nb=0), dict(hkv=0)):
        assert call(lib, name, good, **change) == INVALID, change
    for change in (dict(v=NULL), dict(v=BAD), dict(slots=NULL), dict(slots=BAD), dict(vs=64)):
        assert call(lib, name, one, **change) == INVALID, change
    if name == "pkv_norm_rope_append_fp8kv":
        assert call(lib, name, good, kscale=NULL) == INVALID and call(lib, name, good, vscale=BAD) == INVALID
        assert call(lib, name, good, d=64, rotary=64) == UNSUPPORTED


READ = dict(kc=P, vc=P, nb=9, kcodes=P, kscale=P, vcodes=P, vscale=P, src_nb=5, src=P, dst=P, n=0, hkv=2, d=128, bs=16, stream=NULL)


def test_read_refusals(lib):
    f = "pkv_read_blocks_fp8kv"
    assert call(lib, f, READ) == OK and call(lib, f, READ, src=NULL, dst=NULL) == OK
    for change in (dict(n=-1), dict(hkv=0), dict(d=0), dict(bs=0), dict(nb=0), dict(src_nb=0)):
        assert call(lib, f, READ, **change) == INVALID, change
    one = dict(READ, n=1)
    for key in ("kc", "vc", "kcodes", "kscale", "vcodes", "vscale", "src", "dst"):
        assert call(lib, f, one, **{key: NULL}) == INVALID, key
        assert call(lib, f, one, **{key: BAD}) == INVALID, key
    for change in (dict(d=64), dict(hkv=1 << 20, bs=256), dict(n=2 ** 31 - 1, hkv=1024, bs=256)):
        assert call(lib, f, one, **change) == UNSUPPORTED, change


TREE = dict(out=P, lse=NULL, q=P, qs=1024, kc=P, vc=P, bt=P, cl=P, start=P, mask=P, words=2, seqs=0, total=64, longest=64, width=4, hq=8, hkv=2,
            d=128, bs=16, nb=9, scale=1.0, ws=NULL, ws_bytes=0, stream=NULL)


def test_tree_refusals(lib):
    f = "pkv_decode_attention_tree"
    for empty in (dict(), dict(seqs=1, total=0), dict(seqs=1, longest=0)):
        assert call(lib, f, TREE, **empty) == OK, empty
    for change in (dict(seqs=-1), dict(total=-1), dict(longest=-1), dict(hq=7), dict(hkv=0), dict(scale=0.0), dict(scale=-1.0), dict(words=1),
                   dict(words=-1), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(lib, f, TREE, **change) == INVALID, change
    for change in (dict(hq=6), dict(hq=32), dict(d=64), dict(seqs=70000), dict(longest=1025, words=64)):
        assert call(lib, f, TREE, **change) == UNSUPPORTED, change
    one = dict(TREE, seqs=1)
    for key in ("out", "q", "kc", "vc", "bt", "cl", "start", "mask"):
        assert call(lib, f, one, **{key: NULL}) == INVALID, key
        assert call(lib, f, one, **{key: BAD}) == INVALID, key
    assert call(lib, f, one, out=ctypes.c_void_p(4096 + 8)) == INVALID  # 16-byte stores
    for stride in (1016, 1028):
        assert call(lib, f, one, qs=stride) == INVALID
    assert call(lib, f, one, lse=BAD) == INVALID
    assert call(lib, f, one, nb=2 ** 26) == UNSUPPORTED
    assert call(lib, f, dict(one, width=(1 << 30) // 16 + 1, nb=1000)) == UNSUPPORTED
    need = lib.pkv_tree_workspace_size(1, 64, 64, 8, 2, 128, 4096)
    assert need > 0
    long = dict(one, width=256)
    for change in (dict(ws=NULL), dict(ws=P, ws_bytes=need - 1), dict(ws=ctypes.c_void_p(4096 + 128), ws_bytes=need)):
        assert call(lib, f, long, **change) == WORKSPACE, change


def test_tree_workspace(lib):
    f = lib.pkv_tree_workspace_size
    assert f(1, 8, 8, 32, 8, 128, 300) == 0  # short contexts: no item is split
    most = 0
    for hkv in (1, 3, 8, 200):
        for group in (1, 2, 4, 8):
            for seqs in (1, 7, 5000):
                for n in (1, 16, 61, 1024):
                    for context in (1, 513, 4096, 1 << 20, 1 << 30):
                        most = max(most, f(seqs, seqs * n, n, hkv * group, hkv, 128, context))
    # two slots of at most 256 rows of 128 + 2 floats, and 32 bytes, for each of 152 CTAs
    assert most == 152 * (2 * 256 * 130 * 4 + 32) < 41 * 10 ** 6
    for bad in ((0, 16, 16, 32, 8, 128, 4096), (1, 0, 16, 32, 8, 128, 4096), (1, 16, 0, 32, 8, 128, 4096), (1, 16, 16, 24, 8, 128, 4096),
                (1, 16, 16, 32, 8, 64, 4096), (1, 16, 16, 32, 8, 128, 0)):
        assert f(*bad) == 0


MASKS = dict(mask=P, depths=P, parents=P, start=P, seqs=0, total=64, longest=64, words=2, stream=NULL)


def test_mask_refusals(lib):
    f = "pkv_tree_masks"
    for empty in (dict(), dict(seqs=1, total=0), dict(seqs=1, longest=0)):
        assert call(lib, f, MASKS, **empty) == OK, empty
    for change in (dict(seqs=-1), dict(total=-1), dict(longest=-1), dict(words=1), dict(words=-1)):
        assert call(lib, f, MASKS, **change) == INVALID, change
    assert call(lib, f, MASKS, longest=1025, words=64) == UNSUPPORTED
    one = dict(MASKS, seqs=1)
    for key in ("mask", "parents", "start"):
        assert call(lib, f, one, **{key: NULL}) == INVALID, key
        assert call(lib, f, one, **{key: BAD}) == INVALID, key
    assert call(lib, f, one, depths=BAD) == INVALID


KEEP = dict(kc=P, vc=P, new_lens=P, bt=P, cl=P, start=P, path=P, path_lens=P, seqs=0, width=4, most=4, hkv=2, d=128, bs=16, nb=9, stream=NULL)


def test_keep_refusals(lib):
    f = "pkv_keep_path"
    assert call(lib, f, KEEP) == OK
    for change in (dict(seqs=-1), dict(width=0), dict(most=-1), dict(hkv=0), dict(d=0), dict(bs=0), dict(nb=0)):
        assert call(lib, f, KEEP, **change) == INVALID, change
    for change in (dict(d=64), dict(seqs=70000), dict(hkv=70000)):
        assert call(lib, f, KEEP, **change) == UNSUPPORTED, change
    one = dict(KEEP, seqs=1)
    for key in ("kc", "vc", "bt", "cl", "start", "path", "path_lens"):
        assert call(lib, f, one, **{key: NULL}) == INVALID, key
        assert call(lib, f, one, **{key: BAD}) == INVALID, key
    assert call(lib, f, one, new_lens=BAD) == INVALID
