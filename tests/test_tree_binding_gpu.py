"""What the binding refuses of the norm, read-back and tree calls before any launch."""
import pytest
import torch

import paged_kv_cache_278_gb300 as pkv
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def x():
    f16, i32 = dict(dtype=torch.float16, device="cuda"), dict(dtype=torch.int32, device="cuda")
    d = dict(q=torch.zeros((6, 8, 128), **f16), k=torch.zeros((6, 2, 128), **f16), v=torch.zeros((6, 2, 128), **f16),
             kc=torch.zeros((5, 2, 16, 128), **f16), vc=torch.zeros((5, 2, 16, 128), **f16), out=torch.zeros((6, 8, 128), **f16),
             fp8=pkv.empty_fp8kv_cache(4, 2, 16, "cuda"), slots=torch.arange(6, device="cuda"), pos=torch.arange(6, **i32),
             pos3=torch.zeros((6, 3), **i32), axes=torch.zeros(64, **i32), freq=pkv.rope_frequencies(128), w=torch.ones(128, device="cuda"),
             bt=torch.arange(4, **i32).view(2, 2), cl=torch.tensor([20, 10], **i32), qs=torch.tensor([0, 4, 6], **i32),
             mask=torch.ones((6, 1), **i32), parents=torch.tensor([-1, 0, 0, 1, -1, 0], **i32), depths=torch.zeros(6, **i32),
             path=torch.zeros((2, 3), **i32), path_lens=torch.zeros(2, **i32), lse=torch.zeros((6, 8), device="cuda"),
             ids=torch.arange(2, **i32))
    return d


def refused(f, *args, **more):
    with pytest.raises((ValueError, TypeError, pkv.PkvError)):
        f(*args, **more)


def each(f, good, bads, **more):
    f(*good, **more)
    for i, bad in bads:
        refused(f, *good[:i], bad, *good[i + 1:], **more)


def test_norm_rope(x):
    good = [x["out"], torch.empty_like(x["k"]), x["q"], x["k"], x["pos"], x["freq"], x["w"], x["w"], 1e-6]
    each(pkv.norm_rope, good, ((2, x["q"].float()), (2, x["q"].cpu()), (2, x["q"][:, :, ::2]), (2, None), (3, x["k"][:5]), (0, x["out"][:, :4]),
                               (1, x["q"]), (4, x["pos"].long()), (4, x["pos"][:5]), (4, None), (4, x["pos3"]), (4, x["pos3"][:, :2]),
                               (5, x["freq"].int()), (5, x["freq"][:0]), (5, x["freq"][:3]), (6, x["w"].half()), (6, x["w"][:64]), (7, x["w"].cpu()),
                               (7, x["w"][None]), (8, -1.0), (8, float("nan"))))
    refused(pkv.norm_rope, *good, magnitude=float("inf"))
    refused(pkv.norm_rope, *good, axes=x["axes"][:63])
    refused(pkv.norm_rope, *good, axes=x["axes"].long())
    several = [*good[:4], x["pos3"], *good[5:]]
    pkv.norm_rope(*several, axes=x["axes"])
    refused(pkv.norm_rope, *good[:4], torch.zeros((6, 5), dtype=torch.int32, device="cuda"), *good[5:], axes=x["axes"])
    assert_no_device_error()


def test_norm_rope_append(x):
    tail = [x["slots"], x["pos"], x["freq"], x["w"], None, 1e-6]
    good = [x["out"], x["q"], x["k"], x["v"], x["kc"], x["vc"], *tail]
    each(pkv.norm_rope_append, good, ((2, x["q"]), (3, x["v"][:5]), (4, x["kc"].float()), (5, x["vc"][:4]), (6, x["slots"].int()),
                                      (6, x["slots"][:5]), (1, x["q"][..., :64].contiguous())))
    good = [x["out"], x["q"], x["k"], x["v"], *x["fp8"], *tail]
    each(pkv.norm_rope_append_fp8kv, good, ((2, x["q"]), (3, x["v"][:5]), (4, x["fp8"][0].to(torch.int8)), (5, x["fp8"][1][:3]),
                                            (6, x["fp8"][2][:3]), (7, x["fp8"][3].half()), (8, x["slots"].int()), (4, None),
                                            (1, x["q"][..., :64].contiguous())))
    assert_no_device_error()


def test_read_blocks(x):
    good = [x["kc"], x["vc"], *x["fp8"], x["ids"], x["ids"]]
    other = pkv.empty_fp8kv_cache(4, 2, 32, "cuda")
    each(pkv.read_blocks_fp8kv, good, ((0, x["kc"].float()), (1, x["vc"][:4]), (2, other[0]), (2, x["fp8"][0].cpu()), (6, x["ids"].long()),
                                       (7, x["ids"][:1])))
    refused(pkv.read_blocks_fp8kv, x["kc"], x["vc"], *other, x["ids"], x["ids"])
    pkv.read_blocks_fp8kv(*good[:6], x["ids"][:0], x["ids"][:0])
    assert_no_device_error()


def test_tree(x):
    good = [x["out"], x["q"], x["kc"], x["vc"], x["bt"], x["cl"], x["qs"], x["mask"], 4, 0.1]
    each(pkv.decode_attention_tree, good, ((0, x["out"][:5]), (1, x["q"][:5]), (1, x["q"].float()), (2, x["kc"].float()), (4, x["bt"][:1]),
                                           (5, x["cl"].long()), (6, x["qs"][:2]), (7, x["mask"][:5]), (7, x["mask"].long()), (7, x["mask"][:, 0]),
                                           (8, 33), (8, -1), (9, 0.0), (9, float("nan"))))
    refused(pkv.decode_attention_tree, *good, lse=x["lse"][:5])
    refused(pkv.decode_attention_tree, *good, workspace=torch.empty(16, device="cuda"))
    # a table that needs a workspace, without one and with one too small
    long = [*good[:4], torch.zeros((2, 200), dtype=torch.int32, device="cuda"), *good[5:]]
    refused(pkv.decode_attention_tree, *long)
    refused(pkv.decode_attention_tree, *long, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert_no_device_error()


def test_masks_and_paths(x):
    each(pkv.tree_masks, [x["mask"], x["depths"], x["parents"], x["qs"], 4],
         ((0, x["mask"][:5]), (0, x["mask"].long()), (1, x["depths"][:5]), (2, x["parents"].long()), (3, x["qs"][:0]), (4, 33), (4, -1)))
    each(pkv.keep_path, [x["kc"], x["vc"], x["bt"], x["cl"], x["qs"], x["path"], x["path_lens"]],
         ((0, x["kc"].float()), (1, x["vc"][:4]), (2, x["bt"][:1]), (3, x["cl"].long()), (4, x["qs"][:2]), (5, x["path"][:1]), (5, x["path"][0]),
          (6, x["path_lens"][:1])))
    refused(pkv.keep_path, x["kc"], x["vc"], x["bt"], x["cl"], x["qs"], x["path"], x["path_lens"], new_lens=x["cl"][:1])
    pkv.keep_path(x["kc"], x["vc"], x["bt"], x["cl"], x["qs"], x["path"][:, :0], x["path_lens"])  # nothing accepted anywhere
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    pkv.keep_path(x["kc"], x["vc"], x["bt"][:0], none, torch.zeros(1, dtype=torch.int32, device="cuda"), x["path"][:0], none)
    assert_no_device_error()
