"""What the binding refuses before any launch: wrong types, shapes, strides, devices, missing workspaces."""
import pytest
import torch

import paged_kv_cache_278_gb300 as pkv
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def x():
    f16 = dict(dtype=torch.float16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    d = dict(q=torch.zeros((6, 8, 128), **f16), k=torch.zeros((6, 2, 128), **f16), v=torch.zeros((6, 2, 128), **f16),
             kc=torch.zeros((5, 2, 16, 128), **f16), vc=torch.zeros((5, 2, 16, 128), **f16), out=torch.zeros((6, 8, 128), **f16),
             slots=torch.arange(6, device="cuda"), pos=torch.arange(6, **i32), freq=pkv.rope_frequencies(128),
             bt=torch.arange(4, **i32).view(2, 2), cl=torch.tensor([20, 10], **i32), qs=torch.tensor([0, 4, 6], **i32),
             scores=torch.zeros((2, 2, 32), device="cuda"), lse=torch.zeros((6, 8), device="cuda"))
    return d


def refused(f, *args, **more):
    with pytest.raises((ValueError, TypeError, pkv.PkvError)):
        f(*args, **more)


def test_rope(x):
    good = [x["out"], torch.empty_like(x["k"]), x["q"], x["k"], x["pos"], x["freq"]]
    pkv.rope(*good)
    for i, bad in ((2, x["q"].float()), (2, x["q"].cpu()), (2, x["q"][:, :, ::2]), (2, x["q"].transpose(0, 1)), (2, None), (3, x["k"][:5]),
                   (3, x["k"][0]), (0, x["out"][:, :4]), (1, x["q"]), (4, x["pos"].long()), (4, x["pos"][:5]), (5, x["freq"].int()),
                   (5, x["freq"][:0]), (5, x["freq"][:3]), (5, torch.cat([x["freq"]] * 2)), (2, x["q"][:1].expand(6, 8, 128))):
        refused(pkv.rope, *good[:i], bad, *good[i + 1:])
    refused(pkv.rope, *good, magnitude=float("inf"))


def test_rope_append(x):
    good = [x["out"], x["q"], x["k"], x["v"], x["kc"], x["vc"], x["slots"], x["pos"], x["freq"]]
    pkv.rope_append(*good)
    for i, bad in ((2, x["q"]), (3, x["v"][:5]), (4, x["kc"].float()), (5, x["vc"][:4]), (6, x["slots"].int()), (6, x["slots"][:5]),
                   (1, x["q"][..., :64].contiguous())):
        refused(pkv.rope_append, *good[:i], bad, *good[i + 1:])


def test_prefill(x):
    good = [x["out"], x["q"], x["k"], x["v"], x["qs"], 4, 0.1]
    pkv.prefill_attention(*good)
    for i, bad in ((0, x["out"][:5]), (1, x["q"][:5]), (2, x["k"][:5]), (3, x["q"]), (4, x["qs"].long()), (4, x["qs"][:0]), (5, -1), (6, 0.0),
                   (6, -1.0), (2, torch.zeros((6, 3, 128), dtype=torch.float16, device="cuda"))):
        refused(pkv.prefill_attention, *good[:i], bad, *good[i + 1:])
    refused(pkv.prefill_attention, *good, lse=x["lse"][:5])
    refused(pkv.prefill_attention, *good, lse=x["lse"].half())
    good = [x["out"], x["q"], x["kc"], x["vc"], x["bt"], x["cl"], x["qs"], 4, 0.1]
    pkv.prefill_attention_paged(*good)
    for i, bad in ((2, x["kc"][:4]), (4, x["bt"][:1]), (5, x["cl"][:1]), (6, x["qs"][:2]), (4, x["bt"].long()), (8, float("nan")),
                   (4, x["bt"].t())):
        refused(pkv.prefill_attention_paged, *good[:i], bad, *good[i + 1:])


def test_arguments_that_are_no_tensors(x):
    """Every tensor argument of every call, one after the other: a TypeError that names it, nothing else."""
    kept = torch.empty((2, 2, 8), dtype=torch.int32, device="cuda")
    ws = pkv.make_weights_workspace(2, 8, 32, "cuda")
    calls = [(pkv.rope, [x["out"], torch.empty_like(x["k"]), x["q"], x["k"], x["pos"], x["freq"]]),
             (pkv.rope_append, [x["out"], x["q"], x["k"], x["v"], x["kc"], x["vc"], x["slots"], x["pos"], x["freq"]]),
             (pkv.prefill_attention, [x["out"], x["q"], x["k"], x["v"], x["qs"], 4, 0.1]),
             (pkv.prefill_attention_paged, [x["out"], x["q"], x["kc"], x["vc"], x["bt"], x["cl"], x["qs"], 4, 0.1]),
             (pkv.decode_attention_weights, [x["out"][:2], x["scores"], x["q"][:2], x["kc"], x["vc"], x["bt"], x["cl"], 0.1, ws]),
             (pkv.prefill_attention_weights, [x["scores"], x["q"], x["lse"], x["kc"], x["bt"], x["cl"], x["qs"], 4, 0.1]),
             (pkv.evict, [x["kc"], x["vc"], kept, torch.empty_like(x["scores"]), torch.empty_like(x["cl"]), x["scores"], x["bt"],
                          x["cl"], 8])]
    for f, good in calls:
        for i, a in enumerate(good):
            if isinstance(a, torch.Tensor):
                for bad in (None, [1.0]):
                    with pytest.raises(TypeError, match="must be a torch.Tensor"):
                        f(*good[:i], bad, *good[i + 1:])
    assert_no_device_error()


def test_weights_and_evict(x):
    ws = pkv.make_weights_workspace(2, 8, 32, "cuda")
    good = [x["out"][:2], x["scores"], x["q"][:2], x["kc"], x["vc"], x["bt"], x["cl"], 0.1, ws]
    pkv.decode_attention_weights(*good)
    for i, bad in ((1, x["scores"][:, :, :31]), (1, x["scores"][:, :1]), (1, x["scores"].half()), (8, ws[:-256]), (8, None), (6, x["cl"][:1]),
                   (0, x["out"])):
        refused(pkv.decode_attention_weights, *good[:i], bad, *good[i + 1:])
    good = [x["scores"], x["q"], x["lse"], x["kc"], x["bt"], x["cl"], x["qs"], 4, 0.1]
    pkv.prefill_attention_weights(*good)
    for i, bad in ((0, x["scores"][:1]), (2, x["lse"][:, :4]), (2, x["lse"].double()), (6, x["qs"][:2]), (8, 0.0)):
        refused(pkv.prefill_attention_weights, *good[:i], bad, *good[i + 1:])
    kept = torch.empty((2, 2, 8), dtype=torch.int32, device="cuda")
    good = [x["kc"], x["vc"], kept, torch.empty_like(x["scores"]), torch.empty_like(x["cl"]), x["scores"], x["bt"], x["cl"], 8]
    pkv.evict(*good, recent=2)
    for i, bad in ((2, kept[..., :7].contiguous()), (2, kept.long()), (3, x["scores"][:, :, :16].contiguous()), (4, x["cl"][:1]), (8, 7), (8, 0)):
        refused(pkv.evict, *good[:i], bad, *good[i + 1:])
    refused(pkv.evict, *good, recent=9)
    refused(pkv.evict, *good, recent=4, sinks=5)
    refused(pkv.evict, *good, new_tables=x["bt"][:1])
    assert_no_device_error()
