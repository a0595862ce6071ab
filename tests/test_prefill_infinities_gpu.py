"""Infinities and NaN in V under weights that underflow, in attention of prompts and chunks, whole and split."""
import numpy as np
import pytest
import torch

import paged_kv_cache_278_gb300 as pkv
from gpu_util import assert_no_device_error

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
GROUP, BS = 4, 16


@pytest.mark.parametrize("n,c", [(300, 300), (700, 5), (5000, 37), (5000, 129), (20000, 3)])
@pytest.mark.parametrize("kind", ["infinity", "nan", "minus infinity"])
def test_an_infinity_far_below_the_largest_score(n, c, kind):
    """What a position's V holds of them is in every row that sees the position: beside a key 140 nats above all others, and
    among keys whose scores are all minus infinity.  Rows see one position more each.  (A weight is off by 2^-11 of itself, an output
    by as much; all other weights together are below n e^-140.)"""
    rng = np.random.default_rng(n + c)
    q, k = np.zeros((c, GROUP, 128), np.float16), np.zeros((n, 1, 128), np.float16)
    v = rng.standard_normal((n, 1, 128)).astype(np.float16)
    q[..., 0] = 16.0
    last = n - c  # the last position that all rows see
    at, decides = last // 8, last // 8 * 7
    if kind == "minus infinity":
        k[:max(last // 2, 1), :, 0] = -np.inf
        v[at, 0, 5] = np.inf
    else:
        k[decides, :, 0] = 140.0 / (16.0 * SCALE)
        v[at, 0, 5] = np.nan if kind == "nan" else -np.inf
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    nb = -(-n // BS)
    table = torch.randperm(nb, generator=torch.Generator().manual_seed(2)).to(torch.int32).view(1, -1)
    kc, vc = (torch.full((nb, 1, BS, 128), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    slots = pkv.slot_mapping(table.expand(n, -1).contiguous(), torch.arange(n, dtype=torch.int32), BS).cuda()
    pkv.append(kc, vc, slots, t(k), t(v))
    out = torch.full((c, GROUP, 128), 7.0, dtype=torch.float16, device="cuda")
    pkv.prefill_attention_paged(out, t(q), kc, vc, table.cuda(), i32(n), i32(0, c), c, SCALE,
                                workspace=pkv.make_prefill_workspace(1, c, GROUP, 1, nb * BS, "cuda"))
    got = out.double().cpu().numpy()
    assert not np.isfinite(got[..., 5]).any(), got[..., 5]
    rest = np.delete(got, 5, -1)
    first = 1 if kind == "minus infinity" and n == c else 0  # the row that sees a score of minus infinity alone has no softmax
    assert np.isfinite(rest[first:]).all()
    if kind != "minus infinity" and n > c:
        want = np.delete(v[decides].astype(np.float64), 5, -1)[None]
        assert (np.abs(rest - want) <= 2.0 ** -9 * np.abs(want) + 2.0 ** -24).all()
    assert_no_device_error()
