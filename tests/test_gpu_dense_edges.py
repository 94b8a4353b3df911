"""The ends of what the dense cache calls accept: values that are not finite, scales at the
ends of their range, sequences that cannot be used, streams."""
import math

import pytest
import torch

import dense_check as C
from dense_check import D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from two_stage_kv_snapkv_gb300 import build_lib
    build_lib.build()
    from two_stage_kv_snapkv_gb300 import rkv as mod
    return mod


def _status(rkv, cache):
    return rkv.rkv_get_device_status(cache)[1]


# ------------------------------------------------------------------ eviction: weights that are NaN
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("n,nans,keep,recent,room", [
    (150, 143, 12, 0, 0), (1000, 100, 50, 4, 0), (1000, 999, 500, 0, 0), (300, 300, 20, 3, 0),
    (1000, 100, 50, 4, 20000), (3000, 2500, 700, 16, 20000), (9000, 8000, 4000, 0, 0)])
def test_evict_with_more_nan_weights_than_kept(rkv, n, nans, keep, recent, room, in_place):
    """One decoding step with a NaN leaves every sum of its KV head NaN; tokens appended later
    weigh something.  `room` above 8192 positions: a cluster selects instead of one CTA."""
    Hkv, P = 2, 16
    cache, K, V = C.make_cache(rkv, [n], Hkv, P, seed=81, room=room)
    g = C.gen(82)
    acc0 = torch.rand(1, Hkv, cache.max_pages * P, generator=g) + 2.0 ** -10    # no zero among them
    for h in range(Hkv):
        at = torch.randperm(n, generator=g)[:nans] if h else torch.arange(nans)
        acc0[0, h, at] = math.nan
    acc0[:, :, n:] = 0
    kept = torch.full((1, Hkv, keep + 1), -7, dtype=torch.int32, device="cuda")
    to, to_acc = None, None
    if not in_place:
        to, _, _ = C.make_cache(rkv, [0], Hkv, P, seed=83, room=keep)
        to_acc = rkv.accum_sums(to)
    acc = acc0.cuda()
    rkv.rkv_evict_accum(cache, acc, [keep], recent, kept, dst=to, dst_acc=to_acc)
    assert _status(rkv, cache) == 0
    got, sums = (cache, acc) if in_place else (to, to_acc)
    for h in range(Hkv):
        want = C.keep_set(acc0[0, h], n, keep, recent)
        assert kept[0, h].tolist() == want + [-7], f"g{h}"
        assert torch.equal(got.token_kv(0, keep)[0][h].cpu(), K[0][h][want])
        assert torch.equal(sums[0, h, :keep].cpu().view(torch.int32), acc0[0, h][want].view(torch.int32))
