"""The bounded waits of the ragged operators' kernels: with one K tile's copy withheld they record
PKV_DEV_TIMEOUT and end, and the same call, with the hook off, then matches the oracle."""
import pytest
import torch

from paged_kv_cache_431_b200 import pkv
from tests import test_gpu_cross as cross
from tests import test_gpu_groups as groups
from tests.ragged_helpers import DEV, check, reference, tolerance
from tests.test_gpu_timeout import WAIT, expect_timeout

pytestmark = pytest.mark.gpu

CROSS = {
    # name: (pool dtype, head dim, H_q, H_kv, rows, contexts)
    "warp_level_bf16": (pkv.BF16, 128, 8, 2, [2, 1], [300, 700]),
    "warp_level_int8": (pkv.INT8, 128, 8, 2, [2, 1], [300, 700]),
    "tcgen05_shared_tiles_bf16": (pkv.BF16, 128, 8, 2, [90, 70], [500, 400]),
    "tcgen05_shared_tiles_f16_d64": (pkv.F16, 64, 8, 2, [90, 70], [500, 400]),
    "tcgen05_pair_bf16": (pkv.BF16, 128, 8, 2, [20, 12], [1500, 1100]),
    "tcgen05_pair_fp8": (pkv.FP8E4M3, 128, 8, 2, [20, 12], [1500, 1100]),
    "tcgen05_shared_tiles_int4": (pkv.INT4, 128, 8, 2, [90, 70], [500, 400]),
}


@pytest.mark.parametrize("name", list(CROSS))
def test_cross_gives_up_and_recovers(name):
    dt, d, H_q, H_kv, rows, ctx = CROSS[name]
    pool, opool, q, qd, tables = cross.case(dt, d, H_q, H_kv, rows, ctx, 6000 + list(CROSS).index(name))
    args = (pool, 0, q.to(DEV), cross.starts_of(rows).to(DEV), tables.to(DEV),
            torch.tensor(ctx, dtype=torch.int32, device=DEV), 0.1, max(rows), max(ctx))
    pkv.test_withhold_copy(1, WAIT)
    try:
        pkv.paged_cross_attn(*args)
        torch.cuda.synchronize()
    finally:
        pkv.test_withhold_copy(-1)
    expect_timeout(pool)
    out = pkv.paged_cross_attn(*args)
    torch.cuda.synchronize()
    assert pkv.get_device_status(pool) == (0, 0)
    ref = reference(opool, q, qd, tables, ctx, [b for b, r in enumerate(rows) for _ in range(r)], 0.1)
    check(out, ref, tolerance(opool, q, ref, ctx, 0.1, True))


@pytest.mark.parametrize("dt", [pkv.BF16, pkv.INT8], ids=["bf16", "int8"])
def test_groups_give_up_and_recover(dt):
    sizes, prefix, suffix = [30, 3], [1024, 256], [20] * 33
    pool, opool, q, qd, tables, ctx = groups.case(dt, 128, 16, 2, sizes, prefix, suffix, 6100 + dt)
    pkv.test_withhold_copy(1, WAIT)
    try:
        groups.call(pool, q, tables, ctx, sizes, prefix, suffix, 0.1)
        torch.cuda.synchronize()
    finally:
        pkv.test_withhold_copy(-1)
    expect_timeout(pool)
    out = groups.call(pool, q, tables, ctx, sizes, prefix, suffix, 0.1)
    torch.cuda.synchronize()
    assert pkv.get_device_status(pool) == (0, 0)
    ref = reference(opool, q, qd, tables, ctx, range(33), 0.1)
    check(out, ref, tolerance(opool, q, ref, ctx, 0.1, True))
