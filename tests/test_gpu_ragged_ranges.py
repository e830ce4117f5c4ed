"""The ragged operators, and the decode of quantized pools, where magnitudes differ widely within a
call: query rows, V scales, weights."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_431_b200 import pkv
from paged_kv_cache_431_b200 import workloads as wl
from tests import test_gpu_cross as cross
from tests.ragged_helpers import DEV, NAMES, check, make_pool, reference, tables_for, tolerance

pytestmark = pytest.mark.gpu

# query rows per KV head: warp level with 8 and 16, tcgen05 with the rows four times, twice, once in a
# tile (quantized pools), and with shared tiles
ROWS = [[2], [4], [7], [14], [25], [90]]


def call(pool, q, rows, tables, ctx, scale):
    out = pkv.paged_cross_attn(pool, 0, q.to(DEV), cross.starts_of(rows).to(DEV), tables.to(DEV),
                               torch.tensor(ctx, dtype=torch.int32, device=DEV), scale, max(rows), max(ctx))
    torch.cuda.synchronize()
    assert pkv.read_device_status(pool) == 0
    return out


@pytest.mark.parametrize("rows", ROWS, ids=lambda r: f"{r[0]}rows")
@pytest.mark.parametrize("dt", [pkv.BF16, *pkv.QUANTIZED], ids=lambda x: NAMES[x])
def test_rows_2_40_apart_in_size_keep_their_precision(dt, rows):
    """Every other row 2^40 times smaller, once with a scale that suits the small ones, once one that
    suits the large ones; the suited rows are compared.  Zero in place of the small rows would be off by
    far more than the tolerance (checked on the oracle)."""
    ctx = [700]
    pool, opool, q, qd, tables = cross.case(dt, 128, 4, 1, rows, ctx, 8000 + dt + rows[0])
    small = torch.arange(rows[0]) % 2 == 0
    q[small] *= 2.0 ** -40
    for some, scale in ((small, 0.1 * 2.0 ** 40), (~small, 0.1)):
        out = call(pool, q, rows, tables, ctx, scale)
        qs, n = q[some].contiguous(), int(some.sum())
        ref = reference(opool, qs, qd, tables, ctx, [0] * n, scale)
        tol = tolerance(opool, qs, ref, ctx, scale, True)
        check(out[some], ref, tol)
        none = reference(opool, torch.zeros_like(qs), qd, tables, ctx, [0] * n, scale)
        assert (np.abs(none - ref) > tol).mean() > 0.5


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")], ids=["nan", "inf", "minus_inf"])
@pytest.mark.parametrize("rows", ROWS, ids=lambda r: f"{r[0]}rows")
@pytest.mark.parametrize("dt", pkv.QUANTIZED, ids=lambda x: NAMES[x])
def test_rows_not_finite_leave_the_others_alone(dt, rows, value):
    """A row of q with an element that is not finite is NaN, its neighbours are as without it."""
    ctx = [300]
    pool, opool, q, qd, tables = cross.case(dt, 64, 4, 1, rows, ctx, 8050 + dt + rows[0])
    q[1, 2, 5] = value
    out = call(pool, q, rows, tables, ctx, 0.1)
    assert torch.isnan(out[1, 2]).all()
    clean = q.clone()
    clean[1, 2] = 0
    ref = reference(opool, clean, qd, tables, ctx, [0] * rows[0], 0.1)
    tol = tolerance(opool, clean, ref, ctx, 0.1, True)
    out[1, 2], ref[1, 2], tol[1, 2] = 0, 0, 1
    check(out, ref, tol)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")], ids=["nan", "inf", "minus_inf"])
@pytest.mark.parametrize("dt", pkv.QUANTIZED, ids=lambda x: NAMES[x])
def test_decode_heads_not_finite_leave_the_others_alone(dt, value):
    """The same for the heads of one sequence in the plain decode."""
    g = wl.generator(8090 + dt)
    ctx = [300, 90]
    tables, N = tables_for(ctx, g)
    pool, opool = make_pool(tables, ctx, N, 2, 128, dt, g)
    q = wl.normal((2, 8, 128), torch.bfloat16, g)
    q[1, 2, 5] = value
    lens = torch.tensor(ctx, dtype=torch.int32)
    out = pkv.paged_decode_attn(pool, 0, q.to(DEV), tables.to(DEV), lens.to(DEV), 0.1, max(ctx)).cpu().double().numpy()
    clean = q.clone()
    clean[1, 2] = 0
    ref = oracle.paged_decode(opool, clean, pkv.BF16, tables, lens, np.float32(0.1))
    assert np.isnan(out[1, 2]).all()
    out[1, 2] = ref[1, 2]
    assert np.abs(out - ref).max() <= 2e-3


@pytest.mark.parametrize("gain", [2.0 ** 20, 2.0 ** 60], ids=["2^20", "2^60"])
@pytest.mark.parametrize("rows", ROWS, ids=lambda r: f"{r[0]}rows")
@pytest.mark.parametrize("dt", list(NAMES), ids=lambda x: NAMES[x])
def test_huge_scores_leave_one_key(dt, rows, gain):
    """Scores of 10^6 and 10^18 times the usual size: a row takes the values of its best key (rows whose
    two best keys are closer than the scores' own rounding may mix them, and are only finite)."""
    ctx = [700]
    pool, opool, q, qd, tables = cross.case(dt, 128, 4, 1, rows, ctx, 8100 + dt + rows[0])
    scale = 0.1 * gain
    out = call(pool, q, rows, tables, ctx, scale)
    assert torch.isfinite(out).all()
    blocks = tables[0, :-(-ctx[0] // 16)].long()
    k = torch.as_tensor(opool.dequant("k"))[blocks].transpose(1, 2).reshape(-1, 128)[:ctx[0]]
    best = (q.double() @ k.T).topk(2, dim=-1).values
    # fp32 sums of 128 terms: (128 + 2) 2^-24 |q| |k|; quantized pools' q: 2^-14 / sqrt(128) of it more
    err = q.double().norm(dim=-1) * k.norm(dim=-1).max() * (130 * 2.0 ** -24 + 2.0 ** -14 / 128 ** 0.5)
    clear = ((best[..., 0] - best[..., 1] - 2 * err) * scale > 40).numpy()
    assert clear.mean() > 0.9
    ref = reference(opool, q, qd, tables, ctx, [0] * rows[0], scale)
    # a weight of 1, rounded nowhere, times a value whose scale is rounded into P; and the output's half step
    got = out.cpu().double().numpy()
    bound = torch.finfo(q.dtype).eps / 2 * np.abs(ref) + 2.0 ** -11 * np.abs(ref) + 2.0 ** -24
    assert (np.abs(got - ref) <= bound)[clear].all()


def steer(pool, opool, blocks, d, up):
    """Codes of K's dim 0 in the listed blocks: the largest positive one, or the largest negative one."""
    code = {pkv.INT8: (0x7F, 0x81), pkv.INT4: (0x7, 0x9), pkv.FP8E4M3: (0x7E, 0xFE)}[opool.dtype][0 if up else 1]
    for blk in blocks:
        if opool.dtype == pkv.INT4:
            opool.k[blk, :, :, 0] = (opool.k[blk, :, :, 0] & 0xF0) | code
        else:
            opool.k[blk, :, :, 0] = code
        opool.k_scale[blk] = opool.k_scale[blocks[0]]
        pool.k_data[0, blk] = torch.as_tensor(opool.k[blk])
        pool.k_scale[0, blk] = torch.as_tensor(opool.k_scale[blk])


@pytest.mark.parametrize("ratio", [2.0 ** -20, 2.0 ** -12], ids=["2^-20", "2^-12"])
@pytest.mark.parametrize("rows", ROWS, ids=lambda r: f"{r[0]}rows")
@pytest.mark.parametrize("dt", pkv.QUANTIZED, ids=lambda x: NAMES[x])
def test_weight_on_blocks_with_small_v_scales(dt, rows, ratio):
    """Every other block's V scale 2^-20 of its neighbour's, the rows' weight on these blocks: the output
    is as exact as if the others, which weigh less than 2^-60, were not there."""
    ctx, d = [700], 128
    pool, opool, q, qd, tables = cross.case(dt, d, 4, 1, rows, ctx, 8300 + dt + rows[0], gain=6.0)
    blocks = tables[0, :-(-ctx[0] // 16)].tolist()
    for blk in blocks[::2]:
        opool.v_scale[blk] *= ratio
        pool.v_scale[0, blk] = torch.as_tensor(opool.v_scale[blk])
    steer(pool, opool, blocks[::2], d, True)
    steer(pool, opool, blocks[1::2], d, False)
    q[..., 0] = 256.0
    scale = d ** -0.5
    out = call(pool, q, rows, tables, ctx, scale)
    ref = reference(opool, q, qd, tables, ctx, [0] * rows[0], scale)
    small = opool.copy()
    small.v_scale[blocks[1::2]] = 0
    near = reference(small, q, qd, tables, ctx, [0] * rows[0], scale)
    tol = tolerance(small, q, near, ctx, scale, True)
    assert np.abs(ref - near).max() < 1e-3 * tol.min()
    check(out, ref, tol)


@pytest.mark.parametrize("spread", [1e-9, 1e-6, 1e6], ids=["1e-9", "1e-6", "1e6"])
@pytest.mark.parametrize("H_q,H_kv", [(8, 2), (16, 2), (24, 2), (32, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", pkv.QUANTIZED, ids=lambda x: NAMES[x])
def test_decode_of_small_and_large_pools(dt, d, H_q, H_kv, spread):
    """The plain decode over pools whose scales are far from 1, in one partition and in several (the
    output's bound of 2e-3 in proportion to the pool's magnitude)."""
    g = wl.generator(8400 + dt + d + H_q)
    ctx = [700, 33, 1, 5000]
    tables, N = tables_for(ctx, g)
    pool, opool = make_pool(tables, ctx, N, H_kv, d, dt, g, spread)
    q = wl.normal((len(ctx), H_q, d), torch.bfloat16, g)
    lens = torch.tensor(ctx, dtype=torch.int32)
    scale = d ** -0.5 / spread
    ref = oracle.paged_decode(opool, q, pkv.BF16, tables, lens, np.float32(scale))
    for part in (0, 512):
        out = pkv.paged_decode_attn(pool, 0, q.to(DEV), tables.to(DEV), lens.to(DEV), scale, max(ctx), partition_tokens=part)
        assert np.abs(out.cpu().double().numpy() - ref).max() <= 2e-3 * spread


@pytest.mark.parametrize("rows", [[2, 1], [7, 3], [25, 9], [90, 40]], ids=lambda r: f"{r[0]}rows")
@pytest.mark.parametrize("dt", [pkv.BF16, pkv.INT8], ids=lambda x: NAMES[x])
def test_cross_lengths_past_the_bound(dt, rows):
    """max_context_len counts in whole blocks, whatever kernel and partition the shape gets: one token past
    them is reported and left out, up to them nothing is."""
    ctx = [305, 304]
    pool, _, q, _, tables = cross.case(dt, 128, 4, 1, rows, ctx, 8500 + dt + rows[0])

    def at(lens, bound):
        out = pkv.paged_cross_attn(pool, 0, q.to(DEV), cross.starts_of(rows).to(DEV), tables.to(DEV),
                                   torch.tensor(lens, dtype=torch.int32, device=DEV), 0.1, max(rows), bound)
        torch.cuda.synchronize()
        return out, pkv.read_device_status(pool)
    for bound in (289, 304):
        whole, status = at([304, 304], bound)
        assert status == 0
        clipped, status = at(ctx, bound)
        assert status == pkv.DEV_BAD_LENGTH and torch.equal(clipped, whole)


@pytest.mark.parametrize("H_q", [8, 64], ids=["warp_level", "tcgen05"])
def test_groups_suffixes_past_the_bound(H_q):
    from tests import test_gpu_groups as groups
    sizes, prefix, suffix = [3, 2], [64, 32], [33, 20, 32, 1, 33]
    pool, _, q, _, tables, ctx = groups.case(pkv.BF16, 128, H_q, 2, sizes, prefix, suffix, 8600 + H_q)

    def at(lens, bound):
        out = groups.call(pool, q, tables, lens, sizes, prefix, [bound] * 5, 0.1)
        torch.cuda.synchronize()
        return out, pkv.read_device_status(pool)
    for bound in (17, 32):
        whole, status = at([96, 84, 96, 33, 64], bound)
        assert status == 0
        clipped, status = at(ctx, bound)
        assert status == pkv.DEV_BAD_LENGTH and torch.equal(clipped, whole)
