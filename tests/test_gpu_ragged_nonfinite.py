"""Values that are not finite in visible keys: the ragged operators give NaN exactly where the oracle
(softmax in 64 bits: a score of NaN or +inf makes the row NaN, one of -inf weighs nothing) gives it,
whichever kernel a shape runs on, and every other element stays within its tolerance."""
import numpy as np
import pytest
import torch

from paged_kv_cache_431_b200 import pkv
from paged_kv_cache_431_b200 import workloads as wl
from tests import test_gpu_cross as cross
from tests import test_gpu_groups as groups
from tests.ragged_helpers import DEV, NAMES, check, reference, tolerance

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
B16 = [pkv.BF16, pkv.F16]
TENSOR_CORE = {
    # form: (H_q, H_kv, rows, context) of each of 16 sequences: query rows per KV head 280, 28 and 80
    "shared_tiles": (8, 2, 70, 200),
    "lone_tile": (8, 2, 7, 150),
    "two_partitions": (8, 2, 20, 1500),
}
# 8 and 16 query rows per KV head, with partitions of a few tiles
WARP_LEVEL = {"eight_rows": (8, 2, 2, 500), "sixteen_rows": (8, 2, 4, 300)}
FORMS = {**TENSOR_CORE, **WARP_LEVEL}


def check_with_nan(out, ref, tol):
    """NaN in the same places, the rest within the tolerance."""
    got = out.detach().cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref)), \
        f"{np.isnan(got).sum()} NaN, expected {np.isnan(ref).sum()}; first difference at " \
        f"{np.argwhere(np.isnan(got) != np.isnan(ref))[:3].tolist()}"
    ok = ~np.isnan(ref)
    assert np.isfinite(got[ok]).all()
    over = np.abs(got - ref)[ok] - np.broadcast_to(tol, ref.shape)[ok]
    assert over.max(initial=-1.0) <= 0, f"off by {over.max()} more than allowed"


def put(pool, opool, side, blk, head, off, dim, value):
    """One element of K or V of a 16-bit pool, on both sides."""
    t = pool.k_data if side == "k" else pool.v_data
    t[0, blk, head, off, dim] = value
    raw = opool.k if side == "k" else opool.v
    bits = torch.tensor([value], dtype=wl.TORCH_DTYPE[opool.dtype]).view(torch.int16).numpy().view(np.uint8)
    raw[blk, head, off, 2 * dim:2 * dim + 2] = bits


def put_key(pool, opool, tables, b, pos, head, dim, value, side="k"):
    put(pool, opool, side, int(tables[b, pos // 16]), head, pos % 16, dim, value)


def cross_case(dt, d, form, seed, n=16):
    H_q, H_kv, rows, ctx = form
    rows, ctx = [rows] * n, [ctx + (5 * i) % 17 for i in range(n)]
    pool, opool, q, qd, tables = cross.case(dt, d, H_q, H_kv, rows, ctx, seed)
    return pool, opool, q, qd, tables, rows, ctx


def cross_compare(pool, opool, q, qd, tables, rows, ctx):
    scale = q.shape[-1] ** -0.5
    out = pkv.paged_cross_attn(pool, 0, q.to(DEV), cross.starts_of(rows).to(DEV), tables.to(DEV),
                               torch.tensor(ctx, dtype=torch.int32, device=DEV), scale, max(rows), max(ctx))
    torch.cuda.synchronize()
    ref = reference(opool, q, qd, tables, ctx, [b for b, r in enumerate(rows) for _ in range(r)], scale)
    # (rows of q that are not finite are NaN as a whole: their size adds nothing to the others' tolerance)
    check_with_nan(out, ref, tolerance(opool, torch.nan_to_num(q, 0.0, 0.0, 0.0), np.nan_to_num(ref), ctx, scale, True))
    return out, ref


@pytest.mark.parametrize("value", [NAN, INF, -INF], ids=["nan", "inf", "minus_inf"])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", B16, ids=lambda x: NAMES[x])
def test_one_key_not_finite(dt, d, form, value):
    """16 sequences, one key of each not finite, at 16 neighbouring positions; the other KV head keeps
    its finite keys.  An infinite element makes the score +inf or -inf by the sign of q's."""
    pool, opool, q, qd, tables, rows, ctx = cross_case(dt, d, FORMS[form], 7000 + dt + d)
    for b in range(16):
        put_key(pool, opool, tables, b, 37 + b, b % 2, (7 * b) % d, value)
    _, ref = cross_compare(pool, opool, q, qd, tables, rows, ctx)
    share = np.isnan(ref).mean()
    assert share == 0.5 if np.isnan(value) else 0.1 < share < 0.4


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dt", B16, ids=lambda x: NAMES[x])
def test_last_keys_and_values_not_finite(dt, form):
    """The last visible key, next to slots beyond the context; a NaN among the values, which reaches
    its own dim alone; query elements that are not finite."""
    pool, opool, q, qd, tables, rows, ctx = cross_case(dt, 128, FORMS[form], 7100 + dt)
    for b in range(16):
        if b < 6:
            put_key(pool, opool, tables, b, ctx[b] - 1, 0, 5 * b, (NAN, INF, -INF)[b % 3])
        elif b < 11:
            put_key(pool, opool, tables, b, 6 + b, 1, 9 * b, NAN, side="v")
        else:
            q[rows[0] * b + 1, b % 8, 3] = (NAN, INF, -INF)[b % 3]
    cross_compare(pool, opool, q, qd, tables, rows, ctx)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dt", B16, ids=lambda x: NAMES[x])
def test_scores_of_minus_infinity(dt, form):
    """Whole tiles, and whole sequences, of scores that are -inf: tiles weigh nothing, a sequence of
    nothing else is 0 / 0."""
    pool, opool, q, qd, tables, rows, ctx = cross_case(dt, 64, FORMS[form], 7200 + dt)
    q[..., 11] = q[..., 11].abs() + 1                     # so that -inf in dim 11 is a score of -inf
    for b in range(16):
        n = (0, 128, 130, ctx[b])[b % 4] if form in TENSOR_CORE else (0, 16, 130, ctx[b])[b % 4]
        for pos in range(n):
            put_key(pool, opool, tables, b, pos, b // 8, 11, -INF)
    _, ref = cross_compare(pool, opool, q, qd, tables, rows, ctx)
    assert 0 < np.isnan(ref).mean() < 0.2


@pytest.mark.parametrize("dt", pkv.QUANTIZED, ids=lambda x: NAMES[x])
@pytest.mark.parametrize("form", list(FORMS))
def test_scales_and_codes_not_finite(dt, form):
    """Quantized pools: a block's K or V scale NaN, its K scale infinite, and an e4m3 code that is NaN."""
    pool, opool, q, qd, tables, rows, ctx = cross_case(dt, 128, FORMS[form], 7300 + dt)
    for b in range(16):
        blk, head = int(tables[b, 1 + b % 8]), b % 2
        if b % 4 < 2:
            pool.k_scale[0, blk, head] = opool.k_scale[blk, head] = (NAN, INF)[b % 4]
        elif b % 4 == 2:
            pool.v_scale[0, blk, head] = opool.v_scale[blk, head] = NAN
        elif dt == pkv.FP8E4M3:
            pool.k_data[0, blk, head, b, 40] = 0x7f
            opool.k[blk, head, b, 40] = 0x7f
    _, ref = cross_compare(pool, opool, q, qd, tables, rows, ctx)
    assert np.isnan(ref).mean() >= 0.25


GROUPS = {
    # the prefix pass on the tensor cores, the suffix pass at the warp level, or (32 heads per KV head) too
    "few_heads": (8, 2, 6),
    "many_heads": (64, 2, 1),
}


@pytest.mark.parametrize("value", [NAN, INF, -INF], ids=["nan", "inf", "minus_inf"])
@pytest.mark.parametrize("where", ["prefix", "suffix"])
@pytest.mark.parametrize("form", list(GROUPS))
@pytest.mark.parametrize("dt", B16, ids=lambda x: NAMES[x])
def test_groups_one_key_not_finite(dt, form, where, value):
    """One key of each of 16 groups' prefixes, or of each group's first suffix."""
    H_q, H_kv, size = GROUPS[form]
    sizes, prefix = [size] * 16, [48 + 16 * (i % 3) for i in range(16)]
    suffix = [20 + i % 9 for i in range(16 * size)]
    pool, opool, q, qd, tables, ctx = groups.case(dt, 64, H_q, H_kv, sizes, prefix, suffix, 7400 + dt)
    for i in range(16):
        pos = 16 + i if where == "prefix" else prefix[i] + i
        put_key(pool, opool, tables, i * size, pos, i % 2, 3 * i, value)
    out = groups.call(pool, q, tables, ctx, sizes, prefix, suffix, 0.125)
    torch.cuda.synchronize()
    ref = reference(opool, q, qd, tables, ctx, range(len(ctx)), 0.125)
    check_with_nan(out, ref, tolerance(opool, q, np.nan_to_num(ref), ctx, 0.125, True))
    assert np.isnan(ref).any()


@pytest.mark.parametrize("dt", [pkv.BF16, pkv.INT8], ids=lambda x: NAMES[x])
def test_groups_suffix_of_minus_infinity(dt):
    """Sequences whose own tokens, one or more tiles of them, all have scores of -inf keep what their
    prefix gives (an e4m3 or integer code cannot be infinite: there a block's K scale is NaN)."""
    sizes, prefix, suffix = [3, 2], [32, 64], [1, 16, 40, 300, 7]
    pool, opool, q, qd, tables, ctx = groups.case(dt, 64, 8, 2, sizes, prefix, suffix, 7600 + dt)
    q[..., 11] = q[..., 11].abs() + 1
    for b in (0, 1, 3):
        pre = prefix[0] if b < 3 else prefix[1]
        if dt == pkv.BF16:
            for pos in range(pre, ctx[b]):
                put_key(pool, opool, tables, b, pos, 1, 11, -INF)
        else:
            blk = int(tables[b, pre // 16])
            pool.k_scale[0, blk, 1] = opool.k_scale[blk, 1] = NAN
    out = groups.call(pool, q, tables, ctx, sizes, prefix, suffix, 0.125)
    torch.cuda.synchronize()
    ref = reference(opool, q, qd, tables, ctx, range(len(ctx)), 0.125)
    check_with_nan(out, ref, tolerance(opool, q, np.nan_to_num(ref), ctx, 0.125, True))
    assert np.isnan(ref).any() == (dt == pkv.INT8)


def test_tiny_weights_of_large_values():
    """A key 2^-200 times less likely than another weighs nothing, even with values of 3e38: the
    polynomial exponentials end in 0, not in the smallest normal number."""
    dt, d = pkv.BF16, 128
    pool, opool, q, qd, tables, rows, ctx = cross_case(dt, d, TENSOR_CORE["shared_tiles"], 7500)
    q[..., 0] = 32.0
    for b in range(16):
        for pos in range(ctx[b]):
            put_key(pool, opool, tables, b, pos, 0, 0, 0.0)
        # log2 of the weight: 32 (-63 + 0) / sqrt(128) log2(e) = -257
        put_key(pool, opool, tables, b, 32 + b, 0, 0, -63.0)
        for j in range(d):
            put_key(pool, opool, tables, b, 32 + b, 0, j, 3e38, side="v")
    scale = d ** -0.5
    out = pkv.paged_cross_attn(pool, 0, q.to(DEV), cross.starts_of(rows).to(DEV), tables.to(DEV),
                               torch.tensor(ctx, dtype=torch.int32, device=DEV), scale, max(rows), max(ctx))
    torch.cuda.synchronize()
    ref = reference(opool, q, qd, tables, ctx, [b for b, r in enumerate(rows) for _ in range(r)], scale)
    # the values that count are those of the other keys, at most 6 in size
    for b in range(16):
        for j in range(d):
            put_key(pool, opool, tables, b, 32 + b, 0, j, 0.0, side="v")
    check(out, ref, tolerance(opool, q, ref, ctx, scale, True))
