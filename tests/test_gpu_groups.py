"""GPU parity for paged_decode_attn_groups: groups with prefixes of their own, against the oracle's
plain decode over each sequence's whole context."""
import pytest
import torch

from paged_kv_cache_431_b200 import pkv
from paged_kv_cache_431_b200 import workloads as wl
from tests.ragged_helpers import DEV, NAMES, check, make_pool, q_dtype, reference, tables_for, tolerance
from tests.test_gpu_cross import starts_of

pytestmark = pytest.mark.gpu


def case(dt, d, H_q, H_kv, sizes, prefix, suffix, seed, pad=0, bf16=True):
    """suffix: one list of own lengths per sequence, in order; pad: sequences behind the last group."""
    g = wl.generator(seed)
    of = [(i, p) for i, (n, p) in enumerate(zip(sizes, prefix)) for _ in range(n)]
    ctx = [p + s for (_, p), s in zip(of, suffix)]
    tables, N = tables_for(ctx, g, of)
    pool, opool = make_pool(tables, ctx, N, H_kv, d, dt, g)
    qd = q_dtype(dt, bf16)
    q = (2 * torch.randn(len(ctx) + pad, H_q, d, generator=g)).to(wl.TORCH_DTYPE[qd])
    return pool, opool, q, qd, tables, ctx


def call(pool, q, tables, ctx, sizes, prefix, suffix, scale, pad=0, bound=0, **kw):
    tb = torch.cat([tables, torch.full((pad, tables.shape[1]), -1, dtype=torch.int32)]).to(DEV)
    cl = torch.tensor(ctx + [77] * pad, dtype=torch.int32, device=DEV)
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)
    return pkv.paged_decode_attn_groups(pool, 0, q.to(DEV), tb, cl, starts_of(sizes).to(DEV),
                                        torch.tensor(prefix, dtype=torch.int32, device=DEV), scale,
                                        max(sizes) + bound, max(prefix) + 16 * bound, max(suffix) + bound, out=out, **kw)


def run(dt, d, H_q, H_kv, sizes, prefix, suffix, seed, pad=0, bf16=True, bound=0):
    pool, opool, q, qd, tables, ctx = case(dt, d, H_q, H_kv, sizes, prefix, suffix, seed, pad, bf16)
    scale = d ** -0.5
    out = call(pool, q, tables, ctx, sizes, prefix, suffix, scale, pad, bound)
    torch.cuda.synchronize()
    assert pkv.read_device_status(pool) == 0
    n = len(ctx)
    assert (out[n:] == 9).all()
    ref = reference(opool, q[:n], qd, tables, ctx, range(n), scale)
    check(out[:n], ref, tolerance(opool, q, ref, ctx, scale, True))


def drawn(seed, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=wl.generator(seed)).tolist()


SHAPES = [
    # (H_q, H_kv, group sizes, prefixes, suffixes)
    (8, 2, [2, 3], [32, 64], [1, 2, 3, 16, 17]),
    (4, 4, [1, 4, 0, 2], [16, 0, 48, 512], [5, 0, 1, 200, 33, 0, 1]),      # no prefix, no members, no suffix
    (12, 4, [5, 1], [300 * 16, 16], [40, 1, 500, 0, 3, 129]),              # 3 heads per KV head, split prefix
    (64, 8, [20, 9], [1024, 400], drawn(1, 29, 0, 90)),                    # the 70B head shape
    (16, 1, [40], [272], drawn(2, 40, 0, 40)),                            # one KV head, 640 rows
    (64, 1, [3, 2], [512, 32], [130, 0, 1, 17, 300]),                      # MQA: 64 rows per sequence
    (96, 1, [2], [160], [200, 5]),                                         # 96 heads on one KV head
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", list(NAMES), ids=lambda x: NAMES[x])
def test_groups_parity(dt, d, shape):
    H_q, H_kv, sizes, prefix, suffix = SHAPES[shape]
    run(dt, d, H_q, H_kv, sizes, prefix, suffix, 5000 + 50 * dt + d + shape, pad=shape % 3, bf16=shape % 2 == 0,
        bound=shape % 2)


@pytest.mark.parametrize("dt", [pkv.BF16, pkv.INT8], ids=lambda x: NAMES[x])
def test_groups_many(dt):
    """More groups than one look at 32 items."""
    sizes = drawn(3, 70, 0, 4)
    prefix = [16 * x for x in drawn(4, 70, 0, 12)]
    run(dt, 128, 8, 2, sizes, prefix, drawn(5, sum(sizes), 0, 200), 5500 + dt, pad=3)


def test_groups_without_any_prefix_is_the_plain_decode():
    run(pkv.F16, 64, 8, 2, [3, 2], [0, 0], [40, 1, 300, 0, 16], 5600)


def test_groups_match_the_single_prefix_call():
    """One group over the whole batch against the cascade call (fp32 out, two-part P)."""
    pool, _, q, _, tables, ctx = case(pkv.BF16, 128, 64, 8, [24], [512], drawn(6, 24, 1, 100), 5700)
    out = call(pool, q, tables, ctx, [24], [512], [100], 0.09)
    want = pkv.paged_decode_attn_cascade(pool, 0, q.to(DEV), tables.to(DEV),
                                         torch.tensor(ctx, dtype=torch.int32, device=DEV), 0.09, max(ctx), 512)
    torch.testing.assert_close(out.float(), want, rtol=2 ** -7, atol=2e-2)


def test_groups_reports():
    sizes, prefix, suffix = [3, 2], [64, 32], [5, 6, 7, 8, 9]
    pool, opool, q, qd, tables, ctx = case(pkv.BF16, 128, 8, 2, sizes, prefix, suffix, 5800)
    good = call(pool, q, tables, ctx, sizes, prefix, suffix, 0.1)
    assert pkv.read_device_status(pool) == 0
    t = tables.clone()
    t[1, 2] = t[0, 4]                       # sequence 1 leaves its group's prefix
    call(pool, q, t, ctx, sizes, prefix, suffix, 0.1)
    assert pkv.read_device_status(pool) == pkv.DEV_BAD_PREFIX
    out = call(pool, q, tables, ctx, sizes, [50, 32], [21] * 5, 0.1)     # no multiple of 16: rounded down
    assert pkv.read_device_status(pool) == pkv.DEV_BAD_PREFIX
    torch.testing.assert_close(out.float(), good.float(), rtol=2 ** -7, atol=2e-2)
    out = call(pool, q, tables, ctx, sizes, [-3, 32], [80] * 5, 0.1)
    assert pkv.read_device_status(pool) == pkv.DEV_BAD_LENGTH
    torch.testing.assert_close(out.float(), good.float(), rtol=2 ** -7, atol=2e-2)
    short = list(ctx)
    short[1] = 60                           # shorter than its prefix
    call(pool, q, tables, short, sizes, prefix, suffix, 0.1)
    assert pkv.read_device_status(pool) == pkv.DEV_BAD_LENGTH


def test_groups_larger_than_their_bound_are_reported():
    """Sequences past max_group_size are reported and left unwritten; the others are as they were."""
    sizes, prefix, suffix = [3, 2], [64, 32], [5, 6, 7, 8, 9]
    pool, opool, q, qd, tables, ctx = case(pkv.BF16, 128, 8, 2, sizes, prefix, suffix, 5850)
    args = (tables.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), starts_of(sizes).to(DEV),
            torch.tensor(prefix, dtype=torch.int32, device=DEV), 0.1)
    good = pkv.paged_decode_attn_groups(pool, 0, q.to(DEV), *args, 3, 64, 9)
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)
    pkv.paged_decode_attn_groups(pool, 0, q.to(DEV), *args, 2, 64, 9, out=out)
    torch.cuda.synchronize()
    assert pkv.read_device_status(pool) == pkv.DEV_BAD_LENGTH
    assert (out[2] == 9).all()
    keep = [0, 1, 3, 4]
    assert torch.equal(out[keep], good[keep])


def test_groups_captured_and_replayed():
    sizes, prefix, suffix = [6, 3], [512, 96], drawn(7, 9, 0, 150)
    pool, opool, q, qd, tables, ctx = case(pkv.FP8E4M3, 128, 16, 2, sizes, prefix, suffix, 5900)
    st, tb = starts_of(sizes).to(DEV), tables.to(DEV)
    cl, pl = torch.tensor(ctx, dtype=torch.int32, device=DEV), torch.tensor(prefix, dtype=torch.int32, device=DEV)
    qs = [q.to(DEV), (q.to(DEV) * 0.25).contiguous()]
    want = [pkv.paged_decode_attn_groups(pool, 0, x, tb, cl, st, pl, 0.1, 6, 512, 150) for x in qs]
    buf, res = torch.empty_like(qs[0]), torch.empty_like(qs[0])
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(pkv.paged_decode_groups_workspace_bytes(pool, 9, 16, 2, 6, 512, 150), dtype=torch.uint8, device=DEV)
    with torch.cuda.graph(graph):
        pkv.paged_decode_attn_groups(pool, 0, buf, tb, cl, st, pl, 0.1, 6, 512, 150, out=res, workspace=ws)
    for x, w in zip(qs, want):
        buf.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, w)


def test_rope_append_then_grouped_decode_and_cross():
    """As used together: states appended with the rotation, a grouped step over them, and a second
    model's rows against the same cache."""
    import numpy as np
    from tests.test_gpu_append_rope import oracle_copy, rotate, table
    g = wl.generator(5950)
    H_q, H_kv, d = 8, 2, 64
    sizes, prefix, suffix = [3, 2], [48, 16], [9, 20, 1, 33, 2]
    of = [(i, p) for i, (n, p) in enumerate(zip(sizes, prefix)) for _ in range(n)]
    ctx = [p + s for (_, p), s in zip(of, suffix)]
    tables, N = tables_for(ctx, g, of)
    for dt in (pkv.BF16, pkv.INT8):
        pool = pkv.KVPool.allocate(1, N, H_kv, d, dt)
        cs = table(d)
        # every token once: a group's prefix through its first sequence
        seq, pos = [], []
        for b, n in enumerate(ctx):
            first = 0 if b in (0, sizes[0]) else of[b][1]
            seq += [b] * (n - first)
            pos += range(first, n)
        slots = wl.slots_for(tables, seq, pos)
        k, v = wl.kv_source(len(seq), H_kv, d, g)
        pkv.kv_append_rope(pool, 0, None, k.to(DEV), v.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV),
                           cs.to(DEV), slots.to(DEV))
        torch.cuda.synchronize()
        opool = oracle_copy(pool)
        q = wl.normal((len(ctx), H_q, d), torch.bfloat16, g)
        at = torch.tensor(ctx, dtype=torch.int32) - 1
        qr = rotate(q, cs[at.long()], False, torch.float32).to(torch.bfloat16)
        out = call(pool, qr, tables, ctx, sizes, prefix, suffix, 0.125)
        ref = reference(opool, qr, pkv.BF16, tables, ctx, range(len(ctx)), 0.125)
        check(out, ref, tolerance(opool, qr, ref, ctx, 0.125, True))
        rows = [2, 0, 1, 4, 1]
        x = wl.normal((sum(rows), H_q, d), torch.bfloat16, g)
        o2 = pkv.paged_cross_attn(pool, 0, x.to(DEV), starts_of(rows).to(DEV), tables.to(DEV),
                                  torch.tensor(ctx, dtype=torch.int32, device=DEV), 0.125, 4, max(ctx))
        r2 = reference(opool, x, pkv.BF16, tables, ctx, [b for b, r in enumerate(rows) for _ in range(r)], 0.125)
        check(o2, r2, tolerance(opool, x, r2, ctx, 0.125, True))
        assert pkv.read_device_status(pool) == 0 and np.isfinite(r2).all()
