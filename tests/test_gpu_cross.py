"""GPU parity for paged_cross_attn: every row against the oracle's attention over all cached tokens of
its sequence, with poison in every slot outside the contexts, empty sequences, sequences without
rows, and padding rows that stay as they were."""
import numpy as np
import pytest
import torch

from paged_kv_cache_431_b200 import pkv
from paged_kv_cache_431_b200 import workloads as wl
from tests.ragged_helpers import DEV, NAMES, check, make_pool, q_dtype, reference, tables_for, tolerance

pytestmark = pytest.mark.gpu


def starts_of(rows):
    return torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)


def case(dt, d, H_q, H_kv, rows, ctx, seed, pad=0, bf16=True, spread=1.0, gain=2.0):
    g = wl.generator(seed)
    tables, N = tables_for(ctx, g)
    pool, opool = make_pool(tables, ctx, N, H_kv, d, dt, g, spread)
    qd = q_dtype(dt, bf16)
    total = sum(rows) + pad
    q = (gain * torch.randn(total, H_q, d, generator=g)).to(wl.TORCH_DTYPE[qd])
    return pool, opool, q, qd, tables


def run(dt, d, H_q, H_kv, rows, ctx, seed, pad=0, bf16=True, spread=1.0, gain=2.0):
    pool, opool, q, qd, tables = case(dt, d, H_q, H_kv, rows, ctx, seed, pad, bf16, spread, gain)
    scale = d ** -0.5
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)
    pkv.paged_cross_attn(pool, 0, q.to(DEV), starts_of(rows).to(DEV), tables.to(DEV),
                         torch.tensor(ctx, dtype=torch.int32, device=DEV), scale, max(rows), max(ctx), out=out)
    torch.cuda.synchronize()
    assert pkv.read_device_status(pool) == 0
    n = sum(rows)
    assert (out[n:] == 9).all()
    row_of = [b for b, r in enumerate(rows) for _ in range(r)]
    ref = reference(opool, q[:n], qd, tables, ctx, row_of, scale)
    check(out[:n], ref, tolerance(opool, q, ref, ctx, scale, True))
    return pool, q, tables, out


SHAPES = [
    # (H_q, H_kv, rows per sequence, context per sequence)
    (8, 2, [1, 1, 1], [17, 1, 64]),                                  # single tokens
    (4, 4, [1, 0, 3, 2], [0, 40, 33, 700]),                          # MHA; an empty state, no rows
    (12, 4, [5, 4, 1, 5], [300, 16, 15, 2050]),                      # beams, 3 heads per KV head
    (8, 1, [7, 20, 1], [129, 1000, 255]),                            # MQA-like
    (16, 2, [33, 8, 50], [128, 513, 90]),                            # up to 400 rows per KV head
    (6, 2, [200, 1, 90, 0], [500, 77, 0, 12]),                       # 600 rows, 3 heads per KV head
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", list(NAMES), ids=lambda x: NAMES[x])
def test_cross_parity(dt, d, shape):
    H_q, H_kv, rows, ctx = SHAPES[shape]
    run(dt, d, H_q, H_kv, rows, ctx, 4000 + 50 * dt + d + shape, pad=shape, bf16=shape % 2 == 0)


@pytest.mark.parametrize("dt", list(NAMES), ids=lambda x: NAMES[x])
def test_cross_many_sequences_and_rows(dt):
    """More sequences than one look at 32 items, lengths drawn from 0 to a few hundred."""
    g = wl.generator(4500 + dt)
    rows = torch.randint(0, 9, (75,), generator=g).tolist()
    ctx = torch.randint(0, 300, (75,), generator=g).tolist()
    run(dt, 128, 8, 2, rows, ctx, 4501 + dt, pad=4)


@pytest.mark.parametrize("dt", pkv.QUANTIZED, ids=lambda x: NAMES[x])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [[4, 3, 1, 2, 0, 4], [4, 3, 8, 1, 6, 5], [4, 3, 8, 12, 6, 16]])
def test_cross_rows_shared_out_over_keys(dt, d, rows):
    """8 to 128 query rows per KV head in one launch (up to 32, up to 64 and more are treated
    differently), with last tiles of 1, 40, 72 and 104 keys and partitions of one tile."""
    run(dt, d, 16, 2, rows, [5000, 129, 2088, 40, 300, 3176], 4600 + dt + d + rows[3], pad=2, gain=4.0)


@pytest.mark.parametrize("dt", pkv.QUANTIZED, ids=lambda x: NAMES[x])
def test_cross_peaked_rows_shared_out_over_keys(dt):
    """Logits of up to several hundred, so that a row's parts differ by factors beyond 2^126."""
    run(dt, 128, 8, 1, [4, 2, 6], [1300, 20000, 515], 4650 + dt, gain=60.0)


@pytest.mark.parametrize("dt", [pkv.BF16, pkv.F16, pkv.FP8E4M3, pkv.INT8], ids=lambda x: NAMES[x])
@pytest.mark.parametrize("rows", [1, 130])
def test_cross_long_state(dt, rows):
    run(dt, 128, 8, 2, [rows, 2], [9000, 4097], 4600 + dt + rows)


@pytest.mark.parametrize("dt", [pkv.BF16, pkv.INT8], ids=lambda x: NAMES[x])
@pytest.mark.parametrize("gain", [0.0, 1e-3, 30.0])
def test_cross_flat_and_peaked_weights(dt, gain):
    """Zero, tiny and large q: uniform weights, and weights that leave one key."""
    for rows in ([3, 1], [150, 40]):
        run(dt, 128, 8, 2, rows, [600, 333], 4700 + dt, gain=gain)


@pytest.mark.parametrize("dt", pkv.QUANTIZED, ids=lambda x: NAMES[x])
@pytest.mark.parametrize("spread", [1e-6, 1e4])
def test_cross_small_and_large_scales(dt, spread):
    """Pools whose scales are far from 1 (the scores stay moderate: q is scaled against them)."""
    for rows in ([2, 1], [140, 3]):
        pool, opool, q, qd, tables = case(dt, 128, 8, 2, rows, [400, 260], 4800 + dt, spread=spread, gain=1.0)
        scale = 128 ** -0.5 / spread
        out = pkv.paged_cross_attn(pool, 0, q.to(DEV), starts_of(rows).to(DEV), tables.to(DEV),
                                   torch.tensor([400, 260], dtype=torch.int32, device=DEV), scale, max(rows), 400)
        torch.cuda.synchronize()
        ref = reference(opool, q, qd, tables, [400, 260], [0] * rows[0] + [1] * rows[1], scale)
        check(out, ref, tolerance(opool, q, ref, [400, 260], scale, True))


@pytest.mark.parametrize("dt", [pkv.BF16, pkv.FP8E4M3], ids=lambda x: NAMES[x])
@pytest.mark.parametrize("scale", [-0.07, 0.0])
def test_cross_negative_and_zero_scale(dt, scale):
    for rows in ([2, 1], [130, 50]):
        pool, opool, q, qd, tables = case(dt, 128, 8, 2, rows, [300, 77], 4850 + dt)
        out = pkv.paged_cross_attn(pool, 0, q.to(DEV), starts_of(rows).to(DEV), tables.to(DEV),
                                   torch.tensor([300, 77], dtype=torch.int32, device=DEV), scale, max(rows), 300)
        ref = reference(opool, q, qd, tables, [300, 77], [0] * rows[0] + [1] * rows[1], scale)
        check(out, ref, tolerance(opool, q, ref, [300, 77], scale, True))


def test_cross_rows_of_very_different_size():
    """Neighbouring query rows 2^24 apart in size: each keeps its own precision."""
    for dt in (pkv.BF16, pkv.INT8, pkv.FP8E4M3):
        for rows in ([4], [40], [150]):
            pool, opool, q, qd, tables = case(dt, 128, 4, 1, rows, [200], 4870 + dt)
            q[::2] *= 2.0 ** -24
            out = pkv.paged_cross_attn(pool, 0, q.to(DEV), starts_of(rows).to(DEV), tables.to(DEV),
                                       torch.tensor([200], dtype=torch.int32, device=DEV), 0.1, rows[0], 200)
            ref = reference(opool, q, qd, tables, [200], [0] * rows[0], 0.1)
            check(out, ref, tolerance(opool, q, ref, [200], 0.1, True))


@pytest.mark.parametrize("dt", [pkv.BF16, pkv.INT4], ids=lambda x: NAMES[x])
def test_cross_one_sequence_with_many_rows(dt):
    """One sequence with thousands of rows against a short state; a batch of many tiny sequences."""
    run(dt, 64, 2, 2, [3000], [20], 4880 + dt)
    run(dt, 64, 4, 2, [1] * 700, [1 + i % 40 for i in range(700)], 4890 + dt)


def test_cross_bounds_larger_than_needed_and_layers():
    """Host bounds may exceed the real lengths; the layer argument picks the layer."""
    g = wl.generator(4900)
    rows, ctx = [3, 60], [100, 300]
    tables, N = tables_for(ctx, g)
    p0, _ = make_pool(tables, ctx, N, 2, 128, pkv.BF16, g)
    p1, opool = make_pool(tables, ctx, N, 2, 128, pkv.BF16, g)
    both = pkv.KVPool.from_layers([p0.k_data[0], p1.k_data[0]], [p0.v_data[0], p1.v_data[0]], pkv.BF16, 128)
    q = wl.normal((63, 8, 128), torch.bfloat16, g)
    ref = reference(opool, q, pkv.BF16, tables, ctx, [0] * 3 + [1] * 60, 0.1)
    tol = tolerance(opool, q, ref, ctx, 0.1, True)
    for mr, mc in ((60, 300), (500, 5000), (61, 301), (200000, 300)):
        tb = torch.cat([tables, torch.full((2, 400), -1, dtype=torch.int32)], 1).contiguous()
        out = pkv.paged_cross_attn(both, 1, q.to(DEV), starts_of(rows).to(DEV), tb.to(DEV),
                                   torch.tensor(ctx, dtype=torch.int32, device=DEV), 0.1, mr, mc)
        check(out, ref, tol)


def test_cross_reports_and_clips():
    """Lengths past the bounds and row starts out of range are reported; nothing else is touched."""
    rows, ctx = [4, 30, 2], [100, 300, 50]
    pool, opool, q, qd, tables = case(pkv.BF16, 128, 8, 2, rows, ctx, 4950)
    st, cl = starts_of(rows), torch.tensor(ctx, dtype=torch.int32)

    def call(starts, lens, mr=30, mc=300, tb=tables):
        out = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)
        pkv.paged_cross_attn(pool, 0, q.to(DEV), starts.to(DEV), tb.to(DEV), lens.to(DEV), 0.1, mr, mc, out=out)
        torch.cuda.synchronize()
        return out.cpu(), pkv.read_device_status(pool)
    good, status = call(st, cl)
    assert status == 0
    out, status = call(st, torch.tensor([100, -5, 50], dtype=torch.int32))
    assert status == pkv.DEV_BAD_LENGTH
    assert torch.equal(out[:4], good[:4]) and (out[4:34] == 0).all() and torch.equal(out[34:], good[34:])
    out, status = call(st, torch.tensor([100, 300, 100000], dtype=torch.int32))
    assert status & pkv.DEV_BAD_LENGTH and torch.equal(out[:34], good[:34])
    # bounds choose the kernel, so other bounds give other roundings: within the tolerance of the oracle
    ref = reference(opool, q, qd, tables, ctx, [0] * 4 + [1] * 30 + [2] * 2, 0.1)
    tol = tolerance(opool, q, ref, ctx, 0.1, True)
    check(good, ref, tol)
    out, status = call(st, cl, mr=10)
    assert status == pkv.DEV_BAD_LENGTH and (out[14:34] == 9).all()
    for rows_ in (slice(0, 14), slice(34, 36)):
        check(out[rows_], ref[rows_], tol[rows_])
    bad = torch.tensor([0, 4, 2, 5000], dtype=torch.int32)       # descending, then past the end
    out, status = call(bad, cl)
    assert status == pkv.DEV_BAD_LENGTH
    check(out[:2], ref[:2], tol[:2])
    tb = tables.clone()
    tb[2, 1] = 10 ** 6
    out, status = call(st, cl, tb=tb)
    assert status == pkv.DEV_BAD_BLOCK and torch.equal(out[:34], good[:34])


def test_cross_two_calls_streams_and_graph():
    """Two calls at once on streams of their own, and a captured call replayed on new rows."""
    rows, ctx = [5, 40, 1, 0], [900, 130, 2000, 30]
    pool, opool, q, qd, tables = case(pkv.BF16, 128, 8, 2, rows, ctx, 4960)
    args = (starts_of(rows).to(DEV), tables.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), 0.09, 40, 2000)
    qa = q.to(DEV)
    qb = (qa * 0.5).contiguous()
    want_a, want_b = (pkv.paged_cross_attn(pool, 0, x, *args) for x in (qa, qb))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a = pkv.paged_cross_attn(pool, 0, qa, *args, stream=s1)
        b = pkv.paged_cross_attn(pool, 0, qb, *args, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a, want_a) and torch.equal(b, want_b)
    buf, res = qa.clone(), torch.empty_like(qa)
    ws = torch.empty(pkv.paged_cross_workspace_bytes(pool, qa.shape[0], 8, 4, 40, 2000), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_cross_attn(pool, 0, buf, *args, out=res, workspace=ws)
    for x, want in ((qb, want_b), (qa, want_a)):
        buf.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, want)


def test_cross_python_refusals():
    pool = pkv.KVPool.allocate(1, 8, 2, 128, pkv.BF16)
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device=DEV)
    st = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    tb = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    cl = torch.tensor([20], dtype=torch.int32, device=DEV)
    ok = dict(q=q, row_starts=st, block_tables=tb, context_lens=cl)
    for bad in (dict(q=q[..., :64].contiguous()), dict(q=q.transpose(0, 1)), dict(row_starts=st[:1].contiguous()),
                dict(row_starts=st.long()), dict(block_tables=tb.cpu()), dict(context_lens=cl.repeat(2)),
                dict(block_tables=tb[0])):
        a = dict(ok, **bad)
        with pytest.raises(ValueError):
            pkv.paged_cross_attn(pool, 0, a["q"], a["row_starts"], a["block_tables"], a["context_lens"], 0.1, 4, 20)
    with pytest.raises(ValueError):
        pkv.paged_cross_attn(pool, 0, q, st, tb, cl, 0.1, 4, 20, out=torch.zeros_like(q, dtype=torch.float32))
    with pytest.raises(pkv.PkvError):
        pkv.paged_cross_attn(pool, 0, q.half(), st, tb, cl, 0.1, 4, 20)
    none = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=DEV)
    assert pkv.paged_cross_attn(pool, 0, none, torch.zeros(1, dtype=torch.int32, device=DEV), tb[:0], cl[:0], 0.1, 0,
                                0).shape == none.shape
