"""GPU parity for kv_append_rope: the rotation against its definition in 64 bits, the pool bit-exact
against the oracle's append of the rotated rows, padding and out-of-range tokens left alone."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_431_b200 import pkv
from paged_kv_cache_431_b200 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = {pkv.F16: "f16", pkv.BF16: "bf16", pkv.INT8: "int8", pkv.INT4: "int4", pkv.FP8E4M3: "fp8"}
POS = 5000


def table(rot, positions=POS):
    half = rot // 2
    a = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float()


def pairs(rot, inter):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)


def rotate(x, cs, inter, dtype):
    """The rotation of x [T, H, d] by the angles of cs [T, rot], in `dtype`, every operation rounded."""
    rot = cs.shape[1]
    x, cs = x.to(dtype), cs.to(dtype)
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    p1, p2 = pairs(rot, inter)
    a, b = x[..., p1], x[..., p2]
    y = x.clone()
    y[..., p1] = a * c - b * s
    y[..., p2] = b * c + a * s
    return y


def stale_pool(N, H_kv, d, dt, g, layers=1):
    pool = pkv.KVPool.allocate(layers, N, H_kv, d, dt)
    for x in (pool.k_data, pool.v_data):
        if dt in pkv.QUANTIZED:
            c = torch.randint(0, 256, x.shape, generator=g, dtype=torch.int32).to(torch.uint8)
            if dt == pkv.FP8E4M3:
                c[(c & 0x7F) == 0x7F] = 0x7E      # no NaN codes
            x.copy_(c)
        else:
            x.copy_(wl.normal(x.shape, x.dtype, g))
    if dt in pkv.QUANTIZED:
        pool.k_scale.copy_(torch.rand(pool.k_scale.shape, generator=g) * 0.05)
        pool.v_scale.copy_(torch.rand(pool.v_scale.shape, generator=g) * 0.05)
    return pool


def raw(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def oracle_copy(pool, layer=0):
    ks = None if pool.k_scale is None else pool.k_scale[layer].cpu().numpy().copy()
    vs = None if pool.v_scale is None else pool.v_scale[layer].cpu().numpy().copy()
    return oracle.Pool(pool.num_blocks, pool.num_kv_heads, pool.head_dim, pool.kv_dtype, raw(pool.k_data[layer]).copy(),
                       raw(pool.v_data[layer]).copy(), ks, vs)


def same_pool(pool, opool, layer=0):
    got = oracle_copy(pool, layer)
    assert np.array_equal(got.k_scale.view(np.uint32), opool.k_scale.view(np.uint32)), "K scales differ"
    assert np.array_equal(got.v_scale.view(np.uint32), opool.v_scale.view(np.uint32)), "V scales differ"
    assert np.array_equal(got.k, opool.k), "K differs"
    assert np.array_equal(got.v, opool.v), "V differs"


def check_rotation(got, x, cs, inter):
    """got against the rotation in 64 bits: half a step of the 16-bit type, on top of the fp32
    arithmetic: two products and a sum, each off by at most 2^-24 of its size."""
    want = rotate(x, cs, inter, torch.float64)
    rot = cs.shape[1]
    p1, p2 = pairs(rot, inter)
    size = torch.zeros_like(want)
    both = x[..., p1].double().abs() + x[..., p2].double().abs()
    size[..., p1], size[..., p2] = both, both           # |c|, |s| <= 1
    fp32 = 3 * 2.0 ** -24 * size
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps   # a subnormal step
    tol = torch.finfo(got.dtype).eps / 2 * (want.abs() + fp32) + fp32 + tiny
    assert ((got.cpu().double() - want).abs() <= tol).all()


def tokens_of(T, N, g, run):
    """Slots of T tokens in runs of neighbours through blocks of a permutation, and positions."""
    perm = torch.randperm(N, generator=g)
    slots, b = [], 0
    while len(slots) < T:
        off = int(torch.randint(0, 16, (1,), generator=g))
        for i in range(min(run, T - len(slots))):
            slots.append(int(perm[b + (off + i) // 16]) * 16 + (off + i) % 16)
        b += (off + run - 1) // 16 + 1
    pos = torch.randint(0, POS, (T,), generator=g, dtype=torch.int32)
    return torch.tensor(slots, dtype=torch.int32), pos


def run_case(dt, src, d, rot, inter, T, run, H_q, H_kv, fused, seed, shuffle=False):
    g = wl.generator(seed)
    N = 2 * T + 8 if run < 16 else 2 * (T // 16) + 2 * (T // run) + 8
    pool = stale_pool(N, H_kv, d, dt, g)
    opool = oracle_copy(pool)
    slots, pos = tokens_of(T, N, g, run)
    if shuffle:       # the tokens of a block far apart in the call
        order = torch.randperm(T, generator=g)
        slots = slots[order].contiguous()
    tdt = wl.TORCH_DTYPE[src]
    x = wl.normal((T, H_q + 2 * H_kv, d), tdt, g)
    q, k, v = x.split([H_q, H_kv, H_kv], 1)
    cs = table(rot)
    xd = x.to(DEV)
    qd, kd, vd = xd.split([H_q, H_kv, H_kv], 1) if fused else (q.contiguous().to(DEV), k.contiguous().to(DEV),
                                                               v.contiguous().to(DEV))
    out = pkv.kv_append_rope(pool, 0, qd, kd, vd, pos.to(DEV), cs.to(DEV), slots.to(DEV), interleaved=inter)
    torch.cuda.synchronize()
    assert pkv.read_device_status(pool) == 0
    rows = cs[pos.long()]
    check_rotation(out, q, rows, inter)
    k_rot = rotate(k, rows, inter, torch.float32).to(tdt)
    oracle.kv_append(opool, k_rot.contiguous(), v.contiguous(), src, slots.numpy())
    same_pool(pool, opool)
    return pool, opool


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("T,run", [(1, 1), (7, 1), (33, 5), (190, 47)])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 48), (64, 64), (64, 16)])
@pytest.mark.parametrize("dt", list(NAMES), ids=lambda x: NAMES[x])
def test_rope_append_matches_rotation_and_append(dt, d, rot, T, run, inter):
    src = pkv.F16 if dt == pkv.F16 else pkv.BF16
    run_case(dt, src, d, rot, inter, T, run, 8, 2, fused=T % 2 == 1, seed=3000 + dt * 97 + T + rot + d)


@pytest.mark.parametrize("dt", pkv.QUANTIZED, ids=lambda x: NAMES[x])
@pytest.mark.parametrize("T", [512, 513, 1500])
def test_rope_append_many_tokens_quantized(dt, T):
    """Both ways of finding a block's other tokens (scan, index), tokens of a block out of order."""
    run_case(dt, pkv.F16 if T == 513 else pkv.BF16, 128, 128, False, T, 37, 3, 1, True, 3300 + dt + T, shuffle=True)


@pytest.mark.parametrize("H_q,H_kv", [(64, 8), (64, 1), (5, 5), (3, 1), (0, 2)])
def test_rope_append_head_counts(H_q, H_kv):
    for dt in (pkv.BF16, pkv.INT8):
        if H_q:
            run_case(dt, pkv.BF16, 128, 128, False, 20, 6, H_q, H_kv, True, 3400 + H_q)
            continue
        g = wl.generator(3401)
        pool = stale_pool(50, H_kv, 128, dt, g)
        opool = oracle_copy(pool)
        slots, pos = tokens_of(20, 50, g, 6)
        k, v = wl.kv_source(20, H_kv, 128, g)
        assert pkv.kv_append_rope(pool, 0, None, k.to(DEV), v.to(DEV), pos.to(DEV), table(128).to(DEV),
                                  slots.to(DEV)) is None
        oracle.kv_append(opool, rotate(k, table(128)[pos.long()], False, torch.float32).to(torch.bfloat16), v,
                         pkv.BF16, slots.numpy())
        torch.cuda.synchronize()
        same_pool(pool, opool)


@pytest.mark.parametrize("dt", [pkv.BF16, pkv.FP8E4M3], ids=lambda x: NAMES[x])
@pytest.mark.parametrize("T", [40, 700])
def test_padding_and_out_of_range_tokens_are_left_alone(dt, T):
    g = wl.generator(3500 + T)
    N, H_q, H_kv, d = 2 * T, 4, 2, 64
    pool = stale_pool(N, H_kv, d, dt, g)
    opool = oracle_copy(pool)
    slots, pos = tokens_of(T, N, g, 16)
    skipped = torch.zeros(T, dtype=torch.bool)
    slots[3], slots[T - 1] = -1, -7
    slots[10] = N * 16
    pos[11], pos[12] = POS, -1
    skipped[[3, T - 1, 10, 11, 12]] = True
    q, k, v = (wl.normal((T, h, d), torch.bfloat16, g) for h in (H_q, H_kv, H_kv))
    cs = table(32)
    out = torch.full((T, H_q, d), 7.0, dtype=torch.bfloat16, device=DEV)
    pkv.kv_append_rope(pool, 0, q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), cs.to(DEV), slots.to(DEV), q_out=out)
    torch.cuda.synchronize()
    assert pkv.read_device_status(pool) == pkv.DEV_BAD_SLOT | pkv.DEV_BAD_POSITION
    assert (out.cpu()[skipped] == 7).all()
    keep = ~skipped
    rows = cs[pos[keep].long()]
    check_rotation(out.cpu()[keep], q[keep], rows, False)
    oracle.kv_append(opool, rotate(k[keep], rows, False, torch.float32).to(torch.bfloat16), v[keep].contiguous(),
                     pkv.BF16, slots[keep].numpy())
    same_pool(pool, opool)


def test_rope_in_place_other_stream_and_graph():
    """q rotated in place inside a fused projection's output, on a stream of its own, captured and
    replayed on new contents; an empty call does nothing."""
    g = wl.generator(3600)
    T, H_q, H_kv, d, N = 600, 4, 2, 128, 100
    pool = stale_pool(N, H_kv, d, pkv.INT8, g, layers=2)
    cs = table(128)
    slots, pos = tokens_of(T, N, g, 600)
    x = wl.normal((T, H_q + 2 * H_kv, d), torch.bfloat16, g)
    xd, sd, pd, cd = x.to(DEV), slots.to(DEV), pos.to(DEV), cs.to(DEV)
    ws = torch.empty(pkv.kv_append_rope_workspace_bytes(pool, T), dtype=torch.uint8, device=DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q, k, v = xd.split([H_q, H_kv, H_kv], 1)
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            pkv.kv_append_rope(pool, 1, q, k, v, pd, cd, sd, q_out=q, workspace=ws)
    for seed in (1, 2):
        x = wl.normal(x.shape, torch.bfloat16, wl.generator(seed))
        xd.copy_(x)
        opool, other = oracle_copy(pool, 1), oracle_copy(pool, 0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        rows = cs[pos.long()]
        check_rotation(xd[:, :H_q].cpu(), x[:, :H_q], rows, False)
        assert torch.equal(xd[:, H_q:].cpu(), x[:, H_q:])
        oracle.kv_append(opool, rotate(x[:, H_q:H_q + H_kv], rows, False, torch.float32).to(torch.bfloat16),
                         x[:, H_q + H_kv:].contiguous(), pkv.BF16, slots.numpy())
        same_pool(pool, opool, 1)
        same_pool(pool, other, 0)
    before = oracle_copy(pool, 1)
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    pkv.kv_append_rope(pool, 1, q[:0], k[:0], v[:0], e, cd, e, stream=stream)
    # a stream given by the caller, with the workspace taken from the current stream's allocator
    pkv.kv_append_rope(pool, 0, q.contiguous(), k, v, pd, cd, sd, stream=stream)
    torch.cuda.synchronize()
    same_pool(pool, before, 1)
    assert pkv.read_device_status(pool) == 0


@pytest.mark.parametrize("dt", pkv.QUANTIZED, ids=lambda x: NAMES[x])
@pytest.mark.parametrize("gain", [1e-38, 1e-3, 1.0, 1e30])
def test_rope_append_codes_at_rounding_borders(dt, gain):
    """Values that are codes, or halfway between codes, of the tile's scale, from the smallest
    magnitudes (whose reciprocal scale overflows) to large ones: the codes stay those of the division."""
    g = wl.generator(3700)
    T, H_kv, d, N = 48, 2, 128, 8
    limit = {pkv.INT8: 127, pkv.INT4: 7, pkv.FP8E4M3: 448}[dt]
    steps = torch.randint(-2 * limit, 2 * limit + 1, (T, H_kv, d), generator=g).float() / 2
    steps[:, :, 0] = limit
    k, v = (steps * gain).to(torch.bfloat16), (steps.flip(0) * gain).to(torch.bfloat16)
    pool = stale_pool(N, H_kv, d, dt, g)
    pool.k_scale.fill_(1e-39 * min(gain, 1.0))
    pool.v_scale.fill_(1e-39 * min(gain, 1.0))
    opool = oracle_copy(pool)
    slots = torch.randperm(N * 16, generator=g)[:T].to(torch.int32)
    cs = torch.zeros(1, 128)
    cs[:, :64] = 1                                # a rotation by 0
    pkv.kv_append_rope(pool, 0, None, k.to(DEV), v.to(DEV), torch.zeros(T, dtype=torch.int32, device=DEV), cs.to(DEV),
                       slots.to(DEV))
    torch.cuda.synchronize()
    oracle.kv_append(opool, k, v, pkv.BF16, slots.numpy())
    same_pool(pool, opool)


@pytest.mark.parametrize("dt", [pkv.BF16, pkv.INT8], ids=lambda x: NAMES[x])
def test_rope_append_many_single_tokens(dt):
    """A wide decode step: every token in a block of its own (each block's first token leads alone)."""
    run_case(dt, pkv.BF16, 64, 64, True, 1030, 1, 8, 2, True, 3800 + dt)
