"""Calls given a stream that is not torch's current one, while work is queued on the current one: what
the call takes from torch's allocator must not be memory that the queued work still uses."""
import pytest
import torch

from paged_kv_cache_431_b200 import pkv
from paged_kv_cache_431_b200 import workloads as wl
from tests import test_gpu_cross as cross

pytestmark = pytest.mark.gpu
DEV = "cuda"
BUSY = 40_000_000        # SM cycles, some 20 ms


def beside_queued_work(call, sizes, raw):
    """Runs call(stream) while the current stream is busy and still has to read tensors of `sizes`
    bytes that Python has let go of; the copies it makes of them must come out whole."""
    side = torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    for _ in range(3):
        held = [torch.full((n,), 77, dtype=torch.uint8, device=DEV) for n in sizes]
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        copies = [t.clone() for t in held]
        del held
        got = call(side.cuda_stream if raw else side)
        side.synchronize()
        torch.cuda.synchronize()
        for c in copies:
            assert (c == 77).all()
        assert torch.equal(got, want)
        del copies


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("rows", [2, 130])
def test_cross(rows, raw):
    pool, _, q, _, tables = cross.case(pkv.BF16, 128, 8, 2, [rows] * 4, [3000] * 4, 9000 + rows)
    q, tables = q.to(DEV), tables.to(DEV)
    args = (cross.starts_of([rows] * 4).to(DEV), tables, torch.full((4,), 3000, dtype=torch.int32, device=DEV), 0.1,
            rows, 3000)
    need = pkv.paged_cross_workspace_bytes(pool, 4 * rows, 8, 4, rows, 3000)
    assert need > 0
    beside_queued_work(lambda s: pkv.paged_cross_attn(pool, 0, q, *args, stream=s), [q.numel() * 2, need], raw)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_groups(raw):
    from tests import test_gpu_groups as groups
    sizes, prefix, suffix = [4, 3], [512, 256], [300] * 7
    pool, _, q, _, tables, ctx = groups.case(pkv.BF16, 128, 8, 2, sizes, prefix, suffix, 9100)
    q, tables = q.to(DEV), tables.to(DEV)
    args = (tables, torch.tensor(ctx, dtype=torch.int32, device=DEV), cross.starts_of(sizes).to(DEV),
            torch.tensor(prefix, dtype=torch.int32, device=DEV), 0.1, 4, 512, 300)
    need = pkv.paged_decode_groups_workspace_bytes(pool, 7, 8, 2, 4, 512, 300)
    assert need > 0
    beside_queued_work(lambda s: pkv.paged_decode_attn_groups(pool, 0, q, *args, stream=s), [q.numel() * 2, need], raw)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_append_rope(raw):
    T, g = 600, wl.generator(9200)
    pool = pkv.KVPool.allocate(1, 64, 2, 128, pkv.INT8)
    q, k, v = (wl.normal((T, h, 128), torch.bfloat16, g).to(DEV) for h in (8, 2, 2))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    table = torch.randn(T, 128, device=DEV)
    beside_queued_work(lambda s: pkv.kv_append_rope(pool, 0, q, k, v, pos, table, pos, stream=s),
                       [q.numel() * 2, pkv.kv_append_rope_workspace_bytes(pool, T)], raw)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_decode_and_append(raw):
    """The calls that were there before: their workspaces, let go of while the call's stream still runs,
    and outputs."""
    T, g = 600, wl.generator(9300)
    pool = pkv.KVPool.allocate(1, 64, 2, 128, pkv.INT8)
    k, v = (wl.normal((T, 2, 128), torch.bfloat16, g).to(DEV) for _ in range(2))
    slots = torch.arange(T, dtype=torch.int32, device=DEV)

    pkv.kv_append(pool, 0, k, v, slots)
    q = wl.normal((8, 8, 128), torch.bfloat16, g).to(DEV)
    tables = torch.arange(32, dtype=torch.int32, device=DEV).repeat(8, 1)
    lens = torch.full((8,), 500, dtype=torch.int32, device=DEV)
    need = pkv.paged_decode_workspace_bytes(pool, 8, 8, 500, partition_tokens=64)
    beside_queued_work(lambda s: pkv.paged_decode_attn(pool, 0, q, tables, lens, 0.1, 500, partition_tokens=64, stream=s),
                       [q.numel() * 4, need], raw)
    want = [t.clone() for t in (pool.k_data, pool.v_data, pool.k_scale, pool.v_scale)]
    beside_queued_work(lambda s: (pkv.kv_append(pool, 0, k, v, slots, stream=s), k)[1],
                       [pkv.kv_append_workspace_bytes(pool, T)], raw)
    for t, w in zip((pool.k_data, pool.v_data, pool.k_scale, pool.v_scale), want):
        assert torch.equal(t, w)
