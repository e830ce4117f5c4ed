"""Calls from several host threads at once, each on a stream of its own, with partitions (and so dynamic
shared memory) of different sizes."""
import threading

import pytest
import torch

from paged_kv_cache_431_b200 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def in_threads(calls, n):
    """Every call n times in a thread of its own; the first exception is raised here."""
    errors = []

    def work(call):
        try:
            s = torch.cuda.Stream()
            for _ in range(n):
                call(s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("dt", pkv.QUANTIZED)
def test_partitions_of_different_sizes(dt):
    g = torch.Generator(device=DEV).manual_seed(9400 + dt)
    n, B = 8192, 2
    pool = pkv.KVPool.allocate(1, B * n // 16, 2, 128, dt)
    for t in (pool.k_data, pool.v_data):
        t.random_(0, 100, generator=g)
    for t in (pool.k_scale, pool.v_scale):
        t.fill_(0.01)
    tables = torch.arange(B * n // 16, dtype=torch.int32, device=DEV).view(B, -1)
    lens = torch.full((B,), 4096, dtype=torch.int32, device=DEV)
    q = torch.randn(B, 4, 128, device=DEV, generator=g).to(torch.bfloat16)
    starts = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    calls, results = [], []
    for part in (64, 4096, 512):
        out = torch.empty(B, 4, 128, device=DEV)
        ws = torch.empty(pkv.paged_decode_workspace_bytes(pool, B, 4, 4096, partition_tokens=part) + 16,
                         dtype=torch.uint8, device=DEV)
        calls.append(lambda s, out=out, ws=ws, part=part: pkv.paged_decode_attn(
            pool, 0, q, tables, lens, 0.05, 4096, out=out, workspace=ws, partition_tokens=part, stream=s))
        results.append(out)
    for bound in (100, 8192):                            # the partition follows the bound
        short = torch.full((B,), min(bound, 4096), dtype=torch.int32, device=DEV)
        out = torch.empty_like(q)
        ws = torch.empty(pkv.paged_cross_workspace_bytes(pool, B, 4, B, 1, bound) + 16, dtype=torch.uint8, device=DEV)
        calls.append(lambda s, out=out, ws=ws, short=short, bound=bound: pkv.paged_cross_attn(
            pool, 0, q, starts, tables, short, 0.05, 1, bound, out=out, workspace=ws, stream=s))
        results.append(out)
    for c in calls:
        c(None)
    torch.cuda.synchronize()
    want = [t.clone() for t in results]
    in_threads(calls, 4000)
    for t, w in zip(results, want):
        assert torch.equal(t, w)
