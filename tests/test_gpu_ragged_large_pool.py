"""The ragged operators and the append with rotation on pools whose bytes and offsets pass 32 bits: the
same blocks at the start of a small pool and at the end of a large one give the same bits."""
import pytest
import torch

from paged_kv_cache_431_b200 import pkv
from paged_kv_cache_431_b200 import workloads as wl
from tests.ragged_helpers import DEV
from tests.test_gpu_append_rope import table
from tests.test_gpu_cross import starts_of

pytestmark = pytest.mark.gpu

H_KV, D, USED = 8, 128, 96          # blocks that the calls use


def pools(dt):
    """(small pool of USED blocks, large pool whose last USED blocks hold the same)."""
    g = torch.Generator(device=DEV).manual_seed(9500 + dt)
    N = 2 ** 32 // (H_KV * 16 * pkv.row_bytes(dt, D)) + 2 * USED
    small = pkv.KVPool.allocate(1, USED, H_KV, D, dt)
    shape = (1, N, H_KV, 16)
    dtype = wl.TORCH_DTYPE[dt] if dt not in pkv.QUANTIZED else torch.uint8
    width = D if dt not in pkv.QUANTIZED else pkv.row_bytes(dt, D)
    data = [torch.empty(*shape, width, dtype=dtype, device=DEV) for _ in range(2)]
    scales = [torch.empty(1, N, H_KV, device=DEV) for _ in range(2)] if dt in pkv.QUANTIZED else [None, None]
    large = pkv.KVPool(*data, dt, D, *scales, device_status=torch.zeros(1, dtype=torch.int32, device=DEV))
    for a, b in ((small.k_data, large.k_data), (small.v_data, large.v_data)):
        a.random_(0, 120, generator=g) if dt in pkv.QUANTIZED else a.normal_(generator=g)
        b[:, N - USED:] = a
    if dt in pkv.QUANTIZED:
        for a, b in ((small.k_scale, large.k_scale), (small.v_scale, large.v_scale)):
            a.uniform_(0.01, 0.02, generator=g)
            b[:, N - USED:] = a
    assert large.k_data.numel() * large.k_data.element_size() > 2 ** 32
    return small, large, N - USED


@pytest.mark.parametrize("dt", [pkv.BF16, pkv.INT8], ids=["bf16", "int8"])
def test_blocks_at_the_end_of_a_large_pool(dt):
    small, large, shift = pools(dt)
    g = wl.generator(9510 + dt)
    tables = torch.randperm(USED, generator=g).to(torch.int32).view(4, -1).to(DEV)
    lens = torch.tensor([384, 100, 17, 300], dtype=torch.int32, device=DEV)
    for rows in ([2, 1, 0, 3], [9, 5, 4, 1], [70, 3, 8, 20]):       # warp level, both tcgen05 forms
        q = wl.normal((sum(rows), 32, D), torch.bfloat16, g).to(DEV)
        a, b = (pkv.paged_cross_attn(p, 0, q, starts_of(rows).to(DEV), t, lens, 0.05, max(rows), 384)
                for p, t in ((small, tables), (large, tables + shift)))
        assert torch.equal(a, b)
    tables[1:, :6] = tables[0, :6]                                   # one prefix of 96 tokens
    q = wl.normal((4, 32, D), torch.bfloat16, g).to(DEV)
    lens[2] = 97
    one = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    pre = torch.tensor([96], dtype=torch.int32, device=DEV)
    a, b = (pkv.paged_decode_attn_groups(p, 0, q, t, lens, one, pre, 0.05, 4, 96, 288)
            for p, t in ((small, tables), (large, tables + shift)))
    assert torch.equal(a, b)
    for T in (40, 700):                                              # scanned, and looked up
        k, v, x = (wl.normal((T, h, D), torch.bfloat16, g).to(DEV) for h in (H_KV, H_KV, 32))
        slots = torch.randperm(USED * 16, generator=g)[:T].to(torch.int32).to(DEV)
        pos = torch.arange(T, dtype=torch.int32, device=DEV)
        cs = table(D).to(DEV)
        a, b = (pkv.kv_append_rope(p, 0, x, k, v, pos, cs, s) for p, s in ((small, slots), (large, slots + 16 * shift)))
        assert torch.equal(a, b)
        assert torch.equal(small.k_data.view(torch.uint8), large.k_data[:, shift:].contiguous().view(torch.uint8))
        assert torch.equal(small.v_data.view(torch.uint8), large.v_data[:, shift:].contiguous().view(torch.uint8))
        if dt in pkv.QUANTIZED:
            assert torch.equal(small.k_scale, large.k_scale[:, shift:])
            assert torch.equal(small.v_scale, large.v_scale[:, shift:])
    torch.cuda.synchronize()
    assert pkv.read_device_status(small) == 0 and pkv.read_device_status(large) == 0
