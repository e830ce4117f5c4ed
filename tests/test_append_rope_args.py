"""CPU checks of kv_append_rope's refusals (no CUDA call is reached)."""
import ctypes

import pytest

from paged_kv_cache_431_b200 import pkv


@pytest.fixture()
def pools():
    made = []

    def make(dt, d=128):
        h = ctypes.c_void_p()
        scales = dict(k_scale=0x30000, v_scale=0x40000) if dt in pkv.QUANTIZED else dict(k_scale=None, v_scale=None)
        desc = pkv._PoolDesc(1, 64, 16, 2, d, dt, 0x10000, 0x20000, scales["k_scale"], scales["v_scale"], None)
        assert pkv.lib().kv_pool_create(ctypes.byref(desc), ctypes.byref(h)) == 0
        made.append(h)
        return h
    yield make
    for h in made:
        pkv.lib().kv_pool_destroy(h)


GOOD = dict(layer=0, q=0x1000, qs=512, k=0x2000, ks=256, v=0x3000, vs=256, src=pkv.BF16, table=0x4000, rows=100, rot=128,
            inter=0, pos=0x5000, slots=0x6000, T=4, H_q=4, out=0x7000, outs=512, ws=None, wsb=0)


def call(pool, **kw):
    a = dict(GOOD, **kw)
    rope = None if a["table"] == "none" else ctypes.byref(pkv._Rope(a["table"], a["rows"], a["rot"], a["inter"]))
    return pkv.lib().kv_append_rope(pool, a["layer"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["src"], rope,
                                    a["pos"], a["slots"], a["T"], a["H_q"], a["out"], a["outs"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("change,status", [
    (dict(table="none"), -1), (dict(table=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(q=None), -1),
    (dict(out=None), -1), (dict(pos=None), -1), (dict(slots=None), -1),
    (dict(layer=1), -2), (dict(layer=-1), -2), (dict(T=-1), -2), (dict(H_q=-1), -2), (dict(rows=0), -2),
    (dict(inter=2), -2), (dict(q=0x1008), -2), (dict(k=0x2002), -2), (dict(v=0x3008), -2), (dict(out=0x7004), -2),
    (dict(table=0x4008), -2), (dict(qs=516), -2), (dict(ks=260), -2), (dict(outs=513), -2), (dict(T=1 << 30), -2),
    (dict(src=pkv.F16), -3), (dict(src=pkv.INT8), -3),
    (dict(rot=0), -4), (dict(rot=8), -4), (dict(rot=100), -4), (dict(rot=144), -4), (dict(ks=128), -4), (dict(vs=0), -4),
    (dict(qs=256), -4), (dict(outs=0), -4),
])
def test_refusals(pools, change, status):
    assert call(pools(pkv.BF16), **change) == status


def test_no_tokens_is_no_work(pools):
    assert call(pools(pkv.BF16), T=0, k=None, v=None, q=None, out=None) == 0


def test_workspace_of_quantized_pools(pools):
    L = pkv.lib()
    assert L.kv_append_rope_workspace_bytes(pools(pkv.BF16), 100000) == 0
    q = pools(pkv.INT8)
    assert L.kv_append_rope_workspace_bytes(q, 512) == 0
    need = L.kv_append_rope_workspace_bytes(q, 513)
    assert need == 64 * 16 * 4
    assert L.kv_append_rope_workspace_bytes(q, -1) == 0 and L.kv_append_rope_workspace_bytes(None, 600) == 0
    assert call(q, T=513) == -5
    assert call(q, T=513, ws=0x8000, wsb=need - 1) == -5
    assert call(q, T=513, ws=0x8002, wsb=need) == -2
    assert call(None) == -1
