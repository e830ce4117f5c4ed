"""CPU checks of the refusals and workspace sizes of paged_cross_attn and paged_decode_attn_groups (no
CUDA call is reached)."""
import ctypes

import pytest

from paged_kv_cache_431_b200 import pkv
from tests.test_append_rope_args import pools  # noqa: F401

CROSS = dict(layer=0, q=0x10000, qd=pkv.BF16, starts=0x20000, rows=10, H_q=8, tb=0x30000, W=400, cl=0x40000, B=3, mr=5,
             mc=6000, out=0x50000, ws=None, wsb=0)
GROUPS = dict(layer=0, q=0x10000, qd=pkv.BF16, tb=0x30000, W=40, cl=0x40000, B=6, H_q=8, starts=0x20000, pl=0x60000, n=2,
              ms=4, mp=320, mx=100, out=0x50000, ws=None, wsb=0)


def cross(pool, **kw):
    a = dict(CROSS, **kw)
    return pkv.lib().paged_cross_attn(pool, a["layer"], a["q"], a["qd"], a["starts"], a["rows"], a["H_q"], a["tb"], a["W"],
                                      a["cl"], a["B"], a["mr"], a["mc"], 0.1, a["out"], a["ws"], a["wsb"], None)


def groups(pool, **kw):
    a = dict(GROUPS, **kw)
    return pkv.lib().paged_decode_attn_groups(pool, a["layer"], a["q"], a["qd"], a["tb"], a["W"], a["cl"], a["B"],
                                              a["H_q"], a["starts"], a["pl"], a["n"], a["ms"], a["mp"], a["mx"], 0.1,
                                              a["out"], a["ws"], a["wsb"], None)


BOTH = [(dict(q=None), -1), (dict(out=None), -1), (dict(starts=None), -1), (dict(tb=None), -1), (dict(cl=None), -1),
        (dict(layer=1), -2), (dict(layer=-1), -2), (dict(H_q=0), -2), (dict(B=-1), -2), (dict(W=0), -2),
        (dict(q=0x10008), -2), (dict(out=0x50004), -2), (dict(qd=pkv.F16), -3), (dict(qd=pkv.INT8), -3), (dict(H_q=7), -4),
        (dict(W=1 << 27), -9)]


@pytest.mark.parametrize("change,status", BOTH + [
    (dict(rows=-1), -2), (dict(mr=-1), -2), (dict(mc=-1), -2), (dict(B=65536), -9), (dict(rows=1 << 28, H_q=8), -9),
    (dict(mr=1 << 30), -9), (dict(out=0x10000), -2), (dict(mc=(1 << 30) + 1), -9), (dict(mc=(1 << 31) - 1), -9)])
def test_cross_refusals(pools, change, status):  # noqa: F811
    assert cross(pools(pkv.BF16), **change) == status


@pytest.mark.parametrize("change,status", BOTH + [
    (dict(pl=None), -1), (dict(n=-1), -2), (dict(ms=-1), -2), (dict(mp=-1), -2), (dict(mx=-1), -2),
    (dict(mp=1 << 30, mx=1 << 30), -2), (dict(n=65536), -9), (dict(B=65535), -9), (dict(out=0x10000), -2),
    (dict(mp=1 << 30, mx=1), -9), (dict(mx=(1 << 30) + 1), -9)])
def test_groups_refusals(pools, change, status):  # noqa: F811
    assert groups(pools(pkv.BF16), **change) == status


def test_no_pool_and_nothing_to_do(pools):  # noqa: F811
    assert cross(None) == -1 and groups(None) == -1
    p = pools(pkv.INT8)
    empty = dict(q=None, out=None, starts=None, tb=None, cl=None)
    for change in (dict(B=0), dict(rows=0), dict(mr=0)):
        assert cross(p, **empty, **change) == 0
    for change in (dict(B=0), dict(n=0), dict(ms=0)):
        assert groups(p, **empty, **change) == 0


def test_workspaces(pools):  # noqa: F811
    L = pkv.lib()
    for dt in (pkv.BF16, pkv.INT8):
        p = pools(dt)
        need = L.paged_cross_workspace_bytes(p, 10, 8, 3, 5, 6000)
        assert need > 0 and need % (10 * 8 * (128 + 2) * 4) == 0
        assert L.paged_cross_workspace_bytes(p, 10, 8, 3, 5, 60) == 0       # one partition
        q = dict(qd=pkv.BF16)
        assert cross(p, **q) == -5 and cross(p, ws=0x70000, wsb=need - 1) == -5
        assert cross(p, ws=0x70008, wsb=need) == -5
        need = L.paged_decode_groups_workspace_bytes(p, 6, 8, 2, 4, 320, 100)
        assert need > 0 and need % (6 * 8 * (128 + 2) * 4) == 0
        assert L.paged_decode_groups_workspace_bytes(p, 6, 8, 2, 4, 0, 100) == 0
        assert groups(p) == -5 and groups(p, ws=0x70000, wsb=need - 1) == -5
        for bad in ((-1, 8, 3, 5, 600), (10, 7, 3, 5, 600), (10, 0, 3, 5, 600), (10, 8, -1, 5, 600), (10, 8, 3, -1, 600),
                    (10, 8, 3, 5, -1)):
            assert L.paged_cross_workspace_bytes(p, *bad) == 0
        for bad in ((-1, 8, 2, 4, 320, 100), (6, 7, 2, 4, 320, 100), (6, 8, -1, 4, 320, 100), (6, 8, 2, -1, 320, 100),
                    (6, 8, 2, 4, -1, 100), (6, 8, 2, 4, 320, -1)):
            assert L.paged_decode_groups_workspace_bytes(p, *bad) == 0
    assert L.paged_cross_workspace_bytes(None, 10, 8, 3, 5, 600) == 0
    assert L.paged_decode_groups_workspace_bytes(None, 6, 8, 2, 4, 320, 100) == 0


def test_descriptor_of_the_rotation_matches_the_header():
    assert ctypes.sizeof(pkv._Rope) == 24


@pytest.mark.parametrize("groups_,size,prefix,suffix,same", [(4, 16, 8000, 8000, True), (8, 8, 8000, 8000, True),
                                                             (8, 100, 4000, 500, False)])
def test_prefix_pass_has_all_sms_unless_the_suffixes_run_beside_it(pools, groups_, size, prefix, suffix, same):  # noqa: F811
    """Suffixes on tcgen05 (few long ones) come after the prefix pass, which is then split as a cross
    attention of the same rows would be; lighter ones at the warp level run beside it, and where they weigh
    more the prefix pass is split for fewer SMs.  The partitions are read off the workspaces."""
    L, p, H_q, n = pkv.lib(), pools(pkv.BF16), 16, groups_ * size
    row = n * H_q * (128 + 2) * 4
    pre = max(1, L.paged_cross_workspace_bytes(p, n, H_q, groups_, size, prefix) // row)
    own = max(1, L.paged_cross_workspace_bytes(p, n, H_q, n, 1, suffix) // row)
    both = L.paged_decode_groups_workspace_bytes(p, n, H_q, groups_, size, prefix, suffix) // row
    assert (both == pre + own) == same
