"""Inputs and references for the ragged operators (cross attention, grouped-prefix decode): pools with
poison in every slot no context covers, and each query row attended by the oracle in 64 bits as a
sequence of its own."""
import math

import numpy as np
import torch

import oracle
from paged_kv_cache_431_b200 import pkv
from paged_kv_cache_431_b200 import workloads as wl
from tests.helpers import oracle_decode_threaded

DEV = "cuda"
NAMES = {pkv.F16: "f16", pkv.BF16: "bf16", pkv.INT8: "int8", pkv.INT4: "int4", pkv.FP8E4M3: "fp8"}


def q_dtype(dt, bf16=True):
    return dt if dt in (pkv.F16, pkv.BF16) else (pkv.BF16 if bf16 else pkv.F16)


def covered_slots(tables, ctx, N):
    """bool [N, 16]: slots that some sequence's context covers."""
    m = torch.zeros(N, 16, dtype=torch.bool)
    for b, n in enumerate(ctx):
        for j in range(-(-n // 16)):
            m[int(tables[b, j]), :min(16, n - 16 * j)] = True
    return m


def make_pool(tables, ctx, N, H_kv, d, dt, g, spread=1.0):
    """(KVPool, oracle pool): random K/V; slots outside every context hold NaN (16-bit, fp8) or the
    largest code, and scales of unused blocks are NaN."""
    cover = covered_slots(tables, ctx, N)
    if dt in (pkv.F16, pkv.BF16):
        k, v = (wl.normal((N, H_kv, 16, d), wl.TORCH_DTYPE[dt], g) for _ in range(2))
        for x in (k, v):
            x.transpose(1, 2)[~cover] = float("nan")
        pool = pkv.KVPool(k.to(DEV)[None], v.to(DEV)[None], dt, d, device_status=torch.zeros(1, dtype=torch.int32, device=DEV))
        raw = lambda t: t.view(torch.int16).numpy().view(np.uint8)  # noqa: E731
        return pool, oracle.Pool(N, H_kv, d, dt, raw(k), raw(v))
    sides = []
    for _ in range(2):
        x = torch.randn(N, H_kv, 16, d, generator=g)
        if dt == pkv.FP8E4M3:
            c = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            unit, stale = 1 / 100, 0x7F
        elif dt == pkv.INT8:
            c = (x * 40).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
            unit, stale = 1 / 40, 0x80
        else:
            n = (x * 2.5).round().clamp(-7, 7).to(torch.int32) & 15
            c = (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)
            unit, stale = 1 / 2.5, 0x88
        c.transpose(1, 2)[~cover] = stale
        s = (torch.rand(N, H_kv, generator=g) + 0.5) * unit * spread
        s[~cover.any(1)] = float("nan")
        sides.append((c.contiguous(), s))
    (k, ks), (v, vs) = sides
    pool = pkv.KVPool(k.to(DEV)[None], v.to(DEV)[None], dt, d, ks.to(DEV)[None], vs.to(DEV)[None],
                      device_status=torch.zeros(1, dtype=torch.int32, device=DEV))
    return pool, oracle.Pool(N, H_kv, d, dt, k.numpy(), v.numpy(), ks.numpy(), vs.numpy())


def tables_for(ctx, g, prefix_of=None):
    """Block tables over a permutation: prefix_of[b] = (group, shared tokens), or None."""
    need, shared, used = [], {}, 0
    for b, n in enumerate(ctx):
        grp, pre = prefix_of[b] if prefix_of else (None, 0)
        if pre and grp not in shared:
            shared[grp] = (used, pre // 16)
            used += pre // 16
        own = -(-n // 16) - pre // 16
        need.append((shared.get(grp, (0, 0)) if pre else (0, 0), used, max(0, own)))
        used += max(0, own)
    N = used + 3
    perm = torch.randperm(N, generator=g).to(torch.int32)
    W = max(1, max((-(-n // 16) for n in ctx), default=1)) + 1
    t = torch.full((len(ctx), W), -1, dtype=torch.int32)
    for b, ((s0, sn), o0, on) in enumerate(need):
        t[b, :sn] = perm[s0:s0 + sn]
        t[b, sn:sn + on] = perm[o0:o0 + on]
    return t, N


def reference(opool, q, qd, tables, ctx, row_of, scale):
    """[rows, H_q, d] in 64 bits; row_of[i]: the sequence of row i."""
    idx = torch.as_tensor(row_of, dtype=torch.long)
    return oracle_decode_threaded(opool, q, qd, tables[idx], torch.as_tensor(ctx, dtype=torch.int32)[idx],
                                  np.float32(scale))


def tolerance(opool, q, ref, ctx, scale, p_rounded):
    """What fp32 accumulation and the roundings to 16 bits may add up to, element by element.

    A score is a sum of d exact products added up in fp32, so it is off by at most
    (d + 2) 2^-24 sum|q k| scale <= (d + 2) 2^-24 |q| |k| scale (2-norms); a weight is off by that,
    relatively, twice (numerator and sum), plus its own rounding: half a step of the 16-bit type where
    P enters the second product in one part, 2^-15 where it enters in two; the sum over n keys in
    fp32 adds n 2^-24, a quantized q entering as 14 or more bits 2^-13 |q| |k| scale.  All of it
    scales |v| <= vmax.  The output is rounded once: half a step."""
    eps = torch.finfo(q.dtype).eps
    k, v = opool.dequant("k"), opool.dequant("v")
    finite = lambda x: x[np.isfinite(x)]  # noqa: E731
    vmax = float(np.abs(finite(v)).max(initial=0.0))
    kn = float(np.sqrt(np.nan_to_num((k.astype(np.float64) ** 2).sum(-1), nan=0.0, posinf=0.0).max(initial=0.0)))
    qn = float(q.double().square().sum(-1).sqrt().max())
    d = q.shape[-1]
    quant = opool.dtype in pkv.QUANTIZED
    ds = qn * kn * abs(scale) * ((d + 2) * 2.0 ** -24 + (2.0 ** -14 / math.sqrt(d) if quant else 0.0))
    weight = eps / 2 if p_rounded else 2.0 ** -15
    c = vmax * (2 * ds + weight + max(ctx, default=0) * 2.0 ** -24)
    return eps / 2 * (np.abs(ref) + c) + c + float(torch.finfo(q.dtype).smallest_normal)


def check(out, ref, tol, p_rounded=True):
    got = out.detach().cpu().double().numpy()
    assert np.isfinite(got).all(), "non-finite output"
    over = np.abs(got - ref) - tol
    assert over.max(initial=-1.0) <= 0, f"off by {np.abs(got - ref).max()} (allowed {tol[np.unravel_index(over.argmax(), over.shape)]})"
    # and on the whole: the output's half step, and a half step of P spread over many keys
    norm = np.linalg.norm(ref)
    if norm > 0:
        assert np.linalg.norm(got - ref) <= torch.finfo(out.dtype).eps * norm
