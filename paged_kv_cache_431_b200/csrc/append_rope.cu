// append_rope.cu -- kv_append_rope: rotate q and k by their positions, and write k and v into
// their pool slots, in one pass over the data.
//
// "KV cache, continuous batching and paged attention", section "The KV cache": each step caches
// the new tokens' keys and values.  Rotary position encoding turns pairs of a head's dims by an
// angle that grows with the token's position p:
//   y1 = x1 cos(p w_i) - x2 sin(p w_i),   y2 = x2 cos(p w_i) + x1 sin(p w_i)
// Keys are cached rotated (their positions never change), so the rotation belongs to the append.
// Arithmetic: IEEE fp32, each product and sum rounded on its own (no contraction, so a host or
// torch computation in the same order gives the same bits), then ONE rounding to the source
// type; a quantized pool stores that rounded row as kv_append would.
//
// Bound: HBM at prefill sizes (q read and written, k and v read, their slots written, nothing
// else: the table row of a token is shared by all its heads and stays in L1), launch latency at
// decode sizes.
//
// Copy form (q of every pool, k and v of 16-bit pools): a head's row is D/16 units of two
// 16-byte chunks -- the two halves of 8 pairs (split style), or 8 neighbouring pairs -- so a
// thread holds both elements of each pair, and neighbouring threads move neighbouring chunks.
// A thread keeps its unit over all its heads, so it loads 8 cosines and sines once per token.
//
// Quantized pools: the scale of a (block, head) tile is the maximum over all the call's tokens
// in that block, so the tokens have to be brought together.  kv_append does it with two passes
// over the data and atomics on a per-block scratch; here the first written token of each block
// finds the others (at most 16) and one warp per (block, head, K or V) loads, rotates, reduces,
// quantizes and stores them all, each source row read once.  The others are found
//   - for few tokens by scanning the slots,
//   - else through a scratch of one int per slot, entry = token, filled by a first kernel.  It
//     needs no clearing: an entry t counts only if token t's slot is this slot, so what an
//     earlier call left there either is true or is not believed.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "quant_codes.cuh"

namespace pkv {

namespace {

constexpr int kRopeThreads = 256;
// Up to this many tokens every CTA scans the slots (two loads per thread); above it the scan
// would cost more than the extra launch.
constexpr int kScanTokens = 512;
// Tokens per CTA where the tokens of a block are looked up: 8 against 4 and 16 took 16,384 prefill
// tokens from 150 to 138 (133) us and 2,048 single tokens from 34 to 36 (50).
constexpr int kLook = 8;

struct RopeParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;   // elements per token
    const float* table;       // [max_pos][rot]: rot/2 cosines, then their sines
    const int32_t* positions;
    const int32_t* slots;
    int32_t* index;           // [N * 16] scratch, token of each slot, or null (scan)
    uint8_t* k_pool;
    uint8_t* v_pool;
    float* k_scale;
    float* v_scale;
    int32_t* status;
    int T, N, H_q, H_kv, rot, inter, max_pos;
    int rows;                 // rows of the copy form per token (q, and k and v of 16-bit pools)
    int copy_ctas;            // CTAs of the copy form; the rest quantize
    int copy_y;               // CTAs per token of the copy form
};

// Whether token t takes part: a slot and a position in range.  `report` flags what is out of
// range (a negative slot is padding and is skipped silently).
__device__ __forceinline__ bool live(const RopeParams& p, int slot, int pos, bool report)
{
    if (slot < 0) return false;
    const bool bad_slot = slot >= p.N * kBlock, bad_pos = (unsigned)pos >= (unsigned)p.max_pos;
    if (report && (bad_slot || bad_pos))
        flag_status(p.status, (bad_slot ? PKV_DEV_BAD_SLOT : 0) | (bad_pos ? PKV_DEV_BAD_POSITION : 0));
    return !bad_slot && !bad_pos;
}

// a * c - b * s and b * c + a * s, every operation rounded on its own
__device__ __forceinline__ void turn(float& a, float& b, float c, float s)
{
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// One unit: two chunks of 8 elements; split style pairs x0[e] with x1[e], neighbour style pairs
// elements 2e, 2e + 1 of the 16 in order.
template <bool BF16>
__device__ __forceinline__ void turn_unit(uint4& u0, uint4& u1, const float (&c)[8], const float (&s)[8], bool inter)
{
    uint32_t* w0 = reinterpret_cast<uint32_t*>(&u0);
    uint32_t* w1 = reinterpret_cast<uint32_t*>(&u1);
    if (inter) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float2 a = unpack2<BF16>(w0[e]), b = unpack2<BF16>(w1[e]);
            turn(a.x, a.y, c[e], s[e]);
            turn(b.x, b.y, c[4 + e], s[4 + e]);
            w0[e] = pack2<BF16>(a.x, a.y);
            w1[e] = pack2<BF16>(b.x, b.y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float2 a = unpack2<BF16>(w0[e]), b = unpack2<BF16>(w1[e]);
            turn(a.x, b.x, c[2 * e], s[2 * e]);
            turn(a.y, b.y, c[2 * e + 1], s[2 * e + 1]);
            w0[e] = pack2<BF16>(a.x, a.y);
            w1[e] = pack2<BF16>(b.x, b.y);
        }
    }
}

// ---------------------------------------------------------------- copy form --
template <int D, bool BF16>
__device__ __forceinline__ void copy_rows(const RopeParams& p, int cta)
{
    constexpr int UNITS = D / 16;                       // units per row
    constexpr int STEP = kRopeThreads / UNITS;          // rows in flight per CTA
    constexpr int BATCH = 3;                            // rows of a thread in flight together
    const int t = cta / p.copy_y, y = cta % p.copy_y;
    const int u = threadIdx.x % UNITS;
    const int half = p.rot / 2;
    const bool rotated = 16 * u < p.rot;
    // the unit's two chunks, and the first of its 8 angles
    const int d0 = rotated && !p.inter ? 8 * u : 16 * u;
    const int d1 = rotated && !p.inter ? half + 8 * u : 16 * u + 8;
    const int slot = p.slots[t], pos = p.positions[t];
    const int step = p.copy_y * STEP;
    uint4 x[BATCH][2];
    auto source = [&](int row) -> const uint16_t* {
        if (row < p.H_q) return p.q + t * p.q_stride + row * D;
        const int h = row - p.H_q;
        return h < p.H_kv ? p.k + t * p.k_stride + h * D : p.v + t * p.v_stride + (h - p.H_kv) * D;
    };
    auto load = [&](int row0) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int row = row0 + i * step;
            if (row < p.rows) {
                const uint16_t* src = source(row);
                x[i][0] = *reinterpret_cast<const uint4*>(src + d0);
                x[i][1] = *reinterpret_cast<const uint4*>(src + d1);
            }
        }
    };
    const int first = y * STEP + threadIdx.x / UNITS;
    load(first);                                        // in flight with the slot and the position
    if (!live(p, slot, pos, threadIdx.x == 0 && y == 0)) return;
    float c[8], s[8];
    if (rotated) {
        const float4* cs = reinterpret_cast<const float4*>(p.table + (size_t)pos * p.rot + 8 * u);
        const float4* sn = reinterpret_cast<const float4*>(p.table + (size_t)pos * p.rot + half + 8 * u);
        *reinterpret_cast<float4*>(&c[0]) = __ldg(cs);
        *reinterpret_cast<float4*>(&c[4]) = __ldg(cs + 1);
        *reinterpret_cast<float4*>(&s[0]) = __ldg(sn);
        *reinterpret_cast<float4*>(&s[4]) = __ldg(sn + 1);
    }
    const size_t blk = slot / kBlock, off = slot % kBlock;
    for (int row0 = first; row0 < p.rows; row0 += BATCH * step) {
        if (row0 != first) load(row0);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int row = row0 + i * step;
            if (row >= p.rows) break;
            const bool is_q = row < p.H_q, is_v = row >= p.H_q + p.H_kv;
            uint16_t* dst;
            if (is_q) {
                dst = p.q_out + t * p.q_out_stride + row * D;
            } else {
                const int h = row - p.H_q - (is_v ? p.H_kv : 0);
                dst = reinterpret_cast<uint16_t*>(is_v ? p.v_pool : p.k_pool) + ((blk * p.H_kv + h) * kBlock + off) * D;
            }
            if (rotated && !is_v) turn_unit<BF16>(x[i][0], x[i][1], c, s, p.inter);
            *reinterpret_cast<uint4*>(dst + d0) = x[i][0];
            *reinterpret_cast<uint4*>(dst + d1) = x[i][1];
        }
    }
}

// ---------------------------------------------------------------- quantized --
// A CTA looks at `kLook` tokens (one where the slots are scanned); of these it works on the ones that
// are the first written token of their block, on K or on V.  Each warp takes (block, head) tiles in turn:
// D/8 lanes hold one row (8 elements each, two runs of 4), so 32 / (D/8) rows per pass and at most
// D/16 passes over the block's 16 rows; passes without a token are skipped.  The loops are kept small
// (unrolled over all passes the kernel waited for its instructions: 51 against 43 us).
template <int D, bool BF16, int DT>
__device__ __forceinline__ void quantize_block(const RopeParams& p, int cta, bool is_v)
{
    constexpr int LPR = D / 8, RPP = 32 / LPR, PASSES = kBlock / RPP;
    constexpr int RB = DT == PKV_INT4 ? D / 2 : D;
    constexpr int BATCH = 4;                              // passes whose loads are in flight together
    __shared__ int tok_of[kLook][kBlock], pos_of[kLook][kBlock], blk_of[kLook];
    __shared__ uint4 rows[kRopeThreads / 32][kBlock][LPR];   // a tile's source rows, by warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int look = p.index ? kLook : 1;
    if (p.index) {
        const int i = threadIdx.x / kBlock, o16 = threadIdx.x % kBlock;
        if (i < kLook) {
            const int t = cta * kLook + i;
            const int slot = t < p.T ? p.slots[t] : -1;
            const bool in = t < p.T && live(p, slot, p.positions[t], o16 == 0);
            int tok = -1, pos = 0;
            if (in) {
                const int s = slot / kBlock * kBlock + o16;
                const int o = p.index[s];
                if ((unsigned)o < (unsigned)p.T && p.slots[o] == s) {
                    pos = p.positions[o];
                    if (live(p, s, pos, false)) tok = o;
                }
            }
            // the block's first written token: the lowest offset that has one
            const unsigned have = (__ballot_sync(0xffffffffu, tok >= 0) >> (threadIdx.x & 16)) & 0xffffu;
            const int lead = __shfl_sync(0xffffffffu, tok, (threadIdx.x & 16) + (have ? __ffs(have) - 1 : 0));
            tok_of[i][o16] = tok;
            pos_of[i][o16] = pos;
            if (o16 == 0) blk_of[i] = in && lead == t ? slot / kBlock : -1;
        }
        __syncthreads();
    } else {
        const int t = cta;
        const int slot = p.slots[t];
        if (!live(p, slot, p.positions[t], threadIdx.x == 0)) return;
        if (threadIdx.x < kBlock) tok_of[0][threadIdx.x] = -1;
        __syncthreads();
        for (int o = threadIdx.x; o < p.T; o += kRopeThreads) {
            const int s = p.slots[o];
            if (s >= 0 && s / kBlock == slot / kBlock && live(p, s, p.positions[o], false)) atomicMax(&tok_of[0][s % kBlock], o);
        }
        __syncthreads();
        if (warp == 0) {
            const int tok = lane < kBlock ? tok_of[0][lane] : -1;
            const unsigned have = __ballot_sync(0xffffffffu, tok >= 0);
            const int lead = __shfl_sync(0xffffffffu, tok, have ? __ffs(have) - 1 : 0);
            if (lane < kBlock) pos_of[0][lane] = tok >= 0 ? p.positions[tok] : 0;
            if (lane == 0) blk_of[0] = lead == t ? slot / kBlock : -1;
        }
        __syncthreads();
    }

    const int half = p.rot / 2;
    const int sub = lane / LPR, ln = lane % LPR;
    // the lane's dims: two runs of 4; rotated runs hold 4 pairs (split: run against run;
    // neighbours: two pairs in each run), beyond the rotated dims two runs of 4 in order
    const bool rotated = 8 * ln < p.rot;
    const int d0 = rotated && !p.inter ? 4 * ln : 8 * ln;
    const int d1 = rotated && !p.inter ? half + 4 * ln : 8 * ln + 4;
    for (int all = warp; all < look * p.H_kv; all += kRopeThreads / 32) {
        const int which = all / p.H_kv, h = all % p.H_kv;
        const int blk = blk_of[which];
        if (blk < 0) continue;                               // another token leads that block
        const unsigned have = __ballot_sync(0xffffffffu, lane < kBlock && tok_of[which][lane % kBlock] >= 0);
        const size_t th = (size_t)blk * p.H_kv + h;
        uint8_t* tile = (is_v ? p.v_pool : p.k_pool) + th * kBlock * RB;
        float* scale = (is_v ? p.v_scale : p.k_scale) + th;
        const float stored = *scale;                         // in flight with the rows
        auto some = [&](int pass) { return (have >> (RPP * pass)) & ((1u << RPP) - 1u); };   // the pass has tokens
        const uint16_t* src = is_v ? p.v + h * D : p.k + h * D;
        const int64_t stride = is_v ? p.v_stride : p.k_stride;
        // first: the rows, rotated and rounded, into shared memory, and their largest element
        float amax = 0.f;
#pragma unroll 1
        for (int i0 = 0; i0 < PASSES; i0 += BATCH) {
            if (((have >> (RPP * i0)) & ((1u << (RPP * BATCH)) - 1u)) == 0u) continue;
            uint2 x[BATCH][2];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                x[i][0] = x[i][1] = make_uint2(0u, 0u);
                const int o = tok_of[which][RPP * (i0 + i) + sub];
                if (o >= 0) {
                    x[i][0] = *reinterpret_cast<const uint2*>(src + o * stride + d0);
                    x[i][1] = *reinterpret_cast<const uint2*>(src + o * stride + d1);
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (!some(i0 + i)) continue;
                const int off = RPP * (i0 + i) + sub;
                float2 a = unpack2<BF16>(x[i][0].x), b = unpack2<BF16>(x[i][0].y);
                float2 e = unpack2<BF16>(x[i][1].x), f = unpack2<BF16>(x[i][1].y);
                if (!is_v && rotated && tok_of[which][off] >= 0) {
                    const float* tab = p.table + (size_t)pos_of[which][off] * p.rot + 4 * ln;
                    const float4 c = __ldg(reinterpret_cast<const float4*>(tab));
                    const float4 s = __ldg(reinterpret_cast<const float4*>(tab + half));
                    if (p.inter) {
                        turn(a.x, a.y, c.x, s.x);
                        turn(b.x, b.y, c.y, s.y);
                        turn(e.x, e.y, c.z, s.z);
                        turn(f.x, f.y, c.w, s.w);
                    } else {
                        turn(a.x, e.x, c.x, s.x);
                        turn(a.y, e.y, c.y, s.y);
                        turn(b.x, f.x, c.z, s.z);
                        turn(b.y, f.y, c.w, s.w);
                    }
                    // rounded to the source type, as the row that kv_append would be given
                    x[i][0] = make_uint2(pack2<BF16>(a.x, a.y), pack2<BF16>(b.x, b.y));
                    x[i][1] = make_uint2(pack2<BF16>(e.x, e.y), pack2<BF16>(f.x, f.y));
                    a = unpack2<BF16>(x[i][0].x), b = unpack2<BF16>(x[i][0].y);
                    e = unpack2<BF16>(x[i][1].x), f = unpack2<BF16>(x[i][1].y);
                }
                rows[warp][off][ln] = make_uint4(x[i][0].x, x[i][0].y, x[i][1].x, x[i][1].y);
                amax = fmaxf(amax, fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))),
                                         fmaxf(fmaxf(fabsf(e.x), fabsf(e.y)), fmaxf(fabsf(f.x), fabsf(f.y)))));
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));

        const float s_old = (have & 1u) ? 0.f : stored;      // offset 0 written: a fresh block
        const float s = fmaxf(s_old, __fdiv_rn(amax, quant_limit<DT>()));
        const bool grown = s > s_old && s_old > 0.f;
        const float inv = __fdiv_rn(1.f, s);
        const bool exact = !(inv < INFINITY);                // s 0 or tiny: a division per element
        // then: their codes; each lane reads back what it wrote
#pragma unroll 1
        for (int i = 0; i < PASSES; ++i) {
            if (!grown && !some(i)) continue;
            const int off = RPP * i + sub;
            uint8_t* row = tile + off * RB;
            uint32_t w[2];
            if (tok_of[which][off] >= 0) {
                const uint4 u = rows[warp][off][ln];
                const float2 a = unpack2<BF16>(u.x), b = unpack2<BF16>(u.y), e = unpack2<BF16>(u.z), f = unpack2<BF16>(u.w);
                const float x[2][4] = {{a.x, a.y, b.x, b.y}, {e.x, e.y, f.x, f.y}};
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    w[r] = exact ? pack_codes<DT>(quant_code<DT>(x[r][0], s), quant_code<DT>(x[r][1], s),
                                                  quant_code<DT>(x[r][2], s), quant_code<DT>(x[r][3], s))
                                 : quant_codes4<DT>(x[r], s, inv);
            } else if (grown) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t c = load_codes4<DT>(row, r ? d1 : d0);
                    w[r] = pack_codes<DT>(requant_code<DT>(code_at<DT>(c, 0), s_old, s),
                                          requant_code<DT>(code_at<DT>(c, 1), s_old, s),
                                          requant_code<DT>(code_at<DT>(c, 2), s_old, s),
                                          requant_code<DT>(code_at<DT>(c, 3), s_old, s));
                }
            } else {
                continue;
            }
            store_codes4<DT>(row, d0, w[0]);
            store_codes4<DT>(row, d1, w[1]);
        }
        __syncwarp();
        if (lane == 0) *scale = s;
    }
}

template <int D, bool BF16, int DT>
__global__ void __launch_bounds__(kRopeThreads, 4) append_rope_kernel(const RopeParams p)
{
    if ((int)blockIdx.x < p.copy_ctas) {
        copy_rows<D, BF16>(p, blockIdx.x);
        return;
    }
    if constexpr (DT == PKV_INT8 || DT == PKV_INT4 || DT == PKV_FP8E4M3) {
        if (p.index) pdl_wait_primary();   // the slots' tokens, written by the kernel before this one
        const int cta = (int)blockIdx.x - p.copy_ctas;
        quantize_block<D, BF16, DT>(p, cta >> 1, cta & 1);
    }
}

// index[slot] = token, for every token that takes part
__global__ void __launch_bounds__(256) append_rope_index_kernel(const RopeParams p)
{
    pdl_launch_dependents();
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t >= p.T) return;
    const int slot = p.slots[t];
    if (live(p, slot, p.positions[t], false)) p.index[slot] = t;
}

template <int D, bool BF16>
int launch_dt(const RopeParams& p, int kv_dtype, unsigned grid, bool after_index, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = after_index ? 1 : 0;
    cudaError_t e;
    switch (kv_dtype) {
    case PKV_INT8: e = cudaLaunchKernelEx(&cfg, append_rope_kernel<D, BF16, PKV_INT8>, p); break;
    case PKV_INT4: e = cudaLaunchKernelEx(&cfg, append_rope_kernel<D, BF16, PKV_INT4>, p); break;
    case PKV_FP8E4M3: e = cudaLaunchKernelEx(&cfg, append_rope_kernel<D, BF16, PKV_FP8E4M3>, p); break;
    default: e = cudaLaunchKernelEx(&cfg, append_rope_kernel<D, BF16, PKV_BF16>, p); break;   // 16-bit: copies only
    }
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

size_t append_rope_workspace_bytes(int N, int kv_dtype, int T)
{
    return is_quantized(kv_dtype) && T > kScanTokens ? (size_t)N * kBlock * sizeof(int32_t) : 0;
}

int launch_append_rope(const AppendArgs& a, const RopeArgs& r, cudaStream_t s)
{
    const bool quant = is_quantized(a.kv_dtype);
    RopeParams p;
    p.q = static_cast<const uint16_t*>(r.q);
    p.k = static_cast<const uint16_t*>(a.k);
    p.v = static_cast<const uint16_t*>(a.v);
    p.q_out = static_cast<uint16_t*>(r.q_out);
    p.q_stride = r.q_stride;
    p.k_stride = r.k_stride;
    p.v_stride = r.v_stride;
    p.q_out_stride = r.q_out_stride;
    p.table = r.table;
    p.positions = r.positions;
    p.slots = a.slots;
    const bool indexed = append_rope_workspace_bytes(a.N, a.kv_dtype, a.T) > 0;
    p.index = indexed ? static_cast<int32_t*>(a.workspace) : nullptr;
    p.k_pool = a.k_pool;
    p.v_pool = a.v_pool;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.status = a.status;
    p.T = a.T;
    p.N = a.N;
    p.H_q = r.H_q;
    p.H_kv = a.H_kv;
    p.rot = r.rotary_dim;
    p.inter = r.interleaved;
    p.max_pos = r.max_positions;
    p.rows = r.H_q + (quant ? 0 : 2 * a.H_kv);
    // few tokens: a token's rows over several CTAs, one row per thread, so that a small step is
    // one round of loads on many SMs; many tokens: one CTA per token
    const int step = kRopeThreads / (a.d / 16);
    p.copy_y = a.T <= 2 * num_sms() ? (p.rows + step - 1) / step : 1;
    if (p.copy_y < 1) p.copy_y = 1;
    p.copy_ctas = p.rows > 0 ? a.T * p.copy_y : 0;
    // quantizing: a CTA for K and one for V of every token, or every kLook tokens
    const unsigned grid = (unsigned)p.copy_ctas + (!quant ? 0u : 2u * (indexed ? (unsigned)((a.T + kLook - 1) / kLook) : (unsigned)a.T));
    if (indexed) {
        append_rope_index_kernel<<<(unsigned)((a.T + 255) / 256), 256, 0, s>>>(p);
        if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
    }
    const bool bf = r.src_dtype == PKV_BF16;
    if (a.d == 128) return bf ? launch_dt<128, true>(p, a.kv_dtype, grid, indexed, s)
                              : launch_dt<128, false>(p, a.kv_dtype, grid, indexed, s);
    return bf ? launch_dt<64, true>(p, a.kv_dtype, grid, indexed, s) : launch_dt<64, false>(p, a.kv_dtype, grid, indexed, s);
}

}  // namespace pkv
