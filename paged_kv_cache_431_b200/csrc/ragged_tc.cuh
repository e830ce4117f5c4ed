// ragged_tc.cuh -- the ragged operators (paged_cross_attn, paged_decode_attn_groups) on the 5th-generation tensor cores (tcgen05 + TMEM).
//
// Rows of one item (a sequence's query rows, or a group's sequences) all see the same keys, so
// with R = rows x G query rows per KV head this is a dense [R x keys] contraction:
//   S = Q.K^T,  P = 2^(scale S - m),  O += P.V,  out = O / sum P
// One CTA (one per SM) holds two query tiles A and B of 128 rows in flight, so that the tensor
// cores work on one while the softmax warps work on the other (one warp issues the MMAs of each):
//   !PAIR  A and B are 256 consecutive rows that share every K/V tile (bound by the tensor cores
//          and by the exponentials: 2 x 128 x 128 of them per key tile on 16 lanes a cycle are as
//          many cycles as the four MMAs);
//   PAIR   (at most 128 rows per item and KV head: bound by the K/V bytes) A and B are the SAME
//          rows against two key partitions, each with its own K/V tiles; both write partials.
// Warps: 0..3 and 4..7 are the softmax of A and B (one thread per query row = TMEM lane), 8 and 10
// fetch K and V (TMA, one box per paged block), 9 and 11 issue the MMAs of A and B; for quantized pools
// 12.. turn fetched code tiles into fp16 tiles (the codes are exact in fp16; the K scale of a (block,
// head) multiplies its 16 scores, its V scale multiplies P, so a tile is converted once for all
// rows).  Per key tile and query tile: S (128 columns of TMEM) -> P back over the same columns as
// 16-bit pairs, the A operand of P.V, in two halves of 64 keys so that P.V starts while the other
// half is exponentiated.  The running max is lazy: O is rescaled only when a new max exceeds the
// old by 2^8.
//
// Roundings: Q, K, V enter as they are (16-bit; codes in fp16; a quantized pool's q in fp16
// after a power of two per row that brings its largest element to [1, 2), exact for bf16 down to
// 2^-17 of that).  S, m, sum P and O are fp32.  P enters P.V rounded to nearest in ONE 16-bit part:
// the output is rounded to 16 bits anyway, and P's half step (2^-9 for bf16, 2^-12 for fp16),
// spread over the keys, is of that size (measured against 64 bits: 1.4 times the error of an
// output that is only rounded).  The fp32-output kernels keep two parts.
#pragma once

#include <cuda_fp8.h>

#include "decode_common.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace ragged {

constexpr int kBM = 128;                         // query rows per tile
constexpr int kBN = 128;                         // keys per tile
constexpr int kBlocks = kBN / kBlock;            // paged blocks per key tile
constexpr float kSlack = 8.f;                    // log2 units the running max may lag
constexpr uint32_t kTmemCols = 512;              // tile x: S and P at 256x, O at 256x + 128
constexpr int kPolyEvery = 4;                    // of so many pairs of exponentials, one is a polynomial
constexpr float kTiny = 1.17549435e-38f;
constexpr float kHuge = 1048576.f;               // scores (log2 units) whose rounding, 2^-4, is still no matter
constexpr int kScaleSlots = 4;                   // key tiles whose scales are kept

template <int D, int DT, bool PAIR>
struct Cfg {
    static constexpr bool QUANT = DT == PKV_INT8 || DT == PKV_INT4 || DT == PKV_FP8E4M3;
    static constexpr bool BF16 = DT == PKV_BF16;                  // MMA operand type (else fp16)
    static constexpr int HALVES = D / 64;                         // 64-dim column groups
    static constexpr int TILE = kBN * D * 2;                      // one 16-bit Q, K or V tile
    static constexpr int QT = PAIR ? 1 : 2;                       // Q tiles
    static constexpr int ROW = DT == PKV_INT4 ? D / 2 : D;        // code bytes per row
    static constexpr int CTILE = QUANT ? kBN * ROW : 0;           // one code tile
    // ring depths: what 227 KB hold; 16-bit pools fetch into the K/V rings themselves
    static constexpr int NS = QUANT ? 2 : (D == 64 ? 4 : PAIR ? 3 : 2);
    static constexpr int NC = QUANT ? (PAIR || D == 64 ? 2 : DT == PKV_INT4 ? 2 : 1) : 1;
    static constexpr int SMEM = QT * TILE + NS * 2 * TILE + NC * 2 * CTILE + 1024;
    static constexpr int CONV = PAIR ? 4 : 2;                     // converter warps for K, and for V (quantized pools)
    static constexpr int THREADS = QUANT ? 384 + 64 * CONV : 384;
    // A softmax thread keeps its row's 128 scores in registers, but for the PAIR form of quantized
    // pools: there eight converter warps are worth more (fp8, 48 rows against 4 x 32,768 keys, before
    // COPIES below: 150 -> 138 us; with shared tiles, converted once for 256 rows, 773 -> 808 us).  The block is
    // launched with 168, 128 or 96 a thread, and the softmax warpgroups take what the others release:
    // 2 x 216 + 72 = 3 x 168;  2 x 168 + 72 + 96 <= 4 x 128;  2 x 136 + 56 + 2 x 72 <= 5 x 96.
    static constexpr bool ONE_PASS = !QUANT || !PAIR;
    static constexpr int SOFTMAX_REGS = !QUANT ? 216 : PAIR ? 136 : 168;
    static constexpr int ISSUE_REGS = QUANT && PAIR ? 56 : 72, CONV_REGS = PAIR ? 72 : 96;
    // Head dim 64 leaves 64 columns of TMEM per tile, which hold P apart from S: S(t+1) is computed
    // as soon as S(t) is in registers, beside the exponentials (else only after P(t).V).
    static constexpr bool P_APART = D == 64 && ONE_PASS;
    // PAIR form of quantized pools: up to 64 (32) query rows are put into the tile two (four) times, and
    // each copy takes the softmax of its half (quarter) of a tile's keys, with P = 0 for the others, a
    // running maximum of its own and its own rows of O; the copies are joined at the end.  Else half
    // (three quarters) of the softmax warps would have no rows, and the rest all the exponentials
    // (4 x 32,768 int8 tokens, 8 KV heads: 48 rows 132 -> 118 us, 32 rows 132 -> 99).  What is left
    // is a chain: the MMAs of A and of B, 128 rows each whatever R is, one after the other (2,200 cycles
    // of 4,700 per pair of tiles), and the softmax of each.
    static constexpr bool COPIES = QUANT && PAIR;
    static constexpr int SWZ = ROW >= 128 ? 7 : ROW == 64 ? 3 : 1;   // TMA swizzle of a code tile
    static_assert(SMEM <= 225 * 1024, "dynamic shared memory, with 2 KB left for the static part");
};

// K or V tile layout, 16 bits: 8-row groups; within one, the 64-dim halves; within those 8 rows of
// 128 bytes (128-byte swizzle).  A paged block of 16 rows is two groups, so it is ONE box of a 4-D
// view of the pool (64 dims, 8 rows, halves, 8-row groups).
template <int D>
struct KV {
    static constexpr int GROUP = 8 * D * 2;          // bytes of an 8-row group
    static constexpr int HALF = 1024;                // between the halves of a group
};

struct Bars {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];    // 16-bit tiles, ready for the MMAs
    uint64_t ck_full[2], ck_empty[2], cv_full[2], cv_empty[2];   // code tiles
    uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots];        // the scales of a key tile
    uint64_t q_full;           // the query tiles are in shared memory
    uint64_t s_full[2];        // S(x, t) is in TMEM, and every earlier MMA of the CTA is done
    uint64_t s_empty[2], pv_done[2];   // P_APART: S(x, t) is in registers; P.V(x, t) is done
    uint64_t p_full[2][2];     // a half of P(x, t) is stored
    uint64_t turn[2];          // P_APART: three quarters of P(x, t) are
    uint64_t o_done[2];
    uint64_t mma_drain[2];
};

__device__ __forceinline__ float2 fmul2(float2 a, float2 b)
{
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2bits(a)), "l"(f2bits(b)));
    return bitsf2(d);
}

__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 2^a for a pair, on the FMA pipe: a = n + f with n the nearest integer (by adding 1.5 x 2^23), 2^f
// on [-1/2, 1/2] by the polynomial 1 + f q(f) of least largest relative error, degree 3 (2^-13.2,
// against the half step 2^-9 of a bf16 P) or 4 (2^-18.4, against 2^-12), n added to the exponent field.
// a is at most kSlack.  From -127 down the result is exactly 0 (the constant term 1 at n = -127 leaves
// a field of 0 and no significand), so that a masked score, -inf, weighs nothing; between -127 and -126
// it is some number below 2^-126.  A NaN comes out as 0: the caller's row sum carries it.
template <int DEG>
__device__ __forceinline__ float2 exp2_poly(float2 a)
{
    constexpr float M = 12582912.f;
    a = make_float2(fmaxf(a.x, -127.f), fmaxf(a.y, -127.f));
    const float2 t = fadd2(a, make_float2(M, M));
    const float2 f = fsub2(a, fsub2(t, make_float2(M, M)));
    auto c2 = [](float c) { return make_float2(c, c); };
    float2 y;
    if constexpr (DEG == 3) {
        y = ffma2(c2(0x1.c2a216p-5f), f, c2(0x1.f00c4cp-3f));
        y = ffma2(y, f, c2(0x1.62f5fap-1f));
    } else {
        y = ffma2(c2(0x1.3a02cep-7f), f, c2(0x1.c9fc46p-5f));
        y = ffma2(y, f, c2(0x1.ec0378p-3f));
        y = ffma2(y, f, c2(0x1.62e12cp-1f));
    }
    y = ffma2(y, f, c2(1.f));
    return make_float2(__int_as_float(__float_as_int(y.x) + (__float_as_int(t.x) << 23)),
                       __int_as_float(__float_as_int(y.y) + (__float_as_int(t.y) << 23)));
}

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((127 + e) << 23); }   // e in [-126, 127]

// Exponent shift that brings x > 0 to [1, 2), kept in [-100, 100]; 0 for x = 0.
__device__ __forceinline__ int unit_shift(float x)
{
    if (!(x > 0.f)) return 0;
    const int e = (int)((__float_as_uint(x) >> 23) & 0xffu) - 127;
    return max(-100, min(100, -e));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint32_t hsub2_const(uint32_t a, float c)
{
    __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), __float2half2_rn(c));
    return *reinterpret_cast<uint32_t*>(&r);
}

// Four 8-bit codes -> two fp16 pairs, exact.  int8: code + 128 moved into the significand of
// 1024, then 1152 subtracted.
template <int DT>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& a, uint32_t& b)
{
    if constexpr (DT == PKV_INT8) {
        const uint32_t x = w ^ 0x80808080u;
        a = hsub2_const(__byte_perm(x, 0x64646464u, 0x4140), 1152.f);
        b = hsub2_const(__byte_perm(x, 0x64646464u, 0x4342), 1152.f);
    } else {
        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
        a = (uint32_t)lo.x | ((uint32_t)lo.y << 16);
        b = (uint32_t)hi.x | ((uint32_t)hi.y << 16);
    }
}

// Eight 4-bit codes -> four fp16 pairs in order, exact.  Nibbles 2i and 2i + 1 are brought to
// bits 0..3 of two halves, code + 8 moved into the significand of 1024, then 1032 subtracted.
__device__ __forceinline__ void codes8_int4(uint32_t w, uint32_t (&h)[4])
{
    const uint32_t x = w ^ 0x88888888u;
    const uint32_t even = x & 0x0f0f0f0fu, odd = (x >> 4) & 0x0f0f0f0fu;   // byte i: elements 2i, 2i + 1
    const uint32_t p01 = __byte_perm(even, odd, 0x5140), p23 = __byte_perm(even, odd, 0x7362);
    h[0] = hsub2_const(__byte_perm(p01, 0x64646464u, 0x4140), 1032.f);
    h[1] = hsub2_const(__byte_perm(p01, 0x64646464u, 0x4342), 1032.f);
    h[2] = hsub2_const(__byte_perm(p23, 0x64646464u, 0x4140), 1032.f);
    h[3] = hsub2_const(__byte_perm(p23, 0x64646464u, 0x4342), 1032.f);
}

template <int D, int DT, bool PAIR>
__global__ void __launch_bounds__((Cfg<D, DT, PAIR>::THREADS), 1)
ragged_tc_kernel(const DecodeParams p, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV)
{
    using C = Cfg<D, DT, PAIR>;
    constexpr int NS = C::NS, NC = C::NC, TILE = C::TILE;
    extern __shared__ uint8_t smem_dyn[];
    __shared__ Bars bars;
    __shared__ uint32_t s_tmem_base;
    __shared__ volatile int s_abort;
    __shared__ float s_rowscale[C::QUANT ? C::QT * kBM : 1];              // per query row: 2^-e of its fp16 q
    __shared__ __align__(8) float2 s_scale[C::QUANT ? kScaleSlots * kBlocks : 1];   // (K, V) scales of a key tile's blocks
    __shared__ int s_vmax;
    __shared__ volatile int s_armed[2];                           // K, V tiles whose full barrier is in their phase

    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = blockIdx.y;
    const int zparts = PAIR ? (p.max_parts + 1) / 2 : p.max_parts;
    const int b = blockIdx.z / zparts, z = blockIdx.z % zparts;
    const RaggedItem it = ragged_item(p.rg, p.ctx_lens, p.W, b, p.status,
                                      threadIdx.x == 0 && blockIdx.x == 0 && z == 0 && g == 0);
    const int R = it.rows * p.G;                                  // query rows of this KV head
    const int r0 = blockIdx.x * (C::QT * kBM);
    if (r0 >= R) return;
    const int nparts = (it.end - it.base + p.part_tokens - 1) / p.part_tokens;
    const int part0 = PAIR ? 2 * z : z;                           // partition of tile A
    if (part0 >= nparts) {
        if (z == 0 && it.whole) {                                 // no keys at all: zero rows
            const int n = min(C::QT * kBM, R - r0) * (D / 8);
            for (int i = threadIdx.x; i < n; i += C::THREADS)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.rg.out16) +
                                          ragged_row(it, p.G, p.H_q, g, r0 + i / (D / 8)) * D + 8 * (i % (D / 8))) =
                    make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    // Tile x: key range [key_lo(x), key_hi(x)) in ntiles(x) key tiles.  `shared`: both query tiles
    // use every K/V tile; else K/V tiles come in the order (A,0) (B,0) (A,1) (B,1) ...
    const bool shared = !PAIR && r0 + kBM < R;
    auto key_lo = [&](int x) { return it.base + (PAIR ? part0 + x : part0) * p.part_tokens; };
    auto key_hi = [&](int x) { return min(it.end, key_lo(x) + p.part_tokens); };
    auto ntiles = [&](int x) {
        if (!PAIR && x == 1 && !shared) return 0;
        return max(0, (key_hi(x) - key_lo(x) + kBN - 1) / kBN);
    };
    const int nA = ntiles(0), nB = ntiles(1);
    auto seq = [&](int x, int t) { return shared ? t : x == 0 ? t + min(t, nB) : t + min(t + 1, nA); };

    // Softmax warps of tile x that have rows (32 each).  The others have nothing to compute: what
    // they would leave in TMEM only reaches rows of O that nobody reads.
    const int copies = !C::COPIES ? 1 : R <= 32 ? 4 : R <= 64 ? 2 : 1;
    auto busy = [&](int x) {
        return copies > 1 ? 4 : min(4, (max(1, R - r0 - (PAIR ? 0 : x * kBM)) + 31) / 32);
    };

    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem);
    const uint32_t sK = sQ + C::QT * TILE;
    const uint32_t sV = sK + NS * TILE;
    const uint32_t sCK = sV + NS * TILE;
    const uint32_t sCV = sCK + NC * C::CTILE;

    if (threadIdx.x == 0) {
        s_abort = 0;
        s_vmax = 0;
        s_armed[0] = s_armed[1] = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&bars.k_full[s]), C::QUANT ? C::CONV : 1);
            mbar_init(smem_u32(&bars.k_empty[s]), shared ? 2 : 1);
            mbar_init(smem_u32(&bars.v_full[s]), C::QUANT ? C::CONV : 1);
            mbar_init(smem_u32(&bars.v_empty[s]), shared ? 2 : 1);
        }
        if constexpr (C::QUANT) {
            for (int s = 0; s < NC; ++s) {
                mbar_init(smem_u32(&bars.ck_full[s]), 1);
                mbar_init(smem_u32(&bars.ck_empty[s]), C::CONV);
                mbar_init(smem_u32(&bars.cv_full[s]), 1);
                mbar_init(smem_u32(&bars.cv_empty[s]), C::CONV);
            }
            for (int s = 0; s < kScaleSlots; ++s) {
                mbar_init(smem_u32(&bars.sc_full[s]), C::CONV);
                mbar_init(smem_u32(&bars.sc_empty[s]), shared ? busy(0) + busy(1) : busy(0));
            }
        }
        mbar_init(smem_u32(&bars.q_full), 8);
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&bars.s_full[x]), 1);
            mbar_init(smem_u32(&bars.s_empty[x]), busy(x));
            mbar_init(smem_u32(&bars.pv_done[x]), 1);
            mbar_init(smem_u32(&bars.p_full[x][0]), busy(x));
            mbar_init(smem_u32(&bars.p_full[x][1]), busy(x));
            mbar_init(smem_u32(&bars.turn[x]), busy(x));
            mbar_init(smem_u32(&bars.o_done[x]), 1);
        }
        for (int x = 0; x < 2; ++x) mbar_init(smem_u32(&bars.mma_drain[x]), 1);
        mbar_fence_init();
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const int32_t* trow = p.tables + (size_t)it.table * p.W;
    auto block_id = [&](int lb) -> int {       // physical block of logical block lb (in bounds)
        int blk = trow[lb];
        if ((unsigned)blk >= (unsigned)p.N) {
            flag_status(p.status, PKV_DEV_BAD_BLOCK);
            blk = 0;
        }
        return blk;
    };
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem_base;

    // A wait of a whole warp: agreed on by its lanes; the abort flag is looked at only where the
    // barrier is not there yet.
    auto wait = [&](uint64_t& bar, uint32_t parity) {
        const bool there = mbar_try_wait(smem_u32(&bar), parity);
        if (__all_sync(0xffffffffu, there)) return true;
        return (bool)__all_sync(0xffffffffu, wait_or_abort(smem_u32(&bar), parity, &s_abort, p.status, p.wait_cycles));
    };

    // Waits for K (V) tile n in the ring.  In the PAIR form A and B take turns on the stages but run
    // at their own pace, and a barrier's parity cannot tell tile n's phase from the one two before:
    // so the wait on it starts only once tile n is armed, which its fetcher does after the stage's
    // previous tile was consumed.
    auto wait_tile = [&](int which, uint64_t* full, int n) {
        if constexpr (PAIR) {
            if (s_armed[which] <= n) {
                const long long t0 = clock64();
                while (s_armed[which] <= n) {
                    if (s_abort) break;
                    if (clock64() - t0 > p.wait_cycles) {
                        s_abort = 1;
                        flag_status(p.status, PKV_DEV_TIMEOUT);
                    }
                }
            }
            if (!__all_sync(0xffffffffu, s_armed[which] > n)) return false;
        }
        return wait(full[n % NS], (n / NS) & 1);
    };

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        regs_inc<C::SOFTMAX_REGS>();
        const int x = warp >> 2;
        const int quarter = warp & 3;                             // the 32 TMEM lanes this warp may touch
        const int r = quarter * 32 + lane;
        const int nx = quarter >= busy(x) ? 0 : x == 0 ? nA : nB;
        const int lo = key_lo(x), hi = key_hi(x);
        const uint32_t tS = tmem + ((uint32_t)(quarter * 32) << 16) + 256 * x;
        const uint32_t tO = tS + 128, tP = C::P_APART ? tS + 192 : tS;
        // This warp's 32 query rows into shared memory, K-major with the 128-byte swizzle, by plain loads
        // (rows are gathered: row of the item, head; any group size packs 128 rows into a tile), several
        // in flight, while the fetchers already run.  A negative scale is moved into q, so that the
        // softmax may take maxima before it scales.
        const int rr = C::COPIES ? r & (kBM / copies - 1) : r0 + (PAIR ? 0 : x * kBM) + r;
        const int copy = C::COPIES ? quarter * copies >> 2 : 0;
        // this copy's 32-key columns of a tile
        const int c_lo = C::COPIES ? copy * (4 / copies) : 0, c_hi = C::COPIES ? c_lo + 4 / copies : 4;
        const int at = rr < R ? (int)ragged_row(it, p.G, p.H_q, g, rr) : -1;   // in rows of D
        if (!PAIR || x == 0) {
            constexpr int CH = D / 8, RPI = 32 / CH, BATCH = 8;   // 16-byte chunks per row, rows per load
            const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
            const uint16_t* qh = static_cast<const uint16_t*>(p.q);
            const int c = lane % CH;
#pragma unroll 1
            for (int i0 = 0; i0 < 32 / RPI; i0 += BATCH) {
                uint4 u[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int a = __shfl_sync(0xffffffffu, at, (i0 + k) * RPI + lane / CH);
                    u[k] = a >= 0 ? __ldg(reinterpret_cast<const uint4*>(qh + (size_t)a * D + 8 * c)) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int row = quarter * 32 + (i0 + k) * RPI + lane / CH;
                    uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
                    if constexpr (C::QUANT) {   // fp16, times a power of two per row (its CH lanes agree on it)
                        float f[8], top = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 q2 = p.q_bf16 ? unpack2<true>(w[e]) : unpack2<false>(w[e]);
                            f[2 * e] = q2.x;
                            f[2 * e + 1] = q2.y;
                            top = fmaxf(top, fmaxf(fabsf(q2.x), fabsf(q2.y)));
                        }
#pragma unroll
                        for (int o = CH / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const int e = unit_shift(top);
                        const float m = exp2_int(e);
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = pack2<false>(f[2 * j] * m, f[2 * j + 1] * m);
                        if (c == 0) s_rowscale[(PAIR ? 0 : x * kBM) + row] = exp2_int(-e);
                    }
                    sts128(sQ + (PAIR ? 0 : x) * TILE + (c >> 3) * (kBM * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                           w[0] ^ flip, w[1] ^ flip, w[2] ^ flip, w[3] ^ flip);
                }
            }
            fence_proxy_async_smem();
        }
        // the largest V scale of the CTA's keys: P enters P.V times (V scale / its power of two)
        if constexpr (C::QUANT) {
            const int lb0 = key_lo(0) / kBlock, lb1 = (max(key_hi(0), nB > 0 ? key_hi(1) : 0) + kBlock - 1) / kBlock;
            float m = 0.f;
            for (int lb = lb0 + (int)threadIdx.x; lb < lb1; lb += 256)
                m = fmaxf(m, p.v_scale[(size_t)block_id(lb) * p.H_kv + g]);
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) atomicMax(&s_vmax, __float_as_int(m));     // non-negative: ordered as integers
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.q_full));
        float sl = fabsf(p.scale_log2);
        float v_unit = 1.f, v_mul = 1.f;
        bool ok = true;
        if constexpr (C::QUANT) {
            ok = wait(bars.q_full, 0);
            sl *= s_rowscale[(PAIR ? 0 : x * kBM) + r];
            // the largest V scale to [2^6, 2^7): P, up to 2^8, times it then stays within fp16, and keeps its
            // 11 bits on blocks whose V scale is down to 2^-20 of that
            const int e = unit_shift(__int_as_float(s_vmax)) + 6;
            v_mul = exp2_int(e);
            v_unit = exp2_int(-e);
        }
        // a factor of 0 would turn a masked score's -inf into NaN; the smallest normal number serves as
        // well (a NaN stays: it is the caller's scale)
        sl = fmax_nan(sl, kTiny);
        float m_used = -INFINITY, l_run = 0.f;
        // Huge scores: factor S - m in one step leaves the rounding of the maximum, which passes the
        // exponents' range from 2^28 on.  There the product is rounded by itself, as the maximum's was, so
        // that the largest score gives 0.  (Quantized pools always do so: in two steps 413 us instead of
        // 372 on 4 x 1,024 rows of head dim 64.)
        bool huge = false;
        for (int t = 0; ok && t < nx; ++t) {
            const int n = seq(x, t);
            ok = wait(bars.s_full[x], t & 1);
            if (!ok) break;
            if constexpr (C::QUANT) {
                ok = wait(bars.sc_full[n % kScaleSlots], (n / kScaleSlots) & 1);
                if (!ok) break;
            }
            tc_fence_after();
            // per paged block of 16 keys (quantized pools): (K, V) scales, read where they are needed
            const float2* sc = s_scale + (C::QUANT ? (n % kScaleSlots) * kBlocks : 0);
            const int left = hi - lo - t * kBN;                   // keys of this tile in the range
            const bool need_mask = left < kBN;
            // the row's 128 scores: kept in registers from here to P, or read twice, 32 at a time
            float v[C::ONE_PASS ? 4 : 1][32];
            if constexpr (C::ONE_PASS) {
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, v[c]);
                tmem_wait_ld();
                if constexpr (C::P_APART) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars.s_empty[x]));
                }
                if (need_mask) {
#pragma unroll
                    for (int j = 0; j < kBN; ++j)
                        if (j >= left) v[j >> 5][j & 31] = -INFINITY;
                }
            }
            // P_APART: whether P.V(t-1) is done, asked here so that the answer comes beside the maxima
            bool pv_there = true;
            if constexpr (C::P_APART) {
                if (t > 0) pv_there = mbar_test_wait(smem_u32(&bars.pv_done[x]), (t - 1) & 1);
            }
            // the row maximum of the scaled scores, in three-input maxima per paged block; NaN if any is
            float mx = -INFINITY;
#pragma unroll(C::ONE_PASS ? 4 : 1)
            for (int c = c_lo; c < c_hi; ++c) {
                float* w = v[C::ONE_PASS ? c : 0];
                if constexpr (!C::ONE_PASS) {
                    tmem_ld32(tS + 32 * c, v[0]);
                    tmem_wait_ld();
                    if (need_mask) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (32 * c + j >= left) w[j] = -INFINITY;
                    }
                }
                float m2[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float* u = w + 16 * k;
                    float m0 = fmax3_nan(u[0], u[1], u[2]), m1 = fmax3_nan(u[3], u[4], u[5]);
                    m0 = fmax3_nan(m0, u[6], u[7]);
                    m1 = fmax3_nan(m1, u[8], u[9]);
                    m0 = fmax3_nan(m0, u[10], u[11]);
                    m1 = fmax3_nan(m1, u[12], u[13]);
                    m2[k] = fmax_nan(fmax3_nan(m0, u[14], u[15]), m1);
                    if constexpr (C::QUANT) m2[k] *= fmax_nan(sl * sc[2 * c + k].x, kTiny);
                }
                mx = fmax3_nan(mx, m2[0], m2[1]);
            }
            if constexpr (!C::QUANT) mx = __fmul_rn(mx, sl);
            // a NaN becomes the row's maximum, and so reaches its sum; one of +inf is looked for behind the loop
            const float m_new = mx <= m_used + kSlack ? m_used : mx;
            const float alpha = m_used == -INFINITY ? 0.f : ex2(m_used - m_new);
            const float mref = m_new == -INFINITY ? 0.f : m_new;
            // the max moved: rescale this row of O (P.V(t-1) is done: s_full(t) says so, or pv_done)
            if constexpr (C::P_APART) {
                if (!__all_sync(0xffffffffu, pv_there)) ok = wait(bars.pv_done[x], (t - 1) & 1);
                if (!ok) break;
                tc_fence_after();
            }
            if (__any_sync(0xffffffffu, alpha != 1.f)) {
                if constexpr (!C::QUANT) huge = __any_sync(0xffffffffu, fabsf(m_new) > kHuge);
#pragma unroll 1
                for (int c = 0; t > 0 && c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= alpha;
                    tmem_st32(tO + 32 * c, o);
                }
            }
            // keys past the range: zero their V rows (P is 0 there, V may be stale or NaN).  Where A and
            // B share V both do it, each before its own P.V.  Converted tiles come zeroed.
            if (!C::QUANT && need_mask) {
                const int s = n % NS;
                ok = wait_tile(1, bars.v_full, n);
                if (!ok) break;
                const int tid = threadIdx.x & 127;
                const int rows = kBN - left;
                for (int i = tid; i < C::HALVES * rows * 8; i += 32 * busy(x)) {
                    const int c16 = i & 7, row = left + (i >> 3) % rows, half = (i >> 3) / rows;
                    sts128(sV + s * TILE + (row >> 3) * KV<D>::GROUP + half * KV<D>::HALF + (row & 7) * 128 + c16 * 16, 0u,
                           0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            // A and B take turns with the exponentials: left alone they fall into step, and then wait
            // for the tensor cores together (head dim 128, 1,024 rows x 8 heads against 4 x 4,096 keys:
            // 598 us without turns, 460 with).  Head dim 64 is bound by the exponentials themselves and
            // their waits, so its turn passes after three quarters (394 -> 372 us; 128: 460 -> 469).
            // Quantized pools are bound by the conversions and run faster without turns.
            if (!C::QUANT && shared) {
                uint64_t& turn = C::P_APART ? bars.turn[1 - x] : bars.p_full[1 - x][1];
                if (x == 1) ok = wait(turn, t & 1);
                else if (t > 0) ok = wait(turn, (t - 1) & 1);
                if (!ok) break;
            }
            if constexpr (!C::QUANT) {
                if (huge) {
#pragma unroll
                    for (int j = 0; j < kBN; ++j) v[j >> 5][j & 31] = __fmul_rn(v[j >> 5][j & 31], sl);
                }
            }
            const float fac = huge ? 1.f : sl;
            // P = 2^(factor S - m) in 16 bits, packed into the tile's first 64 columns, in two halves
            const float2 mref2 = make_float2(-mref, -mref);
            float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            auto columns_of_p = [&](int c) {
                const float* u = v[C::ONE_PASS ? c : 0];
                if constexpr (!C::ONE_PASS) {
                    tmem_ld32(tS + 32 * c, v[0]);
                    tmem_wait_ld();
                    if (need_mask) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (32 * c + j >= left) v[0][j] = -INFINITY;
                    }
                }
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float f = fac;
                    [[maybe_unused]] float vm = 1.f;
                    if constexpr (C::QUANT) {
                        const float2 kv = sc[2 * c + (e >> 3)];
                        f = fmaxf(sl * kv.x, kTiny);
                        vm = v_mul * kv.y;
                    }
                    const float2 s2 = make_float2(u[2 * e], u[2 * e + 1]), f2 = make_float2(f, f);
                    // (+ 0: a product alone would be fused with the sum all the same)
                    const float2 a = C::QUANT ? fadd2(ffma2(s2, f2, make_float2(0.f, 0.f)), mref2) : ffma2(s2, f2, mref2);
                    float2 pp;
                    // some pairs take the FMA pipe, so that it shares the exponentials with the
                    // special-function unit
                    if (!C::QUANT && e % kPolyEvery == kPolyEvery - 1) pp = exp2_poly<C::BF16 ? 3 : 4>(a);
                    else pp = make_float2(ex2(a.x), ex2(a.y));
                    sum2[e & 1] = fadd2(sum2[e & 1], pp);
                    if constexpr (C::QUANT) pp = fmul2(pp, make_float2(vm, vm));
                    w[e] = pack2<C::BF16>(pp.x, pp.y);
                }
                tmem_st16u(tP + 16 * c, w);
                if (C::P_APART && c == 2) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars.turn[x]));
                }
            };
            auto half_done = [&](int half) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[x][half]));
            };
            if constexpr (C::COPIES) {
#pragma unroll 1
                for (int c = c_lo; c < c_hi; ++c) {
                    columns_of_p(c);
                    if (copies == 1 && c == 1) half_done(0);
                }
                if (copies > 1) {                                 // the other copies' keys
                    const uint32_t none[16] = {};
#pragma unroll 1
                    for (int c = 0; c < 4; ++c)
                        if (c < c_lo || c >= c_hi) tmem_st16u(tP + 16 * c, none);
                    half_done(0);
                }
                half_done(1);
            } else {
#pragma unroll(C::ONE_PASS ? 2 : 1)
                for (int half = 0; half < 2; ++half) {
#pragma unroll(C::ONE_PASS ? 2 : 1)
                    for (int cc = 0; cc < 2; ++cc) columns_of_p(2 * half + cc);
                    half_done(half);
                }
            }
            if constexpr (C::QUANT) {
                if (lane == 0) mbar_arrive(smem_u32(&bars.sc_empty[n % kScaleSlots]));
            }
            l_run = l_run * alpha + ((sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y));
            m_used = m_new;
        }
        // a score of +inf makes the row's softmax NaN (inf - inf), which not every exponential above would;
        // scores of -inf just weigh nothing
        if (!(m_used < INFINITY)) l_run = NAN;
        bool done = ok && nx > 0 && wait(bars.o_done[x], 0);
        if (done) tc_fence_after();
        // Join the copies: their O, brought to the common maximum, through the rings, which nothing
        // uses any more once the MMAs of both tiles are done.  Every softmax warp comes here, on an
        // abort too (the rings may then still be written to; what is computed is not used).
        float factor = 1.f;
        const float4* others = nullptr;
        if (C::COPIES && copies > 1) {
            const int rows = kBM / copies;
            float2* ml = reinterpret_cast<float2*>(smem) + x * kBM;
            float4* red = reinterpret_cast<float4*>(smem + TILE + x * NS * TILE);   // [copy - 1][D / 4][rows]
            named_sync(1, 256);
            ml[r] = make_float2(m_used, l_run);
            named_sync(2 + x, 128);
            float m = -INFINITY, l = 0.f;
            for (int k = 0; k < copies; ++k) m = fmaxf(m, ml[k * rows + rr].x);
            for (int k = 0; k < copies; ++k) {
                const float2 u = ml[k * rows + rr];
                l += u.x == -INFINITY ? 0.f : ex2(u.x - m) * u.y;
            }
            factor = m_used == -INFINITY ? 0.f : ex2(m_used - m);
            m_used = m;
            l_run = l;
            if (copy > 0 && done) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        red[((copy - 1) * (D / 4) + 8 * c + i) * rows + rr] = make_float4(
                            o[4 * i] * factor, o[4 * i + 1] * factor, o[4 * i + 2] * factor, o[4 * i + 3] * factor);
                    __syncwarp();
                }
            }
            named_sync(2 + x, 128);
            done = done && copy == 0;
            others = red + rr;
        }
        if (done) {
            const bool valid = at >= 0;
            const bool final_out = it.whole && nparts == 1;
            const size_t row = valid ? at : 0;
            const size_t slot = ws_slot(p, row, part0 + (PAIR ? x : 0));
            const float inv = (final_out ? 1.f / l_run : 1.f) * v_unit;   // l_run 0: every score -inf, NaN as 0 / 0
            if (!final_out && valid)
                st_hint(reinterpret_cast<float2*>(p.ws_ml + slot * 2), make_float2(m_used, l_run), l2_evict_last());
            __syncwarp();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                tmem_ld32(tO + 32 * c, o);
                tmem_wait_ld();
                if constexpr (C::COPIES) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= factor;
#pragma unroll 1
                    for (int k = 1; k < copies; ++k) {
                        const float4* u = others + ((k - 1) * (D / 4) + 8 * c) * (kBM / copies);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 w = u[i * (kBM / copies)];
                            o[4 * i] += w.x;
                            o[4 * i + 1] += w.y;
                            o[4 * i + 2] += w.z;
                            o[4 * i + 3] += w.w;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= inv;
                if (!valid) {
                } else if (final_out) {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.rg.out16) + row * D + 32 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 lo2 = pack4(make_float4(o[8 * i], o[8 * i + 1], o[8 * i + 2], o[8 * i + 3]), p.q_bf16);
                        const uint2 hi2 = pack4(make_float4(o[8 * i + 4], o[8 * i + 5], o[8 * i + 6], o[8 * i + 7]), p.q_bf16);
                        dst[i] = make_uint4(lo2.x, lo2.y, hi2.x, hi2.y);
                    }
                } else {
                    float4* dst = reinterpret_cast<float4*>(p.ws_o + slot * D + 32 * c);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_hint(dst + i, make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]), l2_evict_last());
                }
                __syncwarp();                                     // the next TMEM read needs the whole warp
            }
        }
    } else if (warp < 12) {
        regs_dec<C::ISSUE_REGS>();
        if (warp == 8 || warp == 10) {
        // ------------------------------------------------------------ producers (8: K, 10: V)
        // The lanes hold the block ids of the next 4 key tiles of A and of B (one load per 4 tiles,
        // a chunk ahead); one lane issues the copies, one box per paged block.  Keys past the range
        // fetch block 0: in bounds, masked, and their V rows zeroed.
        const bool is_v = warp == 10;
        int cur[2], nxt[2];
        auto entry = [&](int x, int i) -> int {
            const int lb = key_lo(x) / kBlock + i;
            return lb * kBlock < key_hi(x) ? block_id(lb) : 0;
        };
        for (int x = 0; x < 2; ++x) {
            cur[x] = (x == 0 || nB > 0) ? entry(x, lane) : 0;
            nxt[x] = (x == 0 || nB > 0) ? entry(x, 32 + lane) : 0;
        }
        constexpr int ND = C::QUANT ? NC : NS;                    // depth of the ring the copies go to
        uint64_t* full = C::QUANT ? (is_v ? bars.cv_full : bars.ck_full) : (is_v ? bars.v_full : bars.k_full);
        uint64_t* empty = C::QUANT ? (is_v ? bars.cv_empty : bars.ck_empty) : (is_v ? bars.v_empty : bars.k_empty);
        constexpr uint32_t BYTES = C::QUANT ? C::CTILE : TILE;
        constexpr uint32_t BOX = BYTES / kBlocks;                 // one paged block
        const uint32_t ring = C::QUANT ? (is_v ? sCV : sCK) : (is_v ? sV : sK);
        const CUtensorMap* tm = is_v ? &tmV : &tmK;
        int issued = 0;
        bool go = true;
        const uint64_t pol = l2_evict_first();
        const int tmax = max(nA, nB);
        for (int t = 0; go && t < tmax; ++t) {
            if (t > 0 && t % 4 == 0) {
                for (int x = 0; x < 2; ++x) {
                    cur[x] = nxt[x];
                    if (x == 0 || nB > 0) nxt[x] = entry(x, (t / 4 + 1) * 32 + lane);
                }
            }
            for (int x = 0; go && x < (shared ? 1 : 2); ++x) {
                if (t >= (x == 0 ? nA : nB)) continue;
                const int n = seq(x, t), s = n % ND;
                int rows[kBlocks];
#pragma unroll
                for (int kb = 0; kb < kBlocks; ++kb)
                    rows[kb] = (__shfl_sync(0xffffffffu, cur[x], (t % 4) * kBlocks + kb) * p.H_kv + g) * kBlock;
                if (n >= ND) go = wait(empty[s], ((n - ND) / ND) & 1);
                if (!go) break;
                if (lane == 0) {
                    const uint32_t bar = smem_u32(&full[s]), dst = ring + s * BYTES;
                    mbar_arrive_expect_tx(bar, BYTES);
                    if constexpr (!C::QUANT) s_armed[is_v ? 1 : 0] = n + 1;
                    if (is_v || n != p.hold_tile) {   // test hook: the withheld tile's K bytes never arrive
#pragma unroll
                        for (int kb = 0; kb < kBlocks; ++kb) {
                            if constexpr (C::QUANT) {
                                if constexpr (PAIR) tma_load_2d_hint(dst + kb * BOX, tm, 0, rows[kb], bar, pol);
                                else tma_load_2d(dst + kb * BOX, tm, 0, rows[kb], bar);
                            } else {
                                if constexpr (PAIR) tma_load_4d_hint(dst + kb * BOX, tm, 0, 0, 0, rows[kb] / 8, bar, pol);
                                else tma_load_4d(dst + kb * BOX, tm, 0, 0, 0, rows[kb] / 8, bar);
                            }
                        }
                    }
                }
                issued = n + 1;
            }
        }
        // do not leave while copies into this CTA's shared memory may be in flight
        if (lane == 0)
            for (int n = max(0, issued - ND); n < issued; ++n)
                if (is_v || n != p.hold_tile) mbar_wait_bounded(smem_u32(&full[n % ND]), (n / ND) & 1, p.wait_cycles);
        } else {
        // ------------------------------------------------------------ MMA issuers (9: tile A, 11: tile B)
        // One warp per query tile, so that a wait of one tile's chain (P, the next K tile) does not
        // keep the other tile's MMAs back.  The whole warp runs this loop; one elected lane issues
        // each MMA and commit, all of a tile's from the same lane, so they run in order: S(t+1)
        // overwrites the columns of P(t) after P.V(t) has read them.
        const int x = warp == 9 ? 0 : 1;
        const int nx = x == 0 ? nA : nB;
        const uint32_t id_qk = idesc_f16(C::BF16, false, kBM, kBN);
        const uint32_t id_pv = idesc_f16(C::BF16, true, kBM, D);
        const uint32_t tS = tmem + 256 * x, tO = tS + 128, tP = C::P_APART ? tS + 192 : tS;
        const uint64_t dq = sdesc_k128(sQ + (PAIR ? 0 : x) * TILE);
        const uint64_t dk = sdesc_k128_sbo(sK, KV<D>::GROUP), dv = sdesc_mn128_sbo(sV, KV<D>::HALF, KV<D>::GROUP);
        bool ok = true;
        auto scores = [&](int t) {              // S(x, t), and the release of its K tile
            const int n = seq(x, t), s = n % NS;
            ok = wait_tile(0, bars.k_full, n);
            if (!ok) return;
            tc_fence_after();
            const uint64_t k0 = dk + (uint32_t)(s * (TILE >> 4));
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                umma_w(tS, dq + (((ks >> 2) * (kBM * 128) + (ks & 3) * 32) >> 4),
                       k0 + (((ks >> 2) * KV<D>::HALF + (ks & 3) * 32) >> 4), id_qk, ks > 0);
            umma_commit_w(smem_u32(&bars.s_full[x]));
            umma_commit_w(smem_u32(&bars.k_empty[s]));
        };
        if (nx > 0) {
            ok = wait(bars.q_full, 0);
            if (ok) scores(0);
        }
        for (int t = 0; ok && t < nx; ++t) {
            if constexpr (C::P_APART) {
                if (t + 1 < nx) {
                    ok = wait(bars.s_empty[x], t & 1);
                    if (ok) tc_fence_after();
                    if (ok) scores(t + 1);
                    if (!ok) break;
                }
            }
            const int n = seq(x, t), s = n % NS;
            const uint64_t v0 = dv + (uint32_t)(s * (TILE >> 4));
            ok = wait_tile(1, bars.v_full, n);
#pragma unroll
            for (int half = 0; ok && half < 2; ++half) {
                ok = wait(bars.p_full[x][half], t & 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k) {   // 16 keys: two 8-row groups of V
                    const int ks = 4 * half + k;
                    umma_ts_w(tO, tP + 8 * ks, v0 + ((ks * 2 * KV<D>::GROUP) >> 4), id_pv, t > 0 || ks > 0);
                }
            }
            if (!ok) break;
            if (t + 1 < nx) {
                if constexpr (C::P_APART) umma_commit_w(smem_u32(&bars.pv_done[x]));
                umma_commit_w(smem_u32(&bars.v_empty[s]));
                if constexpr (!C::P_APART) scores(t + 1);
            } else {
                umma_commit_w(smem_u32(&bars.o_done[x]));
                umma_commit_w(smem_u32(&bars.v_empty[s]));
            }
        }
        // every MMA that was issued, also on an abort, is done before TMEM is freed
        umma_commit_w(smem_u32(&bars.mma_drain[x]));
        mbar_wait_bounded(smem_u32(&bars.mma_drain[x]), 0, p.wait_cycles);
        }
    } else if constexpr (C::QUANT) {
        regs_dec<C::CONV_REGS>();
        // ------------------------------------------------------------ converters
        // The first CONV warps convert K tiles, the others V tiles, each at the pace of its ring.  A
        // thread takes one key of a tile (or two): its row of codes -> its row of the fp16 tile (both
        // swizzled by 16-byte chunks, so the 32 rows of a warp spread over the banks).
        const bool is_v = warp >= 12 + C::CONV;
        const int id = (int)threadIdx.x - 384 - (is_v ? 32 * C::CONV : 0);
        auto convert = [&](uint32_t code, uint32_t dst, int key, bool zero) {
            const int base = key * C::ROW;
            const int sw = (base >> 7) & C::SWZ;
            const uint32_t row = dst + (key >> 3) * KV<D>::GROUP + (key & 7) * 128;
            // kept small, like the other loops of this kernel: five kinds of warps share the
            // instruction cache (fully unrolled, warps waited for instructions more than for MMAs)
#pragma unroll 2
            for (int c = 0; c < C::ROW / 16; ++c) {
                uint32_t w[4];
                lds128(w, code + base + ((c ^ sw) << 4));
                if (zero) w[0] = w[1] = w[2] = w[3] = 0u;
                if constexpr (DT == PKV_INT4) {                   // 32 elements: 4 chunks of the fp16 row
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h[4];
                        codes8_int4(w[i], h);
                        const int ch = 4 * c + i;
                        sts128(row + (ch >> 3) * KV<D>::HALF + (((ch & 7) ^ (key & 7)) << 4), h[0], h[1], h[2], h[3]);
                    }
                } else {                                          // 16 elements: 2 chunks
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t h[4];
                        codes4<DT>(w[2 * i], h[0], h[1]);
                        codes4<DT>(w[2 * i + 1], h[2], h[3]);
                        const int ch = 2 * c + i;
                        sts128(row + (ch >> 3) * KV<D>::HALF + (((ch & 7) ^ (key & 7)) << 4), h[0], h[1], h[2], h[3]);
                    }
                }
            }
        };
        // K warps, threads 0..7: the scales of one block of the tile each, in two steps, each a tile ahead
        // of its use, so that nobody waits for a load (fetched in one step, a table entry's use held the
        // conversions up for 700 cycles a tile)
        constexpr int kNone = -0x7fffffff - 1;
        auto entry_of = [&](int x, int t) -> int {
            const int k = key_lo(x) + t * kBN + id * kBlock;
            return is_v || id >= kBlocks || (x == 1 && nB == 0) || k >= key_hi(x) ? kNone : trow[k / kBlock];
        };
        auto scales_at = [&](int blk) {
            if (blk == kNone) return make_float2(0.f, 0.f);
            if ((unsigned)blk >= (unsigned)p.N) blk = 0;          // its fetcher reports it
            const size_t i = (size_t)blk * p.H_kv + g;
            return make_float2(p.k_scale[i], p.v_scale[i]);
        };
        uint64_t* cfull = is_v ? bars.cv_full : bars.ck_full;
        uint64_t* cempty = is_v ? bars.cv_empty : bars.ck_empty;
        uint64_t* full = is_v ? bars.v_full : bars.k_full;
        uint64_t* empty = is_v ? bars.v_empty : bars.k_empty;
        const uint32_t from = is_v ? sCV : sCK, to = is_v ? sV : sK;
        bool ok = true;
        const int tmax = max(nA, nB);
        float2 next[2] = {scales_at(entry_of(0, 0)), scales_at(entry_of(1, 0))};
        int blk[2] = {entry_of(0, 1), entry_of(1, 1)};
        for (int t = 0; ok && t < tmax; ++t) {
            for (int x = 0; ok && x < (shared ? 1 : 2); ++x) {
                const int nx = x == 0 ? nA : nB;
                if (t >= nx) continue;
                const int n = seq(x, t), s = n % NS, cs = n % NC;
                const float2 mine = next[x];
                next[x] = scales_at(blk[x]);
                blk[x] = entry_of(x, t + 2);
                const int left = key_hi(x) - key_lo(x) - t * kBN;
                ok = wait(cfull[cs], (n / NC) & 1) && (n < NS || wait(empty[s], ((n - NS) / NS) & 1));
                // the softmax warps release a slot of scales
                if (!is_v && ok && n >= kScaleSlots) ok = wait(bars.sc_empty[n % kScaleSlots], ((n - kScaleSlots) / kScaleSlots) & 1);
                if (!ok) break;
                if (id == 0) s_armed[is_v ? 1 : 0] = n + 1;
                // an infinite K scale counts as NaN (its codes of 0 have no product); looked at here, where
                // the load is back
                if (!is_v && id < kBlocks)
                    s_scale[(n % kScaleSlots) * kBlocks + id] = make_float2(isinf(mine.x) ? NAN : mine.x, mine.y);
#pragma unroll 1
                for (int key = id; key < kBN; key += 32 * C::CONV)
                    convert(from + cs * C::CTILE, to + s * TILE, key, is_v && key >= left);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (!is_v) mbar_arrive(smem_u32(&bars.sc_full[n % kScaleSlots]));
                    mbar_arrive(smem_u32(&full[s]));
                    mbar_arrive(smem_u32(&cempty[cs]));
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int D, int DT, bool PAIR>
int launch(const DecodeParams& p, int items, int max_rows, const CUtensorMap* tmk, const CUtensorMap* tmv, cudaStream_t s)
{
    using C = Cfg<D, DT, PAIR>;
    auto kern = ragged_tc_kernel<D, DT, PAIR>;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(kern, C::SMEM, done)) return PKV_ERR_CUDA;
    const int zparts = PAIR ? (p.max_parts + 1) / 2 : p.max_parts;
    const dim3 grid((max_rows * p.G + C::QT * kBM - 1) / (C::QT * kBM), p.H_kv, items * zparts);
    kern<<<grid, C::THREADS, C::SMEM, s>>>(p, *tmk, *tmv);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int DT>
int launch_any(const DecodeParams& p, int d, bool pair, int items, int max_rows, const CUtensorMap* tmk,
               const CUtensorMap* tmv, cudaStream_t s)
{
    if (d == 128) return pair ? launch<128, DT, true>(p, items, max_rows, tmk, tmv, s)
                              : launch<128, DT, false>(p, items, max_rows, tmk, tmv, s);
    return pair ? launch<64, DT, true>(p, items, max_rows, tmk, tmv, s)
                : launch<64, DT, false>(p, items, max_rows, tmk, tmv, s);
}

}  // namespace ragged

}  // namespace pkv
