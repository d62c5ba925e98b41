// kv8_attn_kernel.cuh -- sm_100a kernel of the suffix attention over an
// 8-bit prefix cache.
//
// The mathematics (per query row, x over the visible keys): with prefix
// codes k8, v8 and block scales ks, vs,
//   z_x = <q, k8_x> ks_x / sqrt(D),  p_x = exp(z_x - m),  l = sum p_x,
//   out = (1 / l) sum_x (p_x vs_x) v8_x,   lse = m + ln l,
// and suffix rows in bf16 with ks = vs = 1.  The scales multiply logits and
// weights, never the cache, so the codes go to the tensor cores as they are:
//   * tcgen05.mma kind::f8f6f4 takes A and B of 8 bits.  A query row is
//     scaled by a power of two to a largest element in (224, 448] and carried
//     as two e4m3 terms, hi = e4m3(q'), lo = e4m3(q' - hi): a bf16 value has 8
//     significant bits, two e4m3 terms hold 4 each, so every element within
//     2^-10 of the row's largest is exact and smaller ones are off by at
//     most 2^-10 in units of that scale.  A weight is carried the same way
//     (from its fp16 rounding): its error is at most 2^-8 of it and on
//     average under half of what one bf16 rounding leaves.
//   * The same MMAs over a bf16 copy of the codes would need the codes
//     widened in shared memory (three times the shared-memory traffic and
//     half the tile); two 8-bit terms run at twice the 16-bit rate, so they
//     cost the tensor pipe the same.
//   * Measured on one SM: 70 cycles for a 128 x 128 x 32 MMA with both
//     operands in shared memory (66 at N = 64, so tiles are 128 keys), 131
//     for 128 x 256 x 32 with A in tensor memory; 2.1k cycles per 128 keys.
//   * The running maximum is taken over z + log2(vs) (log2 units), that is
//     over the weights the PV product sees, with the same lazy update as the
//     bf16 kernel: a new maximum sits at 2^4 and weights may grow to 2^8.75
//     before O is rescaled, so the smallest step of the second term (2^-9) is
//     at most 2^-13 of the largest weight.  (Any of 32 rows asks for a
//     rescale: with 2^6 and 2^8 most tiles of a batch with peaked keys had one.)
//
// One CTA walks a contiguous run of a unit's key tiles: the suffix tiles (64
// rows of bf16, kind::f16), then prefix tiles of 128 codes, each 32 KB of K
// and of V in two rings of shared memory filled by TMA.  Warps 16 and 18 load
// (Q and K; V), warp 17 issues the MMAs, and warps 0-15 are two softmax groups
// that take the tiles in turn (two warps per 32 query rows, half of a tile's
// columns each).  Q lands in shared memory as bf16; the CTA with suffix tiles
// copies it to tensor memory (into the second S buffer, which is not in use
// yet), and the softmax warps rewrite it in place as the two e4m3 terms.
//
// Few query rows of an unclustered run (R = 4: at most 32, R = 2: at most 64) are laid R times over
// the 128 rows of the MMA, and copy r of a row weighs only the r-th part of
// every tile's keys (its other weights are zeros): the exponentials, which
// every one of 128 rows would otherwise do for every key, are dealt to all
// warps, at the price of joining R partial rows at the end.  (P = 30016, S =
// 10: 37 instead of 42 us; with runs under four tiles the joining costs more.)
//
// A unit's tiles may be split over any number of CTAs (and its query rows
// over blocks, so that a CTA writes fewer partial rows).  Each has its
// unnormalised O with {m, l} per row.  Few splits form a cluster whose CTAs
// read one another's partial rows from shared memory (CL); else the rows go to
// the workspace and merge_kernel, launched behind, joins them.  (Clusters alone
// would limit a unit to 16 CTAs and the grid to what clusters leave resident:
// 68 instead of 42 us at B = 2, P = 30016.)
//
// Times a call (device, Hq = 8 over Hkv = 4): one token, P = 576: 8.1 us; S = 50,
// P = 1024: 11.6 us; B = 32, masked: 28.7 us, bound by a tile's chain of logits,
// maximum, weights and product (3.9k cycles, two tiles at a time); B = 2, P =
// 30016, S = 10: 37 us, its loop at 5.2 TB/s.
#pragma once

#include "prefix_cache_kernels.cuh"

namespace dm05 {

namespace ptx {

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulate, K = 32
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same with A in tensor memory: 32 codes of a row in 8 columns.
__device__ __forceinline__ void mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of a kind::f8f6f4 MMA: e4m3 A and B (type 0), fp32
// D, A K-major, B K-major or MN-major, shape M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, bool b_mn_major)
{
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// 32 lanes x 32 bit, 8 consecutive columns per thread.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}

// 4-D tiled bulk tensor store shared -> global (rows past the tensor's end are
// not written); completion by bulk group.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, const void *smem_src, int c0, int c1, int c2, int c3)
{
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_addr(smem_src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

// a * b, lane-wise, rounded to nearest
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The largest of three (a NaN operand is passed over).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

}  // namespace ptx

namespace kv8 {

constexpr int kTile = 128;           // prefix rows of a tile
constexpr int kSufTile = 64;         // suffix rows of a tile
constexpr int kSlotBytes = 32768;    // one K or V tile of either kind
constexpr int kSlots = 2;            // of K and of V
constexpr int kSoftWarps = 16;       // two groups of eight, each two warps per TMEM lane quarter
constexpr int kLoadWarp = 16;        // Q and K
constexpr int kIssueWarp = 17;
constexpr int kLoadVWarp = 18;
constexpr int kClearWarp = 19;       // clears hidden V rows
constexpr int kThreads8 = 640;
constexpr uint32_t kTmemO8 = 0;      // O: columns [0, 256)
constexpr uint32_t kTmemS8 = 256;    // two S / P buffers of 128 columns
constexpr float kTopBits = 4.0f;     // a new maximum's weight is 2^4 ...
constexpr float kMaxBits = 8.75f;    // ... and may grow to 2^8.75 before O is rescaled (e4m3 ends at 448 = 2^8.8)
// Codes reach up to 448 where suffix values have their own size, so a suffix
// weight (bf16, any size will do) counts 2^-7 of itself in the maximum: the
// prefix weights of ordinary data then use the upper part of e4m3's range
// (error of a 900-key row 2.3e-3 -> 1.7e-3 relative, 1.65e-3 being the
// output's own rounding).
constexpr float kSuffixBits = 7.0f;

constexpr int kPartRow = kHeadDim * 4 + 16;  // a partial row: D fp32 of O, then {m, l, 0, 0}
constexpr int kMaxSplits8 = 64;

struct Smem {
    static constexpr int kQBytes = kMRows * 512;  // bf16, then two e4m3 terms in the same bytes
    static constexpr int kK = kQBytes;
    static constexpr int kV = kK + kSlots * kSlotBytes;
    static constexpr int kDataEnd = kV + kSlots * kSlotBytes;
    static constexpr int kBarQFull = 0;
    static constexpr int kBarQFree = 1;   // Q copied to tensor memory
    static constexpr int kBarQConv = 2;   // Q rewritten as two e4m3 terms
    static constexpr int kBarKFull = 3;
    static constexpr int kBarKEmpty = kBarKFull + kSlots;
    static constexpr int kBarVFull = kBarKEmpty + kSlots;
    static constexpr int kBarVEmpty = kBarVFull + kSlots;
    static constexpr int kBarSFull = kBarVEmpty + kSlots;
    static constexpr int kBarPReady = kBarSFull + 2;
    static constexpr int kBarPFree = kBarPReady + 2;
    static constexpr int kBarMmaFinal = kBarPFree + 2;
    static constexpr int kBarRow = kBarMmaFinal + 1;  // per lane quarter: its four warps
    static constexpr int kBarPair = kBarRow + 4;    // per group and lane quarter: its two warps
    static constexpr int kBarMax = kBarPair + 8;    // per lane quarter: tile t's reference maximum is known
    static constexpr int kBarOut = kBarMax + 4;     // every row staged on its way out
    static constexpr int kBarClear = kBarOut + 1;   // per V slot: its hidden rows cleared
    static constexpr int kNumBars = kBarClear + kSlots;
    static constexpr int kBarOff = kDataEnd;
    static constexpr int kTmemSlotOff = kBarOff + kNumBars * 8;
    // tile maxima [2 groups][2 halves][128], reference maxima [2][128], sums
    // [4][128], visibility limits [16 warps][64]
    static constexpr int kXchgOff = (kTmemSlotOff + 16 + 15) / 16 * 16;
    static constexpr int kEnd = kXchgOff + (4 + 2 + 4) * kMRows * 4 + kSoftWarps * 64 * 4;
    static constexpr int kAllocBytes = kEnd + 1024;
    static_assert(kDataEnd >= kMRows * kPartRow, "the rows staged on their way out");
    static_assert(kAllocBytes <= 232448, "shared memory of a CTA");
};

struct Params {
    const float *k_scale, *v_scale;  // [units, nblk]
    const int32_t *valid_len;
    const uint8_t *mask;
    __nv_bfloat16 *out;
    float *lse;
    uint32_t *err;
    uint8_t *part;                   // splits > 1: partial rows [units][splits][GS], kPartRow bytes each
    int Hkv, P, S, GS;               // GS: query rows of a unit
    int qrows;                       // query rows of a block, a multiple of 8: rows of a Q chunk in shared memory
    int row_blocks;                  // blocks of a unit
    int splits;                      // CTAs per unit and block
    int nblk, shift;
    float scale_log2;
};

// Local tile t of a CTA whose first ns tiles are suffix tiles: its S / P
// buffer and how often that buffer was used before.  Suffix tiles share
// buffer 0 (buffer 1 holds the bf16 Q while they run); prefix tiles
// alternate.
__device__ __forceinline__ int buffer_of(int t, int ns) { return t < ns ? 0 : (ns > 0 ? (t - ns + 1) & 1 : t & 1); }
__device__ __forceinline__ int uses_before(int t, int ns)
{
    if (t < ns) return t;
    const int k = t - ns;
    if (ns == 0 || (k & 1) == 0) return k >> 1;
    return ns + (k >> 1);
}

// Four values as two e4m3 terms each (four codes a word): x = fp16(v), hi =
// e4m3(x), lo = e4m3(x - hi), where x - hi is exact.
__device__ __forceinline__ void two_terms(float v0, float v1, float v2, float v3, uint32_t &hi, uint32_t &lo)
{
    asm("{\n\t.reg .b16 h0, h1, l0, l1;\n\t.reg .b32 x0, x1, b0, b1;\n\t"
        "cvt.rn.f16x2.f32 x0, %3, %2;\n\t"
        "cvt.rn.f16x2.f32 x1, %5, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 h0, x0;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 h1, x1;\n\t"
        "mov.b32 %0, {h0, h1};\n\t"
        "cvt.rn.f16x2.e4m3x2 b0, h0;\n\t"
        "cvt.rn.f16x2.e4m3x2 b1, h1;\n\t"
        "sub.rn.f16x2 x0, x0, b0;\n\t"
        "sub.rn.f16x2 x1, x1, b1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 l0, x0;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 l1, x1;\n\t"
        "mov.b32 %1, {l0, l1};\n\t}"
        : "=r"(hi), "=r"(lo)
        : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
}

// Rewrites n query rows (four chunks of 64 bf16 a row, qpitch bytes apart,
// each 128 swizzled bytes) as two e4m3 terms of the row scaled by a power of
// two to a largest element in (224, 448].  The 64 bytes of 32 bf16 values
// become their 32 first terms, then their 32 second ones.  Warp w of 16 takes
// RW rows, lanes 8 / RW parts of a row's chunk (conflict-free).  factor[row]
// becomes the row's scale times `unit`, or NaN for a row with an infinity (NaN
// elements stay NaN codes).  With COPY < 128 the result is written 128 / COPY
// times, COPY rows apart.
template <int COPY, int RW>
__device__ __forceinline__ void split_rows(uint8_t *q, int qpitch, int n, int warp, float unit, float *factor)
{
    constexpr int kParts = 8 / RW;    // lanes of a row's chunk
    constexpr int kUnits = 8 / kParts;  // 16-byte units of a lane
    const int lane = threadIdx.x & 31, part = lane & (kParts - 1);
    const int row = warp * RW + ((lane & 7) / kParts);
    if (warp * RW >= n) return;
    const bool mine = row < n;
    uint8_t *chunk = q + (lane >> 3) * qpitch + row * 128;
    auto unit16 = [&](int u) { return reinterpret_cast<uint4 *>(chunk + ((u ^ (row & 7)) << 4)); };
    __nv_bfloat162 top = __floats2bfloat162_rn(0.0f, 0.0f);
    if (mine) {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const uint4 v = *unit16(part * kUnits + u);
            const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) top = __hmax2(top, __habs2(h[e]));
        }
    }
    float amax = fmaxf(__low2float(top), __high2float(top));
#pragma unroll
    for (int m = 1; m < kParts; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
    const float s = amax < INFINITY ? cache::pow2_scale(amax) : 1.0f;
    if (mine && lane < 8 && part == 0) {
#pragma unroll
        for (int c = 0; c < 128; c += COPY) factor[c + row] = amax < INFINITY ? s * unit : __int_as_float(0x7fffffff);
    }
    const float inv = cache::pow2_inverse(s);
    constexpr int kStep = kUnits < 4 ? kUnits : 4;  // units rewritten together
#pragma unroll 1
    for (int u0 = part * kUnits; u0 < (part + 1) * kUnits; u0 += kStep) {
        uint4 v[kStep];
        uint32_t hi[2 * kStep], lo[2 * kStep];
        if (mine) {
#pragma unroll
            for (int u = 0; u < kStep; ++u) v[u] = *unit16(u0 + u);
#pragma unroll
            for (int e = 0; e < 2 * kStep; ++e) {
                const uint4 &src = v[e >> 1];
                const uint32_t w0 = (e & 1) ? src.z : src.x, w1 = (e & 1) ? src.w : src.y;
                two_terms(__uint_as_float(w0 << 16) * inv, __uint_as_float(w0 & 0xffff0000u) * inv,
                          __uint_as_float(w1 << 16) * inv, __uint_as_float(w1 & 0xffff0000u) * inv, hi[e], lo[e]);
            }
        }
        // two lanes share four units: both have read before either writes
        if (kStep < 4) __syncwarp();
        if (mine) {
            const int out = (u0 & 4) + (u0 & 3) / 2;  // unit of the first terms; the second ones' is two behind
#pragma unroll
            for (int c = 0; c < 128; c += COPY)
#pragma unroll
                for (int e = 0; e < kStep / 2; ++e) {
                    unit16(out + e)[c * 8] = make_uint4(hi[4 * e], hi[4 * e + 1], hi[4 * e + 2], hi[4 * e + 3]);
                    unit16(out + 2 + e)[c * 8] = make_uint4(lo[4 * e], lo[4 * e + 1], lo[4 * e + 2], lo[4 * e + 3]);
                }
        }
    }
}

// As few rows a warp as sixteen warps allow: the fewer, the shorter a lane's chain.
template <int COPY = 128>
__device__ __forceinline__ void split_query_rows(uint8_t *q, int qpitch, int n, int warp, float unit, float *factor)
{
    if (COPY <= 32 || n <= 32)
        split_rows<COPY, 2>(q, qpitch, n, warp, unit, factor);
    else if (COPY <= 64 || n <= 64)
        split_rows<COPY, 4>(q, qpitch, n, warp, unit, factor);
    else
        split_rows<COPY, 8>(q, qpitch, n, warp, unit, factor);
}

// Joins the `splits` partials of one row, two warps a row (thread col4 of 64
// owns four columns): with M = max_c m_c and w_c = 2^(m_c - M), out = sum_c w_c
// O_c / sum_c w_c l_c and lse = (M + log2 sum_c w_c l_c) ln 2.  A partial without
// keys (l = 0) has no weight, whatever its O holds.  part(c): the four
// columns of partial c; state(c): its {m, l}.  Latency is all there is: the
// first AHEAD partials are requested before their weights are known.
template <int AHEAD, class Part, class State>
__device__ __forceinline__ void join_partials(int splits, Part &&part, State &&state, __nv_bfloat16 *out, float *lse,
                                              size_t r, int col4)
{
    const int lane = threadIdx.x & 31;
    float4 o[AHEAD];
#pragma unroll
    for (int c = 0; c < AHEAD; ++c)
        if (c < splits) o[c] = part(c);
    float m[2], l[2], M = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = lane + 32 * h;
        float2 st = make_float2(-INFINITY, 0.0f);
        if (c < splits) st = state(c);
        m[h] = st.x;
        l[h] = st.y;
        if (l[h] != 0.0f) M = fmaxf(M, m[h]);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
    float w[2], total = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        w[h] = l[h] != 0.0f ? ptx::ex2(m[h] - M) : 0.0f;
        total = fmaf(w[h], l[h], total);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](int c, const float4 &v) {
        const float wc = __shfl_sync(0xffffffffu, c < 32 ? w[0] : w[1], c & 31);
        const bool use = wc != 0.0f;
        acc.x = fmaf(wc, use ? v.x : 0.0f, acc.x);
        acc.y = fmaf(wc, use ? v.y : 0.0f, acc.y);
        acc.z = fmaf(wc, use ? v.z : 0.0f, acc.z);
        acc.w = fmaf(wc, use ? v.w : 0.0f, acc.w);
    };
#pragma unroll
    for (int c = 0; c < AHEAD; ++c)
        if (c < splits) add(c, o[c]);
#pragma unroll 4
    for (int c = AHEAD; c < splits; ++c) add(c, part(c));
    const float inv = 1.0f / total;
    *reinterpret_cast<uint2 *>(out + r * kHeadDim + col4 * 4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (col4 == 0 && lse != nullptr) lse[r] = (M + ptx::lg2(total)) * 0.69314718055994531f;
}

template <int R, bool CL>
__global__ void __launch_bounds__(kThreads8, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kp,
                const __grid_constant__ CUtensorMap tm_vp, const __grid_constant__ CUtensorMap tm_ks,
                const __grid_constant__ CUtensorMap tm_vs, const __grid_constant__ CUtensorMap tm_out,
                const Params p)
{
    static_assert(!CL || R == 1, "copies are joined before partial rows leave");
    using L = Smem;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmemSlotOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = p.splits;
    const int cl = blockIdx.x / C, rank = blockIdx.x - cl * C;
    const int unit = cl / p.row_blocks, q0 = (cl - unit * p.row_blocks) * p.qrows;
    const int nr = min(p.qrows, p.GS - q0);  // query rows [q0, q0 + nr) of the unit
    const int b = unit / p.Hkv;
    constexpr int kCopy = kMRows / R;  // MMA rows of a copy of the query rows
    const int qpitch = R == 1 ? p.qrows * 128 : kMRows * 128;  // bytes of a 64-column chunk of Q

    if (threadIdx.x == 0) {
        ptx::mbar_init(&bars[L::kBarQFull], 1);
        ptx::mbar_init(&bars[L::kBarQFree], 1);
        ptx::mbar_init(&bars[L::kBarQConv], kSoftWarps * 32);
        for (int i = 0; i < kSlots; ++i) {
            ptx::mbar_init(&bars[L::kBarKFull + i], 1);
            ptx::mbar_init(&bars[L::kBarKEmpty + i], 1);
            ptx::mbar_init(&bars[L::kBarVFull + i], 1);
            ptx::mbar_init(&bars[L::kBarVEmpty + i], 1);
            ptx::mbar_init(&bars[L::kBarClear + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bars[L::kBarSFull + i], 1);
            ptx::mbar_init(&bars[L::kBarPReady + i], kSoftWarps / 2 * 32);
            ptx::mbar_init(&bars[L::kBarPFree + i], 1);
        }
        ptx::mbar_init(&bars[L::kBarMmaFinal], 1);
        ptx::mbar_init(&bars[L::kBarOut], kSoftWarps * 32);
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(&bars[L::kBarRow + i], 128);
            ptx::mbar_init(&bars[L::kBarPair + i], 64);
            ptx::mbar_init(&bars[L::kBarPair + 4 + i], 64);
            ptx::mbar_init(&bars[L::kBarMax + i], 64);
        }
        ptx::fence_mbar_init();
    }
    if (warp == kLoadWarp && lane == 0) {
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_kp);
        ptx::prefetch_tensormap(&tm_vp);
        ptx::prefetch_tensormap(&tm_ks);
        ptx::prefetch_tensormap(&tm_vs);
    }
    if (warp == kIssueWarp) {
        ptx::tmem_alloc(tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::griddep_launch_dependents();
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    ptx::griddep_wait();

    // Q, and the first suffix tile of the CTA that starts with it, do not
    // depend on the valid length: requested before it has been read.
    auto k_slot = [&](int t) { return smem + L::kK + (t % kSlots) * kSlotBytes; };
    auto v_slot = [&](int t) { return smem + L::kV + (t % kSlots) * kSlotBytes; };
    const bool first = rank == 0;
    uint64_t pol = 0;
    if (warp == kLoadWarp && lane == 0) {
        pol = ptx::policy_evict_first();
        // rows of the MMA past qrows read whatever lies behind: rows of their own
        ptx::mbar_arrive_expect_tx(&bars[L::kBarQFull], static_cast<uint32_t>(4 * p.qrows * 128));
        if (R == 1) {
            ptx::tma_load_4d(smem, &tm_q, &bars[L::kBarQFull], 0, q0, 0, unit);
        } else {
            for (int c = 0; c < 4; ++c) ptx::tma_load_4d(smem + c * qpitch, &tm_q, &bars[L::kBarQFull], 0, q0, c, unit);
        }
        if (first) {
            ptx::mbar_arrive_expect_tx(&bars[L::kBarKFull], kSlotBytes);
            ptx::tma_load_4d_hint(k_slot(0), &tm_ks, &bars[L::kBarKFull], 0, 0, 0, unit, pol);
        }
    }
    if (warp == kLoadVWarp && lane == 0) {
        pol = ptx::policy_evict_first();
        if (first) {
            ptx::mbar_arrive_expect_tx(&bars[L::kBarVFull], kSlotBytes);
            ptx::tma_load_4d_hint(v_slot(0), &tm_vs, &bars[L::kBarVFull], 0, 0, 0, unit, pol);
        }
    }

    const int vl = cache::clamped_len(p.valid_len, b, p.P, p.err,
                                      threadIdx.x == 0 && rank == 0 && q0 == 0 && unit % p.Hkv == 0);
    const int TS = (p.S + kSufTile - 1) / kSufTile;
    const int t_all = TS + (vl + kTile - 1) / kTile;
    const int t_begin = static_cast<int>((static_cast<long long>(t_all) * rank) / C);
    const int t_end = static_cast<int>((static_cast<long long>(t_all) * (rank + 1)) / C);
    const int T = t_end - t_begin;
    const int ns = max(0, min(TS, t_end) - t_begin);  // suffix tiles of this CTA
    // first row of local tile t and how many of its rows are in range
    auto row0_of = [&](int t) { return t < ns ? (t_begin + t) * kSufTile : (t_begin + t - TS) * kTile; };
    auto rows_of = [&](int t) { return t < ns ? min(kSufTile, p.S - row0_of(t)) : min(kTile, vl - row0_of(t)); };
    const uint8_t *mask_row = p.mask ? p.mask + static_cast<size_t>(b) * p.P : nullptr;
    // prefix tiles that may hold rows no query sees
    auto partial_at = [&](int t) { return mask_row != nullptr || rows_of(t) < kTile; };
    bool failed = false;

    if (warp == kClearWarp) {
        // ================================================== hidden V rows
        // Hidden rows, and rows past the valid length that a tile's last 32-row
        // step reads, may hold NaN codes, and 0 * NaN would poison O: they are
        // cleared once the tile has landed (by the softmax warps, after their
        // weights, this took 1k cycles a tile).  Every tile is passed on, so
        // that no phase of its barrier goes by unseen here.
        uint32_t see_next[4];
        auto load_next = [&](int t) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int c = w * 32 + lane;
                const bool in = t >= ns && t < T && c < rows_of(t);
                see_next[w] = !in ? 0u : mask_row != nullptr ? ptx::load(mask_row + row0_of(t) + c) : 1u;
            }
        };
        load_next(0);
        for (int t = 0; t < T; ++t) {
            uint32_t hidden[4];
            const int n32 = (rows_of(t) + 31) / 32;  // 32-row steps that PV reads
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                hidden[w] = __ballot_sync(0xffffffffu, see_next[w] == 0u);
                if (w >= n32 || t < ns) hidden[w] = 0u;
            }
            load_next(t + 1);
            if (!warp_wait(&bars[L::kBarVFull + t % kSlots], (t / kSlots) & 1)) {
                failed = true;
                break;
            }
            // two rows at a time, 16 lanes each
            uint8_t *vt = v_slot(t) + ((lane & 15) >> 3) * (kTile * 128) + (lane & 7) * 16;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                for (uint32_t h = hidden[w]; h != 0u;) {
                    const int r0 = __ffs(static_cast<int>(h)) - 1;
                    h &= h - 1u;
                    const int r1 = h != 0u ? __ffs(static_cast<int>(h)) - 1 : r0;
                    h &= h - 1u;
                    *reinterpret_cast<uint4 *>(vt + (w * 32 + (lane < 16 ? r0 : r1)) * 128) = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars[L::kBarClear + t % kSlots]);
        }
    } else if (warp == kLoadWarp || warp == kLoadVWarp) {
        // ================================================== TMA producers (K, V)
        if (lane == 0) {
            const bool is_v = warp == kLoadVWarp;
            uint64_t *full = &bars[is_v ? L::kBarVFull : L::kBarKFull];
            uint64_t *empty = &bars[is_v ? L::kBarVEmpty : L::kBarKEmpty];
            const CUtensorMap *ms = is_v ? &tm_vs : &tm_ks, *mp = is_v ? &tm_vp : &tm_kp;
            uint8_t *ring = smem + (is_v ? L::kV : L::kK);
            // (rank 0 has no tile when there are more CTAs than tiles: its early
            // one is then only drained)
            int issued = first ? 1 : 0;
            for (int t = issued; t < T; ++t) {
                const int s = t % kSlots, n = t / kSlots;
                if (n > 0 && !ptx::mbar_wait(&empty[s], (n - 1) & 1, kWaitLimitNs)) {
                    failed = true;
                    break;
                }
                ptx::mbar_arrive_expect_tx(&full[s], kSlotBytes);
                ptx::tma_load_4d_hint(ring + s * kSlotBytes, t < ns ? ms : mp, &full[s], 0, row0_of(t), 0, unit, pol);
                issued = t + 1;
            }
            // every copy this thread issued has landed before the CTA may exit
            if (!is_v && !ptx::mbar_wait(&bars[L::kBarQFull], 0, kWaitLimitNs)) failed = true;
            for (int t = max(0, issued - kSlots); t < issued; ++t)
                if (!ptx::mbar_wait(&full[t % kSlots], (t / kSlots) & 1, kWaitLimitNs)) failed = true;
        }
    } else if (warp == kIssueWarp) {
        // ================================================== MMA issuer
        if (lane == 0 && T > 0) {
            constexpr uint32_t id_qk = ptx::idesc_e4m3_f32(kMRows, kTile, false);
            constexpr uint32_t id_pv = ptx::idesc_e4m3_f32(kMRows, kHeadDim, true);
            constexpr uint32_t id_qk16 = ptx::idesc_bf16_f32(kMRows, kSufTile, false);
            constexpr uint32_t id_pv16 = ptx::idesc_bf16_f32(kMRows, kHeadDim, true);
            const uint64_t qdesc = ptx::sw128_desc(ptx::smem_addr(smem), 16, 1024);
            const uint64_t kdesc0 = ptx::sw128_desc(ptx::smem_addr(smem + L::kK), 16, 1024);  // K-major, 128-byte chunks
            // MN-major, column chunks apart
            const uint64_t vdesc0 = ptx::sw128_desc(ptx::smem_addr(smem + L::kV), kTile * 128, 1024);
            const uint64_t vdesc16 = ptx::sw128_desc(ptx::smem_addr(smem + L::kV), kSufTile * 128, 1024);
            auto slot_off = [&](int t) { return static_cast<uint64_t>(((t % kSlots) * kSlotBytes) >> 4); };
            auto issue_pv = [&](int u) -> bool {
                const int pb = buffer_of(u, ns), s = u % kSlots;
                if (!ptx::mbar_wait(&bars[L::kBarPReady + pb], uses_before(u, ns) & 1, kWaitLimitNs)) return false;
                if (!ptx::mbar_wait(&bars[L::kBarVFull + s], (u / kSlots) & 1, kWaitLimitNs)) return false;
                if (!ptx::mbar_wait(&bars[L::kBarClear + s], (u / kSlots) & 1, kWaitLimitNs)) return false;
                ptx::tc_fence_after_sync();
                const uint32_t a = tmem + kTmemS8 + pb * kTile;
                const int n = rows_of(u);
                if (u < ns) {
                    const uint64_t vd = vdesc16 + slot_off(u);
                    const int nk = (n + 15) / 16;
#pragma unroll
                    for (int kk = 0; kk < kSufTile / 16; ++kk) {
                        if (kk >= nk) break;
                        ptx::mma_bf16_ts(tmem + kTmemO8, a + (kk >> 1) * 32 + (kk & 1) * 8,
                                         vd + static_cast<uint64_t>((kk * 16 * 128) >> 4), id_pv16,
                                         (u > 0 || kk > 0) ? 1u : 0u);
                    }
                } else {
                    const uint64_t vd = vdesc0 + slot_off(u);
                    const int nk = (n + 31) / 32;  // 32-row steps that hold rows in range
#pragma unroll
                    for (int kk = 0; kk < kTile / 32; ++kk) {
                        if (kk >= nk) break;
                        const uint64_t vk = vd + static_cast<uint64_t>((kk * 32 * 128) >> 4);
                        const uint32_t ak = a + (kk >> 1) * 64 + (kk & 1) * 16;
                        ptx::mma_f8_ts(tmem + kTmemO8, ak, vk, id_pv, (u > 0 || kk > 0) ? 1u : 0u);
                        ptx::mma_f8_ts(tmem + kTmemO8, ak + 8, vk, id_pv, 1u);
                    }
                }
                ptx::mma_commit(&bars[L::kBarVEmpty + s]);
                ptx::mma_commit(&bars[L::kBarPFree + pb]);
                return true;
            };
            bool ok = ptx::mbar_wait(&bars[L::kBarQFull], 0, kWaitLimitNs);
            if (ok && ns > 0) {
                ptx::tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < kHeadDim / 16; ++kk)
                    ptx::tmem_cp_128x256b(tmem + kTmemS8 + kTile + kk * 8,
                                          qdesc + static_cast<uint64_t>(((kk >> 2) * qpitch + (kk & 3) * 32) >> 4));
                ptx::mma_commit(&bars[L::kBarQFree]);
            }
            for (int t = 0; t < T && ok; ++t) {
                const int sb = buffer_of(t, ns), before = uses_before(t, ns), s = t % kSlots;
                // a second suffix tile shares its predecessor's buffer: that PV goes first
                const bool pv_first = t > 0 && t < ns;
                if (pv_first && !issue_pv(t - 1)) {
                    ok = false;
                    break;
                }
                if (!ptx::mbar_wait(&bars[L::kBarKFull + s], (t / kSlots) & 1, kWaitLimitNs)) ok = false;
                // S(t) overwrites the P its buffer held: that PV must have completed
                if (ok && before > 0 && !ptx::mbar_wait(&bars[L::kBarPFree + sb], (before - 1) & 1, kWaitLimitNs)) ok = false;
                if (ok && t == ns) {
                    // the first prefix tile needs the two-term Q, and its buffer
                    // may hold the bf16 Q that the last suffix QK still reads
                    if (!ptx::mbar_wait(&bars[L::kBarQConv], 0, kWaitLimitNs)) ok = false;
                    if (ok && ns > 0 && !ptx::mbar_wait(&bars[L::kBarSFull], (ns - 1) & 1, kWaitLimitNs)) ok = false;
                }
                if (!ok) break;
                ptx::tc_fence_after_sync();
                const uint64_t kd = kdesc0 + slot_off(t);
                const uint32_t d = tmem + kTmemS8 + sb * kTile;
                if (t < ns) {
#pragma unroll
                    for (int kk = 0; kk < kHeadDim / 16; ++kk)
                        ptx::mma_bf16_ts(d, tmem + kTmemS8 + kTile + kk * 8,
                                         kd + static_cast<uint64_t>(((kk >> 2) * kSufTile * 128 + (kk & 3) * 32) >> 4),
                                         id_qk16, kk > 0 ? 1u : 0u);
                } else {
#pragma unroll
                    for (int kk = 0; kk < 16; ++kk) {
                        // 32 columns j of K against the first, then the second term of
                        // Q's: 32 of the 64 bytes that their bf16 form took
                        const int j = kk >> 1;
                        const uint32_t qo = ((j >> 1) * qpitch + (j & 1) * 64 + (kk & 1) * 32) >> 4;
                        const uint32_t ko = ((j >> 2) * (kTile * 128) + (j & 3) * 32) >> 4;
                        ptx::mma_f8_ss(d, qdesc + qo, kd + ko, id_qk, kk > 0 ? 1u : 0u);
                    }
                }
                ptx::mma_commit(&bars[L::kBarKEmpty + s]);
                ptx::mma_commit(&bars[L::kBarSFull + sb]);
                if (t > 0 && !pv_first && !issue_pv(t - 1)) ok = false;
            }
            if (ok) ok = issue_pv(T - 1);
            ptx::mma_commit(&bars[L::kBarMmaFinal]);
            if (!ptx::mbar_wait(&bars[L::kBarMmaFinal], 0, kWaitLimitNs)) ok = false;
            failed = !ok;
        }
    } else {
        // ================================================== softmax warps
        // The two groups take the tiles in turn, so that one group's waits and
        // reductions run beside the other's exponentials.  Warp w of a group:
        // lane quarter w % 4 (32 query rows), half w / 4 of its tiles' columns.
        const int q4 = warp & 3, hf = (warp >> 2) & 1, grp = warp >> 3;
        const int c4 = warp >> 2;  // column quarter of O
        const int row = q4 * 32 + lane;
        const int copy = row / kCopy, qrow = row % kCopy;
        const bool row_valid = qrow < nr;
        constexpr int kCols = 64 / R, kGroups = kCols / 16, kWords = (kCols + 31) / 32;
        const int col0 = copy * (kTile / R) + hf * kCols;  // this thread's columns of a prefix tile
        const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
        const float *ksc = p.k_scale + static_cast<size_t>(unit) * p.nblk;
        const float *vsc = p.v_scale + static_cast<size_t>(unit) * p.nblk;
        float *xmax = reinterpret_cast<float *>(smem + L::kXchgOff) + grp * 2 * kMRows;  // [2 halves][128] of this group
        float *mref = reinterpret_cast<float *>(smem + L::kXchgOff) + 4 * kMRows;        // [2 tile parity][128]
        float *xl = mref + 2 * kMRows;                                                   // [4][128]
        float *lim = xl + 4 * kMRows + warp * 64;  // this warp's columns: +inf visible, -inf hidden
        uint64_t *row_bar = &bars[L::kBarRow + q4], *pair_bar = &bars[L::kBarPair + grp * 4 + q4];
        uint64_t *max_bar = &bars[L::kBarMax + q4];
        int row_phase = 0, pair_phase = 0;
        auto pair_sync = [&]() -> bool {  // the two of this group
            ptx::mbar_arrive(pair_bar);
            return warp_wait(pair_bar, pair_phase++ & 1);
        };
        float sqs = 0.0f;  // this row's query scale * log2(e) / sqrt(D)
        if (T > 0) {
            failed = !warp_wait(&bars[L::kBarQFull], 0);
            if (!failed && ns > 0) failed = !warp_wait(&bars[L::kBarQFree], 0);
            if (!failed) {
                split_query_rows<kCopy>(smem, qpitch, nr, warp, p.scale_log2, xl);
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(&bars[L::kBarQConv]);
                failed = !warp_wait(&bars[L::kBarQConv], 0);
                if (row_valid) sqs = xl[row];
            }
        }
        float m_l = -INFINITY;  // what this thread's sum refers to
        float l = 0.0f;         // its sum of p, in units of 2^m_l
        // What tile t needs from global memory, one of the group's tiles ahead:
        // the mask bytes of this lane's columns, and (the first lanes) the scales
        // of the thread's 16-column groups (a block never ends inside one).
        uint32_t mask_next[kWords];
        float ks_next, vs_next;
        auto load_next = [&](int t) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) mask_next[w] = 1u;
            ks_next = vs_next = 1.0f;
            if (t < ns || t >= T) return;
            const int r0 = row0_of(t), n = rows_of(t);
            if (mask_row != nullptr) {
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    const int c = col0 + w * 32 + lane;
                    if (w * 32 + lane < kCols && c < n) mask_next[w] = ptx::load(mask_row + r0 + c);
                }
            }
            const int c = col0 + lane * 16;
            if (lane < kGroups && c < n) {
                ks_next = ptx::load(ksc + ((r0 + c) >> p.shift));
                vs_next = ptx::load(vsc + ((r0 + c) >> p.shift));
            }
        };
        load_next(grp);
        for (int t = grp; t < T && !failed; t += 2) {
            const int sb = buffer_of(t, ns), before = uses_before(t, ns);
            uint32_t mask_cur[kWords];
#pragma unroll
            for (int w = 0; w < kWords; ++w) mask_cur[w] = mask_next[w];
            float ks_cur = ks_next, vs_cur = vs_next;
            load_next(t + 2);
            const int n = rows_of(t);
            float ag[kGroups], bg[kGroups];
            float iv = 1.0f;
            const bool partial = t >= ns && partial_at(t);
            if (t >= ns) {
                if (partial) {
                    uint32_t vis[kWords];
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
                        const bool see = w * 32 + lane < kCols && col0 + w * 32 + lane < n && mask_cur[w] != 0u;
                        vis[w] = __ballot_sync(0xffffffffu, see);
                        lim[w * 32 + lane] = see ? INFINITY : -INFINITY;
                    }
                    __syncwarp();
                    // a group without a visible key may have any scale: it gets 1
                    const uint32_t mine = (lane & 2) ? vis[kWords - 1] : vis[0];
                    if (((lane & 1) ? mine >> 16 : mine & 0xffffu) == 0u) ks_cur = vs_cur = 1.0f;
                }
                const float lv = ptx::lg2(vs_cur);
                iv = 1.0f / vs_cur;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    ag[g] = __shfl_sync(0xffffffffu, ks_cur, g) * sqs;
                    bg[g] = __shfl_sync(0xffffffffu, lv, g);
                }
            } else if (t > 0) {
                // the second suffix tile follows the first in one buffer: its
                // barrier's earlier phase is past once the first maximum is known
                if (!warp_wait(max_bar, (t - 1) & 1)) {
                    failed = true;
                    break;
                }
            }
            if (!warp_wait(&bars[L::kBarSFull + sb], before & 1)) {
                failed = true;
                break;
            }
            ptx::tc_fence_after_sync();
            const uint32_t sbuf = tmem + lane_base + kTmemS8 + sb * kTile;
            const uint32_t scol = sbuf + (t < ns ? hf * 32 : col0);
            uint32_t raw[2][16];
            float hmax = -INFINITY;
            // the group's largest exponent (rounding is monotone)
            auto group_max = [&](const uint32_t (&x)[16], int g) {
                float a = __uint_as_float(x[0]), c = __uint_as_float(x[1]);
#pragma unroll
                for (int e = 2; e < 14; e += 4) {
                    a = ptx::max3(a, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                    c = ptx::max3(c, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                }
                a = ptx::max3(a, __uint_as_float(x[14]), __uint_as_float(x[15]));
                return fmaf(fmaxf(a, c), ag[g], bg[g]);
            };
            // min(x, -inf) is -inf for any x, NaN included
            auto hide = [&](uint32_t (&x)[16], int c0) {
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(lim + c0 + c);
                    x[c] = __float_as_uint(fminf(__uint_as_float(x[c]), f.x));
                    x[c + 1] = __float_as_uint(fminf(__uint_as_float(x[c + 1]), f.y));
                    x[c + 2] = __float_as_uint(fminf(__uint_as_float(x[c + 2]), f.z));
                    x[c + 3] = __float_as_uint(fminf(__uint_as_float(x[c + 3]), f.w));
                }
            };
            if (t < ns) {
                // suffix keys are the first copy's
                if (R == 1 || copy == 0) {
                    ptx::tmem_ld16(scol, raw[0]);
                    ptx::tmem_ld16(scol + 16, raw[1]);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        uint32_t &x = raw[c >> 4][c & 15];
                        if (hf * 32 + c >= n) x = 0xff800000u;
                        hmax = fmaxf(hmax, __uint_as_float(x));
                    }
                    hmax = fmaf(hmax, p.scale_log2, -kSuffixBits);
                }
            } else if (R == 1) {
                // 64 columns, 32 at a time: read again below (registers); hidden
                // ones are hidden in tensor memory too
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    ptx::tmem_ld16(scol + w * 32, raw[0]);
                    ptx::tmem_ld16(scol + w * 32 + 16, raw[1]);
                    ptx::tmem_ld_wait();
                    if (partial) {
                        hide(raw[0], w * 32);
                        hide(raw[1], w * 32 + 16);
                        ptx::tmem_st16(scol + w * 32, raw[0]);
                        ptx::tmem_st16(scol + w * 32 + 16, raw[1]);
                    }
                    hmax = fmaxf(hmax, fmaxf(group_max(raw[0], (w * 2) % kGroups), group_max(raw[1], (w * 2 + 1) % kGroups)));
                }
                if (partial) ptx::tmem_st_wait();
            } else {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) ptx::tmem_ld16(scol + g * 16, raw[g % 2]);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    if (partial) hide(raw[g % 2], g * 16);
                    hmax = fmaxf(hmax, group_max(raw[g % 2], g));
                }
            }
            if (!row_valid) hmax = -INFINITY;  // not a query row: never a reason to rescale
            xmax[hf * kMRows + row] = hmax;
            if (!pair_sync()) {
                failed = true;
                break;
            }
            const float tmax = fmaxf(hmax, xmax[(hf ^ 1) * kMRows + row]);
            // Tile t - 1's reference, from the other group.  The parity is exact:
            // phase t - 2 completed before this group's S(t) could exist, and
            // phase t needs this warp.
            float m_old = -INFINITY;
            if (t > 0) {
                if (!warp_wait(max_bar, (t - 1) & 1)) {
                    failed = true;
                    break;
                }
                m_old = mref[((t - 1) & 1) * kMRows + row];
            }
            // weights of this tile are 2^(z + log2 vs - m_used)
            const bool grow = t == 0 || tmax > m_old + kMaxBits;
            const float m_used = grow ? tmax - kTopBits : m_old;
            const bool rescale = grow && m_old != -INFINITY;  // (before any weight O is zero)
            if (hf == 0) mref[(t & 1) * kMRows + row] = m_used;
            ptx::mbar_arrive(max_bar);
            if (m_l != m_used) {
                if (l != 0.0f) l *= ptx::ex2(m_l - m_used);
                m_l = m_used;
            }
            const float msub = m_used == -INFINITY ? 0.0f : m_used;
            // a group's weights: their sum without the scale, and two terms each
            auto weigh = [&](const uint32_t (&x)[16], int g, uint32_t *hi, uint32_t *lo) {
                const float cg = bg[g] - msub;
                const uint64_t a2 = ptx::f32x2(ag[g], ag[g]), c2 = ptx::f32x2(cg, cg);
                uint64_t l2 = ptx::f32x2(0.0f, 0.0f);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float2 u = ptx::unpack_f32x2(ptx::fma_f32x2(
                        ptx::f32x2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), a2, c2));
                    const float2 v = ptx::unpack_f32x2(ptx::fma_f32x2(
                        ptx::f32x2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), a2, c2));
                    const float w0 = ptx::ex2(u.x), w1 = ptx::ex2(u.y), w2 = ptx::ex2(v.x), w3 = ptx::ex2(v.y);
                    l2 = ptx::add_f32x2(l2, ptx::f32x2(w0, w1));
                    l2 = ptx::add_f32x2(l2, ptx::f32x2(w2, w3));
                    two_terms(w0, w1, w2, w3, hi[e >> 2], lo[e >> 2]);
                }
                const float2 lp = ptx::unpack_f32x2(l2);
                l = fmaf(lp.x + lp.y, __shfl_sync(0xffffffffu, iv, g), l);
            };
            if (t < ns) {
                uint32_t pk[16];
                if (R == 1 || copy == 0) {
                    const uint64_t a2 = ptx::f32x2(p.scale_log2, p.scale_log2), c2 = ptx::f32x2(-msub, -msub);
                    uint64_t l2 = ptx::f32x2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float2 x = ptx::unpack_f32x2(ptx::fma_f32x2(
                            ptx::f32x2(__uint_as_float(raw[c >> 4][c & 15]), __uint_as_float(raw[c >> 4][(c & 15) + 1])), a2, c2));
                        const float p0 = ptx::ex2(x.x), p1 = ptx::ex2(x.y);
                        pk[c >> 1] = pack_bf16x2(p0, p1);
                        l2 = ptx::add_f32x2(l2, ptx::f32x2(p0, p1));
                    }
                    const float2 lp = ptx::unpack_f32x2(l2);
                    l += lp.x + lp.y;
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) pk[c] = 0u;
                }
                ptx::tmem_st16(scol, pk);
            } else if (R == 1) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    ptx::tmem_ld16(scol + w * 32, raw[0]);
                    ptx::tmem_ld16(scol + w * 32 + 16, raw[1]);
                    ptx::tmem_ld_wait();
                    uint32_t hi[8], lo[8];
                    weigh(raw[0], (w * 2) % kGroups, hi, lo);
                    weigh(raw[1], (w * 2 + 1) % kGroups, hi + 4, lo + 4);
                    // in the first 16 columns of the half for its first 32 keys, then
                    // the next 16: where only this warp's own logits were
                    ptx::tmem_st8(scol + w * 16, hi);
                    ptx::tmem_st8(scol + w * 16 + 8, lo);
                }
            } else {
                // Both halves hold their logits in registers by now.  A 32-key step
                // kk has its weights in 16 columns of its own; the other copies'
                // steps are zero in these rows.
                const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                auto step = [&](int kk) { return sbuf + (kk >> 1) * 64 + (kk & 1) * 16; };
                const int kk = col0 >> 5;
                uint32_t hi[8], lo[8];
                weigh(raw[0], 0, hi, lo);
                if (R == 2) {
                    weigh(raw[1], kGroups - 1, hi + 4, lo + 4);
                    ptx::tmem_st8(step(kk), hi);
                    ptx::tmem_st8(step(kk) + 8, lo);
                    ptx::tmem_st8(step(kk ^ 2), zero);
                    ptx::tmem_st8(step(kk ^ 2) + 8, zero);
                } else {
                    ptx::tmem_st4(step(kk) + hf * 4, hi);
                    ptx::tmem_st4(step(kk) + 8 + hf * 4, lo);
                    const int k1 = (kk + 1 + hf) & 3;
                    ptx::tmem_st8(step(k1), zero);
                    ptx::tmem_st8(step(k1) + 8, zero);
                    ptx::tmem_st8(step((kk + 3) & 3) + hf * 8, zero);
                }
            }
            if (__any_sync(0xffffffffu, rescale)) {
                // O holds the sum through PV(t-1) once that PV has completed; PV(t)
                // waits for this warp's arrival below, so the parity is exact
                if (!warp_wait(&bars[L::kBarPFree + buffer_of(t - 1, ns)], uses_before(t - 1, ns) & 1)) {
                    failed = true;
                    break;
                }
                ptx::tc_fence_after_sync();
                const float factor = rescale ? ptx::ex2(m_old - m_used) : 1.0f;  // 0 when m_old is -inf
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {
                    uint32_t o[4][16];
                    const uint32_t oc = tmem + lane_base + kTmemO8 + hf * (kHeadDim / 2) + j * 64;
#pragma unroll
                    for (int e = 0; e < 4; ++e) ptx::tmem_ld16(oc + e * 16, o[e]);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        o[e >> 4][e & 15] = __float_as_uint(__uint_as_float(o[e >> 4][e & 15]) * factor);
#pragma unroll
                    for (int e = 0; e < 4; ++e) ptx::tmem_st16(oc + e * 16, o[e]);
                }
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before_sync();
            ptx::mbar_arrive(&bars[L::kBarPReady + sb]);
        }

        // The last reference, then the last PV (its barrier's earlier phase is
        // past once the last tile's maximum is known).  Both warps of the pair
        // have published their own last tile before the other group's is awaited.
        float m_end = -INFINITY;
        if (T > 0 && !failed) {
            failed = !pair_sync() || !warp_wait(max_bar, (T - 1) & 1) ||
                     !warp_wait(&bars[L::kBarPFree + buffer_of(T - 1, ns)], uses_before(T - 1, ns) & 1);
            ptx::tc_fence_after_sync();
            m_end = mref[((T - 1) & 1) * kMRows + row];
            if (l != 0.0f && m_l != m_end) l *= ptx::ex2(m_l - m_end);
        }
        if (T == 0) {
            // Q and an early tile still land in the shared memory used below
            failed = !warp_wait(&bars[L::kBarQFull], 0) ||
                     (first && (!warp_wait(&bars[L::kBarKFull], 0) || !warp_wait(&bars[L::kBarVFull], 0)));
        }
        const bool have_o = T > 0 && !failed;
        // a row's four sums meet; only rows that leave normalised need the total before they are staged
        xl[c4 * kMRows + row] = l;
        const bool direct = R == 1 && C == 1;
        float l_row = 0.0f, inv_l = 0.0f;
        auto total = [&]() {
            if (!failed && !warp_wait(row_bar, row_phase++ & 1)) failed = true;
            l_row = (xl[row] + xl[kMRows + row]) + (xl[2 * kMRows + row] + xl[3 * kMRows + row]);
            inv_l = 1.0f / l_row;
        };
        ptx::mbar_arrive(row_bar);
        if (direct) total();
        const int srow = R == 1 ? row : copy * nr + qrow;  // staged row
        // The rows leave through shared memory in one copy: bf16 rows in the
        // layout of a Q tile, partial rows as they lie in the workspace.
        // (16-byte stores of 32 rows at a time took 5k cycles a CTA, one bulk
        // store a row 3.7k.)
        if (have_o && !failed) {
            uint32_t all[2][2][16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t oc = tmem + lane_base + kTmemO8 + c4 * (kHeadDim / 4) + j * 32;
                ptx::tmem_ld16(oc, all[j][0]);
                ptx::tmem_ld16(oc + 16, all[j][1]);
            }
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t (&o)[2][16] = all[j];
                if (!row_valid) break;
                if (direct) {
                    uint8_t *dst = smem + c4 * qpitch + row * 128;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            w[f] = pack_bf16x2(__uint_as_float(o[e >> 1][(e & 1) * 8 + 2 * f]) * inv_l,
                                               __uint_as_float(o[e >> 1][(e & 1) * 8 + 2 * f + 1]) * inv_l);
                        *reinterpret_cast<uint4 *>(dst + (((j * 4 + e) ^ (row & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(smem + srow * kPartRow + (c4 * (kHeadDim / 4) + j * 32) * 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_uint4(o[e >> 2][4 * (e & 3)], o[e >> 2][4 * (e & 3) + 1], o[e >> 2][4 * (e & 3) + 2],
                                            o[e >> 2][4 * (e & 3) + 3]);
                }
            }
        }
        if (!direct) total();
        if (c4 == 0 && row_valid) {
            if (!direct)
                *reinterpret_cast<float4 *>(smem + srow * kPartRow + kHeadDim * 4) =
                    make_float4(m_end, have_o && !failed ? l_row : 0.0f, 0.0f, 0.0f);
            else if (p.lse != nullptr && !failed)
                p.lse[static_cast<size_t>(unit) * p.GS + q0 + row] = (m_end + ptx::lg2(l_row)) * 0.69314718055994531f;
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&bars[L::kBarOut]);
        if (CL) {
            // joined below
        } else if (R > 1) {
            // the copies of a row joined as the splits are, 64 threads a row
            if (!failed && !warp_wait(&bars[L::kBarOut], 0)) failed = true;
            if (!failed) {
                const int col4 = threadIdx.x & 63;
                for (int r = threadIdx.x >> 6; r < nr; r += kSoftWarps / 2) {
                    float2 st[R];
                    float M = -INFINITY;
#pragma unroll
                    for (int c = 0; c < R; ++c) {
                        st[c] = *reinterpret_cast<const float2 *>(smem + (c * nr + r) * kPartRow + kHeadDim * 4);
                        if (st[c].y != 0.0f) M = fmaxf(M, st[c].x);
                    }
                    float total = 0.0f;
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < R; ++c) {
                        const float w = st[c].y != 0.0f ? ptx::ex2(st[c].x - M) : 0.0f;
                        const float4 v = *reinterpret_cast<const float4 *>(smem + (c * nr + r) * kPartRow + col4 * 16);
                        const bool use = w != 0.0f;
                        total = fmaf(w, st[c].y, total);
                        acc.x = fmaf(w, use ? v.x : 0.0f, acc.x);
                        acc.y = fmaf(w, use ? v.y : 0.0f, acc.y);
                        acc.z = fmaf(w, use ? v.z : 0.0f, acc.z);
                        acc.w = fmaf(w, use ? v.w : 0.0f, acc.w);
                    }
                    if (C == 1) {
                        const size_t o = static_cast<size_t>(unit) * p.GS + q0 + r;
                        const float inv = 1.0f / total;
                        *reinterpret_cast<uint2 *>(p.out + o * kHeadDim + col4 * 4) =
                            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                        if (col4 == 0 && p.lse != nullptr) p.lse[o] = (M + ptx::lg2(total)) * 0.69314718055994531f;
                    } else {
                        uint8_t *dst = p.part + ((static_cast<size_t>(unit) * C + rank) * p.GS + q0 + r) * kPartRow;
                        *reinterpret_cast<float4 *>(dst + col4 * 16) = acc;
                        if (col4 == 0) *reinterpret_cast<float4 *>(dst + kHeadDim * 4) = make_float4(M, total, 0.0f, 0.0f);
                    }
                }
            }
        } else if (threadIdx.x == 0 && !failed) {
            if (ptx::mbar_wait(&bars[L::kBarOut], 0, kWaitLimitNs)) {
                if (C == 1)
                    ptx::tma_store_4d(&tm_out, smem, 0, q0, 0, unit);
                else
                    ptx::bulk_store_s2g(p.part + ((static_cast<size_t>(unit) * C + rank) * p.GS + q0) * kPartRow,
                                        ptx::smem_addr(smem), static_cast<uint32_t>(nr * kPartRow));
                ptx::bulk_commit();
                ptx::bulk_wait_all();
                ptx::fence_proxy_async_global();
            } else {
                failed = true;
            }
        }
    }

    if (failed) atomicOr(p.err, kEwTimeout);
    __syncwarp();
    if (CL) {
        // the partial rows staged by the cluster's CTAs, dealt out row by row
        ptx::cluster_sync();
        const int col4 = threadIdx.x & 63;
        for (int r = rank + C * (threadIdx.x >> 6); r < nr; r += C * (kThreads8 / 64)) {
            const uint32_t at = ptx::smem_addr(smem) + static_cast<uint32_t>(r * kPartRow);
            join_partials<8>(
                C, [&](int c) { return ptx::ld_dsmem_f32x4(ptx::mapa(at + static_cast<uint32_t>(col4) * 16u, c)); },
                [&](int c) {
                    const float4 v = ptx::ld_dsmem_f32x4(ptx::mapa(at + static_cast<uint32_t>(kHeadDim) * 4u, c));
                    return make_float2(v.x, v.y);
                },
                p.out, p.lse, static_cast<size_t>(unit) * p.GS + q0 + r, col4);
        }
        ptx::cluster_sync();  // every peer has read this CTA's rows
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kIssueWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

struct MergeParams {
    const uint8_t *part;   // [units][splits][GS] partial rows
    __nv_bfloat16 *out;    // [units * GS, 256]
    float *lse;            // [units * GS] or nullptr
    int rows, GS, splits;  // rows: units * GS
};

// The partial rows of a split call joined behind it (AHEAD: 8 for few
// partials, 16 cost one token's call 0.3 us; 16 for more: 1.5 us less at 18).
template <int AHEAD>
__global__ void __launch_bounds__(256) merge_kernel(const MergeParams p)
{
    ptx::griddep_launch_dependents();
    const int r = blockIdx.x * 4 + (threadIdx.x >> 6), col4 = threadIdx.x & 63;
    if (r >= p.rows) return;
    const int unit = r / p.GS, row = r - unit * p.GS;
    const uint8_t *base = p.part + (static_cast<size_t>(unit) * p.splits * p.GS + row) * kPartRow;
    const size_t step = static_cast<size_t>(p.GS) * kPartRow;
    ptx::griddep_wait();
    join_partials<AHEAD>(
        p.splits, [&](int c) { return *reinterpret_cast<const float4 *>(base + c * step + col4 * 16); },
        [&](int c) { return *reinterpret_cast<const float2 *>(base + c * step + kHeadDim * 4); }, p.out, p.lse,
        static_cast<size_t>(r), col4);
}

}  // namespace kv8
}  // namespace dm05
