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
//     most 2^-10 in units of that scale.
//   * Weights have no such common unit: where one key is far above the others
//     all of those still count, and V's scales have sizes of their own.
//     kind::mxf8f6f4 gives every row of A a power-of-two scale for each 32
//     keys: a weight times its vs is carried in units in which its step's
//     largest lies in (2^7.8, 2^8.8], as e4m3 and, of what that leaves, e5m2
//     (kTermBits further down).  It is off by at most 2^-7 of itself (rms
//     1.4e-3; one bf16 rounding: 2^-8 and 1.66e-3) down to 2^-14 of the step's
//     largest, by at most a sixth down to 2^-28 of it.  (As two e4m3 terms in
//     one unit for the whole row, weights under 2^-14 of the row's largest
//     were lost: outputs off by 20 to 90 % behind a key 10 nats above the
//     rest, at 8.1, 11.6, 28.7 and 37 us below.  A third term costs 3 to 14 %;
//     V widened to bf16 in shared memory, with two bf16 terms, 4 to 27 %.)
//   * What a step's largest weight is off by goes into the sum that divides
//     the output, so that in a row of one such weight it cancels.
//   * Two blocks of 16 share a step.  One without a value (the quantiser gives
//     it scale 1) must not set its unit: where the two scales are far apart,
//     the V tile is looked at first.
//   * The same MMAs over a bf16 copy of the codes would need the codes
//     widened in shared memory (three times the shared-memory traffic); two
//     8-bit terms run at twice the 16-bit rate, so they cost the tensor pipe the same.
//   * Measured on one SM: 70 cycles for a 128 x 128 x 32 MMA with both
//     operands in shared memory (66 at N = 64, so tiles are 128 keys), 131
//     for 128 x 256 x 32 with A in tensor memory, block scales or not; 2.1k cycles per
//     128 keys.
//   * The running maximum is taken over the logits alone, lazily: O is rescaled
//     once it has grown by 2^16.
//
// One CTA walks a contiguous run of a unit's key tiles: the suffix tiles (64
// rows of bf16, kind::f16, weights as two bf16 terms), then prefix tiles of 128 codes, each 32 KB of K
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
// warps, at the price of joining R partial rows at the end.  (B = 2, P = 30016, S
// = 10: 37.6 instead of 43.3 us; with runs under four tiles the joining costs more.)
//
// A unit's tiles may be split over any number of CTAs (and its query rows
// over blocks, so that a CTA writes fewer partial rows).  Each has its
// unnormalised O with {m, l, l'} per row, l' being
// the sum that divides the output.  Few splits form a cluster whose CTAs
// read one another's partial rows from shared memory (CL); else the rows go to
// the workspace and merge_kernel, launched behind, joins them.  (Clusters alone
// would limit a unit to 16 CTAs and the grid to what clusters leave resident:
// 68 instead of 42 us at B = 2, P = 30016, before rows were copied.)
//
// Times a call (device, Hq = 8 over Hkv = 4): one token, P = 576: 8.8 us; S = 50,
// P = 1024: 12.6 us; B = 32, masked: 29.7 us, bound by a tile's chain of logits,
// maximum, weights and product (4.1k cycles, two tiles at a time); B = 2, P =
// 30016, S = 10: 37.6 us in blocks of 64, 40.0 in blocks of 16.
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

// D[tmem] (+)= (A[tmem] * scales of A) * (B[smem] * scales of B)^T, 8-bit inputs (32 codes of
// a row of A in 8 columns), K = 32, one scale for each row of A and of B.
__device__ __forceinline__ void mma_mxf8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t a_scales, uint32_t b_scales, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], [%1], %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of a kind::mxf8f6f4 MMA: A e4m3 or e5m2, B e4m3 and
// MN-major, ue8m0 scales, those of byte `byte` of the scale columns, shape M x N.
__host__ __device__ constexpr uint32_t idesc_mxf8_f32(int M, int N, bool a_e5m2, int byte)
{
    return (static_cast<uint32_t>(byte) << 4) | ((a_e5m2 ? 1u : 0u) << 7) | (1u << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24) |
           (static_cast<uint32_t>(byte) << 29);
}

// Copies 32 rows of 16 bytes (512 bytes of shared memory) to 4 columns of each quarter of
// tensor memory's lanes: the scales of 128 rows, row r's word at (r % 32) * 4 + r / 32.  Ordered
// before the tcgen05.mma operations the same thread issues later.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t saddr)
{
    // eight rows of 16 bytes lie together, 128 bytes apart; no swizzle
    const uint64_t desc = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(16 >> 4) << 16 |
                          static_cast<uint64_t>(128 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
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
constexpr int kTerms = 2;            // 8-bit terms of a prefix weight
constexpr int kTermBits = 11;        // the second one's unit is 2^-11 of the first one's
// The weights of a 32-key step take the first 16 of the 32 columns of an S / P
// buffer where its logits were, eight for each term.  Behind those of the first and of the
// second step lie the scales of all steps: of the weights (four columns a term), of V.
constexpr uint32_t kStepCols = 32;
constexpr uint32_t kScaleColsA = 16, kScaleColsB = kStepCols + 16;
// O is rescaled once a row's largest logit has grown by 2^16: weights, and sums
// of 2^24 of them times values of 2^73, stay far inside fp32's range, and their
// terms, scaled step by step, are as exact at any size.
constexpr float kGrowBits = 16.0f;

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
    // a step's largest weight [2 groups][2 halves][128] (R = 4)
    static constexpr int kStepMaxOff = kXchgOff + (4 + 2 + 4) * kMRows * 4 + kSoftWarps * 64 * 4;
    // scales of the weights [2 buffers][terms][128 rows][4 steps], and of V
    static constexpr int kCarriedOff = kStepMaxOff + 4 * kMRows * 4;  // sums as carried less the sums [4][128]
    static constexpr int kScaleOff = (kCarriedOff + 4 * kMRows * 4 + 127) / 128 * 128;
    static constexpr int kScaleBOff = kScaleOff + 2 * kTerms * 512;
    static constexpr int kZeroOff = kScaleBOff + 1024;  // per V slot: its 16-row groups without a value
    static constexpr int kEnd = kZeroOff + kSlots * 4;
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

// Whether the scales of two groups that share a step differ by more than 2^6 (a
// NaN does).  A group without a value and with a closer scale costs the other's
// weights at most six of the 14 binades that are carried to 2^-7; to look at
// every V tile before its weights costs 3 us at B = 2, P = 30016.
__device__ __forceinline__ bool scales_apart(float a, float b) { return !(a <= 64.0f * b && b <= 64.0f * a); }

// Two fp32 weights as two bf16 terms each (suffix rows): hi = bf16(w), lo =
// bf16(w - hi), off by at most 2^-16 of w, whatever its size.
__device__ __forceinline__ void bf16_terms(uint64_t w, uint32_t &hi, uint32_t &lo)
{
    const float2 f = ptx::unpack_f32x2(w);
    hi = pack_bf16x2(f.x, f.y);
    const float2 r = ptx::unpack_f32x2(ptx::fma_f32x2(
        ptx::f32x2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), ptx::f32x2(-1.0f, -1.0f), w));
    lo = pack_bf16x2(r.x, r.y);
}

// Four prefix weights, scaled to at most 448, as two 8-bit terms (four codes a
// word): x = fp16(v), e4m3(x), and the remainder x - e4m3(x), which is exact, times 2^11 in
// e5m2 (16 * 2^11 at most, and e5m2 goes 2^28 below that).
__device__ __forceinline__ void weight_terms(float v0, float v1, float v2, float v3, uint32_t &hi, uint32_t &lo)
{
    asm("{\n\t.reg .b16 h0, h1, l0, l1;\n\t.reg .b32 x0, x1, b0, b1, s;\n\t"
        "cvt.rn.f16x2.f32 x0, %3, %2;\n\t"
        "cvt.rn.f16x2.f32 x1, %5, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 h0, x0;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 h1, x1;\n\t"
        "mov.b32 %0, {h0, h1};\n\t"
        "cvt.rn.f16x2.e4m3x2 b0, h0;\n\t"
        "cvt.rn.f16x2.e4m3x2 b1, h1;\n\t"
        "sub.rn.f16x2 x0, x0, b0;\n\t"
        "sub.rn.f16x2 x1, x1, b1;\n\t"
        "mov.b32 s, 0x68006800;\n\t"
        "mul.rn.f16x2 x0, x0, s;\n\t"
        "mul.rn.f16x2 x1, x1, s;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 l0, x0;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 l1, x1;\n\t"
        "mov.b32 %1, {l0, l1};\n\t}"
        : "=r"(hi), "=r"(lo)
        : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
}

// What the terms of two such weights are off by.
__device__ __forceinline__ float2 terms_error(float v0, float v1)
{
    float hi0, hi1, lo0, lo1;
    asm("{\n\t.reg .b16 c, a, b;\n\t.reg .b32 x, y, s;\n\t"
        "cvt.rn.f16x2.f32 x, %5, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 c, x;\n\t"
        "cvt.rn.f16x2.e4m3x2 y, c;\n\t"
        "mov.b32 {a, b}, y;\n\t"
        "cvt.f32.f16 %0, a;\n\t"
        "cvt.f32.f16 %1, b;\n\t"
        "sub.rn.f16x2 x, x, y;\n\t"
        "mov.b32 s, 0x68006800;\n\t"
        "mul.rn.f16x2 x, x, s;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 c, x;\n\t"
        "cvt.rn.f16x2.e5m2x2 y, c;\n\t"
        "mov.b32 {a, b}, y;\n\t"
        "cvt.f32.f16 %2, a;\n\t"
        "cvt.f32.f16 %3, b;\n\t}"
        : "=f"(hi0), "=f"(hi1), "=f"(lo0), "=f"(lo1)
        : "f"(v0), "f"(v1));
    return make_float2(fmaf(lo0, 0x1p-11f, hi0 - v0), fmaf(lo1, 0x1p-11f, hi1 - v1));
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
// O_c / sum_c w_c l'_c and lse = (M + log2 sum_c w_c l_c) ln 2.  A partial without
// keys (l = 0) has no weight, whatever its O holds.  part(c): the four
// columns of partial c; state(c): its {m, l, l'}.  Latency is all there is: the
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
    float m[2], l[2], lc[2], M = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = lane + 32 * h;
        float4 st = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
        if (c < splits) st = state(c);
        m[h] = st.x;
        l[h] = st.y;
        lc[h] = st.z;
        if (l[h] != 0.0f) M = fmaxf(M, m[h]);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
    float w[2], total = 0.0f, carried = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        w[h] = l[h] != 0.0f ? ptx::ex2(m[h] - M) : 0.0f;
        total = fmaf(w[h], l[h], total);
        carried = fmaf(w[h], lc[h], carried);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, s);
        carried += __shfl_xor_sync(0xffffffffu, carried, s);
    }
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
    const float inv = 1.0f / carried;
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
    // scales of 1: V's, and those of the rows' steps that are another copy's
    for (int i = threadIdx.x; i < (2 * kTerms * 512 + 1024) / 4; i += kThreads8)
        reinterpret_cast<uint32_t *>(smem + L::kScaleOff)[i] = 0x7f7f7f7fu;
    ptx::fence_proxy_async_smem();
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
        float vs_next = 1.0f;  // blocks of 16: the scale of group `lane`
        const float *vsc = p.v_scale + static_cast<size_t>(unit) * p.nblk;
        auto load_next = [&](int t) {
            vs_next = 1.0f;
            if (p.shift == 4 && t >= ns && t < T && lane < kTile / 16 && lane * 16 < rows_of(t))
                vs_next = ptx::load(vsc + row0_of(t) / 16 + lane);
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
            const bool apart = __any_sync(0xffffffffu, scales_apart(vs_next, __shfl_xor_sync(0xffffffffu, vs_next, 1)));
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
            if (apart) {
                // Groups of 16 keys whose values are all zero: where a step's two
                // scales are far apart, theirs must not set the step's.
                __syncwarp();
                uint32_t zero = 0u;
                const uint8_t *vg = v_slot(t) + ((lane & 15) >> 3) * (kTile * 128) + (lane & 7) * 16 + (lane >> 4) * 128;
#pragma unroll 1
                for (int g = 0; g < 2 * n32; ++g) {
                    bool any = false;
                    for (int r = 0; r < 16 && !any; r += 2) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(vg + (g * 16 + r) * 128);
                        any = __any_sync(0xffffffffu, ((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) != 0u);
                    }
                    if (!any) zero |= 1u << g;
                }
                if (lane == 0) *reinterpret_cast<volatile uint32_t *>(smem + L::kZeroOff + t % kSlots * 4) = zero;
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
                        // the weights' first terms, then their second ones
                        const uint64_t vk = vd + static_cast<uint64_t>((kk * 16 * 128) >> 4);
                        ptx::mma_bf16_ts(tmem + kTmemO8, a + kk * 16, vk, id_pv16, (u > 0 || kk > 0) ? 1u : 0u);
                        ptx::mma_bf16_ts(tmem + kTmemO8, a + kk * 16 + 8, vk, id_pv16, 1u);
                    }
                } else {
                    const uint64_t vd = vdesc0 + slot_off(u);
                    const int nk = (n + 31) / 32;  // 32-row steps that hold rows in range
                    const uint32_t scales = ptx::smem_addr(smem + L::kScaleOff) + pb * (kTerms * 512);
#pragma unroll
                    for (int j = 0; j < kTerms; ++j) ptx::tmem_cp_scales(a + kScaleColsA + j * 4, scales + j * 512);
                    ptx::tmem_cp_scales(a + kScaleColsB, ptx::smem_addr(smem + L::kScaleBOff));
                    ptx::tmem_cp_scales(a + kScaleColsB + 4, ptx::smem_addr(smem + L::kScaleBOff) + 512);
#pragma unroll
                    for (int kk = 0; kk < kTile / 32; ++kk) {
                        if (kk >= nk) break;
                        const uint64_t vk = vd + static_cast<uint64_t>((kk * 32 * 128) >> 4);
#pragma unroll
                        for (int j = 0; j < kTerms; ++j)
                            ptx::mma_mxf8_ts(tmem + kTmemO8, a + kk * kStepCols + j * 8, vk,
                                             ptx::idesc_mxf8_f32(kMRows, kHeadDim, j > 0, kk), a + kScaleColsA + j * 4,
                                             a + kScaleColsB, (u > 0 || kk > 0 || j > 0) ? 1u : 0u);
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
        float *xstep = reinterpret_cast<float *>(smem + L::kStepMaxOff) + grp * 2 * kMRows;
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
        // What the steps' largest weights are off by, as carried, in these units: the output
        // is divided by the sum with them, so that one weight above all others cancels (its error would be
        // the whole row's, up to 2^-7); the others' differ in sign.
        float lc = 0.0f;
        // What tile t needs from global memory, one of the group's tiles ahead:
        // the mask bytes of this lane's columns, and (the first lanes) the scales
        // of the thread's 16-column groups (a block never ends inside one).
        uint32_t mask_next[kWords];
        float ks_next, vs_next;
        constexpr int kScales = R == 4 ? 2 : kGroups;
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
            // (R = 4: both groups of the step, of which this thread's is number hf)
            const int c = (R == 4 ? col0 & ~31 : col0) + lane * 16;
            if (lane < kScales && c < n) {
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
            // per 16 keys: what takes a product to log2 units; V's scale, and its logarithm
            float ag[kGroups], vg[kGroups], bg[kGroups];
            const bool partial = t >= ns && partial_at(t);
            bool apart = false;
            if (t >= ns) {
                apart = p.shift == 4 &&
                        __any_sync(0xffffffffu, scales_apart(vs_cur, __shfl_xor_sync(0xffffffffu, vs_cur, 1)));
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
                    if (((R != 4 && (lane & 1)) ? mine >> 16 : mine & 0xffffu) == 0u) ks_cur = vs_cur = 1.0f;
                }
                const float lv = ptx::lg2(vs_cur);
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int from = R == 4 ? hf : g;
                    ag[g] = __shfl_sync(0xffffffffu, ks_cur, from) * sqs;
                    vg[g] = __shfl_sync(0xffffffffu, vs_cur, from);
                    bg[g] = __shfl_sync(0xffffffffu, lv, from);
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
            if (apart) {
                // A group without a value does not count in its step's scale.  (S(t)
                // exists, so PV(t - 2) has run, and the phase of the tile before in this
                // slot is past.)
                if (!warp_wait(&bars[L::kBarClear + t % kSlots], (t / kSlots) & 1)) {
                    failed = true;
                    break;
                }
                const uint32_t zero = *reinterpret_cast<volatile uint32_t *>(smem + L::kZeroOff + t % kSlots * 4);
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    if (zero >> (col0 / 16 + g) & 1u) {
                        vg[g] = 0.0f;
                        bg[g] = -INFINITY;
                    }
                }
            }
            ptx::tc_fence_after_sync();
            const uint32_t sbuf = tmem + lane_base + kTmemS8 + sb * kTile;
            const uint32_t scol = sbuf + (t < ns ? hf * 32 : col0);
            uint32_t raw[2][16];
            float hmax = -INFINITY;
            float gmax[kGroups];  // per 16 keys: the largest product of q and k
            auto group_max = [&](const uint32_t (&x)[16], int g) {
                float a = __uint_as_float(x[0]), c = __uint_as_float(x[1]);
#pragma unroll
                for (int e = 2; e < 14; e += 4) {
                    a = ptx::max3(a, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                    c = ptx::max3(c, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                }
                a = ptx::max3(a, __uint_as_float(x[14]), __uint_as_float(x[15]));
                gmax[g] = fmaxf(a, c);
                hmax = fmaxf(hmax, gmax[g] * ag[g]);
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
                    hmax *= p.scale_log2;
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
                    group_max(raw[0], (w * 2) % kGroups);
                    group_max(raw[1], (w * 2 + 1) % kGroups);
                }
                if (partial) ptx::tmem_st_wait();
            } else {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) ptx::tmem_ld16(scol + g * 16, raw[g % 2]);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    if (partial) hide(raw[g % 2], g * 16);
                    group_max(raw[g % 2], g);
                }
            }
            if (!row_valid) hmax = -INFINITY;  // not a query row: never a reason to rescale
            xmax[hf * kMRows + row] = hmax;
            if (R == 4 && t >= ns) xstep[hf * kMRows + row] = fmaf(gmax[0], ag[0], bg[0]);  // its two halves are a step
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
            // weights of this tile are 2^(z - m_used), times vs in the product
            const bool grow = t == 0 || tmax > m_old + kGrowBits;
            const float m_used = grow ? tmax : m_old;
            const bool rescale = grow && m_old != -INFINITY;  // (before any weight O is zero)
            if (hf == 0) mref[(t & 1) * kMRows + row] = m_used;
            ptx::mbar_arrive(max_bar);
            if (m_l != m_used) {
                if (l != 0.0f) {
                    const float f = ptx::ex2(m_l - m_used);
                    l *= f;
                    lc *= f;
                }
                m_l = m_used;
            }
            const float msub = m_used == -INFINITY ? 0.0f : m_used;
            // four weights and their sum
            auto weigh4 = [&](const uint32_t (&x)[16], int e, uint64_t a2, uint64_t c2, uint64_t &l2, uint64_t &w01, uint64_t &w23) {
                const float2 u = ptx::unpack_f32x2(
                    ptx::fma_f32x2(ptx::f32x2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), a2, c2));
                const float2 v = ptx::unpack_f32x2(
                    ptx::fma_f32x2(ptx::f32x2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), a2, c2));
                w01 = ptx::f32x2(ptx::ex2(u.x), ptx::ex2(u.y));
                w23 = ptx::f32x2(ptx::ex2(v.x), ptx::ex2(v.y));
                l2 = ptx::add_f32x2(ptx::add_f32x2(l2, w01), w23);
            };
            const uint64_t c2 = ptx::f32x2(-msub, -msub);
            // 16 weights of a step, whose products with fv are at most 448
            auto weigh = [&](const uint32_t (&x)[16], float a, float fv, uint32_t (&w)[kTerms][8], int at) {
                const uint64_t a2 = ptx::f32x2(a, a), f2 = ptx::f32x2(fv, fv);
                uint64_t l2 = ptx::f32x2(0.0f, 0.0f), w01, w23;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    weigh4(x, 4 * e, a2, c2, l2, w01, w23);
                    const float2 u = ptx::unpack_f32x2(ptx::mul_f32x2(w01, f2)), v = ptx::unpack_f32x2(ptx::mul_f32x2(w23, f2));
                    weight_terms(u.x, u.y, v.x, v.y, w[0][at + e], w[1][at + e]);
                }
                const float2 lp = ptx::unpack_f32x2(l2);
                l += lp.x + lp.y;
            };
            // A step's scale 2^k, its largest weight times V's scale in (2^-0.2, 2^0.8] of it
            // (any scale for a row without weight there, or of NaN).
            auto step_bits = [&](float top) {
                return __float_as_int(fminf(fmaxf(top - msub, -100.0f), 110.0f) - 0.3f + 12582912.0f) - 0x4b400000;
            };
            auto store_scales = [&](int code, int step, auto type) {
                auto *sc = smem + L::kScaleOff + sb * (kTerms * 512) + ((row & 31) * 4 + (row >> 5)) * 4 + step;
                using T = decltype(type);
                constexpr int kOnes = sizeof(T) == 2 ? 0x101 : 1;
#pragma unroll
                for (int j = 0; j < kTerms; ++j)
                    *reinterpret_cast<T *>(sc + j * 512) = static_cast<T>(code - j * kTermBits * kOnes);
            };
            // V's scale times 2^(8 - k)  (finite: 0 * inf where the weights are that far below the reference)
            auto factor_of = [&](int g, int k) { return fminf(vg[g] * __int_as_float((127 + 8 - k) << 23), 3e38f); };
            // log2 of a group's largest weight times V's scale, but for the reference
            auto group_top = [&](int g) { return fmaf(gmax[g], ag[g], bg[g]); };
            // that weight of a step's two groups (the one that sets the step's scale) as carried, and its factor
            auto largest = [&](int g, int h, bool second, float fg, float fh, float &f) {
                f = second ? fh : fg;
                return ptx::ex2(fmaf(second ? gmax[h] : gmax[g], second ? ag[h] : ag[g], -msub)) * f;
            };
            // (a group without a value is carried as zero times zero)
            auto per_factor = [](float e, float f) { return f > 0.0f ? __fdividef(e, f) : 0.0f; };
            // the thread's steps' largest weights as carried, and their factors
            float top0 = 0.0f, top1 = 0.0f, f0 = 0.0f, f1 = 0.0f;
            if (t < ns) {
                // 16 keys: eight columns of first bf16 terms, eight of second ones
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t pk[16];
                    if (R == 1 || copy == 0) {
                        const uint64_t a2 = ptx::f32x2(p.scale_log2, p.scale_log2);
                        uint64_t l2 = ptx::f32x2(0.0f, 0.0f), w01, w23;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            weigh4(raw[g], 4 * e, a2, c2, l2, w01, w23);
                            bf16_terms(w01, pk[2 * e], pk[8 + 2 * e]);
                            bf16_terms(w23, pk[2 * e + 1], pk[8 + 2 * e + 1]);
                        }
                        const float2 lp = ptx::unpack_f32x2(l2);
                        l += lp.x + lp.y;
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; ++c) pk[c] = 0u;
                    }
                    ptx::tmem_st16(scol + g * 16, pk);
                }
            } else if (R == 1) {
                constexpr int g1 = 1 % kGroups, g2 = 2 % kGroups, g3 = 3 % kGroups;
                const float t0 = group_top(0), t1 = group_top(g1), t2 = group_top(g2), t3 = group_top(g3);
                const int k0 = step_bits(fmaxf(t0, t1)), k1 = step_bits(fmaxf(t2, t3));
                store_scales((119 + k0) | (119 + k1) << 8, hf * 2, uint16_t());
                const float fv[4] = {factor_of(0, k0), factor_of(g1, k0), factor_of(g2, k1), factor_of(g3, k1)};
                top0 = largest(0, g1, t1 > t0, fv[0], fv[1], f0);
                top1 = largest(g2, g3, t3 > t2, fv[2], fv[3], f1);
                // not unrolled: less code to fetch (stalls on it 2.3 -> 2.0 warps an issue)
                // and no spills; B = 32 30.4 -> 29.2 us
#pragma unroll 1
                for (int w = 0; w < 2; ++w) {
                    ptx::tmem_ld16(scol + w * 32, raw[0]);
                    ptx::tmem_ld16(scol + w * 32 + 16, raw[1]);
                    ptx::tmem_ld_wait();
                    uint32_t o[kTerms][8];
                    weigh(raw[0], w == 0 ? ag[0] : ag[g2], w == 0 ? fv[0] : fv[2], o, 0);
                    weigh(raw[1], w == 0 ? ag[g1] : ag[g3], w == 0 ? fv[1] : fv[3], o, 4);
#pragma unroll
                    for (int j = 0; j < kTerms; ++j) ptx::tmem_st8(scol + w * kStepCols + j * 8, o[j]);
                }
            } else {
                // Both halves hold their logits in registers by now.  The other
                // copies' steps weigh zero in these rows.
                const int own = col0 >> 5;
                constexpr int g1 = kGroups - 1;
                uint32_t o[kTerms][8];
                const float t0 = R == 2 ? group_top(0) : xstep[hf * kMRows + row];
                const float t1 = R == 2 ? group_top(g1) : xstep[(hf ^ 1) * kMRows + row];
                const int k0 = step_bits(fmaxf(t0, t1));
                if (R == 2 || hf == 0) store_scales(119 + k0, own, uint8_t());
                const float fv0 = factor_of(0, k0), fv1 = factor_of(g1, k0);
                // (R = 4: the half that holds it counts it)
                if (R == 2 || t0 > t1 || (t0 == t1 && hf == 0)) top0 = largest(0, g1, R == 2 && t1 > t0, fv0, fv1, f0);
                weigh(raw[0], ag[0], fv0, o, 0);
                if (R == 2) {
                    weigh(raw[1], ag[g1], fv1, o, 4);
#pragma unroll
                    for (int j = 0; j < kTerms; ++j) ptx::tmem_st8(sbuf + own * kStepCols + j * 8, o[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < kTerms; ++j) ptx::tmem_st4(sbuf + own * kStepCols + j * 8 + hf * 4, o[j]);
                }
                const uint32_t zero[8] = {};
#pragma unroll
                for (int i = 0; i < 4 * kTerms; ++i)
                    if (i / kTerms / (4 / R) != copy && (i & 1) == hf)
                        ptx::tmem_st8(sbuf + i / kTerms * kStepCols + i % kTerms * 8, zero);
            }
            ptx::fence_proxy_async_smem();  // the scales
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
                for (int j = 0; j < 4; ++j) {
                    uint32_t o[2][16];
                    const uint32_t oc = tmem + lane_base + kTmemO8 + hf * (kHeadDim / 2) + j * 32;
#pragma unroll
                    for (int e = 0; e < 2; ++e) ptx::tmem_ld16(oc + e * 16, o[e]);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e >> 4][e & 15] = __float_as_uint(__uint_as_float(o[e >> 4][e & 15]) * factor);
#pragma unroll
                    for (int e = 0; e < 2; ++e) ptx::tmem_st16(oc + e * 16, o[e]);
                }
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before_sync();
            ptx::mbar_arrive(&bars[L::kBarPReady + sb]);
            if (t >= ns) {
                const float2 e = terms_error(top0, top1);
                lc += per_factor(e.x, f0) + per_factor(e.y, f1);
            }
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
            if (l != 0.0f && m_l != m_end) {
                const float f = ptx::ex2(m_l - m_end);
                l *= f;
                lc *= f;
            }
        }
        if (T == 0) {
            // Q and an early tile still land in the shared memory used below
            failed = !warp_wait(&bars[L::kBarQFull], 0) ||
                     (first && (!warp_wait(&bars[L::kBarKFull], 0) || !warp_wait(&bars[L::kBarVFull], 0)));
        }
        const bool have_o = T > 0 && !failed;
        // a row's four sums meet; only rows that leave normalised need the total before they are staged
        float *xc = reinterpret_cast<float *>(smem + L::kCarriedOff);  // [4][128]
        xl[c4 * kMRows + row] = l;
        xc[c4 * kMRows + row] = lc;
        const bool direct = R == 1 && C == 1;
        float l_row = 0.0f, carried = 0.0f, inv_l = 0.0f;
        auto total = [&]() {
            if (!failed && !warp_wait(row_bar, row_phase++ & 1)) failed = true;
            l_row = (xl[row] + xl[kMRows + row]) + (xl[2 * kMRows + row] + xl[3 * kMRows + row]);
            carried = l_row + ((xc[row] + xc[kMRows + row]) + (xc[2 * kMRows + row] + xc[3 * kMRows + row]));
            inv_l = 1.0f / carried;
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
                    make_float4(m_end, have_o && !failed ? l_row : 0.0f, carried, 0.0f);
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
                    float4 st[R];
                    float M = -INFINITY;
#pragma unroll
                    for (int c = 0; c < R; ++c) {
                        st[c] = *reinterpret_cast<const float4 *>(smem + (c * nr + r) * kPartRow + kHeadDim * 4);
                        if (st[c].y != 0.0f) M = fmaxf(M, st[c].x);
                    }
                    float total = 0.0f, carried = 0.0f;
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < R; ++c) {
                        const float w = st[c].y != 0.0f ? ptx::ex2(st[c].x - M) : 0.0f;
                        const float4 v = *reinterpret_cast<const float4 *>(smem + (c * nr + r) * kPartRow + col4 * 16);
                        const bool use = w != 0.0f;
                        total = fmaf(w, st[c].y, total);
                        carried = fmaf(w, st[c].z, carried);
                        acc.x = fmaf(w, use ? v.x : 0.0f, acc.x);
                        acc.y = fmaf(w, use ? v.y : 0.0f, acc.y);
                        acc.z = fmaf(w, use ? v.z : 0.0f, acc.z);
                        acc.w = fmaf(w, use ? v.w : 0.0f, acc.w);
                    }
                    if (C == 1) {
                        const size_t o = static_cast<size_t>(unit) * p.GS + q0 + r;
                        const float inv = 1.0f / carried;
                        *reinterpret_cast<uint2 *>(p.out + o * kHeadDim + col4 * 4) =
                            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                        if (col4 == 0 && p.lse != nullptr) p.lse[o] = (M + ptx::lg2(total)) * 0.69314718055994531f;
                    } else {
                        uint8_t *dst = p.part + ((static_cast<size_t>(unit) * C + rank) * p.GS + q0 + r) * kPartRow;
                        *reinterpret_cast<float4 *>(dst + col4 * 16) = acc;
                        if (col4 == 0) *reinterpret_cast<float4 *>(dst + kHeadDim * 4) = make_float4(M, total, carried, 0.0f);
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
                    return ptx::ld_dsmem_f32x4(ptx::mapa(at + static_cast<uint32_t>(kHeadDim) * 4u, c));
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
        [&](int c) { return *reinterpret_cast<const float4 *>(base + c * step + kHeadDim * 4); }, p.out, p.lse,
        static_cast<size_t>(r), col4);
}

}  // namespace kv8
}  // namespace dm05
