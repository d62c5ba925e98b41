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
//     bf16 kernel: p vs is at most 2^8 and a new maximum sits at 2^6, so the
//     smallest step of the second term (2^-9) is 2^-15 of the largest weight.
//
// One CTA walks a contiguous run of a unit's key tiles: the suffix tiles (64
// rows of bf16, kind::f16), then prefix tiles of 128 codes.  K and V tiles
// (32 KB each) alternate in one ring of shared memory filled by TMA.  Warp
// roles, split over a cluster and the merge are those of the bf16 kernel
// (suffix_attn_kernel.cuh): warp 8 loads, warp 9 issues the MMAs, warps 0-7
// run the softmax (two warps per 32 query rows, half of a tile's columns
// each).  Q lands in shared memory as bf16; the CTA with suffix tiles copies
// it to tensor memory (into the second S buffer, which is not in use yet),
// and the softmax warps rewrite it in place as the two e4m3 terms.
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

}  // namespace ptx

namespace kv8 {

constexpr int kTile = 128;           // prefix rows of a tile
constexpr int kSufTile = 64;         // suffix rows of a tile
constexpr int kSlotBytes = 32768;    // one K or V tile of either kind
constexpr int kSlots = 4;
constexpr uint32_t kTmemO8 = 0;      // O: columns [0, 256)
constexpr uint32_t kTmemS8 = 256;    // two S / P buffers of 128 columns
constexpr float kTopBits = 6.0f;     // a new maximum's weight is 2^6 ...
constexpr float kMaxBits = 8.0f;     // ... and may grow to 2^8 before O is rescaled (e4m3 ends at 448)
// Codes reach up to 448 where suffix values have their own size, so a suffix
// weight (bf16, any size will do) counts 2^-7 of itself in the maximum: the
// prefix weights of ordinary data then use the upper part of e4m3's range
// (error of a 900-key row 2.3e-3 -> 1.7e-3 relative, 1.65e-3 being the
// output's own rounding).
constexpr float kSuffixBits = 7.0f;

struct Smem {
    static constexpr int kQChunkBytes = kMRows * 128;
    static constexpr int kQBytes = 4 * kQChunkBytes;  // bf16, then [hi: 2 chunks][lo: 2 chunks] of e4m3
    static constexpr int kRing = kQBytes;
    static constexpr int kDataEnd = kRing + kSlots * kSlotBytes;
    static constexpr int kBarQFull = 0;
    static constexpr int kBarQFree = 1;   // Q copied to tensor memory
    static constexpr int kBarQConv = 2;   // Q rewritten as two e4m3 terms
    static constexpr int kBarFull = 3;
    static constexpr int kBarEmpty = kBarFull + kSlots;
    static constexpr int kBarSFull = kBarEmpty + kSlots;
    static constexpr int kBarPReady = kBarSFull + 2;
    static constexpr int kBarPFree = kBarPReady + 2;
    static constexpr int kBarMmaFinal = kBarPFree + 2;
    static constexpr int kBarMerge = kBarMmaFinal + 1;
    static constexpr int kBarPair = kBarMerge + 1;
    static constexpr int kNumBars = kBarPair + 4;
    static constexpr int kBarOff = kDataEnd;
    static constexpr int kTmemSlotOff = kBarOff + kNumBars * 8;
    static constexpr int kXchgOff = (kTmemSlotOff + 16 + 15) / 16 * 16;  // row maxima [2][2][128], sums [2][128]
    static constexpr int kEnd = kXchgOff + (4 + 2) * kMRows * 4;
    static constexpr int kAllocBytes = kEnd + 1024;
    static constexpr int kStageStride = kHeadDim * 4 + 16;  // a partial row: D fp32 of O, then {m, l, l, 0}
    static_assert(kDataEnd >= (kMRows + 16) * kStageStride, "the merge receives at most 144 rows");
    static_assert(6 * kMRows * 4 >= kMRows * 8, "the merge keeps one output row index per row in the exchange area");
};

struct Params {
    const float *k_scale, *v_scale;  // [units, nblk]
    const int32_t *valid_len;
    const uint8_t *mask;
    __nv_bfloat16 *out;
    float *lse;
    uint32_t *err;
    float *part;                     // splits > 1: partial rows, as in the bf16 kernel
    int Hkv, P, S, GS, G;
    int row_blocks, SQ, splits;
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

// Two fp32 values as two e4m3 terms each: hi | lo << 16 (two codes each).
__device__ __forceinline__ uint32_t two_terms(float a, float b)
{
    const __half2 x = __floats2half2_rn(a, b);
    const __nv_fp8x2_storage_t hi = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
    const __half2 back = __half2(__nv_cvt_fp8x2_to_halfraw2(hi, __NV_E4M3));
    const __nv_fp8x2_storage_t lo =
        __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hsub2(x, back)), __NV_SATFINITE, __NV_E4M3);
    return static_cast<uint32_t>(hi) | static_cast<uint32_t>(lo) << 16;
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kp,
                const __grid_constant__ CUtensorMap tm_vp, const __grid_constant__ CUtensorMap tm_ks,
                const __grid_constant__ CUtensorMap tm_vs, const Params p)
{
    using L = Smem;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmemSlotOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = p.splits;
    const int cl = blockIdx.x / C, rank = blockIdx.x - cl * C;
    const int unit = cl / p.row_blocks, rb = cl - unit * p.row_blocks;
    const int b = unit / p.Hkv;
    // row m of the MMA <-> head m / rph, query q0 + m % rph; compact row = head * nq + m % rph
    const int q0 = rb * p.SQ;
    const int nq = min(p.SQ, p.S - q0);
    const int rph = p.row_blocks == 1 ? p.S : (p.SQ + 7) / 8 * 8;
    const int NR = p.G * nq;
    const size_t unit_row0 = static_cast<size_t>(unit) * p.GS;

    if (threadIdx.x == 0) {
        ptx::mbar_init(&bars[L::kBarQFull], 1);
        ptx::mbar_init(&bars[L::kBarQFree], 1);
        ptx::mbar_init(&bars[L::kBarQConv], kSoftmaxWarps * 32);
        for (int s = 0; s < kSlots; ++s) {
            ptx::mbar_init(&bars[L::kBarFull + s], 1);
            ptx::mbar_init(&bars[L::kBarEmpty + s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bars[L::kBarSFull + i], 1);
            ptx::mbar_init(&bars[L::kBarPReady + i], kSoftmaxWarps * 32);
            ptx::mbar_init(&bars[L::kBarPFree + i], 1);
        }
        ptx::mbar_init(&bars[L::kBarMmaFinal], 1);
        ptx::mbar_init(&bars[L::kBarMerge], 1);
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&bars[L::kBarPair + i], 64);
        ptx::fence_mbar_init();
    }
    if (warp == kProducerWarp && lane == 0) {
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_kp);
        ptx::prefetch_tensormap(&tm_vp);
        ptx::prefetch_tensormap(&tm_ks);
        ptx::prefetch_tensormap(&tm_vs);
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::griddep_launch_dependents();
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    ptx::griddep_wait();

    const int vl = cache::clamped_len(p.valid_len, b, p.P, p.err,
                                      threadIdx.x == 0 && rank == 0 && rb == 0 && unit % p.Hkv == 0);
    const int TS = (p.S + kSufTile - 1) / kSufTile;
    const int t_all = TS + (vl + kTile - 1) / kTile;
    const int t_begin = static_cast<int>((static_cast<long long>(t_all) * rank) / C);
    const int t_end = static_cast<int>((static_cast<long long>(t_all) * (rank + 1)) / C);
    const int T = t_end - t_begin;
    const int ns = max(0, min(TS, t_end) - t_begin);  // suffix tiles of this CTA
    // first row of local tile t and how many of its rows are in range
    auto row0_of = [&](int t) { return t < ns ? (t_begin + t) * kSufTile : (t_begin + t - TS) * kTile; };
    auto rows_of = [&](int t) { return t < ns ? min(kSufTile, p.S - row0_of(t)) : min(kTile, vl - row0_of(t)); };
    auto slot_at = [&](int i) { return smem + L::kRing + (i % kSlots) * kSlotBytes; };  // item 2t: K of tile t, 2t+1: V
    bool failed = false;

    if (warp == kProducerWarp) {
        // ================================================== TMA producer
        if (lane == 0 && T > 0) {
            const uint64_t pol = ptx::policy_evict_first();
            if (p.row_blocks == 1) {
                ptx::mbar_arrive_expect_tx(&bars[L::kBarQFull], L::kQBytes);
                ptx::tma_load_4d(smem, &tm_q, &bars[L::kBarQFull], 0, 0, 0, unit);
            } else {
                ptx::mbar_arrive_expect_tx(&bars[L::kBarQFull], static_cast<uint32_t>(p.G * kChunks * p.SQ * 128));
                for (int h = 0; h < p.G; ++h)
                    for (int c = 0; c < kChunks; ++c)
                        ptx::tma_load_3d(smem + c * L::kQChunkBytes + h * rph * 128, &tm_q, &bars[L::kBarQFull],
                                         c * kChunkElems, h * p.S + q0, unit);
            }
            int issued = 0;
            for (int i = 0; i < 2 * T; ++i) {
                const int s = i % kSlots, n = i / kSlots;
                if (n > 0 && !ptx::mbar_wait(&bars[L::kBarEmpty + s], (n - 1) & 1, kWaitLimitNs)) {
                    failed = true;
                    break;
                }
                const int t = i >> 1;
                const CUtensorMap *map = t < ns ? ((i & 1) ? &tm_vs : &tm_ks) : ((i & 1) ? &tm_vp : &tm_kp);
                ptx::mbar_arrive_expect_tx(&bars[L::kBarFull + s], kSlotBytes);
                ptx::tma_load_4d_hint(slot_at(i), map, &bars[L::kBarFull + s], 0, row0_of(t), 0, unit, pol);
                issued = i + 1;
            }
            // every copy this thread issued has landed before the CTA may exit
            if (!ptx::mbar_wait(&bars[L::kBarQFull], 0, kWaitLimitNs)) failed = true;
            for (int i = max(0, issued - kSlots); i < issued; ++i)
                if (!ptx::mbar_wait(&bars[L::kBarFull + i % kSlots], (i / kSlots) & 1, kWaitLimitNs)) failed = true;
        }
    } else if (warp == kMmaWarp) {
        // ================================================== MMA issuer
        if (lane == 0 && T > 0) {
            constexpr uint32_t id_qk = ptx::idesc_e4m3_f32(kMRows, kTile, false);
            constexpr uint32_t id_pv = ptx::idesc_e4m3_f32(kMRows, kHeadDim, true);
            constexpr uint32_t id_qk16 = ptx::idesc_bf16_f32(kMRows, kSufTile, false);
            constexpr uint32_t id_pv16 = ptx::idesc_bf16_f32(kMRows, kHeadDim, true);
            const uint32_t ring = ptx::smem_addr(smem + L::kRing);
            const uint64_t qdesc = ptx::sw128_desc(ptx::smem_addr(smem), 16, 1024);
            const uint64_t kdesc0 = ptx::sw128_desc(ring, 16, 1024);                // K-major, 128-byte chunks
            const uint64_t vdesc0 = ptx::sw128_desc(ring, kTile * 128, 1024);       // MN-major, column chunks apart
            const uint64_t vdesc16 = ptx::sw128_desc(ring, kSufTile * 128, 1024);
            auto slot_off = [&](int i) { return static_cast<uint64_t>(((i % kSlots) * kSlotBytes) >> 4); };
            auto issue_pv = [&](int u) -> bool {
                const int pb = buffer_of(u, ns), i = 2 * u + 1;
                if (!ptx::mbar_wait(&bars[L::kBarPReady + pb], uses_before(u, ns) & 1, kWaitLimitNs)) return false;
                if (!ptx::mbar_wait(&bars[L::kBarFull + i % kSlots], (i / kSlots) & 1, kWaitLimitNs)) return false;
                ptx::tc_fence_after_sync();
                const uint32_t a = tmem + kTmemS8 + pb * kTile;
                const int n = rows_of(u);
                if (u < ns) {
                    const uint64_t vd = vdesc16 + slot_off(i);
                    const int nk = (n + 15) / 16;
#pragma unroll
                    for (int kk = 0; kk < kSufTile / 16; ++kk) {
                        if (kk >= nk) break;
                        ptx::mma_bf16_ts(tmem + kTmemO8, a + kk * 8, vd + static_cast<uint64_t>((kk * 16 * 128) >> 4),
                                         id_pv16, (u > 0 || kk > 0) ? 1u : 0u);
                    }
                } else {
                    const uint64_t vd = vdesc0 + slot_off(i);
                    const int nk = (n + 31) / 32;  // 32-row steps that hold rows in range
#pragma unroll
                    for (int kk = 0; kk < kTile / 32; ++kk) {
                        if (kk >= nk) break;
                        const uint64_t vk = vd + static_cast<uint64_t>((kk * 32 * 128) >> 4);
                        ptx::mma_f8_ts(tmem + kTmemO8, a + kk * 8, vk, id_pv, (u > 0 || kk > 0) ? 1u : 0u);
                        ptx::mma_f8_ts(tmem + kTmemO8, a + 32 + kk * 8, vk, id_pv, 1u);
                    }
                }
                ptx::mma_commit(&bars[L::kBarEmpty + i % kSlots]);
                ptx::mma_commit(&bars[L::kBarPFree + pb]);
                return true;
            };
            bool ok = ptx::mbar_wait(&bars[L::kBarQFull], 0, kWaitLimitNs);
            if (ok && ns > 0) {
                ptx::tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < kHeadDim / 16; ++kk)
                    ptx::tmem_cp_128x256b(tmem + kTmemS8 + kTile + kk * 8,
                                          qdesc + static_cast<uint64_t>(((kk >> 2) * L::kQChunkBytes + (kk & 3) * 32) >> 4));
                ptx::mma_commit(&bars[L::kBarQFree]);
            }
            for (int t = 0; t < T && ok; ++t) {
                const int sb = buffer_of(t, ns), before = uses_before(t, ns), i = 2 * t;
                // a second suffix tile shares its predecessor's buffer: that PV goes first
                const bool pv_first = t > 0 && t < ns;
                if (pv_first && !issue_pv(t - 1)) {
                    ok = false;
                    break;
                }
                if (!ptx::mbar_wait(&bars[L::kBarFull + i % kSlots], (i / kSlots) & 1, kWaitLimitNs)) ok = false;
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
                const uint64_t kd = kdesc0 + slot_off(i);
                const uint32_t d = tmem + kTmemS8 + sb * kTile;
                if (t < ns) {
#pragma unroll
                    for (int kk = 0; kk < kHeadDim / 16; ++kk)
                        ptx::mma_bf16_ts(d, tmem + kTmemS8 + kTile + kk * 8,
                                         kd + static_cast<uint64_t>(((kk >> 2) * kSufTile * 128 + (kk & 3) * 32) >> 4),
                                         id_qk16, kk > 0 ? 1u : 0u);
                } else {
#pragma unroll
                    for (int kk = 0; kk < 16; ++kk) {  // eight 32-column steps of hi, then of lo
                        const uint32_t off = (((kk & 7) >> 2) * 16384 + (kk & 3) * 32) >> 4;
                        ptx::mma_f8_ss(d, qdesc + off + static_cast<uint64_t>(kk < 8 ? 0 : (2 * L::kQChunkBytes) >> 4),
                                       kd + off, id_qk, kk > 0 ? 1u : 0u);
                    }
                }
                ptx::mma_commit(&bars[L::kBarEmpty + i % kSlots]);
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
        const int q4 = warp & 3, hf = warp >> 2;
        const int row = q4 * 32 + lane;
        const int row_h = row / rph, row_j = row - row_h * rph;
        const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
        const uint8_t *mask_row = p.mask ? p.mask + static_cast<size_t>(b) * p.P : nullptr;
        const float *ksc = p.k_scale + static_cast<size_t>(unit) * p.nblk;
        const float *vsc = p.v_scale + static_cast<size_t>(unit) * p.nblk;
        float *xmax = reinterpret_cast<float *>(smem + L::kXchgOff);  // [2 tile parity][2 half][128 rows]
        float *xl = xmax + 2 * 2 * kMRows;                            // [2 half][128]
        uint64_t *pair_bar = &bars[L::kBarPair + q4];
        int pair_phase = 0;
        auto pair_sync = [&]() -> bool {
            ptx::mbar_arrive(pair_bar);
            const bool ok = warp_wait(pair_bar, pair_phase & 1);
            ++pair_phase;
            return ok;
        };
        float sqs = 0.0f;  // this row's query scale * log2(e) / sqrt(D)
        if (T > 0) {
            // ---- Q as two e4m3 terms, in place: this thread's half row (128 values)
            failed = !warp_wait(&bars[L::kBarQFull], 0);
            if (!failed && ns > 0) failed = !warp_wait(&bars[L::kBarQFree], 0);
            uint4 v[16];
            uint32_t top = 0u;
            uint8_t *qrow = smem + row * 128;
            const uint32_t sw = static_cast<uint32_t>(row & 7);
            if (!failed) {
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    v[u] = *reinterpret_cast<const uint4 *>(qrow + (2 * hf + (u >> 3)) * L::kQChunkBytes +
                                                            (((u & 7) ^ sw) << 4));
                    top = __vmaxu2(top, v[u].x & 0x7fff7fffu);
                    top = __vmaxu2(top, v[u].y & 0x7fff7fffu);
                    top = __vmaxu2(top, v[u].z & 0x7fff7fffu);
                    top = __vmaxu2(top, v[u].w & 0x7fff7fffu);
                }
                xmax[hf * kMRows + row] = __uint_as_float(max(top & 0xffffu, top >> 16) << 16);
                failed = !pair_sync();
            }
            if (!failed) {
                // magnitudes order like their bits; a row with a non-finite element becomes NaN
                const float amax = __uint_as_float(max(__float_as_uint(xmax[row]), __float_as_uint(xmax[kMRows + row])));
                const float s = amax < INFINITY ? cache::pow2_scale(amax) : 1.0f;
                const float inv = cache::pow2_inverse(s);
                sqs = amax < INFINITY ? s * p.scale_log2 : __int_as_float(0x7fffffff);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4 &src = v[2 * u + (e >> 1)];
                        const uint32_t w0 = (e & 1) ? src.z : src.x, w1 = (e & 1) ? src.w : src.y;
                        const uint32_t a = two_terms(__uint_as_float(w0 << 16) * inv, __uint_as_float(w0 & 0xffff0000u) * inv);
                        const uint32_t c = two_terms(__uint_as_float(w1 << 16) * inv, __uint_as_float(w1 & 0xffff0000u) * inv);
                        hi[e] = __byte_perm(a, c, 0x5410);
                        lo[e] = __byte_perm(a, c, 0x7632);
                    }
                    uint8_t *dst = qrow + hf * L::kQChunkBytes + ((static_cast<uint32_t>(u) ^ sw) << 4);
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(dst + 2 * L::kQChunkBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(&bars[L::kBarQConv]);
                // xmax is read above and written again by tile 0: both halves are past it
                failed = !pair_sync();
            }
        }
        float m_used = -INFINITY;  // weights are 2^(z + log2 vs - m_used)
        float l = 0.0f;            // this half's sum of p in the same units
        // What tile t needs from global memory, one tile ahead: the mask bytes
        // of this lane's columns, and (lanes 0-3) the scales of the half's
        // four 16-column groups (a block never ends inside a group).
        uint32_t mask_next[2];
        float ks_next = 1.0f, vs_next = 1.0f;
        auto load_next = [&](int t) {
            mask_next[0] = mask_next[1] = 1u;
            ks_next = vs_next = 1.0f;
            if (t < ns || t >= T) return;
            const int r0 = row0_of(t), n = rows_of(t);
            if (mask_row != nullptr) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int c = hf * 64 + w * 32 + lane;
                    if (c < n) mask_next[w] = __ldg(mask_row + r0 + c);
                }
            }
            const int c = hf * 64 + lane * 16;
            if (lane < 4 && c < n) {
                ks_next = __ldg(ksc + ((r0 + c) >> p.shift));
                vs_next = __ldg(vsc + ((r0 + c) >> p.shift));
            }
        };
        load_next(0);
        for (int t = 0; t < T && !failed; ++t) {
            const int sb = buffer_of(t, ns), before = uses_before(t, ns);
            const uint32_t mask_cur[2] = {mask_next[0], mask_next[1]};
            float ks_cur = ks_next, vs_cur = vs_next;
            load_next(t + 1);
            if (!warp_wait(&bars[L::kBarSFull + sb], before & 1)) {
                failed = true;
                break;
            }
            ptx::tc_fence_after_sync();
            const uint32_t scol = tmem + lane_base + kTmemS8 + sb * kTile;
            const int n = rows_of(t);
            float hmax;
            float s[64];
            float ag[4], bg[4], ig[4];
            uint32_t vis[2] = {0xffffffffu, 0xffffffffu};
            if (t < ns) {
                uint32_t raw[2][16];
                ptx::tmem_ld16(scol + hf * 32, raw[0]);
                ptx::tmem_ld16(scol + hf * 32 + 16, raw[1]);
                ptx::tmem_ld_wait();
                float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    s[c] = hf * 32 + c < n ? __uint_as_float(raw[c >> 4][c & 15]) : -INFINITY;
                    m2[c & 1] = fmaxf(m2[c & 1], s[c]);
                }
                hmax = fmaf(fmaxf(m2[0], m2[1]), p.scale_log2, -kSuffixBits);
            } else {
                uint32_t raw[4][16];
#pragma unroll
                for (int j = 0; j < 4; ++j) ptx::tmem_ld16(scol + hf * 64 + j * 16, raw[j]);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 64; ++c) s[c] = __uint_as_float(raw[c >> 4][c & 15]);
                if (n < kTile || mask_row != nullptr) {
#pragma unroll
                    for (int w = 0; w < 2; ++w)
                        vis[w] = __ballot_sync(0xffffffffu, hf * 64 + w * 32 + lane < n && mask_cur[w] != 0u);
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (!((vis[c >> 5] >> (c & 31)) & 1u)) s[c] = -INFINITY;
                    // a group without a visible key may have any scale: it gets 1
                    const uint32_t mine = (lane & 2) ? vis[1] : vis[0];
                    if (((lane & 1) ? mine >> 16 : mine & 0xffffu) == 0u) ks_cur = vs_cur = 1.0f;
                }
                const float lv = ptx::lg2(vs_cur), iv = 1.0f / vs_cur;
                hmax = -INFINITY;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    ag[g] = __shfl_sync(0xffffffffu, ks_cur, g) * sqs;
                    bg[g] = __shfl_sync(0xffffffffu, lv, g);
                    ig[g] = __shfl_sync(0xffffffffu, iv, g);
                    float a = s[g * 16], c = s[g * 16 + 1];
#pragma unroll
                    for (int e = 2; e < 16; e += 2) {
                        a = fmaxf(a, s[g * 16 + e]);
                        c = fmaxf(c, s[g * 16 + e + 1]);
                    }
                    // rounding is monotone: this is the largest of the group's exponents
                    hmax = fmaxf(hmax, fmaf(fmaxf(a, c), ag[g], bg[g]));
                }
            }
            xmax[((t & 1) * 2 + hf) * kMRows + row] = hmax;
            if (!pair_sync()) {
                failed = true;
                break;
            }
            const float tmax = fmaxf(hmax, xmax[((t & 1) * 2 + (hf ^ 1)) * kMRows + row]);
            float factor = 1.0f;
            bool rescale = false;
            if (t == 0) {
                m_used = tmax - kTopBits;
            } else if (tmax > m_used + kMaxBits) {
                factor = ptx::ex2(m_used - (tmax - kTopBits));  // 0 when m_used is -inf
                rescale = true;
                l *= factor;
                m_used = tmax - kTopBits;
            }
            const float msub = m_used == -INFINITY ? 0.0f : m_used;
            if (t < ns) {
                const uint64_t a2 = ptx::f32x2(p.scale_log2, p.scale_log2), c2 = ptx::f32x2(-msub, -msub);
                uint64_t l2 = ptx::f32x2(0.0f, 0.0f);
                uint32_t pk[16];
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float2 x = ptx::unpack_f32x2(ptx::fma_f32x2(ptx::f32x2(s[c], s[c + 1]), a2, c2));
                    const float p0 = ptx::ex2(x.x), p1 = ptx::ex2(x.y);
                    pk[c >> 1] = pack_bf16x2(p0, p1);
                    l2 = ptx::add_f32x2(l2, ptx::f32x2(p0, p1));
                }
                const float2 lp = ptx::unpack_f32x2(l2);
                l += lp.x + lp.y;
                ptx::tmem_st16(scol + hf * 16, pk);
            } else {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float cg = bg[g] - msub;
                    const uint64_t a2 = ptx::f32x2(ag[g], ag[g]), c2 = ptx::f32x2(cg, cg);
                    uint64_t l2 = ptx::f32x2(0.0f, 0.0f);
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const int c = g * 16 + e;
                        const float2 x = ptx::unpack_f32x2(ptx::fma_f32x2(ptx::f32x2(s[c], s[c + 1]), a2, c2));
                        const float2 y = ptx::unpack_f32x2(ptx::fma_f32x2(ptx::f32x2(s[c + 2], s[c + 3]), a2, c2));
                        const float w0 = ptx::ex2(x.x), w1 = ptx::ex2(x.y), w2 = ptx::ex2(y.x), w3 = ptx::ex2(y.y);
                        l2 = ptx::add_f32x2(l2, ptx::f32x2(w0, w1));
                        l2 = ptx::add_f32x2(l2, ptx::f32x2(w2, w3));
                        const uint32_t u = two_terms(w0, w1), v = two_terms(w2, w3);
                        hi[c >> 2] = __byte_perm(u, v, 0x5410);
                        lo[c >> 2] = __byte_perm(u, v, 0x7632);
                    }
                    const float2 lp = ptx::unpack_f32x2(l2);
                    l = fmaf(lp.x + lp.y, ig[g], l);  // the weights without their scale
                }
                ptx::tmem_st16(scol + hf * 16, hi);
                ptx::tmem_st16(scol + 32 + hf * 16, lo);
            }
            if (t > 0 && __any_sync(0xffffffffu, rescale)) {
                // O holds the sum through PV(t-1) once that PV has completed; PV(t)
                // waits for this warp's arrival below, so the parity is exact
                if (!warp_wait(&bars[L::kBarPFree + buffer_of(t - 1, ns)], uses_before(t - 1, ns) & 1)) {
                    failed = true;
                    break;
                }
                ptx::tc_fence_after_sync();
#pragma unroll 1
                for (int j = 0; j < kHeadDim / 32; ++j) {
                    uint32_t o[16];
                    const uint32_t oc = tmem + lane_base + kTmemO8 + hf * (kHeadDim / 2) + j * 16;
                    ptx::tmem_ld16(oc, o);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
                    ptx::tmem_st16(oc, o);
                }
            }
            ptx::tmem_st_wait();
            if (t >= ns) {
                // hidden rows, and rows past the valid length that the last
                // 32-row step reads, may hold NaN codes, and 0 * NaN would
                // poison O: they are cleared.  The half's four warps take them in turn.
                const int left = (n + 31) / 32 * 32 - hf * 64;  // columns of this half that PV reads
                uint64_t hidden = ~(static_cast<uint64_t>(vis[1]) << 32 | vis[0]);
                hidden &= left <= 0 ? 0ull : left >= 64 ? ~0ull : (1ull << left) - 1ull;
                if (hidden != 0ull) {
                    const int i = 2 * t + 1;
                    if (!warp_wait(&bars[L::kBarFull + i % kSlots], (i / kSlots) & 1)) {
                        failed = true;
                        break;
                    }
                    uint8_t *vt = slot_at(i) + hf * 64 * 128;
                    for (int k = 0; hidden != 0ull; ++k, hidden &= hidden - 1ull) {
                        const int r = __ffsll(static_cast<long long>(hidden)) - 1;
                        if ((k & 3) == q4 && lane < 16)
                            *reinterpret_cast<uint4 *>(vt + (lane >> 3) * (kTile * 128) + r * 128 + (lane & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    ptx::fence_proxy_async_smem();
                }
            }
            ptx::tc_fence_before_sync();
            ptx::mbar_arrive(&bars[L::kBarPReady + sb]);
        }

        const bool have_o = T > 0 && !failed;
        if (have_o) {
            if (!warp_wait(&bars[L::kBarPFree + buffer_of(T - 1, ns)], uses_before(T - 1, ns) & 1)) failed = true;
            ptx::tc_fence_after_sync();
        }
        xl[hf * kMRows + row] = l;
        if (!failed && !pair_sync()) failed = true;
        const float l_row = l + xl[(hf ^ 1) * kMRows + row];
        const bool row_valid = row_h < p.G && row_j < nq;
        const int row_k = row_h * nq + row_j;
        const size_t out_row = unit_row0 + static_cast<size_t>(row_h) * p.S + q0 + row_j;
        const float inv_l = C == 1 ? 1.0f / l_row : 1.0f;
        uint8_t *srow = smem + row * L::kStageStride;
        if (have_o && !failed) {
#pragma unroll 1
            for (int j = 0; j < kHeadDim / 64; ++j) {
                uint32_t o[2][16];
                const int col = hf * (kHeadDim / 2) + j * 32;
                ptx::tmem_ld16(tmem + lane_base + kTmemO8 + col, o[0]);
                ptx::tmem_ld16(tmem + lane_base + kTmemO8 + col + 16, o[1]);
                ptx::tmem_ld_wait();
                if (!row_valid) continue;
                if (C == 1) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e] = pack_bf16x2(__uint_as_float(o[e >> 3][2 * (e & 7)]) * inv_l,
                                           __uint_as_float(o[e >> 3][2 * (e & 7) + 1]) * inv_l);
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + out_row * kHeadDim + col);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(srow + col * 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_uint4(o[e >> 2][4 * (e & 3)], o[e >> 2][4 * (e & 3) + 1], o[e >> 2][4 * (e & 3) + 2],
                                            o[e >> 2][4 * (e & 3) + 3]);
                }
            }
        }
        if (C == 1) {
            if (hf == 0 && row_valid && p.lse != nullptr)
                p.lse[out_row] = (m_used + ptx::lg2(l_row)) * 0.69314718055994531f;
        } else {
            if (row_valid) {
                const float used = have_o && !failed ? l_row : 0.0f;
                if (hf == 0)
                    *reinterpret_cast<float4 *>(srow + kHeadDim * 4) = make_float4(m_used, used, used, 0.0f);
                ptx::fence_proxy_async_smem();
            }
            if (!failed && !pair_sync()) failed = true;  // both halves of the row staged
            if (row_valid && hf == 0) {
                const size_t prow = (static_cast<size_t>(cl) * C + rank) * (p.G * p.SQ) + row_k;
                ptx::bulk_store_s2g(reinterpret_cast<uint8_t *>(p.part) + prow * L::kStageStride, ptx::smem_addr(srow),
                                    L::kStageStride);
                ptx::bulk_commit();
                ptx::bulk_wait_all();
                ptx::fence_proxy_async_global();
            }
        }
    }

    __syncwarp();
    if (C > 1) {
        // ================================================== split merge, as in the bf16 kernel
        ptx::cluster_sync();
        const int r_lo = (NR * rank) / C, r_hi = (NR * (rank + 1)) / C;
        const int nr = r_hi - r_lo;
        long long *orow_s = reinterpret_cast<long long *>(smem + L::kXchgOff);
        if (nr > 0 && warp == 0) {
            if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[L::kBarMerge], static_cast<uint32_t>(C * nr * L::kStageStride));
            __syncwarp();
            if (lane < C) {
                ptx::fence_proxy_async_global();
                ptx::bulk_load_g2s(ptx::smem_addr(smem) + static_cast<uint32_t>(lane * nr * L::kStageStride),
                                   reinterpret_cast<const uint8_t *>(p.part) +
                                       ((static_cast<size_t>(cl) * C + lane) * (p.G * p.SQ) + r_lo) * L::kStageStride,
                                   static_cast<uint32_t>(nr * L::kStageStride), &bars[L::kBarMerge]);
            }
        }
        if (nr > 0) {
            if (!warp_wait(&bars[L::kBarMerge], 0)) failed = true;
            merge_weights<L>(smem, C, nr, p.lse, unit_row0, r_lo, nq, p.S, q0, nq, orow_s);
            __syncthreads();
            merge_rows<L>(smem, C, nr, p.out, orow_s);
        }
    }
    if (failed) atomicOr(p.err, kEwTimeout);
    __syncwarp();
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace kv8
}  // namespace dm05
