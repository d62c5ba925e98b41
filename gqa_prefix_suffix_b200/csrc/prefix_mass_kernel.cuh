// prefix_mass_kernel.cuh -- sm_100a kernel of the attention weight that each
// prefix position received:
//   mass[j] = mass_in[j] + sum_i exp(<q_i, k_j> / sqrt(D) - lse_i)
// over the GS query rows i of a (sample, KV head) unit.
//
// With the logits transposed, S^T = K Q^T, a tile of 128 keys is the MMA's M
// and the unit's query rows are its N: every thread then owns one key and
// sums along its row, without a reduction over lanes, and a hidden key's
// garbage stays in its own row.  No maximum is needed (the lse is given), so
// a tile is one matrix product, one exponential a logit, and one sum.
// The queries stay in shared memory for all of a CTA's tiles; the tiles of a
// unit are dealt to CTAs in contiguous runs, each key to exactly one, so
// the result has one order of sums and no atomics.
//
// A bf16 cache multiplies in kind::f16 (64 KB a tile); an 8-bit one in
// kind::f8f6f4 straight from its codes (32 KB), with the query rows as two
// e4m3 terms of their scaled values as in the 8-bit attention, the scales of
// key and query applied in the exponent.
//
// Warp roles: warp 16 loads, warp 17 issues the MMAs, warps 0-15 are two
// groups that take the tiles in turn (two warps per 32 keys), so that one
// group's waits run beside the other's exponentials.  The 256 products of a
// logit are summed in two chains, of a bf16 cache in four where they fit,
// joined in fp32 registers: the tensor cores' running sum loses a little with
// every step (bf16, one query against 7281 keys, whose sum is mostly one key of
// large logit: 1.2e-6 relative in two chains, 0.7e-6 in four;
// 8-bit: 0.4e-6 in two and in four).  Two buffers of two chains of 128 columns, or
// of four of 64, fill the tensor memory.
//
// B = 32, P = 1024, 100 rows a unit: 14.1 us from codes (a tile takes 1.65k cycles
// of which the MMAs are 1.1k; the rest waits for a buffer to be read), 13.8 us
// from bf16 (HBM and start-up); B = 1, P = 2048 4.9 us (4.7 in two chains).  The CTA's 18 warps leave a
// thread 96 registers: holding a tile's logits to free its buffer earlier
// spills, and with this much shared memory a spill of 20 bytes costs 1 us.
#pragma once

#include <type_traits>

#include "kv8_attn_kernel.cuh"

namespace dm05 {
namespace mass {

constexpr int kTile = 128;     // keys of a tile
constexpr int kSoftWarps = 16;
constexpr int kLoadWarp = 16;
constexpr int kIssueWarp = 17;
constexpr int kThreadsM = 576;
constexpr int kBufs = 2;       // logit buffers of 256 columns

template <bool KV8>
struct Smem {
    static constexpr int kQBytes = 65536;
    static constexpr int kSlotBytes = KV8 ? 32768 : 65536;
    static constexpr int kSlots = KV8 ? 4 : 2;
    static constexpr int kRing = kQBytes;
    static constexpr int kBarOff = kRing + kSlots * kSlotBytes;
    static constexpr int kBarQFull = 0;
    static constexpr int kBarQReady = 1;   // query rows split (8-bit), row constants written
    static constexpr int kBarFull = 2;
    static constexpr int kBarEmpty = kBarFull + kSlots;
    static constexpr int kBarSFull = kBarEmpty + kSlots;
    static constexpr int kBarSFree = kBarSFull + kBufs;
    static constexpr int kBarPair = kBarSFree + kBufs;  // per group and lane quarter: its two warps
    static constexpr int kBarFinal = kBarPair + 8;
    static constexpr int kNumBars = kBarFinal + 1;
    static constexpr int kTmemSlotOff = kBarOff + kNumBars * 8;
    static constexpr int kRowOff = (kTmemSlotOff + 16 + 15) / 16 * 16;  // per query row: factors [128], -lse [128]
    static constexpr int kSumOff = kRowOff + 2 * 128 * 4;               // partial sums [2 parities][2 groups][128]
    static constexpr int kEnd = kSumOff + 4 * 128 * 4;
    static constexpr int kAllocBytes = kEnd + 1024;
    static_assert(kAllocBytes <= 232448, "shared memory of a CTA");
};

struct Params {
    const float *k_scale;    // 8-bit: [units, nblk]
    const float *lse;        // [units, GS]
    const int32_t *valid_len;
    const uint8_t *mask;     // [B, P] or nullptr
    const float *mass_in;    // [units, P] or nullptr
    float *mass;             // [units, P]
    uint32_t *err;
    int Hkv, P, GS, N;       // N: GS rounded up to 16, the MMA's N
    int nblk, shift;
    float scale;             // 1 / sqrt(D)
};

template <bool KV8>
__global__ void __launch_bounds__(kThreadsM, 1)
    mass_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const Params p)
{
    using L = Smem<KV8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmemSlotOff);
    float *factors = reinterpret_cast<float *>(smem + L::kRowOff);  // per query row: its scale / sqrt(D)
    float *lses = factors + 128;                                    // and -lse
    float *sums = reinterpret_cast<float *>(smem + L::kSumOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.y, b = unit / p.Hkv;

    if (threadIdx.x == 0) {
        ptx::mbar_init(&bars[L::kBarQFull], 1);
        ptx::mbar_init(&bars[L::kBarQReady], kSoftWarps * 32);
        for (int i = 0; i < L::kSlots; ++i) {
            ptx::mbar_init(&bars[L::kBarFull + i], 1);
            ptx::mbar_init(&bars[L::kBarEmpty + i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            ptx::mbar_init(&bars[L::kBarSFull + i], 1);
            ptx::mbar_init(&bars[L::kBarSFree + i], kSoftWarps / 2 * 32);
        }
        for (int i = 0; i < 8; ++i) ptx::mbar_init(&bars[L::kBarPair + i], 64);
        ptx::mbar_init(&bars[L::kBarFinal], 1);
        ptx::fence_mbar_init();
    }
    if (warp == kLoadWarp && lane == 0) {
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
    }
    if (warp == kIssueWarp) {
        ptx::tmem_alloc(tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    ptx::griddep_launch_dependents();
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    if (warp == kLoadWarp && lane == 0) {
        // what will be read first is asked into L2 while the kernel before this
        // one ends (caches and queries may still change until the wait below:
        // L2 then holds the change).  The run is the one of a full prefix.
        if (p.valid_len != nullptr) ptx::prefetch_l2(p.valid_len + b);
        ptx::tma_prefetch_4d(&tm_q, 0, 0, 0, unit);
        const long long all = (p.P + kTile - 1) / kTile;
        const int ta = static_cast<int>(all * blockIdx.x / gridDim.x);
        const int te = static_cast<int>(all * (blockIdx.x + 1) / gridDim.x);
        for (int t = ta; t < min(te, ta + 2); ++t) ptx::tma_prefetch_4d(&tm_k, 0, t * kTile, 0, unit);
    }
    ptx::griddep_wait();
    if (warp == kLoadWarp && lane == 0) {  // needs no valid length
        ptx::mbar_arrive_expect_tx(&bars[L::kBarQFull], static_cast<uint32_t>(p.N) * 512u);
        ptx::tma_load_4d(smem, &tm_q, &bars[L::kBarQFull], 0, 0, 0, unit);
    }

    const int vl = cache::clamped_len(p.valid_len, b, p.P, p.err,
                                      threadIdx.x == 0 && blockIdx.x == 0 && unit % p.Hkv == 0);
    const int t_in = (vl + kTile - 1) / kTile;
    // this CTA's run of the tiles in range, and its share of the rest (whose
    // mass is only carried over)
    const int t0 = static_cast<int>(static_cast<long long>(t_in) * blockIdx.x / gridDim.x);
    const int T = static_cast<int>(static_cast<long long>(t_in) * (blockIdx.x + 1) / gridDim.x) - t0;
    // The 256 products of a bf16 logit are summed in four chains where tensor memory
    // holds them: 64 columns or fewer each, or one tile that needs no second buffer.
    const bool four = !KV8 && (p.N <= 64 || T <= 1);
    const int chain_cols = p.N <= 64 ? 64 : 128;
    bool failed = false;

    if (warp == kLoadWarp) {
        if (lane == 0) {
            const uint64_t pol = ptx::policy_evict_first();
            int issued = 0;
            for (int t = 0; t < T; ++t) {
                const int s = t % L::kSlots, n = t / L::kSlots;
                if (n > 0 && !ptx::mbar_wait(&bars[L::kBarEmpty + s], (n - 1) & 1, kWaitLimitNs)) {
                    failed = true;
                    break;
                }
                ptx::mbar_arrive_expect_tx(&bars[L::kBarFull + s], L::kSlotBytes);
                ptx::tma_load_4d_hint(smem + L::kRing + s * L::kSlotBytes, &tm_k, &bars[L::kBarFull + s], 0,
                                      (t0 + t) * kTile, 0, unit, pol);
                issued = t + 1;
            }
            // every copy this thread issued has landed before the CTA may exit
            if (!ptx::mbar_wait(&bars[L::kBarQFull], 0, kWaitLimitNs)) failed = true;
            for (int t = max(0, issued - L::kSlots); t < issued; ++t)
                if (!ptx::mbar_wait(&bars[L::kBarFull + t % L::kSlots], (t / L::kSlots) & 1, kWaitLimitNs)) failed = true;
        }
    } else if (warp == kIssueWarp) {
        if (lane == 0 && T > 0) {
            const int qpitch = p.N * 128;  // bytes of a 64-column chunk of the query rows
            const uint32_t idesc = KV8 ? ptx::idesc_e4m3_f32(kTile, p.N, false) : ptx::idesc_bf16_f32(kTile, p.N, false);
            const uint64_t qdesc = ptx::sw128_desc(ptx::smem_addr(smem), 16, 1024);
            const uint64_t kdesc = ptx::sw128_desc(ptx::smem_addr(smem + L::kRing), 16, 1024);
            bool ok = ptx::mbar_wait(&bars[L::kBarQFull], 0, kWaitLimitNs) &&
                      ptx::mbar_wait(&bars[L::kBarQReady], 0, kWaitLimitNs);
            for (int t = 0; t < T && ok; ++t) {
                const int s = t % L::kSlots, sb = t % kBufs;
                ok = ptx::mbar_wait(&bars[L::kBarFull + s], (t / L::kSlots) & 1, kWaitLimitNs) &&
                     (t < kBufs || ptx::mbar_wait(&bars[L::kBarSFree + sb], (t / kBufs - 1) & 1, kWaitLimitNs));
                if (!ok) break;
                ptx::tc_fence_after_sync();
                const uint64_t kd = kdesc + static_cast<uint64_t>((s * L::kSlotBytes) >> 4);
                const uint32_t d = tmem + sb * 256;
                auto issue = [&](auto chain, int cols) {
                    constexpr int kLen = decltype(chain)::value;  // MMAs of a chain
#pragma unroll
                    for (int kk = 0; kk < 16; ++kk) {
                        const uint32_t dk = d + kk / kLen * cols, add = kk % kLen > 0 ? 1u : 0u;
                        if (KV8) {
                            // 32 columns j against both terms of the queries
                            const int j = kk >> 1;
                            const uint32_t qo = ((j >> 1) * qpitch + (j & 1) * 64 + (kk & 1) * 32) >> 4;
                            const uint32_t ko = ((j >> 2) * (kTile * 128) + (j & 3) * 32) >> 4;
                            ptx::mma_f8_ss(dk, kd + ko, qdesc + qo, idesc, add);
                        } else {
                            const uint32_t qo = ((kk >> 2) * qpitch + (kk & 3) * 32) >> 4;
                            const uint32_t ko = ((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
                            ptx::mma_bf16_ss(dk, kd + ko, qdesc + qo, idesc, add);
                        }
                    }
                };
                if (four)
                    issue(std::integral_constant<int, 4>(), chain_cols);
                else
                    issue(std::integral_constant<int, 8>(), 128);
                ptx::mma_commit(&bars[L::kBarEmpty + s]);
                ptx::mma_commit(&bars[L::kBarSFull + sb]);
            }
            // every MMA issued above has completed before tensor memory is freed
            ptx::mma_commit(&bars[L::kBarFinal]);
            if (!ptx::mbar_wait(&bars[L::kBarFinal], 0, kWaitLimitNs)) ok = false;
            failed = !ok;
        }
    } else {
        const int q4 = warp & 3, c4 = warp >> 2;
        const int row = q4 * 32 + lane;  // a key of the tile; a query row while those are prepared
        const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
        if (T > 0) {
            // ---- query rows: their constants, and the two terms for an 8-bit cache
            if (KV8) {
                failed = !warp_wait(&bars[L::kBarQFull], 0);
                if (!failed) kv8::split_query_rows(smem, p.N * 128, p.GS, warp, p.scale, factors);
                ptx::fence_proxy_async_smem();
            } else if (c4 == 0) {
                factors[row] = p.scale;
            }
            // the MMA's columns behind the last query row hold zeros; their factor
            // must be a number too
            if (KV8 && c4 == 0 && row >= p.GS) factors[row] = 0.0f;
            if (c4 == 1) {
                // rows that do not exist, and rows that saw no key (-inf), add e^-inf
                float l = INFINITY;
                if (row < p.GS) l = ptx::load(p.lse + static_cast<size_t>(unit) * p.GS + row);
                lses[row] = l == -INFINITY ? -INFINITY : -l;
            }
            ptx::mbar_arrive(&bars[L::kBarQReady]);
            if (!failed) failed = !warp_wait(&bars[L::kBarQReady], 0);
        }
        // The two groups of eight warps take the tiles in turn; a group's two
        // warps of 32 keys take the 16-column groups hf, hf + 2, ...
        const int hf = c4 & 1, grp = c4 >> 1;
        const int groups = p.N >> 4;
        const size_t unit_key0 = static_cast<size_t>(unit) * p.P;
        uint64_t *pair_bar = &bars[L::kBarPair + grp * 4 + q4];
        // what a tile needs of global memory, requested one of the group's tiles ahead
        float before_next = 0.0f, ks_next = 1.0f;
        uint32_t see_next = 0u;
        auto load_next = [&](int t) {
            const int j = (t0 + t) * kTile + row;
            if (t >= T) return;
            if (KV8 && j < vl) ks_next = ptx::load(p.k_scale + static_cast<size_t>(unit) * p.nblk + (j >> p.shift));
            if (hf == 0) {
                see_next = j < vl ? 1u : 0u;
                if (j < vl && p.mask != nullptr) see_next = ptx::load(p.mask + static_cast<size_t>(b) * p.P + j);
                if (j < p.P && p.mass_in != nullptr) before_next = p.mass_in[unit_key0 + j];
            }
        };
        load_next(grp);
        for (int t = grp; t < T && !failed; t += 2) {
            const int sb = t % kBufs;
            const int j = (t0 + t) * kTile + row;
            const float before = before_next, ks = ks_next;
            const uint32_t see = see_next;
            load_next(t + 2);
            if (!warp_wait(&bars[L::kBarSFull + sb], (t / kBufs) & 1)) {
                failed = true;
                break;
            }
            ptx::tc_fence_after_sync();
            const uint32_t col = tmem + lane_base + sb * 256;
            const uint64_t ks2 = ptx::f32x2(ks, ks), log2e = ptx::f32x2(1.4426950408889634f, 1.4426950408889634f);
            uint64_t acc[2] = {ptx::f32x2(0.0f, 0.0f), ptx::f32x2(0.0f, 0.0f)};
            const int last = groups - 1 - ((groups - 1 - hf) & 1);  // this warp's last column group
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int g = hf + 2 * h;
                if (g >= groups) break;
                uint32_t raw[2][16];  // the chains' sums: all but the last, the last
                ptx::tmem_ld16(col + g * 16, raw[0]);
                ptx::tmem_ld16(col + (four ? chain_cols : 128) + g * 16, raw[1]);
                ptx::tmem_ld_wait();
                if (four) {
#pragma unroll
                    for (int c = 2; c < 4; ++c) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            raw[0][i] = __float_as_uint(__uint_as_float(raw[0][i]) + __uint_as_float(raw[1][i]));
                        ptx::tmem_ld16(col + c * chain_cols + g * 16, raw[1]);
                        ptx::tmem_ld_wait();
                    }
                }
                if (g == last) {
                    ptx::tc_fence_before_sync();
                    ptx::mbar_arrive(&bars[L::kBarSFree + sb]);
                }
                const float4 *fc = reinterpret_cast<const float4 *>(factors + g * 16);
                const float4 *lc = reinterpret_cast<const float4 *>(lses + g * 16);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 f4 = fc[e >> 2], l4 = lc[e >> 2];
#pragma unroll
                    for (int d = 0; d < 4; d += 2) {
                        uint64_t f = d == 0 ? ptx::f32x2(f4.x, f4.y) : ptx::f32x2(f4.z, f4.w);
                        const uint64_t l = d == 0 ? ptx::f32x2(l4.x, l4.y) : ptx::f32x2(l4.z, l4.w);
                        if (KV8) f = ptx::mul_f32x2(f, ks2);
                        const int i = e + d;
                        const uint64_t dot =
                            ptx::add_f32x2(ptx::f32x2(__uint_as_float(raw[0][i]), __uint_as_float(raw[0][i + 1])),
                                           ptx::f32x2(__uint_as_float(raw[1][i]), __uint_as_float(raw[1][i + 1])));
                        // z - lse is formed in natural units, where 1 / sqrt(D) is a power of
                        // two and the difference of near equals exact, and only then taken
                        // to base 2 (the other way round costs 2^-24 of the lse)
                        const float2 x = ptx::unpack_f32x2(ptx::mul_f32x2(ptx::fma_f32x2(dot, f, l), log2e));
                        acc[d >> 1] = ptx::add_f32x2(acc[d >> 1], ptx::f32x2(ptx::ex2(x.x), ptx::ex2(x.y)));
                    }
                }
            }
            if (hf >= groups) {  // no column group for this warp (N = 16)
                ptx::tc_fence_before_sync();
                ptx::mbar_arrive(&bars[L::kBarSFree + sb]);
            }
            const float2 s2 = ptx::unpack_f32x2(ptx::add_f32x2(acc[0], acc[1]));
            // the halves meet in the first one's warp; two tiles of a group apart,
            // both are past the buffer's last use
            const int turn = t >> 1;
            float *xs = sums + ((turn & 1) * 2 + grp) * 128 + row;
            if (hf == 1) *xs = s2.x + s2.y;
            ptx::mbar_arrive(pair_bar);
            if (!warp_wait(pair_bar, turn & 1)) {
                failed = true;
                break;
            }
            if (hf == 0 && j < p.P) p.mass[unit_key0 + j] = see != 0u ? before + ((s2.x + s2.y) + *xs) : before;
        }
        // positions past the tiles in range keep what they had
        const int first = t_in * kTile;
        for (long long j = first + static_cast<long long>(blockIdx.x) * (kSoftWarps * 32) + threadIdx.x; j < p.P;
             j += static_cast<long long>(gridDim.x) * (kSoftWarps * 32))
            p.mass[unit_key0 + j] = p.mass_in != nullptr ? p.mass_in[unit_key0 + j] : 0.0f;
    }
    if (failed) atomicOr(p.err, kEwTimeout);
    __syncwarp();
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kIssueWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace mass
}  // namespace dm05
