// prefix_cache_kernels.cuh -- sm_100a kernels that fill and shrink the prefix
// KV cache: the 8-bit quantiser and the eviction (selection, then a gather
// of the kept rows).
//
// The 8-bit cache holds e4m3 codes [B, Hkv, P, 256] and, for K and for V, one
// fp32 scale for each block of `block` consecutive rows of a KV head:
// row j stands for scale[j / block] * code[j].  The quantiser writes powers
// of two: e4m3 is a floating format, so a finer scale would not make the
// codes more exact (the relative step is 2^-4 at any scale), and with a power
// of two the division and the product back are exact, the value fits bf16
// unrounded, and codes move between blocks (eviction) without a second
// rounding unless they fall below the new block's smallest step.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "suffix_attn_kernel.cuh"

namespace dm05 {

namespace ptx {
// A plain global load.  What the kernel launched right before may have written
// is not read through the non-coherent path: with programmatic dependent
// launch this kernel was already running then.
template <class T>
__device__ __forceinline__ T load(const T *p)
{
    return *p;
}

// Barrier `id` over `threads` threads of the CTA.
__device__ __forceinline__ void group_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
}  // namespace ptx

namespace cache {

constexpr int kRowBytes8 = kHeadDim;         // one 8-bit row
constexpr int kMinScaleExp = -64;            // smallest scale 2^-64
constexpr float kCodeMax = 448.0f;           // largest e4m3 value
constexpr uint32_t kCodeNan = 0x7fu;

// valid_len of a sample, clamped to [0, P]; the clamp is recorded once.
__device__ __forceinline__ int clamped_len(const int32_t *valid_len, int b, int P, uint32_t *err, bool report)
{
    if (valid_len == nullptr) return P;
    const int raw = ptx::load(valid_len + b);
    const int vl = min(max(raw, 0), P);
    if (raw != vl && report) atomicOr(err, kEwClamped);
    return vl;
}

// The smallest power of two s >= 2^-64 with amax <= 448 s (amax finite and
// >= 0; s = 1 for amax = 0).  448 = 1.75 * 2^8, so with amax = f * 2^e,
// 1 <= f < 2, the exponent is e - 8, one more when f > 1.75.  A subnormal
// amax has a biased exponent field of 0 and gets the smallest scale.
__device__ __forceinline__ float pow2_scale(float amax)
{
    if (amax == 0.0f) return 1.0f;
    const uint32_t u = __float_as_uint(amax);
    int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, kMinScaleExp);
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// 1 / s of a power of two s in [2^-64, 2^120]
__device__ __forceinline__ float pow2_inverse(float s)
{
    return __uint_as_float((254u << 23) - __float_as_uint(s));
}

__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Two codes and their values in fp16 (which holds every e4m3 value).
__device__ __forceinline__ __half2 decode2(uint32_t codes)
{
    return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3));
}
__device__ __forceinline__ uint32_t encode2(__half2 x)
{
    return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
}

// the four values of four codes
__device__ __forceinline__ float4 decode4(uint32_t w)
{
    const __half2 lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
    const __half2 hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
    const float2 a = __half22float2(lo), b = __half22float2(hi);
    return make_float4(a.x, a.y, b.x, b.y);
}

// Largest value over the CTA (256 threads); `slots` holds 8 words.
__device__ __forceinline__ uint32_t block_max_u32(uint32_t v, uint32_t *slots)
{
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t m = slots[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, slots[i]);
    return m;
}

struct QuantParams {
    const __nv_bfloat16 *k, *v;  // [units, P, 256]
    uint8_t *k8, *v8;
    float *k_scale, *v_scale;    // [units, nblk]
    const int32_t *valid_len;
    uint32_t *err;
    int Hkv, P, nblk, blk0;     // blk0: first block written
};

// One CTA per (block of rows, unit, K or V): every value is read once, held
// in registers for the block's maximum and then encoded.  Bound by HBM
// (2 bytes read and 1 written per value): B = 32, 4 heads, P = 1024 in 24.9 us,
// 6.3 TB/s; small caches by launch and one round trip (2.7 us).
template <int BLOCK>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantParams p)
{
    __shared__ uint32_t slots[8];
    const int unit = blockIdx.y, which = blockIdx.z;
    const int n = p.blk0 + blockIdx.x;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int vl = clamped_len(p.valid_len, unit / p.Hkv, p.P, p.err,
                               threadIdx.x == 0 && blockIdx.x == 0 && which == 0 && unit % p.Hkv == 0);
    const int rows = min(BLOCK, vl - n * BLOCK);
    if (rows <= 0) return;
    constexpr int kPasses = BLOCK / 16;  // 16 rows a pass, 16 values a thread
    const int r0 = threadIdx.x >> 4, col = (threadIdx.x & 15) * 16;
    const size_t row0 = static_cast<size_t>(unit) * p.P + static_cast<size_t>(n) * BLOCK;
    const __nv_bfloat16 *src = (which ? p.v : p.k) + row0 * kHeadDim + col;
    uint4 v[kPasses][2];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
        const int r = i * 16 + r0;
        if (r < rows) {
            const uint4 *a = reinterpret_cast<const uint4 *>(src + static_cast<size_t>(r) * kHeadDim);
            v[i][0] = ptx::load(a);
            v[i][1] = ptx::load(a + 1);
        }
    }
    // bf16 magnitudes order like their bit patterns; 0x7f80 and above are
    // infinities and NaN, which set no scale and become NaN codes
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w[4] = {v[i][h].x, v[i][h].y, v[i][h].z, v[i][h].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
        }
    uint32_t amax = block_max_u32(max(top & 0xffffu, top >> 16), slots);
    const bool odd = amax >= 0x7f80u;
    if (odd) {
        uint32_t fin = 0u;
        for (int i = 0; i < kPasses; ++i)
            for (int h = 0; h < 2; ++h) {
                const uint32_t w[4] = {v[i][h].x, v[i][h].y, v[i][h].z, v[i][h].w};
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
                    fin = max(fin, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                }
            }
        __syncthreads();
        amax = block_max_u32(fin, slots);
    }
    const float s = pow2_scale(__uint_as_float(amax << 16)), inv = pow2_inverse(s);
    if (threadIdx.x == 0) (which ? p.v_scale : p.k_scale)[static_cast<size_t>(unit) * p.nblk + n] = s;
    uint8_t *dst = (which ? p.v8 : p.k8) + row0 * kRowBytes8 + col;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * 16 + r0;
        if (r >= rows) break;
        uint32_t o[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w[4] = {v[i][h].x, v[i][h].y, v[i][h].z, v[i][h].w};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t a = w[2 * e], b = w[2 * e + 1];
                uint32_t c = encode4(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xffff0000u) * inv,
                                     __uint_as_float(b << 16) * inv, __uint_as_float(b & 0xffff0000u) * inv);
                if (odd) {
                    if ((a & 0x7fffu) >= 0x7f80u) c |= kCodeNan;
                    if ((a >> 16 & 0x7fffu) >= 0x7f80u) c |= kCodeNan << 8;
                    if ((b & 0x7fffu) >= 0x7f80u) c |= kCodeNan << 16;
                    if ((b >> 16 & 0x7fffu) >= 0x7f80u) c |= kCodeNan << 24;
                }
                o[2 * h + e] = c;
            }
        }
        *reinterpret_cast<uint4 *>(dst + static_cast<size_t>(r) * kRowBytes8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ------------------------------------------------------------------ eviction

struct SelectParams {
    const float *mass;          // [units, P]
    const int32_t *valid_len;
    const uint8_t *mask;        // [B, P] or nullptr
    float *mass_out;            // [units, Pout]
    int32_t *pos;               // [units, Pout]
    int32_t *valid_out;         // [B]
    uint32_t *err;
    int Hkv, P, Pout, n_keep, n_first, n_last;
};

// Sort key of position j with this weight: 0 hidden, 1 NaN, then the weights
// in ascending order (-0 counts as +0), the largest for a protected position.
__device__ __forceinline__ uint32_t select_key(const SelectParams &p, int vl, int j, float weight, bool shown)
{
    if (j >= vl || !shown) return 0u;
    if (j < p.n_first || j >= vl - p.n_last) return 0xffffffffu;
    const float m = weight + 0.0f;
    if (m != m) return 1u;
    const uint32_t u = __float_as_uint(m);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Adds one to the bin of every participating lane's digit, one atomic per
// distinct digit of the warp: for the first digit, where weights of one head
// share their exponent and single adds would queue on a few bins.
__device__ __forceinline__ void count_digit(int *hist, uint32_t digit, bool active)
{
    const uint32_t who = __ballot_sync(0xffffffffu, active);
    if (active) {
        const uint32_t peers = __match_any_sync(who, digit);
        if ((threadIdx.x & 31) == __ffs(static_cast<int>(peers)) - 1) atomicAdd(&hist[digit], __popc(peers));
    }
    __syncwarp();
}

// The digit whose bin, counted from the largest digit down, holds the
// `want`-th key: {digit, the key's rank within the bin, the bin's count}.
// One warp.
__device__ __forceinline__ void pick_digit(const int *hist, int want, int *pick)
{
    const int lane = threadIdx.x & 31;
    // eight runs of 32 bins, lane l holding the (l + 1)-th largest of each
    int bin[8], chosen = 0, above = 0, run = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) bin[e] = hist[255 - e * 32 - lane];
    bool found = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int n = __reduce_add_sync(0xffffffffu, bin[e]);
        if (!found && above + n >= want) {
            found = true;
            chosen = bin[e];
            run = e;
        }
        if (!found) above += n;
    }
    int incl = chosen;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    const int before = above + incl - chosen;
    if (before < want && before + chosen >= want) {
        pick[0] = 255 - run * 32 - lane;
        pick[1] = want - before;
        pick[2] = chosen;
    }
}

// Exclusive scan of table[0, n) by one warp; returns the total (that warp).
__device__ __forceinline__ int warp_scan_table(int *table, int n)
{
    const int lane = threadIdx.x & 31;
    int run = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int v = i0 + lane < n ? table[i0 + lane] : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += t;
        }
        if (i0 + lane < n) table[i0 + lane] = run + s - v;
        run += __shfl_sync(0xffffffffu, s, 31);
    }
    return run;
}

// The key of a unit's n_keep-th wanted position by a radix selection (four
// 8-bit digits, from the top), then the kept positions in ascending order, the
// lowest ones first among equals: emit(keep, index, position, weight) once
// for each.  Returns keep, the number of kept positions.  All 1024 threads.
//
// Latency bounds it, a chain of counts, scans and barriers, so that it stops at
// the first digit whose bin is kept whole (1000 of 2048 kept: 6.3
// instead of 6.9 us for the whole eviction).
//
// KPT > 0: P <= KPT * 1024 and every thread keeps its keys in registers (the
// weights are read once).  KPT == 0: any P; the keys are formed again in
// every pass, and the positions are found 1024 at a time.  Weights (or a
// length) that someone changes meanwhile make its passes disagree: what is kept is
// then anything, but positions stay inside the prefix and their number inside the new cache.
constexpr int kSelectThreads = 1024;

template <int KPT>
struct SelectShared {
    static constexpr int kKeys = KPT > 0 ? KPT : 1;
    int hist[4][256];
    int table[kKeys * 32 + 1];
    int seen, pick[4][3], len;
};

template <int KPT, class Emit>
__device__ __forceinline__ int select_positions(const SelectParams &p, int unit, SelectShared<KPT> &sh, Emit &&emit)
{
    constexpr int kKeys = SelectShared<KPT>::kKeys;
    auto &hist = sh.hist;
    auto &table = sh.table;
    auto &pick = sh.pick;
    int &seen = sh.seen;
    const int b = unit / p.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < 4 * 256; i += kSelectThreads) (&hist[0][0])[i] = 0;
    if (threadIdx.x == 0) seen = 0;
    ptx::griddep_launch_dependents();
    __syncthreads();
    ptx::griddep_wait();
    const float *mass = p.mass + static_cast<size_t>(unit) * p.P;
    const uint8_t *mask = p.mask ? p.mask + static_cast<size_t>(b) * p.P : nullptr;
    float weight[kKeys];
    bool shown[kKeys];
    if (KPT > 0) {
        // requested before the valid length is known
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const int j = i * kSelectThreads + threadIdx.x;
            weight[i] = j < p.P ? mass[j] : 0.0f;
            shown[i] = j < p.P && (mask == nullptr || mask[j] != 0);
        }
    }
    int vl = clamped_len(p.valid_len, b, p.P, p.err, threadIdx.x == 0 && blockIdx.x == 0 && unit % p.Hkv == 0);
    if (KPT == 0) {  // one length for all, whatever happens to it
        if (threadIdx.x == 0) sh.len = vl;
        __syncthreads();
        vl = sh.len;
    }
    const int rounds = KPT > 0 ? KPT : (vl + kSelectThreads - 1) / kSelectThreads;
    uint32_t keys[kKeys];
    auto key_of = [&](int i) -> uint32_t {
        const int j = i * kSelectThreads + threadIdx.x;
        return j < vl ? select_key(p, vl, j, mass[j], mask == nullptr || mask[j] != 0) : 0u;
    };
    int visible = 0;
    if (KPT > 0) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const int j = i * kSelectThreads + threadIdx.x;
            keys[i] = select_key(p, vl, j, weight[i], shown[i]);
            visible += keys[i] != 0u;
            count_digit(hist[0], keys[i] >> 24, keys[i] != 0u);
        }
    } else {
        for (int i = 0; i < rounds; ++i) {
            const uint32_t k = key_of(i);
            visible += k != 0u;
            count_digit(hist[0], k >> 24, k != 0u);
        }
    }
    visible = __reduce_add_sync(0xffffffffu, visible);
    if (lane == 0 && visible != 0) atomicAdd(&seen, visible);
    __syncthreads();
    const int keep = min(p.n_keep, seen);
    if (keep > 0) {
        if (warp == 0) pick_digit(hist[0], keep, pick[0]);
        __syncthreads();
        // Once every key of the chosen bin is kept, the digits behind it decide nothing.
        bool whole = pick[0][1] == pick[0][2];
        int want = pick[0][1];
        uint32_t prefix = static_cast<uint32_t>(pick[0][0]) << 24, known = 0xff000000u;
#pragma unroll
        for (int pass = 1; pass < 4; ++pass) {
            if (whole) break;
            const int shift = 24 - 8 * pass;
            if (KPT > 0) {
#pragma unroll
                for (int i = 0; i < kKeys; ++i)
                    if (keys[i] != 0u && (keys[i] & known) == prefix)
                        atomicAdd(&hist[pass][(keys[i] >> shift) & 255u], 1);
            } else {
                for (int i = 0; i < rounds; ++i) {
                    const uint32_t k = key_of(i);
                    count_digit(hist[pass], (k >> shift) & 255u, k != 0u && (k & known) == prefix);
                }
            }
            __syncthreads();
            if (warp == 0) pick_digit(hist[pass], want, pick[pass]);
            __syncthreads();
            prefix |= static_cast<uint32_t>(pick[pass][0]) << shift;
            known |= 255u << shift;
            want = pick[pass][1];
            whole = want == pick[pass][2];
        }
        // Kept: the keys above `prefix` in their known digits, and `want` of those
        // that equal it (every one if `whole`; else all four digits are known).
        if (KPT > 0) {
            uint32_t kept[kKeys];
            if (!whole) {
#pragma unroll
                for (int i = 0; i < kKeys; ++i) {
                    const uint32_t t = __ballot_sync(0xffffffffu, keys[i] == prefix);
                    if (lane == 0) table[i * 32 + warp] = __popc(t);
                }
                __syncthreads();
                if (warp == 0) warp_scan_table(table, kKeys * 32);
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                bool tie = keys[i] != 0u && (keys[i] & known) == prefix;
                if (!whole) {
                    const uint32_t t = __ballot_sync(0xffffffffu, tie);
                    tie = tie && table[i * 32 + warp] + __popc(t & ((1u << lane) - 1u)) < want;
                }
                kept[i] = __ballot_sync(0xffffffffu, (keys[i] & known) > prefix || tie);
            }
            if (!whole) __syncthreads();  // the tie table has been read
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
                if (lane == 0) table[i * 32 + warp] = __popc(kept[i]);
            __syncthreads();
            if (warp == 0) warp_scan_table(table, kKeys * 32);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                if (kept[i] >> lane & 1u) {
                    const int at = table[i * 32 + warp] + __popc(kept[i] & ((1u << lane) - 1u));
                    const int j = i * kSelectThreads + threadIdx.x;
                    emit(keep, at, j, weight[i]);
                }
            }
        } else {
            int base = 0, ties = 0;
            for (int i = 0; i < rounds; ++i) {
                const uint32_t k = key_of(i);
                const bool equal = k != 0u && (k & known) == prefix;
                const uint32_t t = __ballot_sync(0xffffffffu, equal);
                __syncthreads();  // the table's last use
                if (lane == 0) table[warp] = __popc(t);
                __syncthreads();
                if (warp == 0) {
                    const int n = warp_scan_table(table, 32);
                    if (lane == 0) table[32] = n;
                }
                __syncthreads();
                const bool tie = equal && ties + table[warp] + __popc(t & ((1u << lane) - 1u)) < want;
                ties += table[32];
                const uint32_t m = __ballot_sync(0xffffffffu, (k & known) > prefix || tie);
                __syncthreads();
                if (lane == 0) table[warp] = __popc(m);
                __syncthreads();
                if (warp == 0) {
                    const int n = warp_scan_table(table, 32);
                    if (lane == 0) table[32] = n;
                }
                __syncthreads();
                if (m >> lane & 1u) {
                    const int at = base + table[warp] + __popc(m & ((1u << lane) - 1u));
                    const int j = i * kSelectThreads + threadIdx.x;
                    if (at < keep) emit(keep, at, j, mass[j]);
                }
                base += table[32];
            }
            return min(keep, base);
        }
    }
    return keep;
}

// The positions and weights behind the kept ones, and the new valid length.
__device__ __forceinline__ void finish_selection(const SelectParams &p, int unit, int keep, int first, int step)
{
    if (first == 0 && unit % p.Hkv == 0) p.valid_out[unit / p.Hkv] = keep;
    for (int i = keep + first; i < p.Pout; i += step) {
        p.pos[static_cast<size_t>(unit) * p.Pout + i] = -1;
        p.mass_out[static_cast<size_t>(unit) * p.Pout + i] = 0.0f;
    }
}

// The selection alone, one CTA per unit, in front of a gather kernel.
template <int KPT>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectParams p)
{
    __shared__ SelectShared<KPT> sh;
    const int unit = blockIdx.y;
    int32_t *pos = p.pos + static_cast<size_t>(unit) * p.Pout;
    float *mass_out = p.mass_out + static_cast<size_t>(unit) * p.Pout;
    const int keep = select_positions<KPT>(p, unit, sh, [&](int, int at, int j, float weight) {
        pos[at] = j;
        mass_out[at] = weight;
    });
    finish_selection(p, unit, keep, threadIdx.x, kSelectThreads);
}

struct GatherParams {
    const uint8_t *k, *v;               // [units, P] rows
    uint8_t *k_out, *v_out;             // [units, Pout] rows
    const float *k_scale, *v_scale;     // 8-bit: [units, nblk]
    float *k_scale_out, *v_scale_out;   // 8-bit: [units, nblk_out]
    const int32_t *pos;      // [units, Pout], -1 behind the kept rows
    int Hkv, P, Pout, n_keep, nblk, nblk_out, shift;  // shift: log2 of the block
};

// bf16 rows: one warp moves four rows of K and V at a time, 512 bytes each.
// Bound by HBM (16 samples of 4 heads, 4000 of 8000 rows: 87.6 us with the
// selection, 6.0 TB/s).
__global__ void __launch_bounds__(256) gather_rows_kernel(const GatherParams p)
{
    ptx::griddep_launch_dependents();
    const int unit = blockIdx.y;
    const int lane = threadIdx.x & 31;
    const int i0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 4;
    const size_t in0 = static_cast<size_t>(unit) * p.P, out0 = static_cast<size_t>(unit) * p.Pout;
    ptx::griddep_wait();
    int j[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) j[r] = i0 + r < p.n_keep ? ptx::load(p.pos + out0 + i0 + r) : -1;
    uint4 v[4][2];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (j[r] >= 0) {
            const size_t off = (in0 + static_cast<size_t>(j[r])) * 512 + lane * 16;
            v[r][0] = ptx::load(reinterpret_cast<const uint4 *>(p.k + off));
            v[r][1] = ptx::load(reinterpret_cast<const uint4 *>(p.v + off));
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (j[r] >= 0) {
            const size_t off = (out0 + i0 + r) * 512 + lane * 16;
            *reinterpret_cast<uint4 *>(p.k_out + off) = v[r][0];
            *reinterpret_cast<uint4 *>(p.v_out + off) = v[r][1];
        }
    }
}

// Largest |code| * s of 16 codes, exact in fp16 and fp32 (NaN codes set no scale).
__device__ __forceinline__ float codes_max(const uint4 &v, float s)
{
    const uint32_t c[4] = {v.x, v.y, v.z, v.w};
    __half2 top = __float2half2_rn(0.0f);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        top = __hmax2(__hmax2(top, __habs2(decode2(c[e] & 0xffffu))), __habs2(decode2(c[e] >> 16)));
    return fmaxf(__low2float(top), __high2float(top)) * s;
}

// 16 codes of scale s as codes of scale 1 / inv, a power of two.
__device__ __forceinline__ uint4 recode(const uint4 &v, float s, float inv)
{
    const uint32_t c[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
    // With powers of two the quotient of the scales multiplies exactly, in
    // fp16 too: what it pushes below fp16's range rounds to the code 0.
    const float ratio = s * inv;
    if ((__float_as_uint(ratio) & 0x7fffffu) == 0u && ratio >= 0x1p-24f && ratio <= 0x1p15f) {
        const __half2 f = __float2half2_rn(ratio);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = encode2(__hmul2(decode2(c[e] & 0xffffu), f)) | encode2(__hmul2(decode2(c[e] >> 16), f)) << 16;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 x = decode4(c[e]);
            o[e] = encode4(x.x * s * inv, x.y * s * inv, x.z * s * inv, x.w * s * inv);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// One strip of the 8-bit gather: `Threads` threads move kPasses * Threads / 16
// kept rows of K or of V, 16 threads a row, and find the scales of the strip's
// new blocks.  The rows come from blocks with scales of their own; a new
// block's largest value sets its scale by the quantiser's rule and every code
// is rounded to it.  at(i): the position that becomes row i < end, -1 behind
// the kept rows.  `slots` are free to write; the threads meet at `barrier` once.
template <int BLOCK, int Threads>
struct Strip {
    static constexpr int kPasses = BLOCK * 16 / Threads > 4 ? BLOCK * 16 / Threads : 4;
    static constexpr int kRowsPass = Threads / 16;
    static constexpr int kRows = kPasses * kRowsPass;
    static constexpr int kBlocks = kRows / BLOCK;
    static constexpr int kPassBlock = kPasses / kBlocks;
    static constexpr int kWarps = Threads / 32;
    using Slots = uint32_t[kBlocks][kWarps];
};

template <int BLOCK, int Threads, bool Skip, class At>
__device__ __forceinline__ void gather_strip(const GatherParams &p, int unit, int row0, int end, bool is_v, int tid, int barrier,
                                             typename Strip<BLOCK, Threads>::Slots &slots, At &&at)
{
    using S = Strip<BLOCK, Threads>;
    const int lane = threadIdx.x & 31;
    const int r0 = row0 + (tid >> 4), col = (tid & 15) * 16;
    const uint8_t *src = (is_v ? p.v : p.k) + static_cast<size_t>(unit) * p.P * kRowBytes8 + col;
    const float *scale = (is_v ? p.v_scale : p.k_scale) + static_cast<size_t>(unit) * p.nblk;
    uint32_t here = 0u;  // bit i: row r0 + i * kRowsPass is a kept one
    int j[S::kPasses];
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
        j[i] = r0 + i * S::kRowsPass < end ? at(r0 + i * S::kRowsPass) : -1;
        here |= (j[i] >= 0 ? 1u : 0u) << i;
    }
    uint4 v[S::kPasses];
    float s[S::kPasses];
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        s[i] = 0.0f;
        if (here >> i & 1u) {
            v[i] = ptx::load(reinterpret_cast<const uint4 *>(src + static_cast<size_t>(j[i]) * kRowBytes8));
            s[i] = ptx::load(scale + (j[i] >> p.shift));
        }
    }
#pragma unroll
    for (int n = 0; n < S::kBlocks; ++n) {
        if (Skip && row0 + n * BLOCK >= end) break;
        float amax = 0.0f;
#pragma unroll
        for (int i = n * S::kPassBlock; i < (n + 1) * S::kPassBlock; ++i) amax = fmaxf(amax, codes_max(v[i], s[i]));
        const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
        if (lane == 0) slots[n][tid >> 5] = m;
    }
    ptx::group_sync(barrier, Threads);
    uint8_t *dst = (is_v ? p.v_out : p.k_out) + static_cast<size_t>(unit) * p.Pout * kRowBytes8 + col;
    float *scale_out = (is_v ? p.v_scale_out : p.k_scale_out) + static_cast<size_t>(unit) * p.nblk_out;
#pragma unroll
    for (int n = 0; n < S::kBlocks; ++n) {
        if (Skip && row0 + n * BLOCK >= end) break;
        uint32_t m = 0u;
#pragma unroll
        for (int w = 0; w < S::kWarps; ++w) m = max(m, slots[n][w]);
        const float t = pow2_scale(__uint_as_float(m)), inv = pow2_inverse(t);
        // thread 0 holds the block's first row: it is a kept one, or none is
        if (tid == 0 && (here >> (n * S::kPassBlock) & 1u)) scale_out[(row0 / BLOCK) + n] = t;
#pragma unroll
        for (int i = n * S::kPassBlock; i < (n + 1) * S::kPassBlock; ++i)
            if (here >> i & 1u)
                *reinterpret_cast<uint4 *>(dst + static_cast<size_t>(r0 + i * S::kRowsPass) * kRowBytes8) =
                    recode(v[i], s[i], inv);
    }
}

// 8-bit rows: one CTA per (strip of new rows, unit), half its threads on K,
// half on V.  Four rows a thread in flight whatever the block: strips of one
// block of 16 took 27.5 us instead of 20.6 at 148 heads and 512 rows.  The end
// is tested block by block only where a strip is one block (40 registers, three
// CTAs an SM: 19.1 instead of 20.1 us; with blocks of 16 it costs 22.8
// instead of 21.0).  Bound by the conversions and their latency
// (16 samples of 4 heads, 4000 of 8000 rows in blocks of 64: 52 us with the
// selection, 5.0 TB/s).
template <int BLOCK>
__global__ void __launch_bounds__(512) gather_codes_kernel(const GatherParams p)
{
    __shared__ typename Strip<BLOCK, 256>::Slots slots[2];
    ptx::griddep_launch_dependents();
    const int unit = blockIdx.y;
    const int half = threadIdx.x >> 8;
    const int32_t *pos = p.pos + static_cast<size_t>(unit) * p.Pout;
    ptx::griddep_wait();
    gather_strip<BLOCK, 256, BLOCK >= 64>(p, unit, blockIdx.x * Strip<BLOCK, 256>::kRows, p.n_keep, half != 0, threadIdx.x & 255,
                             1 + half, slots[half], [&](int i) { return ptx::load(pos + i); });
}

// ---- selection and gather in one kernel

struct EvictParams {
    SelectParams s;
    GatherParams g;
};

// For few units, where the start of a second kernel and its wait would cost
// more than the rows: gridDim.x CTAs per unit, each of which makes the whole selection (the
// weights come from L2) and gathers its share of the kept rows, whose
// positions it holds in shared memory.
// BLOCK == 0: bf16 rows, a warp moving four rows of K and V at a time.
// BLOCK > 0: 8-bit rows, groups of 256 threads (512 for blocks of 128) taking
// strips of 64 (128) rows of K or of V.
template <int KPT, int BLOCK>
__global__ void __launch_bounds__(kSelectThreads, 1) evict_kernel(const EvictParams p)
{
    __shared__ SelectShared<KPT> sh;
    __shared__ int kept[KPT * kSelectThreads];
    const int unit = blockIdx.y, c = blockIdx.x, C = gridDim.x;
    const GatherParams &g = p.g;
    const size_t in0 = static_cast<size_t>(unit) * g.P, out0 = static_cast<size_t>(unit) * g.Pout;
    constexpr int kUnit = BLOCK > 0 ? BLOCK : 1;  // rows that go to one CTA together
    auto share = [&](int keep) { return ((keep + kUnit - 1) / kUnit + C - 1) / C * kUnit; };
    const int keep = select_positions<KPT>(p.s, unit, sh, [&](int n, int at, int j, float weight) {
        kept[at] = j;
        const int rows = share(n);
        if (at >= c * rows && at < (c + 1) * rows) {
            p.s.pos[out0 + at] = j;
            p.s.mass_out[out0 + at] = weight;
        }
    });
    __syncthreads();
    const int rows = share(keep);
    const int r_begin = min(c * rows, keep), r_end = min(r_begin + rows, keep);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if constexpr (BLOCK == 0) {
        for (int i0 = r_begin + warp; i0 < r_end; i0 += 128) {
            uint4 v[4][2];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (i0 + r * 32 < r_end) {
                    const size_t off = (in0 + static_cast<size_t>(kept[i0 + r * 32])) * 512 + lane * 16;
                    v[r][0] = ptx::load(reinterpret_cast<const uint4 *>(g.k + off));
                    v[r][1] = ptx::load(reinterpret_cast<const uint4 *>(g.v + off));
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (i0 + r * 32 < r_end) {
                    const size_t off = (out0 + i0 + r * 32) * 512 + lane * 16;
                    *reinterpret_cast<uint4 *>(g.k_out + off) = v[r][0];
                    *reinterpret_cast<uint4 *>(g.v_out + off) = v[r][1];
                }
            }
        }
    } else {
        constexpr int kGroup = BLOCK == 128 ? 512 : 256;  // threads of a strip
        constexpr int kGroups = kSelectThreads / kGroup;
        using S = Strip<BLOCK, kGroup>;
        __shared__ typename S::Slots slots[2][kGroups];
        const int group = threadIdx.x / kGroup;
        const int strips = (r_end - r_begin + S::kRows - 1) / S::kRows;
        int turn = 0;  // a group's slots were last read two strips ago, a barrier before
        for (int item = group; item < 2 * strips; item += kGroups, turn ^= 1)
            gather_strip<BLOCK, kGroup, true>(g, unit, r_begin + (item >> 1) * S::kRows, r_end, item & 1,
                                        threadIdx.x % kGroup, 1 + group, slots[turn][group],
                                        [&](int i) { return kept[i]; });
    }
    finish_selection(p.s, unit, keep, c * kSelectThreads + static_cast<int>(threadIdx.x), C * kSelectThreads);
}

}  // namespace cache
}  // namespace dm05
