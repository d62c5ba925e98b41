// prefix_mass_kernel.cuh -- the attention weight each prefix position
// received: mass[j] = mass_in[j] + sum over a KV head's query heads and the
// S queries of exp(<q, k_j> / sqrt(D) - lse).
#pragma once

#include "prefix_cache_kernels.cuh"

namespace dm05 {
namespace mass {

struct Params {
    const __nv_bfloat16 *q;  // [units, GS, 256]
    const uint8_t *k;        // [units, P, 256] bf16 or e4m3
    const float *k_scale;    // 8-bit: [units, nblk]
    const float *lse;        // [units, GS]
    const int32_t *valid_len;
    const uint8_t *mask;
    const float *mass_in;    // or nullptr
    float *mass;
    uint32_t *err;
    int Hkv, P, GS, nblk, shift;
    float scale_log2;
};

// One warp per key.
template <bool KV8>
__global__ void __launch_bounds__(256) mass_kernel(const Params p)
{
    const int unit = blockIdx.y, b = unit / p.Hkv;
    const int lane = threadIdx.x & 31, j = blockIdx.x * 8 + (threadIdx.x >> 5);
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int vl = cache::clamped_len(p.valid_len, b, p.P, p.err, threadIdx.x == 0 && blockIdx.x == 0 && unit % p.Hkv == 0);
    if (j >= p.P) return;
    const size_t at = static_cast<size_t>(unit) * p.P + j;
    const bool seen = j < vl && (p.mask == nullptr || p.mask[static_cast<size_t>(b) * p.P + j] != 0);
    float total = p.mass_in != nullptr ? p.mass_in[at] : 0.0f;
    if (seen) {
        float k[8];
        if (KV8) {
            const uint2 w = *reinterpret_cast<const uint2 *>(p.k + at * 256 + lane * 8);
            const float s = p.k_scale[static_cast<size_t>(unit) * p.nblk + (j >> p.shift)];
            const float4 a = cache::decode4(w.x), c = cache::decode4(w.y);
            const float v[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
            for (int e = 0; e < 8; ++e) k[e] = v[e] * s;
        } else {
            const __nv_bfloat16 *row = reinterpret_cast<const __nv_bfloat16 *>(p.k) + at * 256 + lane * 8;
            for (int e = 0; e < 8; ++e) k[e] = __bfloat162float(row[e]);
        }
        for (int i = 0; i < p.GS; ++i) {
            const size_t qi = static_cast<size_t>(unit) * p.GS + i;
            const __nv_bfloat16 *row = p.q + qi * 256 + lane * 8;
            float dot = 0.0f;
            for (int e = 0; e < 8; ++e) dot = fmaf(__bfloat162float(row[e]), k[e], dot);
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            const float l = p.lse[qi];
            if (l != -INFINITY) total += exp2f(dot * p.scale_log2 - l * 1.4426950408889634f);
        }
    }
    if (lane == 0) p.mass[at] = total;
}

}  // namespace mass
}  // namespace dm05
