// kv8_attn_kernel.cuh -- the suffix attention over an 8-bit prefix cache.
#pragma once

#include "prefix_cache_kernels.cuh"

namespace dm05 {
namespace kv8 {

struct Params {
    const __nv_bfloat16 *q;         // [units, GS, 256]
    const uint8_t *k, *v;           // [units, P, 256] e4m3
    const float *k_scale, *v_scale; // [units, nblk]
    const __nv_bfloat16 *ks, *vs;   // [units, S, 256]
    const int32_t *valid_len;
    const uint8_t *mask;
    __nv_bfloat16 *out;
    float *lse;
    uint32_t *err;
    int Hkv, P, S, GS, nblk, shift;
    float scale_log2;
};

// One CTA per query row: each of the 8 warps takes every eighth key, keeps
// the running maximum and sum of its own softmax, and the warps' parts are
// joined at the end.
__global__ void __launch_bounds__(256) attn_kernel(const Params p)
{
    __shared__ float sm[8], sl[8], so[8][256];
    const int unit = blockIdx.y, b = unit / p.Hkv, i = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int vl = cache::clamped_len(p.valid_len, b, p.P, p.err, threadIdx.x == 0 && i == 0 && unit % p.Hkv == 0);
    const size_t qi = static_cast<size_t>(unit) * p.GS + i;
    float q[8], o[8];
    for (int e = 0; e < 8; ++e) {
        q[e] = __bfloat162float(p.q[qi * 256 + lane * 8 + e]);
        o[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int x = warp; x < p.S + vl; x += 8) {
        float k[8], v[8];
        if (x < p.S) {
            const size_t at = (static_cast<size_t>(unit) * p.S + x) * 256 + lane * 8;
            for (int e = 0; e < 8; ++e) {
                k[e] = __bfloat162float(p.ks[at + e]);
                v[e] = __bfloat162float(p.vs[at + e]);
            }
        } else {
            const int j = x - p.S;
            if (p.mask != nullptr && p.mask[static_cast<size_t>(b) * p.P + j] == 0) continue;
            const size_t at = (static_cast<size_t>(unit) * p.P + j) * 256 + lane * 8;
            const size_t n = static_cast<size_t>(unit) * p.nblk + (j >> p.shift);
            const uint2 kw = *reinterpret_cast<const uint2 *>(p.k + at), vw = *reinterpret_cast<const uint2 *>(p.v + at);
            const float4 k0 = cache::decode4(kw.x), k1 = cache::decode4(kw.y);
            const float4 v0 = cache::decode4(vw.x), v1 = cache::decode4(vw.y);
            const float kk[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
            const float vv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            const float fk = p.k_scale[n], fv = p.v_scale[n];
            for (int e = 0; e < 8; ++e) {
                k[e] = kk[e] * fk;
                v[e] = vv[e] * fv;
            }
        }
        float dot = 0.0f;
        for (int e = 0; e < 8; ++e) dot = fmaf(q[e], k[e], dot);
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        const float z = dot * p.scale_log2;
        const float top = fmaxf(m, z);
        const float f = exp2f(m - top), w = exp2f(z - top);
        l = l * f + w;
        for (int e = 0; e < 8; ++e) o[e] = fmaf(w, v[e], o[e] * f);
        m = top;
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    for (int e = 0; e < 8; ++e) so[warp][lane * 8 + e] = o[e];
    __syncthreads();
    float top = sm[0];
    for (int w = 1; w < 8; ++w) top = fmaxf(top, sm[w]);
    float total = 0.0f, acc = 0.0f;
    for (int w = 0; w < 8; ++w) {
        const float f = sl[w] > 0.0f ? exp2f(sm[w] - top) : 0.0f;
        total += f * sl[w];
        acc += f * so[w][threadIdx.x];
    }
    p.out[qi * 256 + threadIdx.x] = __float2bfloat16_rn(acc / total);
    if (threadIdx.x == 0 && p.lse != nullptr) p.lse[qi] = (top + log2f(total)) * 0.69314718055994531f;
}

}  // namespace kv8
}  // namespace dm05
