// prefix_cache.cu -- C ABI of the prefix-cache compression: the 8-bit cache
// and the suffix attention over it, the attention weight each position
// received, and the eviction of the positions that received least.  The
// operations are specified in include/dm05_suffix_attn.h.
#include "dm05_suffix_attn.h"

#include <cmath>
#include <cstdint>

#include "dm05_internal.h"
#include "kv8_attn_kernel.cuh"
#include "prefix_cache_kernels.cuh"
#include "prefix_mass_kernel.cuh"

namespace {

using dm05::internal::Device;

constexpr int kMaxUnits = 65535;      // B * Hkv: a grid dimension of these kernels
constexpr int kMaxPrefix = 1 << 24;   // P
constexpr double kLog2e = 1.4426950408889634;

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }

// log2 of a supported block of tokens, or -1
int block_shift(int block)
{
    switch (block) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
    }
}

int blocks_of(int P, int shift) { return (P + (1 << shift) - 1) >> shift; }

int check_cache(int B, int Hkv, int P, int D)
{
    if (B < 1 || Hkv < 1 || P < 1 || P > kMaxPrefix) return DM05_ERR_SHAPE;
    if (static_cast<long long>(B) * Hkv > kMaxUnits) return DM05_ERR_SHAPE;
    return D == dm05::kHeadDim ? DM05_OK : DM05_ERR_UNSUPPORTED;
}

// Launch with programmatic dependent launch, as every kernel of the library.
template <class K, class P>
int launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const P &params)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, params) == cudaSuccess ? DM05_OK : DM05_ERR_CUDA;
}

int mass_call(bool kv8, const void *q, const void *k, const float *k_scale, int shift, const int32_t *valid_len,
              const uint8_t *mask, const float *lse, const float *mass_in, float *mass, int B, int Hq, int Hkv, int P,
              int S, int D, cudaStream_t stream)
{
    if (!q || !k || !lse || !mass || (kv8 && !k_scale)) return DM05_ERR_NULL;
    if (Hq < 1 || S < 1) return DM05_ERR_SHAPE;
    int rc = check_cache(B, Hkv, P, D);
    if (rc != DM05_OK) return rc;
    if (Hq % Hkv != 0) return DM05_ERR_SHAPE;
    if (shift < 0 || static_cast<long long>(Hq / Hkv) * S > dm05::kMRows) return DM05_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(lse, 4) || !aligned(mass, 4) || !aligned(mass_in, 4) ||
        !aligned(valid_len, 4) || !aligned(k_scale, 4))
        return DM05_ERR_ALIGN;
    Device dev;
    rc = dm05::internal::device(stream, true, &dev);
    if (rc != DM05_OK) return rc;
    dm05::mass::Params mp = {};
    mp.q = static_cast<const __nv_bfloat16 *>(q);
    mp.k = static_cast<const uint8_t *>(k);
    mp.k_scale = k_scale;
    mp.lse = lse;
    mp.valid_len = valid_len;
    mp.mask = mask;
    mp.mass_in = mass_in;
    mp.mass = mass;
    mp.err = dev.err;
    mp.Hkv = Hkv;
    mp.P = P;
    mp.GS = Hq / Hkv * S;
    mp.nblk = blocks_of(P, shift);
    mp.shift = shift;
    mp.scale_log2 = static_cast<float>(kLog2e / std::sqrt(static_cast<double>(D)));
    const dim3 grid(static_cast<unsigned>((P + 7) / 8), static_cast<unsigned>(B * Hkv));
    return kv8 ? launch(dm05::mass::mass_kernel<true>, grid, 256, 0, stream, mp)
               : launch(dm05::mass::mass_kernel<false>, grid, 256, 0, stream, mp);
}

int evict_checks(const void *k, const void *v, const float *mass, const int32_t *valid_len, const void *k_out,
                 const void *v_out, const float *mass_out, const int32_t *positions, const int32_t *valid_out, int B,
                 int Hkv, int P, int P_out, int D, int n_keep, int n_first, int n_last)
{
    if (!k || !v || !mass || !k_out || !v_out || !mass_out || !positions || !valid_out) return DM05_ERR_NULL;
    const int rc = check_cache(B, Hkv, P, D);
    if (rc != DM05_OK) return rc;
    if (P_out < 1 || P_out > kMaxPrefix || n_keep < 0 || n_keep > P_out || n_first < 0 || n_last < 0)
        return DM05_ERR_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(mass, 4) ||
        !aligned(mass_out, 4) || !aligned(positions, 4) || !aligned(valid_out, 4) || !aligned(valid_len, 4))
        return DM05_ERR_ALIGN;
    return DM05_OK;
}

int launch_select(const float *mass, const int32_t *valid_len, const uint8_t *mask, float *mass_out,
                  int32_t *positions, int32_t *valid_out, uint32_t *err, int B, int Hkv, int P, int P_out, int n_keep,
                  int n_first, int n_last, cudaStream_t stream)
{
    dm05::cache::SelectParams sp = {};
    sp.mass = mass;
    sp.valid_len = valid_len;
    sp.mask = mask;
    sp.mass_out = mass_out;
    sp.pos = positions;
    sp.valid_out = valid_out;
    sp.err = err;
    sp.Hkv = Hkv;
    sp.P = P;
    sp.Pout = P_out;
    sp.n_keep = n_keep;
    sp.n_first = n_first;
    sp.n_last = n_last;
    return launch(dm05::cache::select_kernel, dim3(static_cast<unsigned>(B * Hkv)), dm05::cache::kSelectThreads, 0,
                  stream, sp);
}

}  // namespace

extern "C" {

int dm05_kv8_quantize(const void *k, const void *v, const int32_t *valid_len, void *k8, void *v8, float *k_scale,
                      float *v_scale, int B, int Hkv, int P, int D, int block, int first, cudaStream_t stream)
{
    if (!k || !v || !k8 || !v8 || !k_scale || !v_scale) return DM05_ERR_NULL;
    int rc = check_cache(B, Hkv, P, D);
    if (rc != DM05_OK) return rc;
    const int shift = block_shift(block);
    if (shift < 0) return DM05_ERR_UNSUPPORTED;
    if (first < 0 || first >= P || first % block != 0) return DM05_ERR_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k8, 16) || !aligned(v8, 16) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4) || !aligned(valid_len, 4))
        return DM05_ERR_ALIGN;
    Device dev;
    rc = dm05::internal::device(stream, true, &dev);
    if (rc != DM05_OK) return rc;
    dm05::cache::QuantParams qp = {};
    qp.k = static_cast<const __nv_bfloat16 *>(k);
    qp.v = static_cast<const __nv_bfloat16 *>(v);
    qp.k8 = static_cast<uint8_t *>(k8);
    qp.v8 = static_cast<uint8_t *>(v8);
    qp.k_scale = k_scale;
    qp.v_scale = v_scale;
    qp.valid_len = valid_len;
    qp.err = dev.err;
    qp.Hkv = Hkv;
    qp.P = P;
    qp.nblk = blocks_of(P, shift);
    qp.blk0 = first >> shift;
    const dim3 grid(static_cast<unsigned>(qp.nblk - qp.blk0), static_cast<unsigned>(B * Hkv), 2);
    switch (block) {
    case 16: return launch(dm05::cache::quantize_kernel<16>, grid, 256, 0, stream, qp);
    case 32: return launch(dm05::cache::quantize_kernel<32>, grid, 256, 0, stream, qp);
    case 64: return launch(dm05::cache::quantize_kernel<64>, grid, 256, 0, stream, qp);
    default: return launch(dm05::cache::quantize_kernel<128>, grid, 256, 0, stream, qp);
    }
}

int dm05_suffix_attn_kv8_plan(int B, int Hq, int Hkv, int P, int S, int D, int *splits_per_head, int *tile_rows,
                              int *row_blocks, size_t *workspace_bytes)
{
    if (B < 1 || Hq < 1 || Hkv < 1 || S < 1 || P < 0 || Hq % Hkv != 0) return DM05_ERR_SHAPE;
    if (splits_per_head) *splits_per_head = 1;
    if (tile_rows) *tile_rows = 1;
    if (row_blocks) *row_blocks = 1;
    if (workspace_bytes) *workspace_bytes = 0;
    return DM05_OK;
}

int dm05_suffix_attn_kv8(const void *q, const void *k8, const void *v8, const float *k_scale, const float *v_scale,
                         int block, const int32_t *prefix_valid_len, const uint8_t *prefix_mask, const void *k_suffix,
                         const void *v_suffix, void *out, float *lse, void *workspace, size_t workspace_bytes, int B,
                         int Hq, int Hkv, int P, int S, int D, cudaStream_t stream)
{
    (void)workspace;
    (void)workspace_bytes;
    if (!q || !k_suffix || !v_suffix || !out) return DM05_ERR_NULL;
    if (P > 0 && (!k8 || !v8 || !k_scale || !v_scale)) return DM05_ERR_NULL;
    if (B < 1 || Hq < 1 || Hkv < 1 || S < 1 || P < 0 || P > kMaxPrefix || Hq % Hkv != 0) return DM05_ERR_SHAPE;
    if (static_cast<long long>(B) * Hkv > kMaxUnits) return DM05_ERR_SHAPE;
    const int shift = block_shift(block);
    if (D != dm05::kHeadDim || shift < 0 || static_cast<long long>(Hq / Hkv) * S > dm05::kMRows)
        return DM05_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k_suffix, 16) || !aligned(v_suffix, 16) || !aligned(out, 16) ||
        !aligned(lse, 4) || !aligned(prefix_valid_len, 4) ||
        (P > 0 && (!aligned(k8, 16) || !aligned(v8, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4))))
        return DM05_ERR_ALIGN;
    Device dev;
    const int rc = dm05::internal::device(stream, true, &dev);
    if (rc != DM05_OK) return rc;
    dm05::kv8::Params ap = {};
    ap.q = static_cast<const __nv_bfloat16 *>(q);
    ap.k = static_cast<const uint8_t *>(k8);
    ap.v = static_cast<const uint8_t *>(v8);
    ap.k_scale = k_scale;
    ap.v_scale = v_scale;
    ap.ks = static_cast<const __nv_bfloat16 *>(k_suffix);
    ap.vs = static_cast<const __nv_bfloat16 *>(v_suffix);
    ap.valid_len = prefix_valid_len;
    ap.mask = prefix_mask;
    ap.out = static_cast<__nv_bfloat16 *>(out);
    ap.lse = lse;
    ap.err = dev.err;
    ap.Hkv = Hkv;
    ap.P = P;
    ap.S = S;
    ap.GS = Hq / Hkv * S;
    ap.nblk = blocks_of(P, shift);
    ap.shift = shift;
    ap.scale_log2 = static_cast<float>(kLog2e / std::sqrt(static_cast<double>(D)));
    return launch(dm05::kv8::attn_kernel, dim3(static_cast<unsigned>(ap.GS), static_cast<unsigned>(B * Hkv)), 256, 0,
                  stream, ap);
}

int dm05_prefix_attn_mass(const void *q, const void *k_prefix, const int32_t *prefix_valid_len,
                          const uint8_t *prefix_mask, const float *lse, const float *mass_in, float *mass, int B,
                          int Hq, int Hkv, int P, int S, int D, cudaStream_t stream)
{
    return mass_call(false, q, k_prefix, nullptr, 0, prefix_valid_len, prefix_mask, lse, mass_in, mass, B, Hq, Hkv, P,
                     S, D, stream);
}

int dm05_prefix_attn_mass_kv8(const void *q, const void *k8, const float *k_scale, int block,
                              const int32_t *prefix_valid_len, const uint8_t *prefix_mask, const float *lse,
                              const float *mass_in, float *mass, int B, int Hq, int Hkv, int P, int S, int D,
                              cudaStream_t stream)
{
    return mass_call(true, q, k8, k_scale, block_shift(block), prefix_valid_len, prefix_mask, lse, mass_in, mass, B,
                     Hq, Hkv, P, S, D, stream);
}

int dm05_prefix_evict(const void *k, const void *v, const float *mass, const int32_t *valid_len, const uint8_t *mask,
                      void *k_out, void *v_out, float *mass_out, int32_t *positions, int32_t *valid_out, int B,
                      int Hkv, int P, int P_out, int D, int n_keep, int n_first, int n_last, cudaStream_t stream)
{
    int rc = evict_checks(k, v, mass, valid_len, k_out, v_out, mass_out, positions, valid_out, B, Hkv, P, P_out, D,
                          n_keep, n_first, n_last);
    if (rc != DM05_OK) return rc;
    Device dev;
    rc = dm05::internal::device(stream, true, &dev);
    if (rc != DM05_OK) return rc;
    rc = launch_select(mass, valid_len, mask, mass_out, positions, valid_out, dev.err, B, Hkv, P, P_out, n_keep,
                       n_first, n_last, stream);
    if (rc != DM05_OK || n_keep == 0) return rc;
    dm05::cache::GatherParams gp = {};
    gp.k = static_cast<const uint8_t *>(k);
    gp.v = static_cast<const uint8_t *>(v);
    gp.k_out = static_cast<uint8_t *>(k_out);
    gp.v_out = static_cast<uint8_t *>(v_out);
    gp.pos = positions;
    gp.valid = valid_out;
    gp.Hkv = Hkv;
    gp.P = P;
    gp.Pout = P_out;
    return launch(dm05::cache::gather_rows_kernel,
                  dim3(static_cast<unsigned>((n_keep + 31) / 32), static_cast<unsigned>(B * Hkv)), 256, 0, stream, gp);
}

int dm05_prefix_evict_kv8(const void *k8, const void *v8, const float *k_scale, const float *v_scale, int block,
                          const float *mass, const int32_t *valid_len, const uint8_t *mask, void *k8_out,
                          void *v8_out, float *k_scale_out, float *v_scale_out, float *mass_out, int32_t *positions,
                          int32_t *valid_out, int B, int Hkv, int P, int P_out, int D, int n_keep, int n_first,
                          int n_last, cudaStream_t stream)
{
    if (!k_scale || !v_scale || !k_scale_out || !v_scale_out) return DM05_ERR_NULL;
    int rc = evict_checks(k8, v8, mass, valid_len, k8_out, v8_out, mass_out, positions, valid_out, B, Hkv, P, P_out,
                          D, n_keep, n_first, n_last);
    if (rc != DM05_OK) return rc;
    const int shift = block_shift(block);
    if (shift < 0) return DM05_ERR_UNSUPPORTED;
    if (!aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(k_scale_out, 4) || !aligned(v_scale_out, 4))
        return DM05_ERR_ALIGN;
    Device dev;
    rc = dm05::internal::device(stream, true, &dev);
    if (rc != DM05_OK) return rc;
    rc = launch_select(mass, valid_len, mask, mass_out, positions, valid_out, dev.err, B, Hkv, P, P_out, n_keep,
                       n_first, n_last, stream);
    if (rc != DM05_OK || n_keep == 0) return rc;
    dm05::cache::GatherParams gp = {};
    gp.k = static_cast<const uint8_t *>(k8);
    gp.v = static_cast<const uint8_t *>(v8);
    gp.k_out = static_cast<uint8_t *>(k8_out);
    gp.v_out = static_cast<uint8_t *>(v8_out);
    gp.k_scale = k_scale;
    gp.v_scale = v_scale;
    gp.k_scale_out = k_scale_out;
    gp.v_scale_out = v_scale_out;
    gp.pos = positions;
    gp.valid = valid_out;
    gp.Hkv = Hkv;
    gp.P = P;
    gp.Pout = P_out;
    gp.nblk = blocks_of(P, shift);
    gp.nblk_out = blocks_of(P_out, shift);
    gp.shift = shift;
    const dim3 grid(static_cast<unsigned>((n_keep + block - 1) >> shift), static_cast<unsigned>(B * Hkv), 2);
    switch (block) {
    case 16: return launch(dm05::cache::gather_codes_kernel<16>, grid, 256, 0, stream, gp);
    case 32: return launch(dm05::cache::gather_codes_kernel<32>, grid, 256, 0, stream, gp);
    case 64: return launch(dm05::cache::gather_codes_kernel<64>, grid, 256, 0, stream, gp);
    default: return launch(dm05::cache::gather_codes_kernel<128>, grid, 256, 0, stream, gp);
    }
}

}  // extern "C"
