// prefix_cache.cu -- C ABI of the prefix-cache compression: the 8-bit cache
// and the suffix attention over it, the attention weight each position
// received, and the eviction of the positions that received least.  The
// operations are specified in include/dm05_suffix_attn.h.
#include "dm05_suffix_attn.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

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

// ---------------------------------------------------------------- kv8 attention plan

constexpr int kMaxDevices = 64;
std::mutex g_attr_mu;
constexpr int kMaxCluster = 16;  // the hardware's largest
bool g_mass_ready[kMaxDevices];
struct Kv8Device {
    bool ready;
    int active[kMaxCluster + 1];  // clusters of this many CTAs that run at once
} g_kv8[kMaxDevices];

auto *kv8_kernel(int copies, bool cluster)
{
    using namespace dm05::kv8;
    if (cluster) return &attn_kernel<1, true>;
    return copies == 4 ? &attn_kernel<4, false> : copies == 2 ? &attn_kernel<2, false> : &attn_kernel<1, false>;
}

// Kernel attributes of the attention or of the weight kernels, once per device.
int set_attributes(const Device &dev, bool mass) noexcept
{
    if (dev.ordinal < 0 || dev.ordinal >= kMaxDevices) return DM05_ERR_CUDA;
    try {
        std::lock_guard<std::mutex> lk(g_attr_mu);
        bool &ready = mass ? g_mass_ready[dev.ordinal] : g_kv8[dev.ordinal].ready;
        if (ready) return DM05_OK;
        constexpr cudaFuncAttribute kSmem = cudaFuncAttributeMaxDynamicSharedMemorySize;
        constexpr int kSmem8 = dm05::kv8::Smem::kAllocBytes;
        bool ok;
        if (mass)
            ok = cudaFuncSetAttribute(&dm05::mass::mass_kernel<false>, kSmem, dm05::mass::Smem<false>::kAllocBytes) ==
                     cudaSuccess &&
                 cudaFuncSetAttribute(&dm05::mass::mass_kernel<true>, kSmem, dm05::mass::Smem<true>::kAllocBytes) ==
                     cudaSuccess;
        else
            ok = cudaFuncSetAttribute(kv8_kernel(1, false), kSmem, kSmem8) == cudaSuccess &&
                 cudaFuncSetAttribute(kv8_kernel(2, false), kSmem, kSmem8) == cudaSuccess &&
                 cudaFuncSetAttribute(kv8_kernel(4, false), kSmem, kSmem8) == cudaSuccess &&
                 cudaFuncSetAttribute(kv8_kernel(1, true), kSmem, kSmem8) == cudaSuccess &&
                 cudaFuncSetAttribute(kv8_kernel(1, true), cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                     cudaSuccess;
        if (!ok) return DM05_ERR_CUDA;
        for (int c = 2; !mass && c <= kMaxCluster; ++c) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(c), 1, 1);
            cfg.blockDim = dim3(dm05::kv8::kThreads8, 1, 1);
            cfg.dynamicSmemBytes = kSmem8;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = static_cast<unsigned>(c);
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kv8_kernel(1, true), &cfg) != cudaSuccess) {
                cudaGetLastError();  // a refused size: never used
                n = 0;
            }
            g_kv8[dev.ordinal].active[c] = n;
        }
        ready = true;
        return DM05_OK;
    } catch (...) {
        return DM05_ERR_CUDA;
    }
}

constexpr int kCopyRun = 4;        // tiles a CTA walks from which few query rows are copied
constexpr int kClusterRows = 384;  // partial rows a cluster joins

struct Kv8Plan {
    int splits = 1;      // CTAs per (sample, KV head) and block of query rows
    int row_blocks = 1;  // blocks of the GS query rows
    int qrows = 8;       // rows of a block (a multiple of 8)
    int copies = 1;      // how often a block's rows are laid over the MMA's 128
    bool cluster = false;  // the splits of a unit are a cluster that joins their rows
    size_t bytes = 0;    // partial results of the others
};

// The fewest CTAs per (sample, KV head) that make the longest run of tiles as
// short as one wave allows; unsplit while that is as short.  A split unit's
// query rows are cut into blocks while SMs are left (at least 32 rows each):
// every CTA then prepares, stages and writes fewer rows, for K and V tiles read
// from L2 once more (B = 1, P = 1024, S = 64: 12.6 instead of 14.4 us; B = 2, S = 50:
// 13.5 instead of 14.9).  Few rows are copied over the MMA's when a CTA walks at least
// four tiles (B = 2, P = 30016: S = 10 37.6 instead of 43.3 us, S = 30 44.0 instead of
// 45.4; always: B = 1, P = 1024, S = 64 13.4 instead of 12.6).
//
// Splits that fit a cluster join their rows inside it as long as all clusters
// run at once (for which the rows may be cut into fewer blocks) and the partial
// rows of a cluster are few.  In a cluster / with a second kernel (us, splits x
// rows): B = 1, P = 576, S = 1, 6 x 8: 8.7 / 9.7; B = 1, P = 1024: S = 10, 9 x 24: 10.0 / 10.3;
// S = 50, 9 x 40: 12.4 / 13.1; S = 25, 9 x 56: 12.1 / 11.4; S = 64, 9 x 48: 12.9 / 12.6; B = 2, P = 576,
// S = 50, 6 x 56: 12.8 / 13.6; B = 2, P = 1024: S = 16, 9 x 32: 11.4 / 11.8; S = 32, 9 x 64:
// 13.6 / 12.6; S = 50, 9 x 104: 17.0 / 13.5.  Call after set_attributes(dev, false).
Kv8Plan kv8_plan(int B, int Hq, int Hkv, int P, int S, const Device &dev)
{
    const long long units = static_cast<long long>(B) * Hkv;
    const int GS = Hq / Hkv * S;
    const int tiles = (P + dm05::kv8::kTile - 1) / dm05::kv8::kTile + (S + dm05::kv8::kSufTile - 1) / dm05::kv8::kSufTile;
    const int most = static_cast<int>(std::min<long long>(
        std::min(tiles, dm05::kv8::kMaxSplits8), std::max<long long>(1, dev.num_sms / units)));
    Kv8Plan pl;
    if (dev.split_override > 0) {
        pl.splits = dev.split_override;
    } else {
        const int longest = (tiles + most - 1) / most;
        pl.splits = (tiles + longest - 1) / longest;
    }
    const int run = (tiles + pl.splits - 1) / pl.splits;
    auto cut = [&](long long blocks) {
        const int n = static_cast<int>(std::max<long long>(1, blocks));
        pl.qrows = ((GS + n - 1) / n + 7) / 8 * 8;
        pl.row_blocks = (GS + pl.qrows - 1) / pl.qrows;
    };
    cut(1);
    if (pl.splits > 1) {
        const long long blocks = std::min<long long>(GS / 32, dev.num_sms / (units * pl.splits));
        const long long at_once = pl.splits <= kMaxCluster ? g_kv8[dev.ordinal].active[pl.splits] : 0;
        cut(std::min(blocks, at_once / units));
        pl.cluster = run < kCopyRun && units <= at_once && pl.qrows * pl.splits <= kClusterRows;
        if (!pl.cluster) cut(blocks);
    }
    pl.copies = run < kCopyRun ? 1 : pl.qrows <= 32 ? 4 : pl.qrows <= 64 ? 2 : 1;
    if (pl.splits > 1 && !pl.cluster) pl.bytes = static_cast<size_t>(units) * pl.splits * GS * dm05::kv8::kPartRow;
    return pl;
}

int kv8_check(int B, int Hq, int Hkv, int P, int S, int D)
{
    if (B < 1 || Hq < 1 || Hkv < 1 || S < 1 || P < 0 || P > kMaxPrefix || Hq % Hkv != 0) return DM05_ERR_SHAPE;
    if (static_cast<long long>(B) * Hkv > kMaxUnits) return DM05_ERR_SHAPE;
    if (D != dm05::kHeadDim || static_cast<long long>(Hq / Hkv) * S > dm05::kMRows) return DM05_ERR_UNSUPPORTED;
    return DM05_OK;
}

// bf16 [units][rows][256] in boxes of box_rows rows: box_chunks 64-column
// chunks of 128 swizzled bytes
int encode_rows16(CUtensorMap *map, const void *base, int rows, int units, int box_rows, int box_chunks = 4)
{
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), 4, static_cast<cuuint64_t>(units)};
    const cuuint64_t strides[3] = {512, 128, static_cast<cuuint64_t>(rows) * 512};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_chunks), 1};
    return dm05::internal::encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box);
}

// codes [units][rows][256] in boxes of box_rows rows: two 128-column chunks
int encode_rows8(CUtensorMap *map, const void *base, int rows, int units, int box_rows)
{
    const cuuint64_t dims[4] = {128, static_cast<cuuint64_t>(rows), 2, static_cast<cuuint64_t>(units)};
    const cuuint64_t strides[3] = {256, 128, static_cast<cuuint64_t>(rows) * 256};
    const cuuint32_t box[4] = {128, static_cast<cuuint32_t>(box_rows), 2, 1};
    return dm05::internal::encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box);
}

// ---------------------------------------------------------------- accumulated weight

// CTAs per unit: the fewest waves x (set-up + tiles a CTA walks), set-up
// counted as two tiles.
int mass_splits(int units, int tiles, int num_sms)
{
    int best = 1;
    long long best_cost = -1;
    for (int s = 1; s <= std::min(tiles, num_sms); ++s) {
        const long long waves = (static_cast<long long>(units) * s + num_sms - 1) / num_sms;
        const long long cost = waves * (2 + (tiles + s - 1) / s);
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best = s;
        }
    }
    return best;
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
    if ((rc = set_attributes(dev, true)) != DM05_OK) return rc;
    const int units = B * Hkv, GS = Hq / Hkv * S, N = (GS + 15) / 16 * 16;
    CUtensorMap tq, tk;
    if (encode_rows16(&tq, q, GS, units, N) != DM05_OK ||
        (kv8 ? encode_rows8(&tk, k, P, units, dm05::mass::kTile) : encode_rows16(&tk, k, P, units, dm05::mass::kTile)) !=
            DM05_OK)
        return DM05_ERR_CUDA;
    dm05::mass::Params mp = {};
    mp.k_scale = k_scale;
    mp.lse = lse;
    mp.valid_len = valid_len;
    mp.mask = mask;
    mp.mass_in = mass_in;
    mp.mass = mass;
    mp.err = dev.err;
    mp.Hkv = Hkv;
    mp.P = P;
    mp.GS = GS;
    mp.N = N;
    mp.nblk = blocks_of(P, shift);
    mp.shift = shift;
    mp.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
    const int splits = mass_splits(units, (P + dm05::mass::kTile - 1) / dm05::mass::kTile, dev.num_sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(splits), static_cast<unsigned>(units), 1);
    cfg.blockDim = dim3(dm05::mass::kThreadsM, 1, 1);
    cfg.dynamicSmemBytes = kv8 ? dm05::mass::Smem<true>::kAllocBytes : dm05::mass::Smem<false>::kAllocBytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = kv8 ? cudaLaunchKernelEx(&cfg, &dm05::mass::mass_kernel<true>, tq, tk, mp)
                              : cudaLaunchKernelEx(&cfg, &dm05::mass::mass_kernel<false>, tq, tk, mp);
    return e == cudaSuccess ? DM05_OK : DM05_ERR_CUDA;
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

struct Range {
    const void *p;
    size_t n;
    bool meets(const Range &o) const
    {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return p != nullptr && o.p != nullptr && n != 0 && o.n != 0 && a < b + o.n && b < a + n;
    }
};

// The arrays of an eviction.  CTAs of a unit, and of a sample's heads, read all
// of the inputs while others already write: no output may lie on an input, nor
// on another output.
struct EvictArrays {
    Range k, v, k_scale, v_scale, mass, valid_len, mask;
    Range k_out, v_out, k_scale_out, v_scale_out, mass_out, positions, valid_out;

    // rows of row_bytes; nblk > 0: an 8-bit cache with so many scales a unit
    EvictArrays(const dm05::cache::EvictParams &ep, int row_bytes, int B, int nblk, int nblk_out)
    {
        const size_t units = static_cast<size_t>(B) * ep.s.Hkv, rows = units * ep.s.P, rows_out = units * ep.s.Pout;
        k = {ep.g.k, rows * row_bytes};
        v = {ep.g.v, rows * row_bytes};
        k_scale = {ep.g.k_scale, units * nblk * 4};
        v_scale = {ep.g.v_scale, units * nblk * 4};
        mass = {ep.s.mass, rows * 4};
        valid_len = {ep.s.valid_len, static_cast<size_t>(B) * 4};
        mask = {ep.s.mask, static_cast<size_t>(B) * ep.s.P};
        k_out = {ep.g.k_out, rows_out * row_bytes};
        v_out = {ep.g.v_out, rows_out * row_bytes};
        k_scale_out = {ep.g.k_scale_out, units * nblk_out * 4};
        v_scale_out = {ep.g.v_scale_out, units * nblk_out * 4};
        mass_out = {ep.s.mass_out, rows_out * 4};
        positions = {ep.s.pos, rows_out * 4};
        valid_out = {ep.s.valid_out, static_cast<size_t>(B) * 4};
    }

    // The new cache, its weights and its lengths: known without a device.
    bool overlap() const
    {
        for (const Range &o : {k_out, v_out, mass_out})
            for (const Range &i : {k, v, k_scale, v_scale, mass, valid_len, mask, positions, valid_out})
                if (o.meets(i)) return true;
        for (const Range &o : {positions, valid_out})
            for (const Range &i : {mass, valid_len, mask})
                if (o.meets(i)) return true;
        return k_out.meets(v_out) || k_out.meets(mass_out) || v_out.meets(mass_out);
    }

    // Every other pair, before the launch.
    bool overlap_rest() const
    {
        const Range outs[] = {k_scale_out, v_scale_out, positions, valid_out, k_out, v_out, mass_out};
        for (int a = 0; a < 4; ++a) {
            for (const Range &i : {k, v, k_scale, v_scale, mass, valid_len, mask})
                if (outs[a].meets(i)) return true;
            for (int b = a + 1; b < 7; ++b)
                if (outs[a].meets(outs[b])) return true;
        }
        return false;
    }
};

// CTAs per unit of the one-kernel eviction: what one wave holds, at most one
// for each block (8-bit) or eight rows (bf16); 0 where the selection and a
// gather of finer grain behind it are faster: many rows a CTA, more units than
// SMs, or more positions than a CTA's registers hold.
int evict_ctas(int units, int P, int n_keep, int block, int num_sms)
{
    if (units > num_sms || n_keep == 0 || P > 8 * dm05::cache::kSelectThreads) return 0;
    const int rows = block > 0 ? block : 8, parts = (n_keep + rows - 1) / rows;
    const int ctas = std::min(num_sms / units, parts);
    return (parts + ctas - 1) / ctas * rows <= 256 ? ctas : 0;
}

template <int BLOCK>
int launch_evict(const dm05::cache::EvictParams &ep, int ctas, int units, cudaStream_t stream)
{
    using namespace dm05::cache;
    constexpr int kT = kSelectThreads;
    const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(units));
    if (ep.s.P <= kT) return launch(evict_kernel<1, BLOCK>, grid, kT, 0, stream, ep);
    if (ep.s.P <= 2 * kT) return launch(evict_kernel<2, BLOCK>, grid, kT, 0, stream, ep);
    if (ep.s.P <= 4 * kT) return launch(evict_kernel<4, BLOCK>, grid, kT, 0, stream, ep);
    return launch(evict_kernel<8, BLOCK>, grid, kT, 0, stream, ep);
}

int launch_select(const dm05::cache::SelectParams &sp, int units, cudaStream_t stream)
{
    using namespace dm05::cache;
    const dim3 grid(1, static_cast<unsigned>(units));
    constexpr int kT = kSelectThreads;
    if (sp.P <= kT) return launch(select_kernel<1>, grid, kT, 0, stream, sp);
    if (sp.P <= 2 * kT) return launch(select_kernel<2>, grid, kT, 0, stream, sp);
    if (sp.P <= 4 * kT) return launch(select_kernel<4>, grid, kT, 0, stream, sp);
    if (sp.P <= 8 * kT) return launch(select_kernel<8>, grid, kT, 0, stream, sp);
    return launch(select_kernel<0>, grid, kT, 0, stream, sp);
}

template <int BLOCK>
int launch_gather(const dm05::cache::GatherParams &gp, int units, int n_keep, cudaStream_t stream)
{
    constexpr int kRows = dm05::cache::Strip<BLOCK, 256>::kRows;
    return launch(dm05::cache::gather_codes_kernel<BLOCK>,
                  dim3(static_cast<unsigned>((n_keep + kRows - 1) / kRows), static_cast<unsigned>(units)), 512, 0, stream,
                  gp);
}

// One kernel or two (microseconds, P = 1024, 512 rows kept, bf16 / blocks of
// 64): 4 samples of 4 heads 7.2 / 6.6 in one, 8.4 / 7.9 in two; 18 samples
// 16.4 / 12.5 and 17.3 / 13.2; 25 samples, with one CTA a unit 22.8 / 17.9
// and 21.8 / 16.0.
int run_evict(const dm05::cache::EvictParams &ep, int units, int n_keep, int block, int num_sms, cudaStream_t stream)
{
    using namespace dm05::cache;
    const int ctas = evict_ctas(units, ep.s.P, n_keep, block, num_sms);
    if (ctas > 0) {
        switch (block) {
        case 0: return launch_evict<0>(ep, ctas, units, stream);
        case 16: return launch_evict<16>(ep, ctas, units, stream);
        case 32: return launch_evict<32>(ep, ctas, units, stream);
        case 64: return launch_evict<64>(ep, ctas, units, stream);
        default: return launch_evict<128>(ep, ctas, units, stream);
        }
    }
    const int rc = launch_select(ep.s, units, stream);
    if (rc != DM05_OK || n_keep == 0) return rc;
    if (block == 0)
        return launch(gather_rows_kernel, dim3(static_cast<unsigned>((n_keep + 31) / 32), static_cast<unsigned>(units)),
                      256, 0, stream, ep.g);
    switch (block) {
    case 16: return launch_gather<16>(ep.g, units, n_keep, stream);
    case 32: return launch_gather<32>(ep.g, units, n_keep, stream);
    case 64: return launch_gather<64>(ep.g, units, n_keep, stream);
    default: return launch_gather<128>(ep.g, units, n_keep, stream);
    }
}

dm05::cache::SelectParams select_params(const float *mass, const int32_t *valid_len, const uint8_t *mask,
                                        float *mass_out, int32_t *positions, int32_t *valid_out, int Hkv, int P,
                                        int P_out, int n_keep, int n_first, int n_last)
{
    dm05::cache::SelectParams sp = {};
    sp.mass = mass;
    sp.valid_len = valid_len;
    sp.mask = mask;
    sp.mass_out = mass_out;
    sp.pos = positions;
    sp.valid_out = valid_out;
    sp.Hkv = Hkv;
    sp.P = P;
    sp.Pout = P_out;
    sp.n_keep = n_keep;
    sp.n_first = n_first;
    sp.n_last = n_last;
    return sp;
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
                              size_t *workspace_bytes)
{
    int rc = kv8_check(B, Hq, Hkv, P, S, D);
    if (rc != DM05_OK) return rc;
    Device dev;
    if ((rc = dm05::internal::device(nullptr, false, &dev)) != DM05_OK || (rc = set_attributes(dev, false)) != DM05_OK)
        return rc;
    const Kv8Plan pl = kv8_plan(B, Hq, Hkv, P, S, dev);
    if (splits_per_head) *splits_per_head = pl.splits;
    if (tile_rows) *tile_rows = dm05::kv8::kTile;
    if (workspace_bytes) *workspace_bytes = pl.bytes;
    return DM05_OK;
}

int dm05_suffix_attn_kv8(const void *q, const void *k8, const void *v8, const float *k_scale, const float *v_scale,
                         int block, const int32_t *prefix_valid_len, const uint8_t *prefix_mask, const void *k_suffix,
                         const void *v_suffix, void *out, float *lse, void *workspace, size_t workspace_bytes, int B,
                         int Hq, int Hkv, int P, int S, int D, cudaStream_t stream)
{
    if (!q || !k_suffix || !v_suffix || !out) return DM05_ERR_NULL;
    if (P > 0 && (!k8 || !v8 || !k_scale || !v_scale)) return DM05_ERR_NULL;
    int rc = kv8_check(B, Hq, Hkv, P, S, D);
    if (rc != DM05_OK) return rc;
    const int shift = block_shift(block);
    if (shift < 0) return DM05_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k_suffix, 16) || !aligned(v_suffix, 16) || !aligned(out, 16) ||
        !aligned(lse, 4) || !aligned(prefix_valid_len, 4) ||
        (P > 0 && (!aligned(k8, 16) || !aligned(v8, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4))))
        return DM05_ERR_ALIGN;
    Device dev;
    if ((rc = dm05::internal::device(stream, true, &dev)) != DM05_OK || (rc = set_attributes(dev, false)) != DM05_OK)
        return rc;
    const Kv8Plan pl = kv8_plan(B, Hq, Hkv, P, S, dev);
    if (pl.bytes > 0) {
        if (workspace == nullptr || workspace_bytes < pl.bytes) return DM05_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return DM05_ERR_ALIGN;
    }
    const int GS = Hq / Hkv * S, units = B * Hkv;
    const long long grid = static_cast<long long>(units) * pl.row_blocks * pl.splits;
    if (grid > 0x7fffffffLL) return DM05_ERR_SHAPE;
    CUtensorMap tq, tkp, tvp, tks, tvs, to;
    if (encode_rows16(&tq, q, GS, units, pl.qrows, pl.copies == 1 ? 4 : 1) != DM05_OK ||
        encode_rows16(&to, out, GS, units, pl.qrows) != DM05_OK ||
        encode_rows16(&tks, k_suffix, S, units, dm05::kv8::kSufTile) != DM05_OK ||
        encode_rows16(&tvs, v_suffix, S, units, dm05::kv8::kSufTile) != DM05_OK)
        return DM05_ERR_CUDA;
    if (P > 0) {
        if (encode_rows8(&tkp, k8, P, units, dm05::kv8::kTile) != DM05_OK ||
            encode_rows8(&tvp, v8, P, units, dm05::kv8::kTile) != DM05_OK)
            return DM05_ERR_CUDA;
    } else {
        tkp = tks;  // never read: there is no prefix tile
        tvp = tvs;
    }
    dm05::kv8::Params ap = {};
    ap.k_scale = k_scale;
    ap.v_scale = v_scale;
    ap.valid_len = prefix_valid_len;
    ap.mask = prefix_mask;
    ap.out = static_cast<__nv_bfloat16 *>(out);
    ap.lse = lse;
    ap.err = dev.err;
    ap.part = static_cast<uint8_t *>(workspace);
    ap.Hkv = Hkv;
    ap.P = P;
    ap.S = S;
    ap.GS = GS;
    ap.qrows = pl.qrows;
    ap.row_blocks = pl.row_blocks;
    ap.splits = pl.splits;
    ap.nblk = blocks_of(P, shift);
    ap.shift = shift;
    ap.scale_log2 = static_cast<float>(kLog2e / std::sqrt(static_cast<double>(D)));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(dm05::kv8::kThreads8, 1, 1);
    cfg.dynamicSmemBytes = dm05::kv8::Smem::kAllocBytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(pl.splits);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = pl.cluster ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kv8_kernel(pl.copies, pl.cluster), tq, tkp, tvp, tks, tvs, to, ap) != cudaSuccess)
        return DM05_ERR_CUDA;
    if (pl.splits == 1 || pl.cluster) return DM05_OK;
    dm05::kv8::MergeParams mp = {};
    mp.part = ap.part;
    mp.out = static_cast<__nv_bfloat16 *>(out);
    mp.lse = lse;
    mp.rows = units * GS;
    mp.GS = GS;
    mp.splits = pl.splits;
    const dim3 blocks(static_cast<unsigned>((mp.rows + 3) / 4));
    return pl.splits <= 8 ? launch(dm05::kv8::merge_kernel<8>, blocks, 256, 0, stream, mp)
                          : launch(dm05::kv8::merge_kernel<16>, blocks, 256, 0, stream, mp);
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
    dm05::cache::EvictParams ep = {};
    ep.s = select_params(mass, valid_len, mask, mass_out, positions, valid_out, Hkv, P, P_out, n_keep, n_first,
                         n_last);
    dm05::cache::GatherParams &gp = ep.g;
    gp.k = static_cast<const uint8_t *>(k);
    gp.v = static_cast<const uint8_t *>(v);
    gp.k_out = static_cast<uint8_t *>(k_out);
    gp.v_out = static_cast<uint8_t *>(v_out);
    gp.pos = positions;
    gp.Hkv = Hkv;
    gp.P = P;
    gp.Pout = P_out;
    gp.n_keep = n_keep;
    const EvictArrays arrays(ep, 512, B, 0, 0);
    if (arrays.overlap()) return DM05_ERR_UNSUPPORTED;
    Device dev;
    rc = dm05::internal::device(stream, true, &dev);
    if (rc != DM05_OK) return rc;
    if (arrays.overlap_rest()) return DM05_ERR_UNSUPPORTED;
    ep.s.err = dev.err;
    return run_evict(ep, B * Hkv, n_keep, 0, dev.num_sms, stream);
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
    dm05::cache::EvictParams ep = {};
    ep.s = select_params(mass, valid_len, mask, mass_out, positions, valid_out, Hkv, P, P_out, n_keep, n_first,
                         n_last);
    dm05::cache::GatherParams &gp = ep.g;
    gp.k = static_cast<const uint8_t *>(k8);
    gp.v = static_cast<const uint8_t *>(v8);
    gp.k_out = static_cast<uint8_t *>(k8_out);
    gp.v_out = static_cast<uint8_t *>(v8_out);
    gp.k_scale = k_scale;
    gp.v_scale = v_scale;
    gp.k_scale_out = k_scale_out;
    gp.v_scale_out = v_scale_out;
    gp.pos = positions;
    gp.Hkv = Hkv;
    gp.P = P;
    gp.Pout = P_out;
    gp.n_keep = n_keep;
    gp.nblk = blocks_of(P, shift);
    gp.nblk_out = blocks_of(P_out, shift);
    gp.shift = shift;
    const EvictArrays arrays(ep, 256, B, gp.nblk, gp.nblk_out);
    if (arrays.overlap()) return DM05_ERR_UNSUPPORTED;
    Device dev;
    rc = dm05::internal::device(stream, true, &dev);
    if (rc != DM05_OK) return rc;
    if (arrays.overlap_rest()) return DM05_ERR_UNSUPPORTED;
    ep.s.err = dev.err;
    return run_evict(ep, B * Hkv, n_keep, block, dev.num_sms, stream);
}

}  // extern "C"
