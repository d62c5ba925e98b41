// dm05_internal.h -- what the library's translation units share: the state
// of the current device and the tensor-map encoder.  Not part of the ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace dm05 {
namespace internal {

struct Device {
    uint32_t *err = nullptr;  // the device error word
    int num_sms = 0;
    int split_override = 0;      // dm05_set_split_override
    int ordinal = 0;
};

// State of the current device.  With `need_err` the error word exists on
// return (created outside stream capture only: DM05_ERR_WORKSPACE otherwise).
__attribute__((visibility("hidden"))) int device(cudaStream_t stream, bool need_err, Device *out) noexcept;

// cuTensorMapEncodeTiled of `rank` dimensions, element strides 1, zero fill
// out of range, 256-byte L2 promotion.  Call after device().
__attribute__((visibility("hidden"))) int encode_tiled(CUtensorMap *map, CUtensorMapDataType type, int rank,
                                                       const void *base, const cuuint64_t *dims,
                                                       const cuuint64_t *strides, const cuuint32_t *box) noexcept;

}  // namespace internal
}  // namespace dm05
