// fq_tensormap.h -- tensor maps for the TMA-fed serving kernels.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace fq {

// A map of bytes with `rank` dimensions (innermost first, which is contiguous), strides[i] bytes between
// neighbours of dimension i + 1, boxes of box[i] elements, reads outside filled with zeros. False if the
// driver refuses.
bool byte_tensor_map(CUtensorMap* map, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box, CUtensorMapSwizzle swizzle);

// The same of 16-bit elements: dims, box and the copies' coordinates in elements, strides in bytes.
bool half_tensor_map(CUtensorMap* map, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box, CUtensorMapSwizzle swizzle);

}  // namespace fq
