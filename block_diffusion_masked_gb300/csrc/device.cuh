// What the entry points of the sampling operators need of the host side in
// api.cu, beside what params.cuh declares: apart from it, so that the sources of
// the training kernels do not include it.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace dfa {

// check_device, and the current device's status word and SM count.
struct DeviceInfo {
  unsigned* status;
  int sms;
};
int device_info(DeviceInfo* info);

// A tensor map of a byte array (a null pointer, an alignment or an extent the
// driver refuses: DFA_ECUDA).
int encode_map_u8(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle);

}  // namespace dfa
