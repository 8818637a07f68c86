// tk_device.h -- what the library's translation units share of the current
// device: set up once per device (tk_attn.cu), read by every entry point.
#pragma once

#include <cuda.h>

#include <cstddef>
#include <cstdint>

namespace tkattn {

constexpr int kMaxDevices = 64;

struct DeviceView {
  int index;      // CUDA device ordinal
  int num_sms;
  int *err_word;  // device error word of this device
};

// The current device, set up on first use.  Returns TK_ATTN_OK or the status
// the calling entry point has to return.
int device_view(DeviceView *out);

// Tensor map of a byte matrix [rows, row_bytes] (row_bytes 64 or 128): boxes of
// box_rows whole rows, swizzled over the row's length.
bool make_map_bytes(CUtensorMap *map, const void *ptr, long long rows, int row_bytes,
                    int box_rows);

// [a, a + na) and [b, b + nb) share a byte.
inline bool ranges_overlap(uintptr_t a, size_t na, uintptr_t b, size_t nb) {
  return na > 0 && nb > 0 && a < b + nb && b < a + na;
}

// Codes of the device error word (0: none).  The first one raised stays until
// tk_attn_last_device_error reads it.
constexpr int kDevErrTimeout = 1;  // a barrier wait was abandoned
constexpr int kDevErrIndex = 2;    // a page, length, position or count out of its range

}  // namespace tkattn
