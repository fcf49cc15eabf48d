// train_api.hip -- version, error texts and the device check shared by the
// training operators' entry points.

#include <mutex>

#include "train_common.hpp"

namespace ssim_train {

int check_current_device() {
  struct Known {
    bool ready;
    int status;
  };
  static std::mutex mu;
  static Known known[64] = {};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return SSIM_ERR_HIP;
  if (dev < 0 || dev >= 64) return SSIM_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(mu);
  Known& d = known[dev];
  if (!d.ready) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return SSIM_ERR_HIP;
    const bool ok = prop.warpSize == kWave && strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    d.status = ok ? SSIM_OK : SSIM_ERR_DEVICE;
    d.ready = true;
  }
  return d.status;
}

}  // namespace ssim_train

extern "C" {

int ssim_train_abi_version(void) { return SSIM_TRAIN_ABI_VERSION; }

const char* ssim_train_strerror(int code) {
  switch (code) {
    case SSIM_OK: return "success";
    case SSIM_ERR_NULL: return "a required pointer is NULL";
    case SSIM_ERR_SHAPE: return "a size is out of range or a pointer is not aligned";
    case SSIM_ERR_OVERFLOW: return "a size overflows";
    case SSIM_ERR_ALIAS: return "an output overlaps an input or another output";
    case SSIM_ERR_HIP: return "a HIP call failed";
    case SSIM_ERR_DEVICE: return "the current device is not a gfx950 GPU";
    case SSIM_ERR_DTYPE: return "an element type is unknown or does not go with another one";
    case SSIM_ERR_VALUE: return "a hyperparameter is not a number or out of its range";
    default: return "unknown error code";
  }
}

}  // extern "C"
