// Host test of the per-device counts, with a fake device query and fake occupancy
// answers: what the library asks the driver once and keeps.
#include <cstdio>

#include "moe_internal.h"

static int g_device = 0;
extern "C" cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}

int main() {
  static moe::DeviceOnce once;
  int asked = 0, bad = 0;
  // the answers of devices 0, 1 and 2; device 3's first query fails
  const int answers[4] = {0, 1, 76, 9};
  for (int turn = 0; turn < 3; ++turn)
    for (g_device = 0; g_device < 4; ++g_device) {
      int n = -1;
      const cudaError_t err = moe::count_per_device(once, &n, [&](int dev, int* v) {
        ++asked;
        if (dev == 3 && turn == 0) return cudaErrorInvalidValue;
        *v = answers[dev];
        return cudaSuccess;
      });
      const bool fails = g_device == 3 && turn == 0;
      if ((err != cudaSuccess) != fails || n != (fails ? 0 : answers[g_device])) {
        std::printf("turn %d device %d: error %d, count %d\n", turn, g_device, (int)err, n);
        ++bad;
      }
    }
  std::printf("asked %d bad %d\n", asked, bad);
  return bad || asked != 5;
}
