// Many kernels on many devices, sizes that rise and fall: a limit never falls, no
// launch exceeds it, and a size that has been had is not set again.
#include <cstdio>
#include <map>
#include <utility>

#include "smem_limits.h"

int main() {
  static bl::SmemLimits limits;
  static char kernels[400];
  std::map<std::pair<const void*, int>, size_t> attr;
  int sets = 0, bad = 0;
  auto call = [&](int k, int dev, size_t bytes) {
    const void* fn = &kernels[k];
    size_t& now = attr[{fn, dev}];
    const bool ok = limits.ensure(fn, dev, bytes, [&](size_t b) {
      ++sets;
      bad += b < now;  // lowered
      now = b;
      return true;
    });
    bad += !ok || now < bytes;  // the launch would fail
  };
  for (int step = 1; step <= 40; ++step)  // more sizes than a list of 512 holds
    for (int dev = 0; dev < 8; ++dev)
      for (int k = 0; k < 400; ++k) {
        call(k, dev, 1024 * step);
        call(k, dev, 512 * step);
      }
  const int rising = sets;
  for (int step = 40; step >= 0; --step)
    for (int dev = 0; dev < 8; ++dev)
      for (int k = 0; k < 400; ++k) call(k, dev, 1024 * step);
  const bool refused = !limits.ensure(&kernels[0], 0, 1 << 20, [](size_t) { return false; });
  std::printf("rising %d again %d bad %d refused %d\n", rising, sets - rising, bad, (int)refused);
  return bad == 0 && sets == rising && rising == 40 * 8 * 400 && refused ? 0 : 1;
}
