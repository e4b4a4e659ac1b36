// asked_once.cuh - answers about a device that are asked for once (host code
// without CUDA).
#pragma once
#include <atomic>

namespace msa {

// What ask() says about (device, key), kept from the first time on: >= 0 the
// answer, < 0 the question failed, which counts as 0 and is kept as well, so
// that no later call goes another way than the first.  Devices past the last
// one kept get 0.
template <int kDevices, int kKeys>
struct AskedOnce {
  std::atomic<int> known[kDevices][kKeys];  // answer + 1; 0: not asked yet

  template <typename Ask>
  int get(int device, int key, Ask ask) {
    if (device < 0 || device >= kDevices) return 0;
    std::atomic<int>& slot = known[device][key];
    int have = slot.load();
    if (have == 0) {
      const int said = ask();
      const int mine = said < 0 ? 1 : said + 1;
      // of two threads that ask at once the first one's answer stands
      have = slot.compare_exchange_strong(have, mine) ? mine : have;
    }
    return have - 1;
  }
};

}  // namespace msa
