// What a device is asked once (to raise a limit, to count resident clusters) and
// whose answer holds for the process.  Host code only.
#pragma once

#include <atomic>

namespace cgk {

// One positive answer per device.  A device without one, or past the table, is asked;
// an answer of 0 or less is not kept.  Threads may ask at the same time.
class DeviceAnswers {
 public:
  template <typename Ask>
  int get(int device, Ask ask) {
    const bool kept = device >= 0 && device < kDevices;
    int answer = kept ? known_[device].load(std::memory_order_relaxed) : 0;
    if (answer > 0) return answer;
    answer = ask();
    if (kept && answer > 0) known_[device].store(answer, std::memory_order_relaxed);
    return answer;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> known_[kDevices] = {};
};

}  // namespace cgk
