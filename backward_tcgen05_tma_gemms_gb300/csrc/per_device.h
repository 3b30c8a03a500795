// per_device.h -- set-up that the first call on each device does.  Attributes of a
// kernel and what the occupancy calculator says of it hold for one device only.
#pragma once
#include <mutex>
#include <vector>

namespace tps {

// One value for each device.  `set_up` makes a device's value and returns
// whether it could; one that it could not make is asked for again by the next
// call.
template <class T>
class PerDevice {
 public:
  template <class F>
  bool get(int device, T* value, F&& set_up) {
    if (device < 0) return false;
    std::lock_guard<std::mutex> lock(mu_);
    if (static_cast<size_t>(device) >= known_.size()) known_.resize(static_cast<size_t>(device) + 1);
    Entry& e = known_[static_cast<size_t>(device)];
    if (!e.have) {
      T made{};
      if (!set_up(&made)) return false;
      e.value = made;
      e.have = true;
    }
    *value = e.value;
    return true;
  }

 private:
  struct Entry {
    T value{};
    bool have = false;
  };
  std::mutex mu_;
  std::vector<Entry> known_;
};

}  // namespace tps
