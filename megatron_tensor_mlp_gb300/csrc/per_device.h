// A value per device, computed at the first use on it (host only; any thread may be first).
#pragma once
#include <atomic>
#include <mutex>

namespace tpmlp {

template <typename T>
class PerDevice {
  public:
    static constexpr int kDevices = 64;

    // The device's value.  compute(value) fills it in and says whether it holds from now on; if not, or past the last
    // device that is kept, the next call computes again.  A thread that finds the value there sees it whole: the flag is
    // published after it (on weakly ordered hosts a plain flag could be seen first).
    template <typename F>
    T get(int device, F&& compute) {
        if (device < 0 || device >= kDevices) {
            T v{};
            compute(v);
            return v;
        }
        Slot& s = slots_[device];
        if (s.ready.load(std::memory_order_acquire)) return s.value;
        std::lock_guard<std::mutex> lock(mutex_);
        if (s.ready.load(std::memory_order_relaxed)) return s.value;
        T v{};
        if (compute(v)) {
            s.value = v;
            s.ready.store(true, std::memory_order_release);
        }
        return v;
    }

  private:
    struct Slot {
        std::atomic<bool> ready{false};
        T value{};
    };
    Slot slots_[kDevices];
    std::mutex mutex_;
};

}  // namespace tpmlp
