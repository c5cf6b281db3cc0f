// per_device.h -- what is asked of a GPU once and kept for each.
#pragma once

#include <map>
#include <mutex>

namespace gemmar {

template <typename T>
class PerDevice {
public:
    // The device's value; where there is none yet, ask(value) says it, or returns false: then nothing is kept.
    template <typename F>
    bool get(int device, T &value, F ask)
    {
        std::lock_guard<std::mutex> lock(mu_);
        const auto at = known_.find(device);
        if (at != known_.end()) {
            value = at->second;
            return true;
        }
        if (!ask(value))
            return false;
        known_.emplace(device, value);
        return true;
    }

private:
    std::mutex mu_;
    std::map<int, T> known_;
};

}  // namespace gemmar
