// What has to be done once on each device of the process, such as raising a
// kernel's shared-memory limit, which is an attribute of a function on a device.
#pragma once

#include <mutex>

namespace moedc_host {

class PerDevice {
public:
    // True when `act` has succeeded for this device, now or before.  A failure is not
    // kept: the next call tries again.
    template <typename Act> bool once(int device, Act act)
    {
        if (device < 0 || device >= kDevices) return act();
        std::lock_guard<std::mutex> lock(mutex_);
        if (!done_[device]) done_[device] = act();
        return done_[device];
    }

private:
    static constexpr int kDevices = 64;
    std::mutex mutex_;
    bool done_[kDevices] = {};
};

}  // namespace moedc_host
