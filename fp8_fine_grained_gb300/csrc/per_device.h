// A property of a kernel on a device, asked for once per device.
#pragma once

#include <atomic>

namespace fp8fg {

class PerDevice {
public:
    // The property of device `dev`, from query() the first time. 0 when the
    // query gives nothing above 0 (or the device is beyond the table): that is
    // not kept, so the next call asks again.
    template <typename Query>
    int get(int dev, Query query)
    {
        if (dev < 0 || dev >= MAX_DEVICES)
            return 0;
        int n = known_[dev].load();
        if (n == 0) {
            n = query();
            if (n < 1)
                return 0;
            known_[dev].store(n);
        }
        return n;
    }

private:
    static constexpr int MAX_DEVICES = 64;
    std::atomic<int> known_[MAX_DEVICES] = {};
};

}  // namespace fp8fg
