/*
 * memo.h -- answers of the CUDA runtime about a kernel that launches ask for again
 * and again (how many of its blocks run at once), kept by everything that they
 * depend on.  A fixed table: nothing is allocated, so nothing is thrown through a C
 * entry point; past its end answers are asked for anew.  Plain C++.
 */
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <mutex>

namespace dlrm {

class KernelMemo {
public:
    struct Key {
        const void* kernel;   // its address: kernels of one signature differ in nothing else
        int device, cluster;
        size_t smem;
        bool operator==(const Key& o) const
        {
            return kernel == o.kernel && device == o.device && cluster == o.cluster && smem == o.smem;
        }
    };

    // The answer for `key`: the kept one, or ask()'s.
    template <typename Ask>
    int get(const Key& key, Ask&& ask)
    {
        std::lock_guard<std::mutex> lock(mu_);
        size_t at = (reinterpret_cast<uintptr_t>(key.kernel) / 16 * 31 + key.smem / 16 * 7 + (size_t)(key.device * 16 + key.cluster)) % kSlots;
        for (int i = 0; i < kProbes; ++i, at = (at + 1) % kSlots) {
            if (!used_[at]) {
                used_[at] = true;
                keys_[at] = key;
                return values_[at] = ask();
            }
            if (keys_[at] == key) return values_[at];
        }
        return ask();
    }

private:
    static constexpr size_t kSlots = 1024;
    static constexpr int kProbes = 16;
    std::mutex mu_;
    bool used_[kSlots] = {};
    Key keys_[kSlots];
    int values_[kSlots];
};

}  // namespace dlrm
