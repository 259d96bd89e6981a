// What is kept per (kernel, device) for the life of the process, however many of each there are.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <functional>
#include <mutex>
#include <unordered_map>

namespace pa {

template <typename Info>
class LaunchCache {
 public:
  bool find(const void* kern, int dev, Info* out) {
    std::lock_guard<std::mutex> lock(mu_);
    auto it = map_.find(Key{kern, dev});
    if (it == map_.end()) return false;
    *out = it->second;
    return true;
  }
  // (without memory for it the entry is not kept: no exception may pass a C entry point)
  void put(const void* kern, int dev, const Info& info) noexcept {
    try {
      std::lock_guard<std::mutex> lock(mu_);
      map_[Key{kern, dev}] = info;
    } catch (...) {
    }
  }

 private:
  struct Key {
    const void* kern;
    int dev;
    bool operator==(const Key& o) const { return kern == o.kern && dev == o.dev; }
  };
  struct Hash {
    size_t operator()(const Key& k) const {
      return std::hash<const void*>()(k.kern) * 31 + static_cast<size_t>(k.dev);
    }
  };
  std::mutex mu_;
  std::unordered_map<Key, Info, Hash> map_;
};

}  // namespace pa
