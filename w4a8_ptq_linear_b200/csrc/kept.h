// Answers of the driver that a launch needs and that do not change (occupancy), asked once.
#pragma once

#include <map>
#include <mutex>

namespace oq {

// The value of `key`, kept from the first time that ask(value) returned true. What it leaves in value
// with false is this call's alone and is asked again the next time: a query can fail for a reason
// that passes.
template <typename K, typename V>
class Kept {
 public:
  template <typename F>
  bool get(const K& key, V* value, F ask) {
    {
      std::lock_guard<std::mutex> lock(mu_);
      auto found = kept_.find(key);
      if (found != kept_.end()) {
        *value = found->second;
        return true;
      }
    }
    V v{};
    const bool keep = ask(&v);
    *value = v;
    if (!keep) return false;
    std::lock_guard<std::mutex> lock(mu_);
    kept_[key] = v;
    return true;
  }

 private:
  std::mutex mu_;
  std::map<K, V> kept_;
};

}  // namespace oq
