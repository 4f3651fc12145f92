// What the C ABI's translation units share: argument checks, the workspace
// allocator, the kernel timing log and the error state of poetx.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

namespace poetx {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// every pointer non-null and 16-byte aligned
inline bool ptrs_ok(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p || !aligned16(p)) return false;
  return true;
}

// Bump allocator over the caller's workspace (256-byte aligned pieces).
struct Carve {
  char* base;
  size_t off = 0;
  explicit Carve(void* p) : base(static_cast<char*>(p)) {}
  template <typename T>
  T* take(int64_t count, size_t esize = sizeof(T)) {
    const size_t o = off;
    off = (off + static_cast<size_t>(count) * esize + 255) & ~static_cast<size_t>(255);
    return base ? reinterpret_cast<T*>(base + o) : nullptr;
  }
};

// Drops a HIP error left pending by earlier calls of other code on this
// thread, so that launch_status() sees only this entry point's launches.
void clear_pending_error();
int launch_status();

// A step of the timing log (poetx_profile_*): HIP events around its launches
// while the log is recording, nothing otherwise.
class ProfScope {
 public:
  ProfScope(const char* name, hipStream_t s);
  ~ProfScope();
  ProfScope(const ProfScope&) = delete;
  ProfScope& operator=(const ProfScope&) = delete;

 private:
  bool on_ = false;
  hipStream_t st_;
  const char* name_;
  hipEvent_t start_ = nullptr, stop_ = nullptr;
};

}  // namespace poetx
