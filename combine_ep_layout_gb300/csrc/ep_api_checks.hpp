// ep_api_checks.hpp -- what the entry points beside ep_api.cpp share: errors with a
// message, nothing thrown across the boundary, alignment.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <exception>
#include <string>

#include "ep_gb300.h"
#include "ep_kernels.hpp"

namespace epg {
namespace api {

inline int fail(int code, const std::string& msg) { return RecordError(code, msg.c_str()); }

inline int fail_cuda(cudaError_t e, const char* what) {
  return fail(EP_ECUDA, std::string(what) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <class F>
int guarded(F&& f) noexcept {
  try {
    return f();
  } catch (const std::exception& ex) {
    return RecordError(EP_EINVAL, ex.what());
  } catch (...) {
    return RecordError(EP_EINVAL, "unknown exception");
  }
}

// What the entry points beside ep_api.cpp use of a handle: the routing of the last
// ep_layout that it uses, and where its fields lie.
struct Routing {
  int num_tokens, topk, experts, hidden;
  int64_t rcap;
  bool no_expand;
  const int32_t* count;      // [E]
  const int32_t* first;      // [E + 1]
  const int32_t* num_recv;   // [1]
  const int32_t* send_slot;  // [N, K]
  const int32_t* meta;       // [rcap, K + 2]
};
// EP_EINVAL unless h is a handle of the current device.
int RoutingOf(ep_handle_t h, Routing* r);
// A call enqueued work on `s` that uses h.
void MarkUsed(ep_handle_t h, cudaStream_t s);

}  // namespace api
}  // namespace epg
