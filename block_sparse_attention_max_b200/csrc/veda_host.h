// veda_host.h -- what the library's translation units share on the host.
#pragma once

#include <exception>
#include <string>

#include "../../include/veda.h"

namespace veda {

// Message of the calling thread's last failing call (veda_last_error).
void set_last_error(const std::string& msg);

// Current device: compute capability 10.0 or an error; its SM count.
veda_status host_device(int& sms);

// Body of a C entry: nothing it throws leaves it.
template <typename F>
veda_status guarded(const char* call, F&& body) noexcept {
  try {
    return body();
  } catch (const std::exception&) {
    try { set_last_error(std::string(call) + ": host error"); } catch (...) {}
    return VEDA_ERR_CUDA;
  } catch (...) {
    return VEDA_ERR_CUDA;
  }
}

}  // namespace veda
