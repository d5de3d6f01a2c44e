// Error translation at the C ABI: nothing but a status code leaves an entry point.
#pragma once

#include <exception>
#include <new>
#include <string>

#include "common.hpp"

namespace cgtp {

template <typename F>
cgtp_status guarded(F&& f) {
  try {
    set_error("");
    f();
    return CGTP_OK;
  } catch (const Error& e) {
    set_error(e.msg);
    return e.code;
  } catch (const std::bad_alloc&) {
    set_error("host allocation failed");
    return CGTP_ERR_ALLOC;
  } catch (const std::exception& e) {
    set_error(e.what());
    return CGTP_ERR_INVALID_ARG;
  } catch (...) {
    set_error("unknown error");
    return CGTP_ERR_INVALID_ARG;
  }
}

inline void need(bool ok, const char* what) {
  if (!ok) throw Error{CGTP_ERR_INVALID_ARG, what};
}

inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace cgtp
