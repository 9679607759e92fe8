// Shared by the decode-step operators' translation units: error text, the device check, cache checks.
#pragma once

#include "moe_decode.h"
#include "moe_internal.h"

namespace moe {

// Sets moe_last_error() (printf-style) and returns st.
moe_status_t decode_fail(moe_status_t st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The current device is a GB300 (asked once per device); num_sms, if not NULL, receives its SM count.
moe_status_t check_device(int* num_sms);

// Checks of a cache descriptor that need no device.  `call` names the entry point in the error text.
moe_status_t check_cache(const moe_kv_cache_t* c, const char* call);

// Division of a token position by the page size as a multiply and a shift: n / page = umulhi(n, mul) >> shift
// for 0 <= n < 2^31 (page_size 1 has mul = 0: the position is the page).
struct PageDiv {
  uint32_t mul, shift;
};
PageDiv page_div(uint32_t page_size);

}  // namespace moe
