// What the step and the prefill of the gated delta rule share: a sequence's
// rows and state slots, checked on the device.
#pragma once

#include "device_common.hpp"
#include "serving.hpp"

namespace gdn {
namespace rule {

struct Sequence {
    int first, len;      // its rows; len 0 where they are not known to lie in the arrays
    int src, dst;        // state slots, src < 0: from zero
    int fault;
};

__device__ __forceinline__ bool slots_ok(const RuleArgs &a, int src, int dst) {
    return src >= -1 && src < a.slots && dst >= 0 && dst < a.slots;
}

__device__ __forceinline__ Sequence sequence(const RuleArgs &a, int b) {
    Sequence s;
    s.first = a.cu[b];
    const int end = a.cu[b + 1];
    s.src = a.src[b], s.dst = a.dst[b];
    s.fault = 0;
    if (s.first < 0 || end < s.first || end > a.rows) {
        s.fault = kFaultBadLength;
        s.first = 0, s.len = 0;
        return s;
    }
    s.len = end - s.first;
    if (!slots_ok(a, s.src, s.dst)) s.fault = kFaultBadSlot;
    return s;
}

__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t *p, float x) {
    *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

}  // namespace rule
}  // namespace gdn
