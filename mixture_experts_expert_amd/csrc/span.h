// The memory of a call's buffers, on the host (internal).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <initializer_list>

namespace moe {
namespace {

// A buffer of a call.  What is written may share memory with nothing else of the
// call, or be one of the buffers that are named, from its first byte to its last:
// parts of it are stored while others are still to be read.
struct Span {
    const void* at;
    size_t bytes;
    bool meets(const Span& o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(at), b = reinterpret_cast<uintptr_t>(o.at);
        return at && o.at && bytes && o.bytes && a < b + o.bytes && b < a + bytes;
    }
    bool apart(std::initializer_list<Span> others) const {
        return std::none_of(others.begin(), others.end(), [&](const Span& o) { return meets(o); });
    }
    bool apart_or_one_of(std::initializer_list<Span> others) const {
        return std::none_of(others.begin(), others.end(), [&](const Span& o) { return meets(o) && (o.at != at || o.bytes != bytes); });
    }
};

}  // namespace
}  // namespace moe
