// Host-side checks that a call's outputs share no memory with anything else it
// reads or writes.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace moe {

struct Span {
  const void* p;
  size_t n;
};

// Whether the two share a byte (a NULL span is empty).
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && x < y + b.n && y < x + a.n;
}

// Whether every output is apart from every other one and from every input.
inline bool outputs_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (auto q = outs.begin(); q != o; ++q)
      if (overlap(*o, *q)) return false;
    for (const Span& i : ins)
      if (overlap(*o, i)) return false;
  }
  return true;
}

// Whether an output is the very tensor `in` (of n bytes, like the output) or apart from it.
inline bool same_or_apart(const void* out, const void* in, size_t n) {
  return out == in || !overlap({out, n}, {in, n});
}

}  // namespace moe
