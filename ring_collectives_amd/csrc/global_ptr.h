// global_ptr.h -- pointers that are known to point into global memory.
#pragma once

namespace ringc {

// Of a pointer that asm has hidden the origin of, the compiler would otherwise
// make flat accesses.
template <class T> using Global = __attribute__((address_space(1))) T*;

}  // namespace ringc
