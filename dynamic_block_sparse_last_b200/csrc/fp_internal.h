// fp_internal.h -- what the library's translation units share on the host.
#pragma once

#include <cuda.h>

namespace fpk {

// The sticky device error word of the current device (null when the device is
// unusable); one word for every kernel of the library.
int *library_error_word();

// The calling thread's current context (null without one): what a set-up step was
// made in, so that it is made again after a device reset.
void *library_context();

// 2-D tensor map over `rows` rows of `row_bytes` bytes, boxes of box_rows rows
// by box_bytes bytes (at most 128, the swizzle span: 64 or 128).
bool make_byte_map(CUtensorMap *m, const void *ptr, uint64_t row_bytes, uint64_t rows, uint32_t box_bytes,
                   uint32_t box_rows);

}  // namespace fpk
