// f8.h -- the block-scaled 8-bit format shared by its quantiser and product.
//
// A matrix of R rows and K columns is held as R rows of 128 * ceil(K / 128)
// e4m3 bytes (zeros past K) and R rows of 4 * ceil(K / 512) scale bytes: byte
// b of a row is the biased exponent (E8M0: 2^(byte - 127)) of elements
// 128 b .. 128 b + 127.  The power of two is the smallest that brings the
// block's largest magnitude to at most 448, the largest e4m3 value.  A power
// of two costs an 8-bit FLOAT no precision (its relative step does not depend
// on the exponent), and both the widening to bf16 and the 8-bit matrix
// instructions apply it themselves, so a product needs no arithmetic on its
// sums between blocks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bnn {

constexpr int kF8Block = 128;
constexpr int64_t kF8MaxK = int64_t(1) << 24;  // columns of a product's operands

__host__ __device__ inline int64_t f8_blocks(int64_t k) { return (k + kF8Block - 1) / kF8Block; }
__host__ __device__ inline int64_t f8_row_bytes(int64_t k) { return f8_blocks(k) * kF8Block; }
__host__ __device__ inline int64_t f8_scale_bytes(int64_t k) { return (f8_blocks(k) + 3) / 4 * 4; }

}  // namespace bnn
