// tmaps.h -- TMA tensor maps of the INT8 GEMMs' operands and outputs (host).
// Defined in gemm.cu; each returns false when the driver refuses the map.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace sq {

// [rows, inner] int8, box [box_rows, 128 bytes], 128-byte swizzle, zero fill.
bool make_tmap(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows);
// [batch, rows, inner] int8, box [1, box_rows, 128 bytes], the same otherwise.
bool make_tmap3(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t batch,
                uint32_t box_rows);
// [rows, cols] of bf16 or fp32, box 32 rows x row_bytes (64 or 128), swizzled
// over row_bytes.
bool make_tmap_out(CUtensorMap* m, void* base, uint64_t cols, uint64_t rows, bool bf16,
                   uint32_t row_bytes = 64);

}  // namespace sq
