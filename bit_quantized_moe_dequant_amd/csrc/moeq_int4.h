// 4-bit integer weights with group scales: their layout, shared by the kernels and the host.
//
//   w[r][k] = scale2 * s[r][k / G] * (q[r][k] - z[r][k / G])       q 0..15, z = 8 or a zero point
//
// A tensor is stored as tiles of 16 rows x 128 columns in the order of the matrix instruction's
// operand (16 x 16 x 32, 8 values to a lane), rows padded to 16 and columns to 128 with s = 0:
//   data    tile (r / 16) * ktiles + k / 128, 1024 bytes: lane n + 16 g (row n of the tile) holds
//           words j = 0..3 with columns 32 j + 8 g + 0..7 of the tile; column 2 p in bits 4 p of a
//           word's low half, column 2 p + 1 in those of its high half (p = 0..3), so that a shift
//           and a mask give a register's pair of operand values
//   scales  per tile [16 rows][128 / G] fp16; behind all of them, where the format has zero
//           points, per tile [16][128 / G] bytes
// A wave reads a tile's codes as one run of 1 KB.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace moeq {

enum {  // beside the FMT_* of moeq_device.h; G 32, 64, 128, then the same with zero points
  FMT_INT4_G32 = 10,
  FMT_INT4_G64 = 11,
  FMT_INT4_G128 = 12,
  FMT_INT4Z_G32 = 13,
  FMT_INT4Z_G64 = 14,
  FMT_INT4Z_G128 = 15
};

constexpr bool is_int4(int fmt) { return fmt >= FMT_INT4_G32 && fmt <= FMT_INT4Z_G128; }
constexpr bool int4_zeros(int fmt) { return fmt >= FMT_INT4Z_G32; }
constexpr int int4_group(int fmt) { return 32 << ((fmt - FMT_INT4_G32) % 3); }
constexpr int int4_ktiles(int cols) { return cols / 128 + (cols % 128 != 0); }
constexpr int int4_rtiles(int rows) { return rows / 16 + (rows % 16 != 0); }
constexpr size_t int4_tiles(int rows, int cols) { return (size_t)int4_rtiles(rows) * int4_ktiles(cols); }
constexpr size_t int4_data_bytes(int rows, int cols) { return int4_tiles(rows, cols) * 1024; }
// bytes of the scales, which the zero points follow
constexpr size_t int4_zeros_at(int fmt, int rows, int cols) { return int4_tiles(rows, cols) * 16 * (128 / int4_group(fmt)) * 2; }
constexpr size_t int4_scale_bytes(int fmt, int rows, int cols) {
  return int4_zeros_at(fmt, rows, cols) / 2 * (int4_zeros(fmt) ? 3 : 2);
}

constexpr int INT4_MAX_ROWS = 1 << 23;
constexpr int INT4_MAX_COLS = 1 << 20;

}  // namespace moeq
