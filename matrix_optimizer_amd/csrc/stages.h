// Which bytes of an operand the waves of the tiled matrix kernels load into a
// stage of shared memory: plain arithmetic, shared with the host's checks.
//
// A load goes through a buffer that begins at the tile (and the stage's column
// or row of it) and ends with the tile's last row.  The whole distance from the
// buffer's begin is the lane's offset and the scalar offset is 0, so that the
// hardware compares that distance itself with the buffer's size: rows and
// columns past the end are not read, whatever the tile's size.
#pragma once
#include <stdint.h>

namespace muon {

// 8-bit product: 256 rows of 128 bytes (one block of k) an operand, 32 rows a
// wave in four loads of eight rows.  16-byte piece c of row r lies in slot
// c ^ (r / 2 % 8), so the lane that fills slot lane % 8 takes that piece.
constexpr uint32_t product_row(int wave, int lane, int load) { return 32u * wave + 8u * load + (lane >> 3); }
constexpr uint32_t product_piece(int lane, int load) { return ((lane & 7) ^ ((4 * load + (lane >> 4)) & 7)) * 16; }
constexpr uint32_t product_offset(int wave, int lane, int load, uint32_t pitch) {
  return product_row(wave, lane, load) * pitch + product_piece(lane, load);
}
// Bytes from a block's first column in the tile's first row to the end of the last of `rows` rows of `width`
// bytes, `done` bytes of each belonging to the blocks before.
constexpr uint32_t product_bytes(uint32_t rows, uint32_t pitch, uint32_t width, uint32_t done) {
  return (rows - 1) * pitch + width - done;
}
// Scales of a block, 4 bytes each: the tile's rows by four waves, and the one or two blocks of the matrix's
// rows by one wave.
constexpr uint32_t product_scale_offset(int wave, int lane, uint32_t pitch) { return (64u * wave + lane) * pitch; }
constexpr uint32_t product_matrix_scale_offset(int lane, uint32_t pitch) { return (lane & 1) * pitch; }

// Weight gradient: 64 rows of 512 bytes (256 columns) an operand, eight rows a wave in four loads of two rows.
// 16-byte piece c of row r lies in slot c ^ 4 (r % 4).
constexpr uint32_t grad_row(int wave, int lane, int load) { return 8u * wave + 2u * load + (lane >> 5); }
constexpr uint32_t grad_piece(int lane, int load) { return ((lane & 31) ^ (4 * (lane >> 5) + 8 * (load & 1))) * 16; }
constexpr uint32_t grad_offset(int wave, int lane, int load, uint32_t pitch) {
  return grad_row(wave, lane, load) * pitch + grad_piece(lane, load);
}
// Bytes from a tile's first column in the stage's first row to the end of the last of `rows` rows (none for rows
// <= 0), which have `left` bytes from that column on.
constexpr uint32_t grad_bytes(int rows, uint32_t pitch, uint32_t left) { return rows > 0 ? (rows - 1) * pitch + left : 0; }

}  // namespace muon
