"""Which bytes the tiled expert kernels load into shared memory
(matrix_optimizer_amd/csrc/stages.h), checked on the host for every wave, lane
and load of tiles of all lengths: what a tile needs lies wholly within its
buffer, the buffer ends with the tile's last row, and no lane of a row past it
has an offset that the buffer's size lets through."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "matrix_optimizer_amd", "csrc")

HEAD = """
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "stages.h"
using namespace muon;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: " #x "\\n", __LINE__); std::exit(1); } } while (0)
"""

PRODUCT = """
int main() {
  const uint32_t all_rows[] = {1, 2, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256};
  const uint32_t widths[] = {144, 256, 272, 400, 1024};
  for (uint32_t K : widths)
    for (uint32_t pitch : {K, K + 16, K + 4096, (1u << 22) - 16})
      for (uint32_t rows : all_rows) {
        const uint32_t KB = (K + 127) / 128, s_pitch = pitch == K ? KB * 4 : (1u << 22) - 4;
        const uint64_t end = uint64_t(rows - 1) * pitch + K, s_end = uint64_t(rows - 1) * s_pitch + KB * 4;
        for (uint32_t kb = 0; kb < KB; ++kb) {
          // what advance() leaves after kb blocks
          const uint32_t bytes = product_bytes(rows, pitch, K, 0) - kb * 128;
          CHECK(bytes == product_bytes(rows, pitch, K, kb * 128));
          CHECK(kb * 128 + uint64_t(bytes) == end);
          const uint32_t s_bytes = product_bytes(rows, s_pitch, KB * 4, 4 * kb);
          CHECK(4 * kb + uint64_t(s_bytes) == s_end);
          for (int w = 0; w < 8; ++w)
            for (int lane = 0; lane < 64; ++lane) {
              for (int j = 0; j < 4; ++j) {
                const uint32_t r = product_row(w, lane, j), c = product_piece(lane, j);
                const uint64_t off = uint64_t(r) * pitch + c;
                CHECK(product_offset(w, lane, j, pitch) == off);              // no carry out of 32 bits
                CHECK(w * 4096 + j * 1024 + lane * 16 == int(r * 128 + ((c / 16) ^ ((r >> 1) & 7)) * 16));
                if (r >= rows) CHECK(off >= bytes);                           // not read
                else if (kb * 128 + c < K) CHECK(off + 16 <= bytes);          // read whole
                else if (off < bytes) CHECK(kb * 128 + off + 16 <= end);      // another row's, within the tile
              }
              if (w < 4) {
                const uint32_t r = 64 * w + lane;
                const uint64_t off = uint64_t(r) * s_pitch;
                CHECK(product_scale_offset(w, lane, s_pitch) == off);
                if (r >= rows) CHECK(off >= s_bytes);
                else CHECK(off + 4 <= s_bytes);
              }
            }
          for (uint32_t blocks : {1u, 2u})
            for (int lane = 0; lane < 64; ++lane) {
              const uint32_t off = product_matrix_scale_offset(lane, KB * 4), left = product_bytes(blocks, KB * 4, KB * 4, 4 * kb);
              CHECK(4 * kb + left == blocks * KB * 4);
              if (uint32_t(lane & 1) < blocks) CHECK(off + 4 <= left);
              else CHECK(off >= left);
            }
        }
      }
  std::puts("ok");
}
"""

GRAD = """
int main() {
  const uint32_t widths[] = {8, 16, 128, 248, 256, 264, 512, 1000};
  for (uint32_t cols : widths)
    for (uint32_t pitch : {2 * cols, 2 * cols + 16, (1u << 23) - 16})
      for (uint32_t first = 0; first < cols; first += 256)      // the tile's first column
        for (int rows = -3; rows <= 64; ++rows) {
          const uint32_t left = (cols - first) * 2, bytes = grad_bytes(rows, pitch, left);
          CHECK(rows > 0 ? 2 * first + bytes == uint64_t(rows - 1) * pitch + 2 * cols : bytes == 0);
          for (int w = 0; w < 8; ++w)
            for (int lane = 0; lane < 64; ++lane)
              for (int j = 0; j < 4; ++j) {
                const uint32_t r = grad_row(w, lane, j), c = grad_piece(lane, j);
                const uint64_t off = uint64_t(r) * pitch + c;
                CHECK(grad_offset(w, lane, j, pitch) == off);                 // no carry out of 32 bits
                CHECK(w * 4096 + j * 1024 + lane * 16 == int(r * 512 + ((c / 16) ^ (4 * (r & 3))) * 16));
                if (int(r) >= rows) CHECK(off >= bytes);                      // not read
                else if (c < left) CHECK(off + 16 <= bytes);                  // read whole
                else if (off < bytes) CHECK(off + 16 <= bytes);               // another row's, within the run
              }
        }
  std::puts("ok");
}
"""


def run(body, tmp_path):
    src, exe = tmp_path / "reach.cpp", tmp_path / "reach"
    src.write_text(HEAD + body)
    done = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(src), "-o", str(exe)],
                          capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    done = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0 and done.stdout == "ok\n", done.stdout


def test_product_tiles_stay_within_their_operands(tmp_path):
    run(PRODUCT, tmp_path)


def test_weight_gradient_tiles_stay_within_their_operands(tmp_path):
    run(GRAD, tmp_path)


def test_product_loads_have_no_scalar_offset():
    """The kernel's lane offsets and buffers are those checked above, and its loads take nothing besides them."""
    src = open(os.path.join(CSRC, "product.hip")).read()
    for call in ("lds_dma16(o.a, a_off[j], ", "lds_dma16(o.w, w_off[j], ", "lds_dma4(o.scales, s_off, "):
        assert call in src
    assert src.count("lds_dma") == 3
    forms = [line for line in open(os.path.join(CSRC, "lds.h")) if "buffer_load_dword " in line]
    assert forms and all("%0, %1, 0 offen lds" in line for line in forms)


def test_weight_gradient_loads_have_no_scalar_offset():
    src = open(os.path.join(CSRC, "weight_grad.hip")).read()
    for call in ("lds_dma16(r.x, x_off[j], ", "lds_dma16(r.dy, d_off[j], "):
        assert call in src
    assert src.count("lds_dma") == 2
    for name in os.listdir(CSRC):
        forms = [line for line in open(os.path.join(CSRC, name)) if "buffer_load_dword" in line]
        assert all("%0, %1, 0 offen lds" in line for line in forms), name
