"""The arithmetic of rows, visible slots and read ranges (csrc/token_rows.hpp),
built for the CPU, against the definition slot by slot: whatever row_start, lengths,
windows and first slots hold, no row or slot outside is named, every visible slot is
read, and the ranges said to be seen or unseen by all columns are."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gguf_block_quant_dequant_amd", "csrc")

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include <vector>
#include "token_rows.hpp"
using namespace gqk;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

static bool sees(int held, int rows, int j, int64_t window, int sinks, int i) {
  const int64_t p = (int64_t)held - rows + j;
  return i >= 0 && i <= p && (window == 0 || i > p - window || i < sinks);
}

int main() {
  const int32_t starts[] = {0, 3, 3, 2, 9, INT_MAX, INT_MIN, -5, 4, 7};
  for (int s = 0; s + 1 < (int)(sizeof(starts) / 4); ++s) {
    const SeqRows r = seq_rows(starts, s, 8);
    CHECK(r.row0 >= 0 && r.rows >= 0 && r.row0 + r.rows <= 8);
  }
  CHECK(seq_rows(starts, 0, 8).rows == 3 && seq_rows(starts, 1, 8).rows == 0 && seq_rows(starts, 2, 8).rows == 0);
  CHECK(seq_rows(starts, 3, 8).row0 == 2 && seq_rows(starts, 3, 8).rows == 6);
  CHECK(seq_rows(nullptr, 5, 8).row0 == 5 && seq_rows(nullptr, 5, 8).rows == 1);
  CHECK(low_bits(-1) == 0 && low_bits(0) == 0 && low_bits(1) == 1 && low_bits(31) == 0x7FFFFFFF && low_bits(32) == ~0u &&
        low_bits(INT64_MAX) == ~0u && low_bits(INT64_MIN) == 0);
  const int helds[] = {0, 1, 2, 5, 31, 32, 33, 64, 100, 257, 400};
  const int rowss[] = {1, 2, 3, 7, 16, 40};
  const int64_t windows[] = {0, 1, 2, 7, 33, 64, 150, 10000, INT64_MAX};
  const int sinkss[] = {0, 1, 4, 32, 40, 200};
  const int groups[] = {1, 3, 4, 16, 20};
  for (int held : helds) for (int rows : rowss) for (int64_t window : windows) for (int sinks : sinkss) {
    for (int j = 0; j < rows; ++j) {
      const SlotRange r = slot_range(held, rows, j, window);
      for (int at = 0; at < held + 40; at += 8) {
        const uint32_t bits = slot_bits(r, sinks, at);
        for (int i = 0; i < 32; ++i) CHECK((bits >> i & 1) == sees(held, rows, j, window, sinks, at + i));
      }
    }
    for (int group : groups) for (int columns : {16, 32, 128}) for (int unit : {32, 64, 256}) {
      for (int tile = 0; tile * columns < rows * group; ++tile) {
        const TileRange t = tile_range(held, rows, group, tile, columns, window, sinks, unit);
        CHECK(t.gap >= 0 && t.gap % unit == 0 && t.n <= held);
        if (t.gap > 0) CHECK(t.pad % unit == 0 && t.pad >= sinks);
        std::vector<char> read(held + 1);
        for (int v = 0; v < t.n; ++v) {
          const int i = v + (v >= t.pad ? t.gap : 0);
          CHECK(i < held);
          read[i] = 1;
        }
        for (int c = tile * columns; c < (tile + 1) * columns && c < rows * group; ++c)
          for (int i = 0; i < held; ++i) {
            const bool see = sees(held, rows, c / group, window, sinks, i);
            CHECK(!see || read[i]);
            if (i >= t.far && i < t.full) CHECK(see);
            if (i >= sinks && i < t.near) CHECK(!see);
          }
      }
    }
  }
  // far ends of the ranges
  const SlotRange e = slot_range(1 << 25, 1, 0, INT64_MAX);
  CHECK(e.lo == 0 && e.hi == 1 << 25);
  const TileRange t = tile_range(1 << 25, 1 << 23, 1, (1 << 19) - 1, 16, 5, 1 << 25, 256);
  CHECK(t.gap == 0 && t.n == 1 << 25);
  std::puts("ok");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_rows_and_slots_stay_inside(tmp_path):
    src, exe = tmp_path / "rows.cpp", tmp_path / "rows"
    src.write_text(PROGRAM)
    build = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined",
                            "-fno-sanitize-recover=undefined", "-I", CSRC, str(src), "-o", str(exe)],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr


SEARCH = r"""
#include <climits>
#include <cstdio>
#include <vector>
#include "token_rows.hpp"
using namespace gqk;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  uint32_t state = 1;
  auto random = [&](int n) { state = state * 1664525u + 1013904223u; return (int)((state >> 8) % (uint32_t)n); };
  for (int trial = 0; trial < 3000; ++trial) {
    const int n_seqs = 1 + random(trial % 10 == 0 ? 200 : 9), n_rows = random(60);
    std::vector<int32_t> starts(n_seqs + 1);
    starts[0] = random(8) - 4;   // before the first row, and rows of nobody in front
    for (int s = 0; s < n_seqs; ++s) starts[s + 1] = starts[s] + (random(3) == 0 ? 0 : random(9));
    for (int row = 0; row < n_rows; ++row) {
      int seq = -1;
      for (int s = 0; s < n_seqs; ++s)
        if (row >= starts[s] && row < starts[s + 1]) seq = s;
      const SeqOf f = seq_of_row(starts.data(), n_seqs, n_rows, row);
      CHECK(f.seq == seq);
      if (seq >= 0) CHECK(f.rows.row0 <= row && row < f.rows.row0 + f.rows.rows && f.rows.row0 == (starts[seq] < 0 ? 0 : starts[seq]));
    }
    // entries in any order: a sequence of the call and rows within, or none
    for (auto& x : starts) x = random(5) == 0 ? (random(2) ? INT_MAX : INT_MIN) : random(80) - 10;
    for (int row = 0; row < n_rows; ++row) {
      const SeqOf f = seq_of_row(starts.data(), n_seqs, n_rows, row);
      CHECK(f.seq >= -1 && f.seq < n_seqs);
      if (f.seq >= 0) CHECK(f.rows.row0 >= 0 && f.rows.row0 <= row && row < f.rows.row0 + f.rows.rows && f.rows.row0 + f.rows.rows <= n_rows);
    }
  }
  for (int64_t row : {0, 5, 8388607}) {
    const SeqOf f = seq_of_row(nullptr, 1 << 20, 1 << 23, row);
    CHECK(f.seq == row && f.rows.row0 == row && f.rows.rows == 1);
  }
  std::puts("ok");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_rows_find_their_sequence(tmp_path):
    src, exe = tmp_path / "search.cpp", tmp_path / "search"
    src.write_text(SEARCH)
    build = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined",
                            "-fno-sanitize-recover=undefined", "-I", CSRC, str(src), "-o", str(exe)],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr
