"""Every load that the 8-bit product's kernels issue against the arrays it may
read: the arithmetic of csrc/linear_loads.hpp on the host, over all blocks,
waves, lanes and stages of a product, and the compiled kernels' loads, whose
whole offset has to be the lane's own (the part that the check against the
array's size covers without doubt).
"""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_draft_select_amd", "csrc")

PROGRAM = r"""
#include "linear_loads.hpp"
#include <algorithm>
#include <cstdio>
using namespace dfk;

static int64_t most;
static bool bad(const char* what, int64_t row, int64_t stage, int64_t off) {
  std::printf("%s: row %lld stage %lld offset %lld\n", what, (long long)row, (long long)stage, (long long)off);
  return true;
}

// one load of a lane: row and first piece of 16 bytes that it is for, from a buffer that begins at row `from`
static bool check(int64_t from, int64_t rows, int64_t stride, int H, int64_t row, int64_t byte, int stage, bool real, int64_t off) {
  const int64_t bytes = buffer_bytes(from, rows, stride, H), end = (rows - 1) * stride + (H + 15) / 16 * 16;
  if (bytes <= 0 || bytes > INT32_MAX || from * stride + bytes > end) return bad("buffer", from, stage, bytes);
  if (off < 0 || off > INT32_MAX || off % 16 || off != row * stride + byte) return bad("offset", row, stage, off);
  if (off < bytes && off + 16 > bytes) return bad("across the end", row, stage, off);
  if (real && from + row < rows && byte < H && off + 16 > bytes) return bad("not read", row, stage, off);
  most = std::max(most, off);
  return false;
}

template <int TT>
static bool tiles(int64_t R, int N, int H, int64_t xs, int64_t ws) {
  using L = TileLoads<TT>;
  const int n_st = (H + 127) / 128;
  for (int ct = 0; ct * kTileCh < N; ++ct)
    for (int rot : {0, (ct >> 3) * 5 % n_st, n_st - 1})
      for (int64_t row0 = 0; row0 < R; row0 += L::BM)
        for (int wave = 0; wave < 8; ++wave)
          for (int lane = 0; lane < 64; ++lane)
            for (int i = 0; i < L::PER; ++i)
              for (int s = 0; s < n_st + L::NB; ++s) {
                const int chb = std::min(ct * kTileCh, N - 64), chw = std::min(ct * kTileCh + (wave >> 1) * 64, N - 64) - chb;
                const int at = tile_stage(s, rot, n_st);
                if (s < n_st && (at < 0 || at >= n_st)) return bad("stage", s, rot, at);
                const int64_t row = i < 4 ? chw + tile_channel(wave, lane, i) : tile_token<TT>(wave, lane, i);
                if (row < 0 || row >= (i < 4 ? std::min(kTileCh, N - chb) : L::BM)) return bad("row", row, s, i);
                const int64_t stride = i < 4 ? ws : xs;
                const int64_t byte = load_piece(lane) + at * 128;
                const int off = (int)row * (int)stride + load_piece(lane) + at * 128;
                if (check(i < 4 ? chb : row0, i < 4 ? N : R, stride, H, row, byte, at, s < n_st, off)) return true;
              }
  return false;
}

static bool stream(int N, int H, int64_t ws) {
  const int steps = (H + 127) / 128;
  for (int group = 0; group * 16 < N; ++group)
    for (int lane = 0; lane < 64; ++lane)
      for (int i = 0; i < 2; ++i)
        for (int s = 0; s < steps; ++s) {
          const int row = stream_channel(lane, i);
          const int off = row * (int)ws + load_piece(lane) + s * 128;
          if (check(group * 16, N, ws, H, row, load_piece(lane) + s * 128, s, true, off)) return true;
        }
  return false;
}

int main() {
  long long R, xs, ws;
  int N, H;
  while (std::scanf("%lld %d %d %lld %lld", &R, &N, &H, &xs, &ws) == 5) {
    most = 0;
    bool wrong = stream(N, H, ws);
    if (N >= 64) wrong = wrong || tiles<2>(R, N, H, xs, ws) || tiles<4>(R, N, H, xs, ws) || tiles<8>(R, N, H, xs, ws);
    if (wrong) return std::printf("%lld x %d x %d, strides %lld %lld\n", R, H, N, xs, ws), 1;
    std::printf("%lld\n", (long long)most);
  }
  return 0;
}
"""

# R, N, H, strides (a multiple of 16, at least H; at most 2^22)
CASES = [(R, N, H, -(-H // 16) * 16 + px, -(-H // 16) * 16 + pw)
         for R, N in ((1, 64), (2, 65), (17, 70), (63, 127), (64, 128), (65, 256), (129, 257), (255, 300), (257, 513))
         for H, px, pw in ((1, 0, 0), (16, 0, 16), (100, 16, 0), (128, 0, 0), (129, 0, 64), (400, 0, 0))]
CASES += [(1, 64, 40, 0, 48), (1, 1, 300, 0, 0), (3, 9, 300, 304, 304), (300, 30, 5, 16, 16)]  # one row: stride 0
CASES += [(300, 300, 1000, 1 << 22, 1 << 22)]


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("linear_loads")
    src, exe = d / "loads.cpp", d / "loads"
    src.write_text(PROGRAM)
    subprocess.run([cc, "-O2", "-std=c++17", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)

    def run(cases):
        text = "\n".join(" ".join(str(v) for v in c) for c in cases) + "\n"
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout[-500:]
        return [int(v) for v in r.stdout.split()]
    return run


def test_every_load_lies_in_its_array_or_behind_its_size(program):
    assert len(program(CASES)) == len(CASES)


def test_the_largest_offset_fits_its_register(program):
    # 256 rows 2^22 bytes apart, the longest rows, and stages behind them
    most, = program([(256, 256, 65536, 1 << 22, 1 << 22)])
    assert 255 << 22 < most < 1 << 31


def test_compiled_loads_take_no_scalar_offset(tmp_path):
    import importlib.util
    spec = importlib.util.spec_from_file_location("_dflash_build_flags", os.path.join(ROOT, "block_draft_select_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    out = tmp_path / "linear.s"
    subprocess.run([cc, *build.COMMON_FLAGS, "-S", "--cuda-device-only", os.path.join(CSRC, "linear.hip"), "-o", str(out)], check=True,
                   capture_output=True)
    loads = [x.strip() for x in out.read_text().splitlines() if re.match(r"\s+buffer_load", x)]
    assert loads
    for x in loads:
        assert re.fullmatch(r"buffer_load_dwordx4 v\d+, s\[\d+:\d+\], 0 offen( offset:\d+)? lds", x), x
