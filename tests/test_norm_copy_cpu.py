"""The shared copy of a row whose ends lie anywhere, on the host: every byte of the row once, and
none outside its tensor."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <stdio.h>
#include <string.h>
#include <vector>
#include "qmm_norm_copy.h"

// A tensor of M rows of N elements, `ld` apart, that begins `base` bytes behind a boundary of 16.
static int check(int size, int N, int64_t M, int64_t ld, int base, int threads) {
  const int64_t first = base, last = base + ((M - 1) * ld + N) * size;  // of the tensor, from that boundary on
  for (int64_t m = 0; m < M; ++m) {
    const int64_t row = base + m * ld * size, from = row & ~15ll;
    const int skew = (int)(row & 15), bytes = N * size;
    std::vector<int> times(skew + bytes + 16, 0);
    bool good = true;
    auto take = [&](int at, int n) {
      good &= n > 0 && from + at >= first && from + at + n <= last && at >= 0 && at + n <= (int)times.size();
      for (int i = at; good && i < at + n; ++i) ++times[i];
    };
    for (int t = 0; t < threads; ++t)
      qmm::copy_row(t, threads, m, skew, bytes,
                    [&](int at, int n) { good &= at % 16 == 0 && n <= 16; take(at, n); }, [&](int at) { take(at, 2); });
    for (int i = skew; i < skew + bytes; ++i) good &= times[i] == 1;
    if (!good) {
      printf("size %d N %d M %lld ld %lld base %d threads %d: row %lld\n", size, N, (long long)M, (long long)ld, base, threads, (long long)m);
      return 1;
    }
  }
  return 0;
}

int main() {
  int bad = 0;
  const int sizes[] = {65, 66, 71, 72, 127, 128, 777, 1001};
  for (int size = 2; size <= 4; size += 2)
    for (int N : sizes)
      for (int gap = 0; gap < 9; ++gap)
        for (int base = 0; base < 16; base += size)
          for (int threads = 32; threads <= 1024; threads *= 4)
            for (int M = 1; M <= 4; M += 3) bad += check(size, N, M, N + gap, base, threads);
  return bad != 0;
}
"""


def test_every_byte_once_and_none_outside(tmp_path):
    src, exe = tmp_path / "copy.cc", tmp_path / "copy"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "speculative_decode_verification_qmm_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout[:2000]
