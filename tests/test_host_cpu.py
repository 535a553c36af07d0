"""What the calls do on the host, without a GPU."""
import os
import subprocess

import pytest


@pytest.fixture(scope="module")
def lib():
    from dynamic_embedding_tables_amd import recis
    recis.load_library()
    return recis


def test_a_forked_process_asks_torch_before_it_launches(lib, monkeypatch):
    """torch refuses the GPU in a process that was forked off one that uses it: the handles kept to ask for the stream
    directly, which would not, are not a forked process's."""
    monkeypatch.setattr(lib, "_raw_stream", lambda device: 7 + device)
    monkeypatch.setattr(lib, "_current_device", lambda: 3)
    assert lib._stream() == 10
    pid = os.fork()
    if pid == 0:
        os._exit(0 if lib._raw_stream is None else 1)
    assert os.waitstatus_to_exitcode(os.waitpid(pid, 0)[1]) == 0
    assert lib._stream() == 10


DIVIDE = r"""
#include <cstdio>
#include <initializer_list>
#define __device__
#define __forceinline__ inline
static unsigned __umulhi(unsigned a, unsigned b) { return (unsigned)(((unsigned long long)a * b) >> 32); }
#include "divide.h"
using namespace recis;

int main() {
  const long long top = (1ll << 31) - 1;
  long long wrong = 0, checked = 0;
  auto quick = [&](long long d) {
    const Quick q(d);
    auto one = [&](long long x) {
      if (x < 0 || x > top) return;
      ++checked;
      wrong += divided((int)x, q) != (int)(x / d);
    };
    for (long long x = 0; x < 70; ++x) one(x), one(top - x);
    for (long long m : {1ll, 2ll, 3ll, 1000ll, top / d / 2, top / d - 1, top / d})
      for (long long x = m * d - 2; x <= m * d + 2; ++x) one(x);
  };
  for (long long d = 1; d < 5000; ++d) quick(d);
  for (int bits = 12; bits <= 31; ++bits)
    for (long long d = (1ll << bits) - 3; d <= (1ll << bits) + 3 && d <= top; ++d) quick(d);
  auto small = [&](long long d) {   // for x * d < 2^32
    const Div v = div_by(d);
    const long long most = ((1ll << 32) - 1) / d;
    auto one = [&](long long x) {
      if (x < 0 || x > most) return;
      ++checked;
      wrong += divided((unsigned)x, v) != (unsigned)(x / d);
    };
    for (long long x = 0; x < 70; ++x) one(x), one(most - x);
    for (long long m : {1ll, 2ll, 3ll, 1000ll, most / d / 2, most / d - 1, most / d})
      for (long long x = m * d - 2; x <= m * d + 2; ++x) one(x);
  };
  for (long long d = 1; d < 5000; ++d) small(d);
  for (int bits = 12; bits <= 18; ++bits)
    for (long long d = (1ll << bits) - 3; d <= (1ll << bits) + 3; ++d) small(d);
  printf("%lld %lld\n", wrong, checked);
}
"""


def test_divisions_by_multiplication(tmp_path):
    """csrc/divide.h itself, on the host: every divisor up to 5000 and those beside powers of two, at the ends of the
    range, and around multiples where a quotient changes."""
    src, exe = tmp_path / "divide.cpp", tmp_path / "divide"
    src.write_text(DIVIDE)
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dynamic_embedding_tables_amd", "csrc")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)])
    wrong, checked = map(int, subprocess.check_output([str(exe)], text=True).split())
    assert wrong == 0 and checked > 1_000_000
