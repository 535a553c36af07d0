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


def test_in_place_with_other_strides_is_refused(lib):
    """out may be x, q_out q: then each element is read where it is written. With other strides it is not."""
    import ctypes as C

    from test_history_cpu import APPEND, INVALID, P, ROTARY, described
    L = lib.load_library()
    still = dict(ROTARY, rot_dim=0, freqs=None)   # (in place, with nothing that turns, there is no work to do)
    assert L.recis_rotary(C.byref(described(lib.recis_rotary_desc, still)), 0, P, P, None) == 0
    one = dict(still, batch=1)
    assert L.recis_rotary(C.byref(described(lib.recis_rotary_desc, one, out_strides=(7, 32, 8))), 0, P, P, None) == 0
    for strides in ((160, 8, 32), (160, 32, 9), (0, 32, 8)):
        for values in (ROTARY, still):
            d = described(lib.recis_rotary_desc, values, out_strides=strides)
            for backward in (0, 1):
                assert L.recis_rotary(C.byref(d), backward, P, P, None) == INVALID, strides
        d = described(lib.recis_append_desc, APPEND, q_out_strides=strides)
        assert L.recis_cache_append(C.byref(d), P, P, P, P, P, P, None) == INVALID, strides
