"""Host check of the places that linear attention's workspace has for the segments of packed
sequences (csrc/places.h), compiled with the host compiler: over arrays of sequence ends
that decrease, pass the tokens or are negative, no segment lies past the last place; and the workspace's size."""
import ctypes
import os
import shutil
import subprocess

import pytest

import softmax_attention_backward_gb300 as A
from softmax_attention_backward_gb300 import build as B

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "softmax_attention_backward_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdint>
#include <vector>
#include "places.h"
using namespace attn;
static uint64_t state = 88172645463325252ull;
static uint32_t next32() { state ^= state << 13; state ^= state >> 7; state ^= state << 17; return (uint32_t)state; }
static long bad = 0, checked = 0;
static void check(const std::vector<int>& cu, int tokens) {
  const int n = (int)cu.size() - 1;
  for (int seg = 1; seg < 40; seg += 1 + seg / 4) {
    int64_t sum = 0, walks = 0, places = 0;
    int at = packed_end(cu[0], 0, tokens);
    bool ok = at >= 0 && at <= tokens;
    for (int i = 0; i < n; ++i) {
      const int end = packed_end(cu[i + 1], at, tokens);
      ok = ok && end >= at && end <= tokens;
      const int count = segments_of(end - at, seg), chunks = chunks_of(end - at);
      ok = ok && count >= 1 && (int64_t)count * seg >= chunks && (int64_t)(count - 1) * seg < (chunks > 0 ? chunks : 1);
      sum += end - at;
      walks += count;
      places += count - 1;
      at = end;
    }
    ok = ok && sum <= tokens && walks <= packed_walks(tokens, n, seg) && places <= packed_places(tokens, seg);
    ++checked;
    if (!ok && bad++ < 5) std::printf("n %d tokens %d seg %d: %lld tokens, %lld walks, %lld places\n", n, tokens, seg, (long long)sum, (long long)walks, (long long)places);
  }
}
int main() {
  for (int T : {1, 127, 128, 129, 4096, 8192, 100000, 1 << 30, 2147483647}) {
    check({0, T}, T);
    check({0, T, 0, T}, T);
    check({0, T, 0, T, 0, T}, T);
    check({T, 0, T}, T);
    check({-5, T / 2, T}, T);
    check({0, 2147483647, -2147483647 - 1, T}, T);
    std::vector<int> far(40, 0);
    far[1] = far[39] = T;
    check(far, T);
    std::vector<int> one(T < 5000 ? T + 1 : 1);          // as many sequences as tokens
    for (size_t i = 0; i < one.size(); ++i) one[i] = (int)i;
    if (one.size() > 1) check(one, T);
    for (int k = 0; k < 300; ++k) {
      std::vector<int> cu(2 + next32() % 100);
      for (int& x : cu) x = next32() % 8 ? (int)(next32() % ((uint32_t)T + 1)) : (int)next32();
      check(cu, T);
    }
  }
  std::printf("checked %ld bad %ld\n", checked, bad);
  return bad ? 1 : 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host C++ compiler")
def test_segments_have_places_whatever_the_array_holds(tmp_path):
    src = tmp_path / "places.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "places"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "bad 0" in r.stdout


@pytest.mark.parametrize("n,length", [(1, 8192), (200, 8), (1000, 128), (2000, 8), (12, 2048), (4096, 1)])
@pytest.mark.parametrize("hq,hkv", [(32, 32), (32, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_workspace_holds_only_states_that_can_be_handed_on(n, length, hq, hkv, D):
    # a segment has a chunk at least, so that there is at most one such state for every 128 tokens and KV head: one
    # array of them forwards, three backwards; without cu_seqlens, none where a sequence is one chunk
    B.build()
    L = A.lib()
    state = 4 * hkv * D * D
    for packed in (False, True):
        p = A._LinearProblem(n, 0 if packed else length, n * length, hq, hkv, D, 0.1, 0, 0, 0, 0, 0x10000 if packed else None,
                             0x10000, None)
        fwd, bwd = (f(ctypes.byref(p)) for f in (L.linear_attn_fwd_workspace_size, L.linear_attn_bwd_workspace_size))
        most = n * length // 128 if packed else n * ((length + 127) // 128 - 1)
        assert fwd <= most * state and bwd <= 3 * most * state
