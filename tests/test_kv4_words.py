"""How append and read of the 4-bit cache divide their work: every piece of
every token, for every shape that a cache may have, checked on the host."""

import ctypes
import os
import shutil
import subprocess

import pytest

cpa = pytest.importorskip("context_long_sequence_zigzag_gb300")

CSRC = os.path.join(os.path.dirname(os.path.abspath(cpa.__file__)), "csrc")

CHECK = r"""
#include <cstdio>
#include "kv4_words.h"
using namespace cpattn;
int main() {
  int bad = 0;
  for (int dqk : {64, 128, 192})
    for (int dv : {64, 128})
      for (int hkv = 1; hkv <= 1024; ++hkv) {
        const Words n = words_of(hkv, dqk, dv);
        // the most tokens that a CTA takes, over lengths of a call and sizes of a GPU
        int per = 0;
        for (int sms : {1, 152})
          for (int64_t tokens : {int64_t(1), int64_t(1000), int64_t(20000), int64_t(1) << 20, (int64_t(1) << 31) - 1}) {
            const int p = kv4_tokens_per_block(n.words, tokens, sms);
            if (p < 1 || p > kKv4MostTokens) { std::printf("per %d\n", p); return 1; }
            per = std::max(per, p);
          }
        bool wrong = false;
        int i = 0;
        for (int t = 0; t < per; ++t)
          for (int v = 0; v < 2; ++v)
            for (int h = 0, r = 0; h < hkv; ++h)
              for (int w = 0; w < (v ? n.nv : n.nk); ++w, ++r, ++i) {
                const Word x = word_of(n, i);
                wrong |= x.token != t || x.is_v != bool(v) || x.r != r || x.head != h || x.word != w;
              }
        if (wrong && ++bad < 20) std::printf("d %d/%d, %d heads, %d tokens a CTA\n", dqk, dv, hkv, per);
      }
  std::printf("%d shapes wrong\n", bad);
  return bad != 0;
}
"""


def test_every_piece_of_every_shape(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    (tmp_path / "check.cpp").write_text(CHECK)
    built = subprocess.run([gxx, "-O2", "-std=c++17", "-I", CSRC, "-o", str(tmp_path / "check"), str(tmp_path / "check.cpp")],
                           capture_output=True, text=True, timeout=120)
    assert built.returncode == 0, built.stderr
    done = subprocess.run([str(tmp_path / "check")], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stdout


def test_no_more_heads_than_were_checked():
    c = cpa.cp_kv4_t(num_seqs=1, hq=1024, hkv=1024, d_qk=192, d_v=128, gqa=0, dtype=cpa.CP_DT_BF16, scale=0.1, num_pages=1,
                     max_pages=1, pages=4096, weights=None, page_table=64)
    assert cpa._lib.cp_kv4_validate(ctypes.byref(c)) == cpa.CP_OK
    c.hq = c.hkv = 1025
    assert cpa._lib.cp_kv4_validate(ctypes.byref(c)) == cpa.CP_ERR_UNSUPPORTED
