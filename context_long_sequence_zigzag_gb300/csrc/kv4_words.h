// kv4_words.h — how append and read divide a CTA's work: tokens a CTA takes,
// and which token, head and channels a piece belongs to.  Plain C++ (the
// divisions are checked on the host for every shape that a cache may have).
#pragma once

#include <algorithm>
#include <cstdint>

#ifdef __CUDACC__
#define KV4_HD __host__ __device__ __forceinline__
#else
#define KV4_HD inline
#endif

namespace cpattn {

// What piece i (16 channels, two words) of a CTA's tokens is: of which token, k or v, head, piece.  The
// divisions are products with rounded-up reciprocals, exact while i times the
// divisor stays below 2^32; kv4_tokens_per_block sees to it.
struct Words {
  int nk, nv, words, all_k;  // pieces of a head's k, of its v, of a token, of all its k
  uint32_t by_words, by_nk, by_nv;
};
struct Word {
  int token, r, head, word;  // r: piece of all heads' k, or of all their v
  bool is_v;
};

KV4_HD uint32_t kv4_mul_high(uint32_t a, uint32_t b) {
#ifdef __CUDA_ARCH__
  return __umulhi(a, b);
#else
  return uint32_t((uint64_t(a) * b) >> 32);
#endif
}

KV4_HD Word word_of(const Words& n, int i) {
  Word x;
  x.token = int(n.words == 1 ? uint32_t(i) : kv4_mul_high(uint32_t(i), n.by_words));
  x.r = i - x.token * n.words;
  x.is_v = x.r >= n.all_k;
  if (x.is_v) x.r -= n.all_k;
  x.head = int(kv4_mul_high(uint32_t(x.r), x.is_v ? n.by_nv : n.by_nk));
  x.word = x.r - x.head * (x.is_v ? n.nv : n.nk);
  return x;
}

inline Words words_of(int hkv, int dqk, int dv) {
  Words n;
  n.nk = dqk / 16;
  n.nv = dv / 16;
  n.all_k = hkv * n.nk;
  n.words = hkv * (n.nk + n.nv);
  auto inverse = [](int d) { return uint32_t(((uint64_t(1) << 32) + d - 1) / d); };
  n.by_words = inverse(n.words);
  n.by_nk = inverse(n.nk);
  n.by_nv = inverse(n.nv);
  return n;
}

constexpr int kKv4Threads = 256;     // of a CTA of append and read
constexpr int kKv4MostTokens = 32;   // of a CTA

// Tokens a CTA of append or read takes: several words a thread once every SM
// has CTAs enough, whole tokens in any case, and no more than word_of divides.
inline int kv4_tokens_per_block(int words, int64_t tokens, int sms) {
  const int64_t fill = (kKv4Threads + words - 1) / words;        // a word a thread
  const int64_t many = tokens / (int64_t(sms) * 8);              // 8 CTAs an SM
  const int64_t exact = (int64_t(1) << 32) / (int64_t(words) * words);  // i < per * words, i * words < 2^32
  const int64_t per = std::max<int64_t>(std::max<int64_t>(1, kKv4Threads / words), std::min(many, fill * 16));
  return int(std::min<int64_t>({int64_t(kKv4MostTokens), per, std::max<int64_t>(1, exact)}));
}

}  // namespace cpattn

#undef KV4_HD
