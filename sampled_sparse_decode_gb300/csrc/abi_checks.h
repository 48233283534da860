// abi_checks.h — argument checks that the ABI files share (internal to libsanta).
#pragma once

#include <algorithm>
#include <cstdint>

#include "kernels.h"
#include "q8.cuh"

namespace santa {
namespace abi {

constexpr int kMaxTeams = 16384;
constexpr int kMaxDraws = 4096;
constexpr int kMaxRopeDim = 128;
constexpr int64_t kMaxPages = 0x7fffffff;           // page ids are int32
constexpr int64_t kMaxTokens = int64_t(1) << 24;    // tokens of one chunk call
constexpr size_t kAlign = 256;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int map_cuda(cudaError_t e) { return e == cudaSuccess ? SANTA_OK : SANTA_ERR_CUDA; }

inline int check_cache_shape(int dtype, int batch, int hkv, int d, int T, int max_teams) {
  if (dtype != SANTA_F32 && dtype != SANTA_BF16) return SANTA_ERR_UNSUPPORTED;
  if (batch < 1 || hkv < 1 || max_teams < 1) return SANTA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SANTA_ERR_UNSUPPORTED;
  if (T != 64 && T != 128) return SANTA_ERR_UNSUPPORTED;
  if (max_teams > kMaxTeams || batch > 65535 || hkv > 65535) return SANTA_ERR_UNSUPPORTED;
  return SANTA_OK;
}
inline int check_heads(int hq, int hkv) {
  if (hq < 1 || hq % hkv != 0) return SANTA_ERR_INVALID_ARG;
  return hq / hkv > santa::kMaxGroup ? SANTA_ERR_UNSUPPORTED : SANTA_OK;
}
inline int check_tokens(int64_t num_tokens) {
  if (num_tokens < 0) return SANTA_ERR_INVALID_ARG;
  return num_tokens > kMaxTokens ? SANTA_ERR_UNSUPPORTED : SANTA_OK;
}
// Whether [a, a + bytes) meets one of the `rows` rows of row_bytes that lie stride_bytes
// (>= row_bytes) apart from b on.
inline bool meets(const void* a, int64_t bytes, const void* b, int64_t rows, int64_t row_bytes,
                  int64_t stride_bytes) {
  if (!a || !b || bytes <= 0 || rows <= 0 || row_bytes <= 0) return false;
  const __int128 lo = reinterpret_cast<uintptr_t>(a), at = reinterpret_cast<uintptr_t>(b);
  // the first row that ends behind lo
  const __int128 r = at + row_bytes > lo ? 0 : (lo - at - row_bytes) / stride_bytes + 1;
  return r < rows && at + r * stride_bytes < lo + bytes;
}

// A buffer of a call, for the overlap checks.
struct Span {
  const void* at;
  int64_t bytes;
};
template <int N>
bool meets_any(const Span& out, const Span (&in)[N]) {
  return std::any_of(in, in + N, [&](const Span& s) {
    return meets(out.at, out.bytes, s.at, 1, s.bytes, s.bytes);
  });
}

// CodeType of an 8-bit santa_dtype.
inline int code_of(int type, int* code) {
  if (type != SANTA_I8 && type != SANTA_E4M3) return SANTA_ERR_UNSUPPORTED;
  *code = type == SANTA_I8 ? kCodeI8 : kCodeE4M3;
  return SANTA_OK;
}

}  // namespace abi
}  // namespace santa
