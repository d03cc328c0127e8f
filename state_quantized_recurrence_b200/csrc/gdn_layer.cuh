// Device helpers shared by the convolution, the scan and the norm: 16-byte
// vectors of bf16 or fp32, the logistic gate, and the split of packed
// sequences into tiles.
#pragma once

#include "gdn_common.cuh"

namespace gdn {
namespace layer {

// V consecutive elements as fp32.  V = 1 loads one element at its own
// alignment; V = 4 (fp32, bf16) and V = 8 (bf16) load one aligned vector.
template <typename T, int V>
struct Vec;
template <typename T>
struct Vec<T, 1> {
  T raw;
  __device__ __forceinline__ void load(const T *p) { raw = *p; }
  __device__ __forceinline__ void store(T *p) const { *p = raw; }
  __device__ __forceinline__ void zero() { raw = T(0.0f); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32(raw); }
  __device__ __forceinline__ void set(const float (&f)[1]) { raw = T(f[0]); }
};
template <>
struct Vec<float, 4> {
  float4 raw;
  __device__ __forceinline__ void load(const float *p) { raw = *reinterpret_cast<const float4 *>(p); }
  __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = raw.x; f[1] = raw.y; f[2] = raw.z; f[3] = raw.w; }
  __device__ __forceinline__ void set(const float (&f)[4]) { raw = make_float4(f[0], f[1], f[2], f[3]); }
};
__device__ __forceinline__ void bf2_get(uint32_t w, float &lo, float &hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t bf2_set(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&p);
}
template <>
struct Vec<__nv_bfloat16, 4> {
  uint2 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { raw = *reinterpret_cast<const uint2 *>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint2 *>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = make_uint2(0, 0); }
  __device__ __forceinline__ void get(float (&f)[4]) const { bf2_get(raw.x, f[0], f[1]); bf2_get(raw.y, f[2], f[3]); }
  __device__ __forceinline__ void set(const float (&f)[4]) { raw = make_uint2(bf2_set(f[0], f[1]), bf2_set(f[2], f[3])); }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { raw = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    bf2_get(raw.x, f[0], f[1]); bf2_get(raw.y, f[2], f[3]);
    bf2_get(raw.z, f[4], f[5]); bf2_get(raw.w, f[6], f[7]);
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    raw = make_uint4(bf2_set(f[0], f[1]), bf2_set(f[2], f[3]), bf2_set(f[4], f[5]), bf2_set(f[6], f[7]));
  }
};

// V fp32 parameters (weights); aligned16 says that p is 16-byte aligned and
// V is a multiple of 4.
template <int V>
__device__ __forceinline__ void load_params(const float *p, bool aligned16, float (&f)[V]) {
  if constexpr (V % 4 == 0) {
    if (aligned16) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p + i));
        f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = __ldg(p + i);
}

// 1 / (1 + exp(-x)).  fp32 inputs take the correctly rounded division and
// expf; bf16 inputs, whose result is rounded to 8 bits, the fast forms (a
// few fp32 ulps).  Past |x| = 126 ln 2 the fast division gives 0, the limit.
template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
  if constexpr (sizeof(T) == 4) return 1.0f / (1.0f + expf(-x));
  return __fdividef(1.0f, 1.0f + __expf(-x));
}

// ------------------------------------------------------------- sequences ----
// Packed sequences are cut into tiles of L tokens counted from each
// sequence's own start.  Sequence s takes the slots from s + cu[s] / L on;
// the next sequence's first slot is at least ceil(n / L) (and at least one)
// further, so every tile has a slot of its own, every sequence has one slot
// at least, and n_seq + T / L slots hold them all.
struct Tile {
  int seq;          // -1: nothing to do in this slot
  int tile;         // index of the tile in its sequence (0 for an empty one)
  long long start;  // first row of the sequence
  long long len;    // its tokens
};

// Whether sequence s of cu is a range inside the T packed tokens that the
// first sequence starts and the last one ends, and that does not step back
// behind the start of the one in front of it, whose tokens it would write over.
__device__ __forceinline__ bool seq_ok(const int *__restrict__ cu, int n_seq, int s, int T) {
  const int a = cu[s], b = cu[s + 1];
  return a >= (s != 0 ? max(cu[s - 1], 0) : 0) && b >= a && b <= T && (s != 0 || a == 0) &&
         (s != n_seq - 1 || b == T);
}

// The tile of `slot`, found by a whole warp: each round probes 32 sequences
// and keeps the interval in which the slots pass `slot`, so that 1024
// sequences take two dependent loads.  Every index stays in [0, n_seq]
// whatever cu holds; a malformed cu finds no tile or a sequence that seq_ok
// accepts.
__device__ __forceinline__ Tile find_tile(const int *__restrict__ cu, int n_seq, int T, int L,
                                          long long slot) {
  Tile t;
  t.seq = -1;
  t.tile = 0;
  t.start = t.len = 0;
  if (!cu) {
    const long long per = T > 0 ? (T + L - 1LL) / L : 1;
    t.seq = (int)(slot / per);
    t.tile = (int)(slot - t.seq * per);
    t.start = (long long)t.seq * T;
    t.len = T;
    return t;
  }
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n_seq;  // the last sequence whose first slot is <= slot lies in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int probe = lo + lane * step;
    const bool below = probe < hi && (long long)probe + cu[probe] / L <= slot;
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int k = m ? 31 - __clz(m) : 0;
    hi = min(hi, lo + (k + 1) * step);
    lo = lo + k * step;
  }
  if (lo >= n_seq || !seq_ok(cu, n_seq, lo, T)) return t;
  const long long a = cu[lo], n = cu[lo + 1] - a, i = slot - (lo + a / L);
  if (i < 0 || (i > 0 && i * L >= n)) return t;
  t.seq = lo;
  t.tile = (int)i;
  t.start = a;
  t.len = n;
  return t;
}

// Slots of a call on the host: dense sequences have ceil(T / L) (at least
// one) tiles each.
inline long long slot_count(int n_seq, long long T, int L, bool packed) {
  if (n_seq == 0) return 0;
  if (packed) return n_seq + T / L;
  return n_seq * (T > 0 ? (T + L - 1) / L : 1);
}

// Reports a malformed cu; run by one block's threads at most.
__device__ __forceinline__ void check_seqlens(const int *__restrict__ cu, int n_seq, int T,
                                              unsigned *err) {
  for (int s = threadIdx.x; s < n_seq; s += blockDim.x)
    if (!seq_ok(cu, n_seq, s, T)) atomicOr(err, kErrBadSeqlens);
}

}  // namespace layer
}  // namespace gdn
