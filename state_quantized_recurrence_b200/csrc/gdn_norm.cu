// Root-mean-square norm of rows, with the residual stream's addition in
// front, the output gate behind, and the result in the input's type or in 8
// bits with the state's codecs:
//   s = round(x + residual)            (s = x without a residual)
//   n = s / sqrt(mean(s^2) + eps),  y = n * w * silu(gate)
//   FP8 row: scale = amax |y| / 448, code = E4M3(y / scale)
//   INT8 group: scale = amax of the group / 127, code = rint(y / scale)
// and its gradient, with dn = dy * w * silu(gate):
//   ds = (dn - n mean(dn n)) / sqrt(mean(s^2) + eps) + dresidual
//   dw = sum over rows of dy silu(gate) n,  dgate = dy n w silu'(gate)
//
// Both are bound by HBM: every element is read once, kept in registers
// across the row's reductions, and written once.  A row belongs to TPR
// neighbouring threads with VPT vectors each (16 bytes forward), chosen by
// the row's length so that short rows (a head's 128 values: 16 lanes) fill
// their warps and long rows spread over a CTA.
#include "gdn_layer.cuh"
#include "gdn_host.cuh"
#include "gdn_layer.h"

namespace gdn {
namespace norm {

using namespace layer;

// Rows [tokens, heads, d]: heads and elements contiguous, tokens `stride`
// elements apart.
struct Rows {
  long long stride;
  __device__ __forceinline__ long long at(long long row, int heads, int d) const {
    if (heads == 1) return row * stride;
    const long long t = row / heads;
    return t * stride + (row - t * heads) * (long long)d;
  }
};

// 1 / sqrt(v), and 0 for v = 0: a row of zeros without an eps has outputs, codes
// and gradients of zero.
__device__ __forceinline__ float inverse_root(float v) { return v == 0.0f ? 0.0f : __frsqrt_rn(v); }

// max that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Reductions over the TPR threads of a row; `red` holds one value a warp.
// Every thread of the block calls them.  The values are added in a fixed
// order.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float *red) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if constexpr (TPR > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    const int w0 = threadIdx.x / TPR * (TPR / 32);
    x = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) x += red[w0 + w];
  }
  return x;
}
template <int TPR>
__device__ __forceinline__ float row_max(float x, float *red) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
    x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  if constexpr (TPR > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    const int w0 = threadIdx.x / TPR * (TPR / 32);
    x = red[w0];
#pragma unroll
    for (int w = 1; w < TPR / 32; ++w) x = max_nan(x, red[w0 + w]);
  }
  return x;
}

enum Out : int { kSame = 0, kFp8Row = 1, kInt8 = 2 };

template <int TPR>
constexpr int kBlock = TPR < 128 ? 128 : TPR;

template <typename T>
struct FwdArgs {
  const T *x, *residual, *gate;
  Rows xr, rr, gr;
  const float *w;
  long long rows;
  int heads, d, group;
  float eps;
  T *y, *res_out;
  uint8_t *codes;
  float *scales;
};

// Codes of V values with one scale: E4M3 (round to nearest even,
// saturating) or INT8 (round half to even, clamped), by the correctly
// rounded quotient.  A zero scale gives code 0; a scale that is not finite
// gives codes that mean nothing beside it.
__device__ __forceinline__ uint32_t code_pair(float a, float b, const ScaleRecip &sr, bool some, bool fp8) {
  float qa = 0.0f, qb = 0.0f;
  if (some) div_by_scale2(a, b, sr, qa, qb);
  if (fp8) return __nv_cvt_float2_to_fp8x2(make_float2(qa, qb), __NV_SATFINITE, __NV_E4M3);
  const int ia = __float2int_rn(fminf(fmaxf(qa, -127.0f), 127.0f));
  const int ib = __float2int_rn(fminf(fmaxf(qb, -127.0f), 127.0f));
  return (ia & 0xff) | (ib & 0xff) << 8;
}
template <int V>
__device__ __forceinline__ void store_codes(const float (&y)[V], float s, bool fp8, uint8_t *p) {
  const bool some = s > 0.0f;
  const ScaleRecip sr = make_scale(some ? s : 1.0f);
  if constexpr (V == 1) {
    *p = (uint8_t)code_pair(y[0], 0.0f, sr, some, fp8);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      w[i] = code_pair(y[4 * i], y[4 * i + 1], sr, some, fp8) |
             code_pair(y[4 * i + 2], y[4 * i + 3], sr, some, fp8) << 16;
    if constexpr (V == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(p) = w[0];
  }
}

template <typename T, int V, int TPR, int VPT, int OUT>
__global__ void __launch_bounds__(kBlock<TPR>)
norm_fwd_kernel(const FwdArgs<T> a) {
  constexpr int kThreads = kBlock<TPR>;
  __shared__ float red[kThreads / 32];
  const int lane = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  const bool live = row < a.rows;
  const int nv = a.d / V;
  const T *xp = a.x + (live ? a.xr.at(row, a.heads, a.d) : 0);
  Vec<T, V> sv[VPT], gv[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = k * TPR + lane;
    if (live && i < nv) sv[k].load(xp + (long long)i * V);
    else sv[k].zero();
  }
  if (a.gate) {
    const T *gp = a.gate + (live ? a.gr.at(row, a.heads, a.d) : 0);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = k * TPR + lane;
      if (live && i < nv) gv[k].load(gp + (long long)i * V);
      else gv[k].zero();
    }
  }
  if (a.residual) {
    const T *rp = a.residual + (live ? a.rr.at(row, a.heads, a.d) : 0);
    Vec<T, V> rv[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = k * TPR + lane;
      if (live && i < nv) rv[k].load(rp + (long long)i * V);
      else rv[k].zero();
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = k * TPR + lane;
      float f[V], r[V];
      sv[k].get(f);
      rv[k].get(r);
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] += r[v];
      sv[k].set(f);  // the stream's own type: the norm and its gradient see what is kept
      if (live && i < nv) sv[k].store(a.res_out + row * a.d + (long long)i * V);
    }
  }
  float sq = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    float f[V];
    sv[k].get(f);
#pragma unroll
    for (int v = 0; v < V; ++v) sq = fmaf(f[v], f[v], sq);
  }
  sq = row_sum<TPR>(sq, red);
  const float r = inverse_root(sq / (float)a.d + a.eps);
  const bool wal = (reinterpret_cast<uintptr_t>(a.w) & 15) == 0;

  float y[OUT == kSame ? 1 : VPT][V];
  float amax[OUT == kSame ? 1 : VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = k * TPR + lane;
    float(&o)[V] = y[OUT == kSame ? 0 : k];
    sv[k].get(o);
    if (i < nv) {
      float w[V];
      load_params<V>(a.w + (long long)i * V, wal, w);
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = o[v] * r * w[v];
    }
    if (a.gate) {
      float g[V];
      gv[k].get(g);
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] *= g[v] * sigmoid<T>(g[v]);
    }
    if constexpr (OUT == kSame) {
      Vec<T, V> out;
      out.set(o);
      if (live && i < nv) out.store(a.y + row * a.d + (long long)i * V);
    } else {
      float m = 0.0f;
      if (i < nv) {
#pragma unroll
        for (int v = 0; v < V; ++v) m = max_nan(m, fabsf(o[v]));
      }
      amax[k] = m;
    }
  }
  if constexpr (OUT == kFp8Row) {
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) m = max_nan(m, amax[k]);
    const float s = fp8_scale(row_max<TPR>(m, red));
    if (live && lane == 0) a.scales[row] = s;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = k * TPR + lane;
      if (live && i < nv) store_codes<V>(y[k], s, true, a.codes + row * a.d + (long long)i * V);
    }
  }
  if constexpr (OUT == kInt8) {  // a group is 2 .. 16 neighbouring lanes' vectors
    const int lanes = a.group / V;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = k * TPR + lane;
      float m = amax[k];
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, m, o);
        if (o < lanes) m = max_nan(m, other);
      }
      const float s = int8_scale(m);
      if (live && i < nv) {
        if (i % lanes == 0) a.scales[row * (a.d / a.group) + i / lanes] = s;
        store_codes<V>(y[k], s, false, a.codes + row * a.d + (long long)i * V);
      }
    }
  }
}

template <typename T>
struct BwdArgs {
  const T *s, *dy, *gate, *dres;
  Rows sr, dyr, gr, dr;
  const float *w;
  long long rows;
  int heads, d;
  float eps;
  T *dx, *dgate;
  float *partial;  // [CTAs][d]
};

// A CTA takes rows b, b + grid, .. of its row groups and keeps its columns'
// weights and dw in registers; the next row's loads are in flight while a
// row is reduced (both sums in one pass, one barrier where a row spans
// several warps).  The groups are added in shared memory, the CTAs by
// norm_reduce_kernel, both in order.
template <typename T, int V, int TPR, int VPT, bool GATE, bool RES>
__global__ void __launch_bounds__(kBlock<TPR>)
norm_bwd_kernel(const BwdArgs<T> a) {
  constexpr int kThreads = kBlock<TPR>, kGroups = kThreads / TPR, kWarps = kThreads / 32;
  __shared__ float red[2][2][kWarps];
  __shared__ float cols[kGroups > 1 ? kGroups : 1][kGroups > 1 ? TPR * VPT * V : 1];
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int nv = a.d / V;
  const bool wal = (reinterpret_cast<uintptr_t>(a.w) & 15) == 0;
  float dw[VPT][V], w[VPT][V];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = k * TPR + lane;
#pragma unroll
    for (int v = 0; v < V; ++v) dw[k][v] = w[k][v] = 0.0f;
    if (i < nv) load_params<V>(a.w + (long long)i * V, wal, w[k]);
  }
  struct Row {
    Vec<T, V> s[VPT], dy[VPT], gate[GATE ? VPT : 1], res[RES ? VPT : 1];
  };
  auto load = [&](long long row, Row &r) {
    const bool live = row < a.rows;
    const T *sp = a.s + (live ? a.sr.at(row, a.heads, a.d) : 0);
    const T *dp = a.dy + (live ? a.dyr.at(row, a.heads, a.d) : 0);
    const T *gp = GATE ? a.gate + (live ? a.gr.at(row, a.heads, a.d) : 0) : nullptr;
    const T *rp = RES ? a.dres + (live ? a.dr.at(row, a.heads, a.d) : 0) : nullptr;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = k * TPR + lane;
      const bool in = live && i < nv;
      const long long o = (long long)i * V;
      if (in) r.s[k].load(sp + o); else r.s[k].zero();
      if (in) r.dy[k].load(dp + o); else r.dy[k].zero();
      if constexpr (GATE) { if (in) r.gate[k].load(gp + o); else r.gate[k].zero(); }
      if constexpr (RES) { if (in) r.res[k].load(rp + o); else r.res[k].zero(); }
    }
  };
  const long long step = (long long)gridDim.x * kGroups;
  Row next;
  load((long long)blockIdx.x * kGroups + group, next);
  int turn = 0;
#pragma unroll 1
  for (long long base = (long long)blockIdx.x * kGroups; base < a.rows; base += step, turn ^= 1) {
    const long long row = base + group;
    const Row cur = next;
    load(row + step, next);
    float sq = 0.0f, dot = 0.0f;  // sum s^2 and sum dn s
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float s[V], g[V];
      cur.s[k].get(s);
      cur.dy[k].get(g);
      if constexpr (GATE) {
        float z[V];
        cur.gate[k].get(z);
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] *= z[v] * sigmoid<T>(z[v]);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sq = fmaf(s[v], s[v], sq);
        dot = fmaf(g[v] * w[k][v], s[v], dot);
      }
    }
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
      sq += __shfl_xor_sync(0xffffffffu, sq, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    if constexpr (TPR > 32) {  // two sets of sums in turn: one barrier a row
      if ((threadIdx.x & 31) == 0) {
        red[turn][0][threadIdx.x >> 5] = sq;
        red[turn][1][threadIdx.x >> 5] = dot;
      }
      __syncthreads();
      const int w0 = threadIdx.x / TPR * (TPR / 32);
      sq = dot = 0.0f;
#pragma unroll
      for (int i = 0; i < TPR / 32; ++i) {
        sq += red[turn][0][w0 + i];
        dot += red[turn][1][w0 + i];
      }
    }
    const float r = inverse_root(sq / (float)a.d + a.eps);
    const float c = dot * r * r / (float)a.d;  // ds = r (dn - s c)
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = k * TPR + lane;
      if (row >= a.rows || i >= nv) continue;
      const long long o = row * a.d + (long long)i * V;
      float s[V], g[V], e[V];
      cur.s[k].get(s);
      cur.dy[k].get(g);
      if constexpr (RES) cur.res[k].get(e);
      if constexpr (GATE) {
        float z[V], dz[V];
        cur.gate[k].get(z);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float sg = sigmoid<T>(z[v]);
          dz[v] = g[v] * (s[v] * r) * w[k][v] * (sg * (1.0f + z[v] * (1.0f - sg)));
          g[v] *= z[v] * sg;
        }
        Vec<T, V> out;
        out.set(dz);
        out.store(a.dgate + o);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        dw[k][v] = fmaf(g[v], s[v] * r, dw[k][v]);
        const float ds = fmaf(g[v], w[k][v], -s[v] * c);
        e[v] = RES ? fmaf(r, ds, e[v]) : r * ds;
      }
      Vec<T, V> out;
      out.set(e);
      out.store(a.dx + o);
    }
  }
  if constexpr (kGroups > 1) {
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) cols[group][(k * TPR + lane) * V + v] = dw[k][v];
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      float s = 0.0f;
      for (int g = 0; g < kGroups; ++g) s += cols[g][c];
      a.partial[(long long)blockIdx.x * a.d + c] = s;
    }
  } else {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = k * TPR + lane;
      if (i >= nv) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) a.partial[(long long)blockIdx.x * a.d + (long long)i * V + v] = dw[k][v];
    }
  }
}

// dw[c] = sum over the CTAs' partials: a warp's lanes are columns, the 16
// warps take every 16th partial and are added in order.
__global__ void __launch_bounds__(512)
norm_reduce_kernel(const float *__restrict__ partial, int ctas, int d, float *__restrict__ dw) {
  __shared__ float sums[16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < d) {
#pragma unroll 4
    for (int i = warp; i < ctas; i += 16) s += __ldg(partial + (long long)i * d + c);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < d) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += sums[w][lane];
    dw[c] = s;
  }
}

// ------------------------------------------------------------------ host ----
// CTAs of the gradient, four on every SM: 16384 x 2048 bf16 with a residual's
// gradient 54.5 us, 75 % of the copy rate; six, which do not fit at once, 65.
constexpr int kMaxCtas = 148 * 4;

// Threads a row and vectors a thread by the row's vectors: whole rows in a
// warp up to 128 vectors (no block barrier), then 64 to 1024 threads with
// four vectors each in flight (16384 x 2048 bf16 with a residual to E4M3: 44
// us, 81 % of the copy rate, with 64 threads of four; 47 with a warp of
// eight, 48 with 128 of two, 53 with 256 of one).  The gradient, which holds three to four
// tensors of two rows, keeps to two vectors a thread where it can.  CTAs of 512
// threads and more leave it too few registers for them: bf16 rows above 4096
// with a gate spill 216 to 280 bytes, all above 8192 256 to 892, above 16384, with
// four vectors, 0.9 to 2.3 KB.  33.5 million elements, bf16, with a residual's
// gradient and a gate: 101 us at d = 4096, 114 at 8192, 373 at 16384 (the bytes
// take 61); without a gate 54 at 2048, 146 at 16384 (41).
#define GDN_NORM_SHAPE(nv, CALL)          \
  ((nv) <= 8      ? CALL(8, 1)            \
   : (nv) <= 16   ? CALL(16, 1)           \
   : (nv) <= 32   ? CALL(32, 1)           \
   : (nv) <= 64   ? CALL(32, 2)           \
   : (nv) <= 128  ? CALL(32, 4)           \
   : (nv) <= 256  ? CALL(64, 4)           \
   : (nv) <= 512  ? CALL(128, 4)          \
   : (nv) <= 1024 ? CALL(256, 4)          \
   : (nv) <= 2048 ? CALL(512, 4)          \
   : (nv) <= 4096 ? CALL(1024, 4)         \
                  : CALL(1024, 8))
// 8192 elements one by one, 4096 vectors of them (eight vectors a thread
// would not fit a CTA of 1024).
template <int V>
constexpr int max_vectors() { return V == 1 ? 8192 : 4096; }

template <typename T, int V, int TPR, int VPT>
gdn_status fwd_shape(const FwdArgs<T> &a, int out, cudaStream_t st) {
  if constexpr (V > 1 && VPT > 4) return GDN_ERR_UNSUPPORTED;
  else {
  constexpr int kThreads = kBlock<TPR>;
  const long long blocks = (a.rows + kThreads / TPR - 1) / (kThreads / TPR);
  if (blocks > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  const unsigned nb = (unsigned)blocks;
  if (out == kSame) norm_fwd_kernel<T, V, TPR, VPT, kSame><<<nb, kThreads, 0, st>>>(a);
  else if (out == kFp8Row) norm_fwd_kernel<T, V, TPR, VPT, kFp8Row><<<nb, kThreads, 0, st>>>(a);
  else if constexpr (V > 1) norm_fwd_kernel<T, V, TPR, VPT, kInt8><<<nb, kThreads, 0, st>>>(a);
  else return GDN_ERR_INVALID_ARG;
  return launched();
  }
}

template <typename T, int V>
gdn_status fwd_vec(const FwdArgs<T> &a, int out, cudaStream_t st) {
  const int nv = a.d / V;
  if (nv > max_vectors<V>()) return GDN_ERR_UNSUPPORTED;
#define GDN_NORM_F(TPR, VPT) fwd_shape<T, V, TPR, VPT>(a, out, st)
  return GDN_NORM_SHAPE(nv, GDN_NORM_F);
#undef GDN_NORM_F
}

template <typename T, int V, int TPR, int VPT>
gdn_status bwd_shape(const BwdArgs<T> &a, int ctas, cudaStream_t st) {
  if constexpr (V > 1 && VPT > 4) return GDN_ERR_UNSUPPORTED;
  else {
    if (a.gate && a.dres) norm_bwd_kernel<T, V, TPR, VPT, true, true><<<ctas, kBlock<TPR>, 0, st>>>(a);
    else if (a.gate) norm_bwd_kernel<T, V, TPR, VPT, true, false><<<ctas, kBlock<TPR>, 0, st>>>(a);
    else if (a.dres) norm_bwd_kernel<T, V, TPR, VPT, false, true><<<ctas, kBlock<TPR>, 0, st>>>(a);
    else norm_bwd_kernel<T, V, TPR, VPT, false, false><<<ctas, kBlock<TPR>, 0, st>>>(a);
    return launched();
  }
}

template <typename T, int V>
gdn_status bwd_vec(const BwdArgs<T> &a, int ctas, cudaStream_t st) {
  const int nv = a.d / V;
  if (nv > max_vectors<V>()) return GDN_ERR_UNSUPPORTED;
#define GDN_NORM_SHAPE2(nv, CALL)         \
  ((nv) <= 8      ? CALL(8, 1)            \
   : (nv) <= 16   ? CALL(16, 1)           \
   : (nv) <= 32   ? CALL(32, 1)           \
   : (nv) <= 64   ? CALL(32, 2)           \
   : (nv) <= 128  ? CALL(64, 2)           \
   : (nv) <= 256  ? CALL(128, 2)          \
   : (nv) <= 512  ? CALL(256, 2)          \
   : (nv) <= 1024 ? CALL(512, 2)          \
   : (nv) <= 2048 ? CALL(1024, 2)         \
   : (nv) <= 4096 ? CALL(1024, 4)         \
                  : CALL(1024, 8))
#define GDN_NORM_B(TPR, VPT) bwd_shape<T, V, TPR, VPT>(a, ctas, st)
  return GDN_NORM_SHAPE2(nv, GDN_NORM_B);
#undef GDN_NORM_B
}

// CTAs of the gradient: one row each at least, kMaxCtas at most.
int bwd_ctas(long long rows) { return (int)(rows < kMaxCtas ? (rows > 0 ? rows : 1) : kMaxCtas); }

template <typename T, int V>
bool rows_aligned(const void *p, long long stride, int d) {
  return !p || (aligned_to(p, sizeof(T) * V) && stride % V == 0 && d % V == 0);
}

template <typename T, int V>
gdn_status fwd_typed(const FwdArgs<T> &a, int out, cudaStream_t st) {
  const bool v = rows_aligned<T, V>(a.x, a.xr.stride, a.d) &&
                 rows_aligned<T, V>(a.residual, a.rr.stride, a.d) &&
                 rows_aligned<T, V>(a.gate, a.gr.stride, a.d) &&
                 rows_aligned<T, V>(a.y, V, a.d) && rows_aligned<T, V>(a.res_out, V, a.d) &&
                 (!a.codes || aligned_to(a.codes, V));
  if (v) return fwd_vec<T, V>(a, out, st);
  if (out == kInt8) return GDN_ERR_INVALID_ARG;
  return fwd_vec<T, 1>(a, out, st);
}

template <typename T, int V>
gdn_status bwd_typed(const BwdArgs<T> &a, int ctas, cudaStream_t st) {
  const bool v = rows_aligned<T, V>(a.s, a.sr.stride, a.d) &&
                 rows_aligned<T, V>(a.dy, a.dyr.stride, a.d) &&
                 rows_aligned<T, V>(a.gate, a.gr.stride, a.d) &&
                 rows_aligned<T, V>(a.dres, a.dr.stride, a.d) &&
                 rows_aligned<T, V>(a.dx, V, a.d) && rows_aligned<T, V>(a.dgate, V, a.d);
  return v ? bwd_vec<T, V>(a, ctas, st) : bwd_vec<T, 1>(a, ctas, st);
}

gdn_status check(long long tokens, int heads, int d, gdn_dtype dt, float eps) {
  if (tokens < 0 || heads <= 0 || d <= 0 || !(eps >= 0.0f)) return GDN_ERR_INVALID_ARG;
  if (!known_dtype(dt)) return GDN_ERR_UNSUPPORTED;
  if (tokens > 0x7fffffffffffLL / heads) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// A row tensor that is given has its tokens at least heads * d apart (or
// only one token) and its elements aligned.
bool bad_rows(const void *p, int64_t stride, long long tokens, int heads, int d, size_t e) {
  return p && (!aligned_to(p, e) || (tokens > 1 && stride < (int64_t)heads * d));
}

}  // namespace norm
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_norm(const void *x, int64_t x_stride, const void *residual,
                    int64_t residual_stride, const void *gate, int64_t gate_stride,
                    const float *weight, int64_t tokens, int heads, int d, float eps,
                    gdn_dtype dt, gdn_norm_out out, void *y, float *scales, void *residual_out,
                    void *cuda_stream) {
  gdn_status s = norm::check(tokens, heads, d, dt, eps);
  if (s != GDN_OK) return s;
  int kind, group = 0;
  switch (out) {
    case GDN_NORM_SAME: kind = norm::kSame; break;
    case GDN_NORM_FP8_ROW: kind = norm::kFp8Row; break;
    case GDN_NORM_INT8_GROUP16: kind = norm::kInt8; group = 16; break;
    case GDN_NORM_INT8_GROUP32: kind = norm::kInt8; group = 32; break;
    case GDN_NORM_INT8_GROUP64: kind = norm::kInt8; group = 64; break;
    default: return GDN_ERR_UNSUPPORTED;
  }
  if (group && d % group) return GDN_ERR_INVALID_ARG;
  if (tokens == 0) return GDN_OK;
  if (!x || !weight || !y || (kind != norm::kSame && !scales) ||
      (residual != nullptr) != (residual_out != nullptr))
    return GDN_ERR_INVALID_ARG;
  const size_t e = elem_bytes(dt);
  if (norm::bad_rows(x, x_stride, tokens, heads, d, e) ||
      norm::bad_rows(residual, residual_stride, tokens, heads, d, e) ||
      norm::bad_rows(gate, gate_stride, tokens, heads, d, e) || !aligned_to(residual_out, e) ||
      (kind == norm::kSame && !aligned_to(y, e)) || !aligned_to(weight, 4) ||
      !aligned_to(scales, 4))
    return GDN_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const bool same = kind == norm::kSame;
#define GDN_NORM_FWD(T, V)                                                                   \
  norm::fwd_typed<T, V>(                                                                     \
      norm::FwdArgs<T>{static_cast<const T *>(x), static_cast<const T *>(residual),          \
                       static_cast<const T *>(gate), {x_stride}, {residual_stride},          \
                       {gate_stride}, weight, tokens *heads, heads, d, group, eps,           \
                       same ? static_cast<T *>(y) : nullptr, static_cast<T *>(residual_out), \
                       same ? nullptr : static_cast<uint8_t *>(y), scales},                  \
      kind, st)
  return dt == GDN_DTYPE_F32 ? GDN_NORM_FWD(float, 4) : GDN_NORM_FWD(__nv_bfloat16, 8);
#undef GDN_NORM_FWD
}

size_t gdn_norm_backward_workspace_bytes(int64_t tokens, int heads, int d) {
  if (tokens <= 0 || heads <= 0 || d <= 0 || tokens > 0x7fffffffffffLL / heads) return 0;
  return (size_t)norm::bwd_ctas(tokens * heads) * d * sizeof(float);
}

gdn_status gdn_norm_backward(const void *x, int64_t x_stride, const void *gate,
                             int64_t gate_stride, const float *weight, const void *dy,
                             int64_t dy_stride, const void *dresidual, int64_t dresidual_stride,
                             int64_t tokens, int heads, int d, float eps, gdn_dtype dt,
                             void *workspace, size_t workspace_bytes, void *dx, float *dweight,
                             void *dgate, void *cuda_stream) {
  gdn_status s = norm::check(tokens, heads, d, dt, eps);
  if (s != GDN_OK) return s;
  if (!dweight || !aligned_to(dweight, 4)) return GDN_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (tokens == 0)
    return cudaMemsetAsync(dweight, 0, (size_t)d * 4, st) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
  if (!x || !weight || !dy || !dx || (gate != nullptr) != (dgate != nullptr))
    return GDN_ERR_INVALID_ARG;
  const size_t e = elem_bytes(dt);
  if (norm::bad_rows(x, x_stride, tokens, heads, d, e) ||
      norm::bad_rows(gate, gate_stride, tokens, heads, d, e) ||
      norm::bad_rows(dy, dy_stride, tokens, heads, d, e) ||
      norm::bad_rows(dresidual, dresidual_stride, tokens, heads, d, e) || !aligned_to(dx, e) ||
      !aligned_to(dgate, e) || !aligned_to(weight, 4))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned_to(workspace, 16) ||
      workspace_bytes < gdn_norm_backward_workspace_bytes(tokens, heads, d))
    return GDN_ERR_INVALID_ARG;
  const int ctas = norm::bwd_ctas(tokens * heads);
  float *partial = static_cast<float *>(workspace);
#define GDN_NORM_BWD(T, V)                                                                  \
  norm::bwd_typed<T, V>(                                                                    \
      norm::BwdArgs<T>{static_cast<const T *>(x), static_cast<const T *>(dy),               \
                       static_cast<const T *>(gate), static_cast<const T *>(dresidual),     \
                       {x_stride}, {dy_stride}, {gate_stride}, {dresidual_stride}, weight,  \
                       tokens *heads, heads, d, eps, static_cast<T *>(dx),                  \
                       static_cast<T *>(dgate), partial},                                   \
      ctas, st)
  s = dt == GDN_DTYPE_F32 ? GDN_NORM_BWD(float, 4) : GDN_NORM_BWD(__nv_bfloat16, 8);
#undef GDN_NORM_BWD
  if (s != GDN_OK) return s;
  norm::norm_reduce_kernel<<<(d + 31) / 32, 512, 0, st>>>(partial, ctas, d, dweight);
  return launched();
}

}  // extern "C"
