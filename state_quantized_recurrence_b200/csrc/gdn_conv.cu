// Short causal convolution over tokens, a channel at a time, with its state
// (the last W - 1 inputs) carried between calls, its one-token form and its
// gradient:
//   pre_t = bias + sum_{j < W} w_j x_{t - W + 1 + j},   y_t = act(pre_t)
//   dp_t = dy_t act'(pre_t),  dx_u = sum_j w_j dp_{u + W - 1 - j},
//   dw_j = sum_t dp_t x_{t - W + 1 + j},  dbias = sum_t dp_t
// with the state's rows in the places of the tokens before the first one.
//
// All three are bound by HBM (two planes of the sequence forward, three
// backward, 2 W - 1 flops a byte at most).  A thread owns a vector of
// channels (16 bytes forward) and walks a run of tokens with the last W - 1
// inputs in registers, so that x is read once but for the W - 1 rows in
// front of a run; a warp's lanes are neighbouring vectors.
#include "gdn_layer.cuh"
#include "gdn_host.cuh"
#include "gdn_layer.h"

namespace gdn {
namespace conv {

using namespace layer;

constexpr int kWarps = 8;  // runs of one CTA, one a warp

template <typename T>
__device__ __forceinline__ float act_fwd(float p, bool silu) {
  return silu ? p * sigmoid<T>(p) : p;
}
template <typename T>
__device__ __forceinline__ float act_grad(float p, bool silu) {
  if (!silu) return 1.0f;
  const float s = sigmoid<T>(p);
  return s * (1.0f + p * (1.0f - s));
}

// w[v][j] of V channels from c0 on (rows of W, fp32; a row of four taps in
// one load where the pointer allows it).
template <int V, int W>
__device__ __forceinline__ void load_taps(const float *w, long long c0, float (&t)[V][W]) {
  if constexpr (W == 4) {
    if ((reinterpret_cast<uintptr_t>(w) & 15) == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float4 r = __ldg(reinterpret_cast<const float4 *>(w + (c0 + v) * 4));
        t[v][0] = r.x; t[v][1] = r.y; t[v][2] = r.z; t[v][3] = r.w;
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < W; ++j) t[v][j] = __ldg(w + (c0 + v) * W + j);
}

template <int V>
__device__ __forceinline__ void load_bias(const float *b, long long c0, float (&f)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) f[v] = b ? __ldg(b + c0 + v) : 0.0f;
}

// Row `pos` (0 = first token of the sequence) of V channels; negative
// positions are the state's rows, or zero without a state.
template <typename T, int V, int W>
__device__ __forceinline__ Vec<T, V> row_or_state(const T *x, long long xs, long long start,
                                                  long long pos, const T *state, long long seq,
                                                  int C, long long c0) {
  Vec<T, V> r;
  if (pos >= 0) r.load(x + (start + pos) * xs + c0);
  else if (state) r.load(state + (seq * (W - 1) + (W - 1 + pos)) * C + c0);
  else r.zero();
  return r;
}

// Forward.  grid = (slots, channel blocks); warp w of a CTA takes tokens
// [RUN w, RUN (w + 1)) of the slot's tile.  RUN rows are loaded U at a time,
// so a thread keeps U 16-byte loads in flight.  The thread of a sequence's
// first run also writes the new state, after it has read the old one, which
// may be the same memory.
template <typename T, int V, int W, int RUN>
__global__ void __launch_bounds__(32 * kWarps)
conv_fwd_kernel(const T *x, long long xs, const float *__restrict__ weight,
                const float *__restrict__ bias, const T *state_in,
                const int *__restrict__ cu, int n_seq, int T_, int C, bool silu, T *y,
                T *state_out, unsigned *err) {
  constexpr int U = RUN < 8 ? RUN : 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (cu && blockIdx.x == 0 && blockIdx.y == 0) check_seqlens(cu, n_seq, T_, err);
  const Tile t = find_tile(cu, n_seq, T_, RUN * kWarps, blockIdx.x);
  if (t.seq < 0) return;
  const long long c0 = ((long long)blockIdx.y * 32 + lane) * V;
  if (c0 >= C) return;
  const long long p0 = (long long)t.tile * (RUN * kWarps) + warp * RUN;
  if (p0 >= t.len && !(p0 == 0)) return;

  float win[W - 1][V];
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    row_or_state<T, V, W>(x, xs, t.start, p0 - (W - 1) + k, state_in, t.seq, C, c0).get(win[k]);

  if (p0 == 0) {  // the new state: the last W - 1 rows of [old state; x]
    Vec<T, V> last[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      last[k] = row_or_state<T, V, W>(x, xs, t.start, t.len - (W - 1) + k, state_in, t.seq, C, c0);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      last[k].store(state_out + ((long long)t.seq * (W - 1) + k) * C + c0);
  }

  float taps[V][W], b[V];
  load_taps<V, W>(weight, c0, taps);
  load_bias<V>(bias, c0, b);
  const long long n = min((long long)RUN, t.len - p0);
  const T *xp = x + (t.start + p0) * xs + c0;
  T *yp = y + (t.start + p0) * C + c0;
  for (int base = 0; base < n; base += U) {
    Vec<T, V> in[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (base + u < n) in[u].load(xp + (base + u) * xs);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u >= n) break;
      float f[V], o[V];
      in[u].get(f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float p = b[v];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) p = fmaf(taps[v][j], win[j][v], p);
        p = fmaf(taps[v][W - 1], f[v], p);
        o[v] = act_fwd<T>(p, silu);
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][v] = win[j + 1][v];
        win[W - 2][v] = f[v];
      }
      Vec<T, V> out;
      out.set(o);
      out.store(yp + (long long)(base + u) * C);
    }
  }
}

// One token a sequence; the state moves up by one row in place.
template <typename T, int V, int W>
__global__ void __launch_bounds__(128)
conv_decode_kernel(const T *x, long long xs, const float *__restrict__ weight,
                   const float *__restrict__ bias, T *state, int C, bool silu, T *y) {
  const long long s = blockIdx.x;
  const long long c0 = ((long long)blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (c0 >= C) return;
  Vec<T, V> rows[W];
  T *st = state + s * (W - 1) * C + c0;
#pragma unroll
  for (int k = 0; k < W - 1; ++k) rows[k].load(st + (long long)k * C);
  rows[W - 1].load(x + s * xs + c0);
  float taps[V][W], p[V];
  load_taps<V, W>(weight, c0, taps);
  load_bias<V>(bias, c0, p);
#pragma unroll
  for (int k = 0; k < W; ++k) {
    float f[V];
    rows[k].get(f);
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = fmaf(taps[v][k], f[v], p[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] = act_fwd<T>(p[v], silu);
  Vec<T, V> out;
  out.set(p);
  out.store(y + s * C + c0);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) rows[k + 1].store(st + (long long)k * C);
}

// Gradient.  A warp walks its run of tokens [p0, p1) and W - 1 tokens more:
// at step t it forms pre_t and dp_t, and with dp_{t-W+1} .. dp_t at hand
// writes dx_{t-W+1}.  The first run of a sequence starts W - 1 rows early
// and writes the gradient of the state's rows.  The weights' gradients are
// summed in registers over the run, over the CTA's warps in shared memory,
// and go to partial[slot] ([W + 1][C], the bias last); conv_reduce_kernel
// adds the slots in order, so that results do not depend on timing.
template <typename T, int V, int W, int RUN>
__global__ void __launch_bounds__(32 * kWarps)
conv_bwd_kernel(const T *x, long long xs, const float *__restrict__ weight,
                const float *__restrict__ bias, const T *__restrict__ state_in,
                const int *__restrict__ cu, int n_seq, int T_, int C, bool silu,
                const T *__restrict__ dy, const T *__restrict__ dstate_out,
                float *__restrict__ partial, T *__restrict__ dx, T *__restrict__ dstate_in,
                unsigned *err) {
  __shared__ float sums[kWarps][W + 1][32 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (cu && blockIdx.x == 0 && blockIdx.y == 0) check_seqlens(cu, n_seq, T_, err);
  const Tile t = find_tile(cu, n_seq, T_, RUN * kWarps, blockIdx.x);
  const long long c0 = ((long long)blockIdx.y * 32 + lane) * V;
  const long long p0 = (long long)t.tile * (RUN * kWarps) + warp * RUN;
  float dw[V][W], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[v][j] = 0.0f;
  }
  if (t.seq >= 0 && c0 < C && (p0 < t.len || p0 == 0)) {
    const long long p1 = min(p0 + RUN, t.len);
    float taps[V][W], b[V], xw[W - 1][V], dpw[W - 1][V];
    load_taps<V, W>(weight, c0, taps);
    load_bias<V>(bias, c0, b);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      row_or_state<T, V, W>(x, xs, t.start, p0 - (W - 1) + k, state_in, t.seq, C, c0).get(xw[k]);
#pragma unroll
      for (int v = 0; v < V; ++v) dpw[k][v] = 0.0f;
    }
    const long long first = p0 == 0 ? -(W - 1) : p0;  // first row written
    // Rows p0 .. p1 - 1 + (W - 1); past the sequence's end dp is zero.
    constexpr int U = 4;
    for (long long base = p0; base < p1 + (W - 1); base += U) {
      Vec<T, V> xin[U], gin[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = base + u < t.len && base + u < p1 + (W - 1);
        if (in) {
          xin[u].load(x + (t.start + base + u) * xs + c0);
          gin[u].load(dy + (t.start + base + u) * C + c0);
        } else {
          xin[u].zero();
          gin[u].zero();
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long pos = base + u;
        if (pos >= p1 + (W - 1)) break;
        const bool in = pos < t.len;
        float f[V], g[V], dp[V];
        xin[u].get(f);
        gin[u].get(g);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float p = b[v];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) p = fmaf(taps[v][j], xw[j][v], p);
          p = fmaf(taps[v][W - 1], f[v], p);
          dp[v] = in ? g[v] * act_grad<T>(p, silu) : 0.0f;
          if (pos < p1) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) dw[v][j] = fmaf(dp[v], xw[j][v], dw[v][j]);
            dw[v][W - 1] = fmaf(dp[v], f[v], dw[v][W - 1]);
            db[v] += dp[v];
          }
#pragma unroll
          for (int j = 0; j + 1 < W - 1; ++j) xw[j][v] = xw[j + 1][v];
          xw[W - 2][v] = f[v];
        }
        const long long u0 = pos - (W - 1);  // dx_{u0} has all its terms now
        if (u0 >= first) {
          float o[V];
#pragma unroll
          for (int v = 0; v < V; ++v) {
            // w_j meets dp_{u0 + W - 1 - j}: j = 0 the newest
            float s = taps[v][0] * dp[v];
#pragma unroll
            for (int j = 1; j < W; ++j) s = fmaf(taps[v][j], dpw[W - 1 - j][v], s);
            o[v] = s;
          }
          if (dstate_out && u0 >= t.len - (W - 1)) {  // this row is in the new state
            Vec<T, V> e;
            e.load(dstate_out + ((long long)t.seq * (W - 1) + (u0 - (t.len - (W - 1)))) * C + c0);
            float f2[V];
            e.get(f2);
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] += f2[v];
          }
          Vec<T, V> out;
          out.set(o);
          if (u0 >= 0) out.store(dx + (t.start + u0) * C + c0);
          else out.store(dstate_in + ((long long)t.seq * (W - 1) + (W - 1 + u0)) * C + c0);
        }
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) dpw[j][v] = dpw[j + 1][v];
#pragma unroll
        for (int v = 0; v < V; ++v) dpw[W - 2][v] = dp[v];
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j < W; ++j) sums[warp][j][lane * V + v] = dw[v][j];
    sums[warp][W][lane * V + v] = db[v];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (W + 1) * 32 * V; i += blockDim.x) {
    const int j = i / (32 * V), c = i % (32 * V);
    const long long ch = (long long)blockIdx.y * 32 * V + c;
    if (ch >= C) continue;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][j][c];
    partial[((long long)blockIdx.x * (W + 1) + j) * C + ch] = s;
  }
}

// dw[c][j], dbias[c] = sums over the slots: a warp's lanes are channels, the
// CTA's warps take every kWarps-th slot and are added in order.
__global__ void __launch_bounds__(32 * kWarps)
conv_reduce_kernel(const float *__restrict__ partial, long long slots, int C, int W,
                   float *__restrict__ dw, float *__restrict__ dbias) {
  __shared__ float sums[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.y;
  const long long c = (long long)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 4
    for (long long i = warp; i < slots; i += kWarps) s += __ldg(partial + (i * (W + 1) + j) * C + c);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < C) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][lane];
    if (j < W) dw[c * W + j] = s;
    else dbias[c] = s;
  }
}

// ------------------------------------------------------------------ host ----
constexpr int kRun = 32, kRunShort = 8, kRunBwd = 32;

struct Args {
  const void *x;
  long long xs;
  const float *w, *b;
  const void *state_in;
  const int *cu;
  int n_seq, T, C, W;
  bool silu;
};

gdn_status check(const Args &a, gdn_dtype dt, int act) {
  if (a.n_seq < 0 || a.T < 0 || a.C <= 0 || a.xs < a.C) return GDN_ERR_INVALID_ARG;
  if (!known_dtype(dt) || (act != GDN_ACT_NONE && act != GDN_ACT_SILU)) return GDN_ERR_UNSUPPORTED;
  if (a.W < 2 || a.W > 4) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

bool vector_ok(const void *p, size_t bytes) { return !p || aligned_to(p, bytes); }

template <typename T, int V, int W, int RUN>
gdn_status fwd_launch(const Args &a, void *y, void *so, unsigned *err, cudaStream_t st) {
  const long long slots = slot_count(a.n_seq, a.T, RUN * kWarps, a.cu != nullptr);
  const long long cb = (a.C + 32LL * V - 1) / (32 * V);
  if (slots > 0x7fffffffLL || cb > 65535) return GDN_ERR_UNSUPPORTED;
  conv_fwd_kernel<T, V, W, RUN><<<dim3((unsigned)slots, (unsigned)cb), 32 * kWarps, 0, st>>>(
      static_cast<const T *>(a.x), a.xs, a.w, a.b, static_cast<const T *>(a.state_in), a.cu,
      a.n_seq, a.T, a.C, a.silu, static_cast<T *>(y), static_cast<T *>(so), err);
  return launched();
}

template <typename T, int V, int W>
gdn_status fwd_run(const Args &a, void *y, void *so, unsigned *err, cudaStream_t st) {
  // Runs of 32 tokens re-read 3 rows in 32; a call too small to give every
  // SM two such CTAs takes runs of 8, which spreads it over four times as many.
  const long long cb = (a.C + 32LL * V - 1) / (32 * V);
  if (slot_count(a.n_seq, a.T, kRun * kWarps, a.cu != nullptr) * cb < 2 * 148)
    return fwd_launch<T, V, W, kRunShort>(a, y, so, err, st);
  return fwd_launch<T, V, W, kRun>(a, y, so, err, st);
}

template <typename T, int V, int W>
gdn_status decode_run(const Args &a, void *state, void *y, cudaStream_t st) {
  const long long nv = (a.C + V - 1) / V;
  const int threads = nv >= 128 ? 128 : (int)((nv + 31) / 32 * 32);
  const long long cb = (nv + threads - 1) / threads;
  if (cb > 65535) return GDN_ERR_UNSUPPORTED;
  conv_decode_kernel<T, V, W><<<dim3((unsigned)a.n_seq, (unsigned)cb), threads, 0, st>>>(
      static_cast<const T *>(a.x), a.xs, a.w, a.b, static_cast<T *>(state), a.C, a.silu,
      static_cast<T *>(y));
  return launched();
}

struct BwdArgs {
  const void *dy, *dso;
  float *partial;
  void *dx;
  float *dw, *db;
  void *dsi;
};

template <typename T, int V, int W>
gdn_status bwd_run(const Args &a, const BwdArgs &g, unsigned *err, cudaStream_t st) {
  const long long slots = slot_count(a.n_seq, a.T, kRunBwd * kWarps, a.cu != nullptr);
  const long long cb = (a.C + 32LL * V - 1) / (32 * V);
  if (slots > 0x7fffffffLL || cb > 65535) return GDN_ERR_UNSUPPORTED;
  conv_bwd_kernel<T, V, W, kRunBwd><<<dim3((unsigned)slots, (unsigned)cb), 32 * kWarps, 0, st>>>(
      static_cast<const T *>(a.x), a.xs, a.w, a.b, static_cast<const T *>(a.state_in), a.cu,
      a.n_seq, a.T, a.C, a.silu, static_cast<const T *>(g.dy), static_cast<const T *>(g.dso),
      g.partial, static_cast<T *>(g.dx), static_cast<T *>(g.dsi), err);
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  conv_reduce_kernel<<<dim3((unsigned)((a.C + 31) / 32), (unsigned)(W + 1)), 32 * kWarps, 0, st>>>(
      g.partial, slots, a.C, W, g.dw, g.db);
  return launched();
}

#define GDN_CONV_W(FN, T, V, ...)                         \
  (a.W == 4 ? FN<T, V, 4>(__VA_ARGS__)                    \
            : a.W == 3 ? FN<T, V, 3>(__VA_ARGS__) : FN<T, V, 2>(__VA_ARGS__))

// Vectors need aligned pointers and a channel count and token stride that
// keep every row aligned; other calls go element by element.
bool vec(const Args &a, size_t e, int v, std::initializer_list<const void *> ps) {
  if (a.C % v || a.xs % v) return false;
  for (const void *p : ps)
    if (!vector_ok(p, e * v)) return false;
  return true;
}

}  // namespace conv
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_conv_prefill(const void *x, int64_t x_stride, const float *weight,
                            const float *bias, const void *state_in, const int32_t *cu_seqlens,
                            int n_seq, int T, int C, int W, gdn_dtype dt, gdn_activation act,
                            void *y, void *state_out, void *cuda_stream) {
  const conv::Args a{x, x_stride, weight, bias, state_in, cu_seqlens, n_seq, T, C, W,
                     act == GDN_ACT_SILU};
  gdn_status s = conv::check(a, dt, act);
  if (s != GDN_OK || n_seq == 0) return s;
  const size_t e = elem_bytes(dt);
  if (!weight || !state_out || (T > 0 && (!x || !y))) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(state_in, e) ||
      !aligned_to(state_out, e) || !aligned_to(weight, 4) || !aligned_to(bias, 4) ||
      !aligned_to(cu_seqlens, 4))
    return GDN_ERR_INVALID_ARG;
  unsigned *err = nullptr;
  if (cu_seqlens && (s = error_word(&err)) != GDN_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (dt == GDN_DTYPE_F32) {
    if (conv::vec(a, e, 4, {x, y, state_in, state_out}))
      return GDN_CONV_W(conv::fwd_run, float, 4, a, y, state_out, err, st);
    return GDN_CONV_W(conv::fwd_run, float, 1, a, y, state_out, err, st);
  }
  if (conv::vec(a, e, 8, {x, y, state_in, state_out}))
    return GDN_CONV_W(conv::fwd_run, __nv_bfloat16, 8, a, y, state_out, err, st);
  return GDN_CONV_W(conv::fwd_run, __nv_bfloat16, 1, a, y, state_out, err, st);
}

gdn_status gdn_conv_decode(const void *x, int64_t x_stride, const float *weight,
                           const float *bias, void *state_inout, int n_seq, int C, int W,
                           gdn_dtype dt, gdn_activation act, void *y, void *cuda_stream) {
  const conv::Args a{x, x_stride, weight, bias, nullptr, nullptr, n_seq, 1, C, W,
                     act == GDN_ACT_SILU};
  gdn_status s = conv::check(a, dt, act);
  if (s != GDN_OK || n_seq == 0) return s;
  const size_t e = elem_bytes(dt);
  if (!weight || !state_inout || !x || !y) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(state_inout, e) ||
      !aligned_to(weight, 4) || !aligned_to(bias, 4))
    return GDN_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (dt == GDN_DTYPE_F32) {
    if (conv::vec(a, e, 4, {x, y, state_inout}))
      return GDN_CONV_W(conv::decode_run, float, 4, a, state_inout, y, st);
    return GDN_CONV_W(conv::decode_run, float, 1, a, state_inout, y, st);
  }
  if (conv::vec(a, e, 8, {x, y, state_inout}))
    return GDN_CONV_W(conv::decode_run, __nv_bfloat16, 8, a, state_inout, y, st);
  return GDN_CONV_W(conv::decode_run, __nv_bfloat16, 1, a, state_inout, y, st);
}

size_t gdn_conv_backward_workspace_bytes(int n_seq, int T, int C, int W, int packed) {
  if (n_seq <= 0 || T < 0 || C <= 0 || W < 2 || W > 4) return 0;
  return (size_t)layer::slot_count(n_seq, T, conv::kRunBwd * conv::kWarps, packed != 0) *
         (size_t)(W + 1) * C * sizeof(float);
}

gdn_status gdn_conv_backward(const void *x, int64_t x_stride, const float *weight,
                             const float *bias, const void *state_in, const int32_t *cu_seqlens,
                             int n_seq, int T, int C, int W, gdn_dtype dt, gdn_activation act,
                             const void *dy, const void *dstate_out, void *workspace,
                             size_t workspace_bytes, void *dx, float *dweight, float *dbias,
                             void *dstate_in, void *cuda_stream) {
  const conv::Args a{x, x_stride, weight, bias, state_in, cu_seqlens, n_seq, T, C, W,
                     act == GDN_ACT_SILU};
  gdn_status s = conv::check(a, dt, act);
  if (s != GDN_OK) return s;
  if (!dweight || !dbias || !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
    return GDN_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (n_seq == 0) {
    if (cudaMemsetAsync(dweight, 0, (size_t)C * W * 4, st) != cudaSuccess ||
        cudaMemsetAsync(dbias, 0, (size_t)C * 4, st) != cudaSuccess)
      return GDN_ERR_CUDA;
    return GDN_OK;
  }
  const size_t e = elem_bytes(dt);
  if (!weight || !dstate_in || (T > 0 && (!x || !dy || !dx))) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(x, e) || !aligned_to(dy, e) || !aligned_to(dx, e) || !aligned_to(state_in, e) ||
      !aligned_to(dstate_out, e) || !aligned_to(dstate_in, e) || !aligned_to(weight, 4) ||
      !aligned_to(bias, 4) || !aligned_to(cu_seqlens, 4))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned_to(workspace, 16) ||
      workspace_bytes < gdn_conv_backward_workspace_bytes(n_seq, T, C, W, cu_seqlens != nullptr))
    return GDN_ERR_INVALID_ARG;
  unsigned *err = nullptr;
  if (cu_seqlens && (s = error_word(&err)) != GDN_OK) return s;
  const conv::BwdArgs g{dy, dstate_out, static_cast<float *>(workspace), dx, dweight, dbias,
                        dstate_in};
  const bool v4 = conv::vec(a, e, 4, {x, dy, dx, state_in, dstate_out, dstate_in});
  if (dt == GDN_DTYPE_F32)
    return v4 ? GDN_CONV_W(conv::bwd_run, float, 4, a, g, err, st)
              : GDN_CONV_W(conv::bwd_run, float, 1, a, g, err, st);
  return v4 ? GDN_CONV_W(conv::bwd_run, __nv_bfloat16, 4, a, g, err, st)
            : GDN_CONV_W(conv::bwd_run, __nv_bfloat16, 1, a, g, err, st);
}

}  // extern "C"
