// Short causal convolution over tokens, a channel at a time, with its state
// (the last W - 1 inputs) carried between calls, its one-token form and its
// gradient:
//   pre_t = bias + sum_{j < W} w_j x_{t - W + 1 + j},   y_t = act(pre_t)
//   dp_t = dy_t act'(pre_t),  dx_u = sum_j w_j dp_{u + W - 1 - j},
//   dw_j = sum_t dp_t x_{t - W + 1 + j},  dbias = sum_t dp_t
// with the state's rows in the places of the tokens before the first one.
//
// All three are bound by HBM (two planes of the sequence forward, three
// backward).  A thread owns four channels (8 bytes of bf16: three CTAs of 256
// threads fit an SM, where 16-byte vectors leave two and ran 70 us against
// 65 on 16384 x 4352) and walks a run of tokens with the last W - 1 inputs
// in registers, so that x is read once but for the W - 1 rows in front of a
// run; a warp's lanes are neighbouring vectors.
#include <type_traits>

#include "gdn_layer.cuh"
#include "gdn_host.cuh"
#include "gdn_layer.h"

namespace gdn {
namespace conv {

using namespace layer;

constexpr int kWarps = 8;     // runs of one CTA, one a warp
constexpr int kWarpsBwd = 2;  // the gradient's: small CTAs, so that a sequence's end idles few warps

// Channels in packed fp32 pairs: V / 2 of them, or one with an idle half.
template <int V>
struct Pairs {
  static constexpr int n = (V + 1) / 2;
  uint64_t p[n];
  __device__ __forceinline__ void from(const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < n; ++i) p[i] = f2_pack(f[2 * i], 2 * i + 1 < V ? f[2 * i + 1 < V ? 2 * i + 1 : 0] : 0.0f);
  }
  __device__ __forceinline__ void to(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float a, b;
      f2_unpack(p[i], a, b);
      f[2 * i] = a;
      if (2 * i + 1 < V) f[2 * i + 1 < V ? 2 * i + 1 : 0] = b;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < n; ++i) p[i] = 0;
  }
};

// 1 / (1 + e^-a), 1 / (1 + e^-b).  bf16 results take the approximate base-2
// exponential and reciprocal (each within 2^-22 or so), fp32 ones the
// accurate forms; past the exponential's range both give the limits 0 and 1.
template <typename T>
__device__ __forceinline__ uint64_t sigmoid2(uint64_t x) {
  float a, b;
  if constexpr (sizeof(T) == 4) {
    f2_unpack(x, a, b);
    return f2_pack(sigmoid<T>(a), sigmoid<T>(b));
  }
  f2_unpack(f2_mul(x, f2_pack(-1.44269504f, -1.44269504f)), a, b);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  f2_unpack(f2_add(f2_pack(a, b), f2_pack(1.0f, 1.0f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return f2_pack(a, b);
}
template <typename T, bool SILU>
__device__ __forceinline__ uint64_t act_fwd(uint64_t p) {
  if constexpr (SILU) return f2_mul(p, sigmoid2<T>(p));
  return p;
}
// s (1 + p (1 - s)) for SiLU
template <typename T, bool SILU>
__device__ __forceinline__ uint64_t act_grad(uint64_t p) {
  const uint64_t one = f2_pack(1.0f, 1.0f);
  if constexpr (SILU) {
    const uint64_t s = sigmoid2<T>(p);
    return f2_mul(s, f2_fma(p, f2_fma(s, f2_pack(-1.0f, -1.0f), one), one));
  }
  return one;
}

// The taps w[j] and the bias of V channels from c0 on (weight rows of W,
// fp32; a row of four taps in one load where the pointer allows it).
template <int V, int W>
__device__ __forceinline__ void load_taps(const float *w, const float *b, long long c0,
                                          Pairs<V> (&taps)[W], Pairs<V> &bias) {
  float t[W][V], f[V];
  bool done = false;
  if constexpr (W == 4) {
    if ((reinterpret_cast<uintptr_t>(w) & 15) == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float4 r = __ldg(reinterpret_cast<const float4 *>(w + (c0 + v) * 4));
        t[0][v] = r.x; t[1][v] = r.y; t[2][v] = r.z; t[3][v] = r.w;
      }
      done = true;
    }
  }
  if (!done) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < W; ++j) t[j][v] = __ldg(w + (c0 + v) * W + j);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) f[v] = b ? __ldg(b + c0 + v) : 0.0f;
#pragma unroll
  for (int j = 0; j < W; ++j) taps[j].from(t[j]);
  bias.from(f);
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
// [RUN w, RUN (w + 1)) of the slot's tile.  Products run on packed fp32
// pairs.  16384 x 4352 bf16: 65 us, 67 % of the copy rate; the special
// function unit (an exponential and a reciprocal an element) is 58 % busy.
// The thread of a sequence's
// first run also writes the new state, after it has read the old one, which
// may be the same memory.
template <typename T, int V, int W, bool SILU, int RUN>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) * V == 8 ? 3 : 1)
conv_fwd_kernel(const T *x, long long xs, const float *__restrict__ weight,
                const float *__restrict__ bias, const T *state_in,
                const int *__restrict__ cu, int n_seq, int T_, int C, T *y,
                T *state_out, unsigned *err) {
  constexpr int U = 8;  // rows a group; the next group's loads are in flight meanwhile
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (cu && blockIdx.x == 0 && blockIdx.y == 0) check_seqlens(cu, n_seq, T_, err);
  const Tile t = find_tile(cu, n_seq, T_, RUN * kWarps, blockIdx.x);
  if (t.seq < 0) return;
  const long long c0 = ((long long)blockIdx.y * 32 + lane) * V;
  if (c0 >= C) return;
  const long long p0 = (long long)t.tile * (RUN * kWarps) + warp * RUN;
  if (p0 >= t.len && !(p0 == 0)) return;

  Pairs<V> hist[W - 1 + U];  // the last W - 1 inputs, then the group's
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    float f[V];
    row_or_state<T, V, W>(x, xs, t.start, p0 - (W - 1) + k, state_in, t.seq, C, c0).get(f);
    hist[k].from(f);
  }
  if (p0 == 0) {  // the new state: the last W - 1 rows of [old state; x]
    Vec<T, V> last[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      last[k] = row_or_state<T, V, W>(x, xs, t.start, t.len - (W - 1) + k, state_in, t.seq, C, c0);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      last[k].store(state_out + ((long long)t.seq * (W - 1) + k) * C + c0);
  }

  Pairs<V> taps[W], bias2;
  load_taps<V, W>(weight, bias, c0, taps, bias2);
  const int n = (int)max(0LL, min((long long)RUN, t.len - p0));
  const T *xp = x + (t.start + p0) * xs + c0;
  T *yp = y + (t.start + p0) * C + c0;
  Vec<T, V> next[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < n) next[u].load(xp + u * xs);
#pragma unroll 1
  for (int base = 0; base < n; base += U) {
    Vec<T, V> in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) in[u] = next[u];
    xp += U * xs;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (base + U + u < n) next[u].load(xp + u * xs);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[V];
      in[u].get(f);
      hist[W - 1 + u].from(f);
      Pairs<V> o;
#pragma unroll
      for (int i = 0; i < Pairs<V>::n; ++i) {
        uint64_t p = bias2.p[i];
#pragma unroll
        for (int j = 0; j < W; ++j) p = f2_fma(taps[j].p[i], hist[u + j].p[i], p);
        o.p[i] = act_fwd<T, SILU>(p);
      }
      o.to(f);
      Vec<T, V> out;
      out.set(f);
      if (base + u < n) out.store(yp + (long long)u * C);
    }
    yp += (long long)U * C;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) hist[k] = hist[U + k];
  }
}

// One token a sequence; the state moves up by one row in place.  A thread
// takes S sequences, so that the taps, 4 W bytes a channel against the
// 4 W bytes of bf16 state, input and output, are read once for all of them.
template <typename T, int V, int W, bool SILU, int S>
__global__ void __launch_bounds__(128)
conv_decode_kernel(const T *x, long long xs, const float *__restrict__ weight,
                   const float *__restrict__ bias, T *state, int n_seq, int C, T *y) {
  const long long s0 = (long long)blockIdx.x * S;
  const long long c0 = ((long long)blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (c0 >= C) return;
  Vec<T, V> rows[S][W];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if (s0 + i >= n_seq) break;
    const T *st = state + (s0 + i) * (W - 1) * C + c0;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) rows[i][k].load(st + (long long)k * C);
    rows[i][W - 1].load(x + (s0 + i) * xs + c0);
  }
  Pairs<V> taps[W], b;
  load_taps<V, W>(weight, bias, c0, taps, b);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if (s0 + i >= n_seq) break;
    Pairs<V> p = b;
    float f[V];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      Pairs<V> r;
      rows[i][k].get(f);
      r.from(f);
#pragma unroll
      for (int j = 0; j < Pairs<V>::n; ++j) p.p[j] = f2_fma(taps[k].p[j], r.p[j], p.p[j]);
    }
#pragma unroll
    for (int j = 0; j < Pairs<V>::n; ++j) p.p[j] = act_fwd<T, SILU>(p.p[j]);
    p.to(f);
    Vec<T, V> out;
    out.set(f);
    out.store(y + (s0 + i) * C + c0);
    T *st = state + (s0 + i) * (W - 1) * C + c0;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) rows[i][k + 1].store(st + (long long)k * C);
  }
}

// Gradient.  A warp walks its run of tokens [p0, p1) and W - 1 tokens more:
// at step t it forms pre_t and dp_t, and with dp_{t-W+1} .. dp_t at hand
// writes dx_{t-W+1}.  The first run of a sequence starts W - 1 rows early
// and writes the gradient of the state's rows.  The weights' gradients are
// summed in registers over the run, over the CTA's warps in shared memory,
// and go to partial[slot] ([W + 1][C], the bias last); conv_reduce_kernel
// adds the slots in order, so that results do not depend on timing.  Groups
// of rows away from the run's ends skip every test.  16 packed sequences,
// 13.6 thousand tokens x 2304 bf16: 66 us, 43 % of the copy rate, bound by
// the latency of 16 warps an SM (128 registers each: the window, dp, taps
// and five sums); runs of 64 in CTAs of two warps against 73 us with runs
// of 45 in CTAs of eight.
template <typename T, int V, int W, bool SILU, int RUN>
__global__ void __launch_bounds__(32 * kWarpsBwd, sizeof(T) * V == 8 ? 8 : 4)
conv_bwd_kernel(const T *x, long long xs, const float *__restrict__ weight,
                const float *__restrict__ bias, const T *__restrict__ state_in,
                const int *__restrict__ cu, int n_seq, int T_, int C,
                const T *__restrict__ dy, const T *__restrict__ dstate_out,
                float *__restrict__ partial, T *__restrict__ dx, T *__restrict__ dstate_in,
                unsigned *err) {
  __shared__ float sums[kWarpsBwd][W + 1][32 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (cu && blockIdx.x == 0 && blockIdx.y == 0) check_seqlens(cu, n_seq, T_, err);
  const Tile t = find_tile(cu, n_seq, T_, RUN * kWarpsBwd, blockIdx.x);
  const long long c0 = ((long long)blockIdx.y * 32 + lane) * V;
  const long long p0 = (long long)t.tile * (RUN * kWarpsBwd) + warp * RUN;
  Pairs<V> dw[W], db;
  db.zero();
#pragma unroll
  for (int j = 0; j < W; ++j) dw[j].zero();
  if (t.seq >= 0 && c0 < C && (p0 < t.len || p0 == 0)) {
    constexpr int U = 4;
    const int n = (int)max(0LL, min((long long)RUN, t.len - p0));     // own rows
    const int all = (int)min((long long)n + W - 1, t.len - p0);       // and those behind them
    Pairs<V> taps[W], bias2, xh[W - 1 + U], dh[W - 1 + U];
    load_taps<V, W>(weight, bias, c0, taps, bias2);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      float f[V];
      row_or_state<T, V, W>(x, xs, t.start, p0 - (W - 1) + k, state_in, t.seq, C, c0).get(f);
      xh[k].from(f);
      dh[k].zero();
    }
    const int first = p0 == 0 ? -(W - 1) : 0;                         // first row written
    const int kept = (int)max(-(long long)W, min(t.len - (W - 1) - p0, 0x7fffffffLL));  // in the new state from here
    const T *xp = x + (t.start + p0) * xs + c0, *gp = dy + (t.start + p0) * C + c0;
    Vec<T, V> xn[U], gn[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      xn[u].zero();
      gn[u].zero();
      if (u < all) {
        xn[u].load(xp + u * xs);
        gn[u].load(gp + (long long)u * C);
      }
    }
    // One group of U rows.  INSIDE: every row is one of the run's own, writes
    // a row of dx, and neither it nor what it writes is in a state.
    auto group = [&](int base, auto inside) {
      constexpr bool INSIDE = decltype(inside)::value;
      Vec<T, V> xin[U], gin[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xin[u] = xn[u];
        gin[u] = gn[u];
      }
      xp += U * xs;
      gp += (long long)U * C;
      if (base + 2 * U <= all) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          xn[u].load(xp + u * xs);
          gn[u].load(gp + (long long)u * C);
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          xn[u].zero();
          gn[u].zero();
          if (base + U + u < all) {
            xn[u].load(xp + u * xs);
            gn[u].load(gp + (long long)u * C);
          }
        }
      }
      T *op = dx + (t.start + p0 + base - (W - 1)) * C + c0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int pos = base + u;
        float f[V];
        Pairs<V> g, o;
        xin[u].get(f);
        xh[W - 1 + u].from(f);
        gin[u].get(f);
        g.from(f);
#pragma unroll
        for (int i = 0; i < Pairs<V>::n; ++i) {
          uint64_t p = bias2.p[i];
#pragma unroll
          for (int j = 0; j < W; ++j) p = f2_fma(taps[j].p[i], xh[u + j].p[i], p);
          uint64_t d = f2_mul(g.p[i], act_grad<T, SILU>(p));
          // rows past the sequence's end: g is zero, but the slope there is
          // of inputs that may not be finite
          if (!INSIDE && pos >= all) d = 0;
          dh[W - 1 + u].p[i] = d;
          if (INSIDE || pos < n) {
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j].p[i] = f2_fma(d, xh[u + j].p[i], dw[j].p[i]);
            db.p[i] = f2_add(db.p[i], d);
          }
          // row pos - (W - 1) has all its terms: w_j meets dp_{pos - j}
          uint64_t s = f2_mul(taps[0].p[i], d);
#pragma unroll
          for (int j = 1; j < W; ++j) s = f2_fma(taps[j].p[i], dh[W - 1 + u - j].p[i], s);
          o.p[i] = s;
        }
        const int u0 = pos - (W - 1);
        if (INSIDE || (u0 >= first && u0 < n)) {
          o.to(f);
          if (!INSIDE && dstate_out && u0 >= kept) {  // this row is in the new state
            Vec<T, V> e;
            e.load(dstate_out + ((long long)t.seq * (W - 1) + (p0 + u0 - (t.len - (W - 1)))) * C + c0);
            float f2[V];
            e.get(f2);
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] += f2[v];
          }
          Vec<T, V> out;
          out.set(f);
          if (INSIDE || u0 >= 0) out.store(op + (long long)u * C);
          else out.store(dstate_in + ((long long)t.seq * (W - 1) + (W - 1 + u0)) * C + c0);
        }
      }
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        xh[k] = xh[U + k];
        dh[k] = dh[U + k];
      }
    };
    const int calm = dstate_out ? min(n, kept + W - 1) : n;  // groups that end here are inside
#pragma unroll 1
    for (int base = 0; base < n + W - 1; base += U) {
      if (base >= W - 1 && base + U <= calm) group(base, std::true_type{});
      else group(base, std::false_type{});
    }
  }
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    float f[V];
    (j < W ? dw[j < W ? j : 0] : db).to(f);
#pragma unroll
    for (int v = 0; v < V; ++v) sums[warp][j][lane * V + v] = f[v];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (W + 1) * 32 * V; i += blockDim.x) {
    const int j = i / (32 * V), c = i % (32 * V);
    const long long ch = (long long)blockIdx.y * 32 * V + c;
    if (ch >= C) continue;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarpsBwd; ++w) s += sums[w][j][c];
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
constexpr int kRun = 32, kRunShort = 8, kRunBwd = 64;

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

template <typename T, int V, int W, bool SILU, int RUN>
gdn_status fwd_launch(const Args &a, void *y, void *so, unsigned *err, cudaStream_t st) {
  const long long slots = slot_count(a.n_seq, a.T, RUN * kWarps, a.cu != nullptr);
  const long long cb = (a.C + 32LL * V - 1) / (32 * V);
  if (slots > 0x7fffffffLL || cb > 65535) return GDN_ERR_UNSUPPORTED;
  conv_fwd_kernel<T, V, W, SILU, RUN><<<dim3((unsigned)slots, (unsigned)cb), 32 * kWarps, 0, st>>>(
      static_cast<const T *>(a.x), a.xs, a.w, a.b, static_cast<const T *>(a.state_in), a.cu,
      a.n_seq, a.T, a.C, static_cast<T *>(y), static_cast<T *>(so), err);
  return launched();
}

template <typename T, int V, int W, bool SILU>
gdn_status fwd_run(const Args &a, void *y, void *so, unsigned *err, cudaStream_t st) {
  // Runs of 32 tokens re-read 3 rows in 32, runs of 8 spread a call over four
  // times as many CTAs.  bf16, us with runs of 8 / 32 by CTAs of the latter:
  // 5.1 / 7.2 at 64, 7.7 / 7.2 at 144, 9.2 / 9.8 at 204, 9.6 / 9.8 at 216,
  // 12.2 / 9.8 at 272, 20.5 / 15.9 at 544, 49 / 34 at 1088.  fp32 calls
  // were faster with runs of 8 at every size (6.7 / 13.3 at 64, 19 / 25 at 272,
  // 75 / 108 at 1088) and always take them.
  if constexpr (sizeof(T) == 2) {
    const long long cb = (a.C + 32LL * V - 1) / (32 * V);
    if (slot_count(a.n_seq, a.T, kRun * kWarps, a.cu != nullptr) * cb >= 148 * 3 / 2)
      return fwd_launch<T, V, W, SILU, kRun>(a, y, so, err, st);
  }
  return fwd_launch<T, V, W, SILU, kRunShort>(a, y, so, err, st);
}

template <typename T, int V, int W, bool SILU>
gdn_status decode_run(const Args &a, void *state, void *y, cudaStream_t st) {
  const long long nv = (a.C + V - 1) / V;
  const int threads = nv >= 128 ? 128 : (int)((nv + 31) / 32 * 32);
  const long long cb = (nv + threads - 1) / threads;
  if (cb > 65535) return GDN_ERR_UNSUPPORTED;
  // Four sequences a thread once one would make this many CTAs.  us of a call
  // in a row of them, one / four, by the CTAs of one: bf16 2.26 / 2.77 at 192,
  // 2.87 / 2.87 at 288, 3.18 / 2.77 at 320, 3.81 / 2.87 at 480, 6.87 / 4.71 at 1280;
  // fp32 2.36 / 3.08 at 288, 2.98 / 3.28 at 640, 3.57 / 3.69 at 960, 4.00 / 3.70 at
  // 1152, 6.26 / 5.13 at 2304.
  if (a.n_seq * cb >= (sizeof(T) == 2 ? 2 : 7) * 148)
    conv_decode_kernel<T, V, W, SILU, 4><<<dim3((unsigned)((a.n_seq + 3LL) / 4), (unsigned)cb), threads, 0, st>>>(
        static_cast<const T *>(a.x), a.xs, a.w, a.b, static_cast<T *>(state), a.n_seq, a.C,
        static_cast<T *>(y));
  else
    conv_decode_kernel<T, V, W, SILU, 1><<<dim3((unsigned)a.n_seq, (unsigned)cb), threads, 0, st>>>(
        static_cast<const T *>(a.x), a.xs, a.w, a.b, static_cast<T *>(state), a.n_seq, a.C,
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

template <typename T, int V, int W, bool SILU>
gdn_status bwd_run(const Args &a, const BwdArgs &g, unsigned *err, cudaStream_t st) {
  const long long slots = slot_count(a.n_seq, a.T, kRunBwd * kWarpsBwd, a.cu != nullptr);
  const long long cb = (a.C + 32LL * V - 1) / (32 * V);
  if (slots > 0x7fffffffLL || cb > 65535) return GDN_ERR_UNSUPPORTED;
  conv_bwd_kernel<T, V, W, SILU, kRunBwd><<<dim3((unsigned)slots, (unsigned)cb), 32 * kWarpsBwd, 0, st>>>(
      static_cast<const T *>(a.x), a.xs, a.w, a.b, static_cast<const T *>(a.state_in), a.cu,
      a.n_seq, a.T, a.C, static_cast<const T *>(g.dy), static_cast<const T *>(g.dso),
      g.partial, static_cast<T *>(g.dx), static_cast<T *>(g.dsi), err);
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  conv_reduce_kernel<<<dim3((unsigned)((a.C + 31) / 32), (unsigned)(W + 1)), 32 * kWarps, 0, st>>>(
      g.partial, slots, a.C, W, g.dw, g.db);
  return launched();
}

#define GDN_CONV_A(FN, T, V, W, ...) \
  (a.silu ? FN<T, V, W, true>(__VA_ARGS__) : FN<T, V, W, false>(__VA_ARGS__))
#define GDN_CONV_W(FN, T, V, ...)                      \
  (a.W == 4   ? GDN_CONV_A(FN, T, V, 4, __VA_ARGS__)   \
   : a.W == 3 ? GDN_CONV_A(FN, T, V, 3, __VA_ARGS__)   \
              : GDN_CONV_A(FN, T, V, 2, __VA_ARGS__))

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
  if (conv::vec(a, e, 4, {x, y, state_in, state_out}))
    return GDN_CONV_W(conv::fwd_run, __nv_bfloat16, 4, a, y, state_out, err, st);
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
  return (size_t)layer::slot_count(n_seq, T, conv::kRunBwd * conv::kWarpsBwd, packed != 0) *
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
