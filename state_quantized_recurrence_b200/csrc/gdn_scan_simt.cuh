// Selective state space scan on the CUDA cores, fp32 prompts and gradients and
// single tokens of either type:
//   S_t = a_t S_{t-1} + B_t u_t^T,  y_t = S_t^T C_t + D x_t,
//   a_t = exp(dt_t A), u_t = dt_t x_t, dt_t = softplus(raw_t + bias)
// token by token with the state in registers (forward, and the states and
// their adjoints at chunk boundaries for the gradient), and the gradient of
// one 64-token chunk in matrix form.  What bf16 calls share is here too: their
// arguments, the starts of runs, and the sums over heads and chunks.
#pragma once

#include "gdn_layer.cuh"

namespace gdn {
namespace scan {

using namespace layer;

constexpr int kChunk = 64;

template <typename T>
struct In {
  const T *x, *raw, *B, *C;
  long long xs, rs, bs, cs;  // token strides
  const float *A, *D, *bias;
  const float *state_in;
  const int *cu;
  int n_seq, T_, H, P, G;
};

// softplus without overflow on either side.
__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
}

// e^x as two floats, neither of them negative and the second not zero unless
// the first is (an infinity times both stays one).  Where 0.7 to 1.4 is kept, e^x - 1 is
// its series (the first term left out is 2^-26 of it), and 1 + em, rounded
// towards zero, and what that drops are exact; a state that keeps less forgets
// the rounding with it.
__device__ __forceinline__ void exp_pair(float x, float &hi, float &lo) {
  float p = fmaf(x, 1.0f / 5040, 1.0f / 720);
  p = fmaf(x, p, 1.0f / 120);
  p = fmaf(x, p, 1.0f / 24);
  p = fmaf(x, p, 1.0f / 6);
  p = fmaf(x, p, 0.5f);
  const float em = fmaf(x * x, p, x), one = __fadd_rz(1.0f, em);
  const bool near = fabsf(x) < 0.35f;
  hi = near ? one : expf(x);
  lo = fmaxf(near ? em - (one - 1.0f) : 0.0f, hi * 0x1p-40f);
}
// The decays of a chain of steps, one float each.  Rounded by itself (2^-24
// relative), the same decay step after step takes a state that forgets little
// as far off as the sum of those roundings, 6e-6 in 16384 tokens; here what a
// step's rounding drops, relative to it, is carried into the next one, so
// that the product of any number of them is within one rounding of the exact.
__device__ __forceinline__ float exp_step(float x, float &carry) {
  float one, lo;
  exp_pair(x, one, lo);
  const bool near = fabsf(x) < 0.35f;
  lo = near ? fmaf(one, carry, lo) : 0.0f;
  const float hi = one + lo;
  carry = near ? __fdividef(lo - (hi - one), hi) : 0.0f;
  return hi;
}

struct Ends {           // of the runs, where sequences are cut into several
  float *state;         // [run slot][H][N][P]; NULL: one run a sequence
  float *log_decay;     // [run slot][H]
};

// From what each run adds to zero (kEnds) to the state that each run starts
// from, in place: run k starts from e^{log_decay_{k-1}} start_{k-1} +
// added_{k-1}.
// A thread follows four state elements through the runs of a sequence.
// Bound by latency; it keeps every run from adding up all that went before
// it.
template <bool REV>
__device__ __forceinline__ void start_states(const int *__restrict__ cu, int n_seq, int T, int H, long long np,
                                             const float *__restrict__ first, int seg_chunks, Ends ends) {
  const int parts = (int)(np / 1024);
  const int part = blockIdx.x % parts, h = blockIdx.x / parts % H;
  const long long s = blockIdx.x / parts / H;
  const long long L = seg_chunks * 64LL;
  long long len = T, slot;
  if (cu) {
    if (!seq_ok(cu, n_seq, (int)s, T)) return;
    len = cu[s + 1] - cu[s];
    slot = s + cu[s] / L;
  } else {
    slot = s * (T > 0 ? (T + L - 1) / L : 1);
  }
  const int segs = (int)max(1LL, (len + L - 1) / L);
  const long long at = part * 1024 + threadIdx.x * 4;
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
  if (first) run = *reinterpret_cast<const float4 *>(first + (s * H + h) * np + at);
  float carry = 0.0f;
  constexpr int kAhead = 8;  // runs loaded before the first is needed
  for (int k0 = 0; k0 < segs; k0 += kAhead) {
    float4 add[kAhead];
    float log_d[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + u;
      if (k >= segs - 1) continue;  // the last run adds to nobody
      const long long w = slot + (REV ? segs - 1 - k : k);
      add[u] = *reinterpret_cast<const float4 *>(ends.state + (w * H + h) * np + at);
      log_d[u] = ends.log_decay[w * H + h];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + u;
      if (k >= segs) break;
      const long long w = slot + (REV ? segs - 1 - k : k);
      *reinterpret_cast<float4 *>(ends.state + (w * H + h) * np + at) = run;
      if (k == segs - 1) break;
      const float d = exp_step(log_d[u], carry);
      run.x = fmaf(d, run.x, add[u].x);
      run.y = fmaf(d, run.y, add[u].y);
      run.z = fmaf(d, run.z, add[u].z);
      run.w = fmaf(d, run.w, add[u].w);
    }
  }
}
// blockIdx.y = 1 (where there are two): the adjoints, from the last run on.
__global__ void __launch_bounds__(256)
start_states_kernel(const int *__restrict__ cu, int n_seq, int T, int H, long long np, const float *first,
                    const float *last, int seg_chunks, Ends fwd, Ends rev) {
  if (blockIdx.y == 0) start_states<false>(cu, n_seq, T, H, np, first, seg_chunks, fwd);
  else start_states<true>(cu, n_seq, T, H, np, last, seg_chunks, rev);
}

// Sweep over one run of chunks of one (sequence, head, 64-column tile of P)
// by 256 threads: thread (p, q) holds rows q N/4 .. of column p.
//   kForward   y and the last state
//   kStates    the state at the start of every chunk -> dump[slot]
//   kAdjoint   backwards, with C and dy in the places of B and u:
//              G <- a_t (G + C_t dy_t^T); the adjoint of the state at the end
//              of every chunk -> dump[slot], the last one -> out_state
//   kAdds, kAddsBack   what the run adds to a zero state -> ends
// Bound by the instruction stream: 4 fp32 operations and half a shared-memory
// load for each state element and token.
enum Sweep : int { kForward = 0, kStates = 1, kAdjoint = 2, kAdds = 3, kAddsBack = 4 };
constexpr int kTok = 16;  // tokens staged at a time

template <int N, int MODE>
__device__ __forceinline__ void sweep(const In<float> &in, const float *__restrict__ dy, const float *first,
                                      int seg_chunks, Ends ends, float *__restrict__ y, float *out_state,
                                      float *__restrict__ dump, unsigned *err) {
  constexpr int R = N / 4;
  constexpr bool kBack = MODE == kAdjoint || MODE == kAddsBack, kAdd = MODE == kAdds || MODE == kAddsBack;
  __shared__ __align__(16) float sb[kTok][N], sc[kTok][N], su[kTok][64], sy[4][kTok][64];
  __shared__ float sa[kTok], sal[kTok], sdt[kTok];
  const int tid = threadIdx.x, p = tid & 63, q = tid >> 6;
  const int npt = in.P / 64;
  const int pt = blockIdx.x % npt, h = blockIdx.x / npt % in.H;
  long long slot = blockIdx.x / npt / in.H;
  const int g = h / (in.H / in.G);
  if (in.cu && blockIdx.x == 0) check_seqlens(in.cu, in.n_seq, in.T_, err);
  // packed sequences that are not cut into runs: the longest first
  if (in.cu && seg_chunks * 64LL >= in.T_ && in.n_seq <= 256 && slot < in.n_seq)
    slot = seq_of_rank(in.cu, in.n_seq, (int)slot);
  const Tile tile = find_tile(in.cu, in.n_seq, in.T_, seg_chunks * kChunk, slot);
  if (tile.seq < 0) return;
  const long long t0 = tile.start, len = tile.len, s = tile.seq, L = (long long)seg_chunks * kChunk;
  const long long segs = max(1LL, (len + L - 1) / L);
  const bool last_run = kBack ? tile.tile == 0 : tile.tile == segs - 1;
  if (kAdd && last_run) return;  // nobody follows
  const long long slot0 = in.cu ? s + t0 / kChunk : s * (len > 0 ? (len + kChunk - 1) / kChunk : 1);
  const long long from = tile.tile * L, to = min(len, from + L);
  const float A = in.A[h], D = in.D ? in.D[h] : 0.0f, bias = in.bias ? in.bias[h] : 0.0f;
  const long long np = (long long)N * in.P, mine = pt * 64 + p;
  const long long at = (s * in.H + h) * np + mine, at_run = (slot * in.H + h) * np + mine;
  float st[R];
  const float *src = kAdd ? nullptr : ends.state ? ends.state + at_run : first ? first + at : nullptr;
#pragma unroll
  for (int i = 0; i < R; ++i) st[i] = src ? src[(long long)(q * R + i) * in.P] : 0.0f;
  double decay = 0.0;  // log of the run's

  const long long tiles = (to - from + kTok - 1) / kTok;
  for (long long k = 0; k < tiles; ++k) {
    const long long b0 = from + (kBack ? tiles - 1 - k : k) * kTok;
    const int n = (int)min((long long)kTok, to - b0);
    __syncthreads();
    for (int i = tid; i < n * N; i += 256) {
      const long long row = t0 + b0 + i / N;
      if (!kBack) sb[i / N][i % N] = in.B[row * in.bs + g * N + i % N];
      if (kBack || MODE == kForward) sc[i / N][i % N] = in.C[row * in.cs + g * N + i % N];
    }
    if (tid < n) {
      const float dt = softplus(in.raw[(t0 + b0 + tid) * in.rs + h] + bias);
      sdt[tid] = dt;
      // The decay as two floats: its rounding alone, multiplied up over a few
      // hundred tokens, costs a slowly forgetting state 1e-6 (and without the
      // second one the gradient of 7 packed sequences of up to 300 tokens, 6
      // heads, took 125 us instead of 148).  Neither is negative and the second
      // is not zero unless the first is, so that an infinity in a state stays
      // one.
      const double a = exp((double)dt * (double)A);
      if (kAdd) decay += (double)dt * (double)A;
      sa[tid] = __double2float_rz(a);
      sal[tid] = fmaxf((float)(a - (double)sa[tid]), sa[tid] * 0x1p-40f);
    }
    for (int i = tid; i < n * 64; i += 256) {
      const long long row = t0 + b0 + i / 64;
      const long long c = (long long)h * in.P + pt * 64 + i % 64;
      su[i / 64][i % 64] = kBack ? dy[row * in.H * in.P + c] : in.x[row * in.xs + c];
    }
    __syncthreads();
    if constexpr (kBack) {
      for (int t = n - 1; t >= 0; --t) {
        if (MODE == kAdjoint && ((b0 + t) % kChunk == kChunk - 1 || b0 + t == len - 1)) {
          float *d = dump + ((slot0 + (b0 + t) / kChunk) * in.H + h) * (long long)N * in.P + pt * 64 + p;
#pragma unroll
          for (int i = 0; i < R; ++i) d[(long long)(q * R + i) * in.P] = st[i];
        }
        const float a = sa[t], al = sal[t], u = su[t][p];
#pragma unroll
        for (int i = 0; i < R; i += 4) {
          const float4 c = *reinterpret_cast<const float4 *>(&sc[t][q * R + i]);
          const float v0 = fmaf(c.x, u, st[i]), v1 = fmaf(c.y, u, st[i + 1]);
          const float v2 = fmaf(c.z, u, st[i + 2]), v3 = fmaf(c.w, u, st[i + 3]);
          st[i] = fmaf(a, v0, al * v0);
          st[i + 1] = fmaf(a, v1, al * v1);
          st[i + 2] = fmaf(a, v2, al * v2);
          st[i + 3] = fmaf(a, v3, al * v3);
        }
      }
    } else {
      for (int t = 0; t < n; ++t) {
        if (MODE == kStates && (b0 + t) % kChunk == 0) {
          float *d = dump + ((slot0 + (b0 + t) / kChunk) * in.H + h) * (long long)N * in.P + pt * 64 + p;
#pragma unroll
          for (int i = 0; i < R; ++i) d[(long long)(q * R + i) * in.P] = st[i];
        }
        const float a = sa[t], al = sal[t], u = sdt[t] * su[t][p];
        float acc = 0.0f;
#pragma unroll
        for (int i = 0; i < R; i += 4) {
          const float4 b = *reinterpret_cast<const float4 *>(&sb[t][q * R + i]);
          st[i] = fmaf(a, st[i], fmaf(al, st[i], b.x * u));
          st[i + 1] = fmaf(a, st[i + 1], fmaf(al, st[i + 1], b.y * u));
          st[i + 2] = fmaf(a, st[i + 2], fmaf(al, st[i + 2], b.z * u));
          st[i + 3] = fmaf(a, st[i + 3], fmaf(al, st[i + 3], b.w * u));
          if constexpr (MODE == kForward) {
            const float4 c = *reinterpret_cast<const float4 *>(&sc[t][q * R + i]);
            acc = fmaf(c.x, st[i], acc);
            acc = fmaf(c.y, st[i + 1], acc);
            acc = fmaf(c.z, st[i + 2], acc);
            acc = fmaf(c.w, st[i + 3], acc);
          }
        }
        if (MODE == kForward) sy[q][t][p] = acc;
      }
      if constexpr (MODE == kForward) {
        __syncthreads();
        for (int i = tid; i < n * 64; i += 256) {
          const int t = i / 64, c = i % 64;
          const float o = (sy[0][t][c] + sy[1][t][c]) + (sy[2][t][c] + sy[3][t][c]) + D * su[t][c];
          y[((t0 + b0 + t) * in.H + h) * in.P + pt * 64 + c] = o;
        }
      }
    }
  }
  float *dst = nullptr;
  if constexpr (kAdd) {
    dst = ends.state + at_run;
    if (tid < 32) {  // the lanes of the staged tokens
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) decay += __shfl_xor_sync(0xffffffffu, decay, o);
      if (tid == 0 && pt == 0) ends.log_decay[slot * in.H + h] = (float)decay;
    }
  } else if (MODE != kStates && last_run) {
    dst = out_state + at;
  }
  if (dst) {
#pragma unroll
    for (int i = 0; i < R; ++i) dst[(long long)(q * R + i) * in.P] = st[i];
  }
}

template <int N>
__global__ void __launch_bounds__(256)
forward_kernel(const In<float> in, int seg_chunks, Ends ends, float *__restrict__ y, float *out_state, unsigned *err) {
  sweep<N, kForward>(in, nullptr, in.state_in, seg_chunks, ends, y, out_state, nullptr, err);
}
template <int N>
__global__ void __launch_bounds__(256)
adds_kernel(const In<float> in, const float *__restrict__ dy, int seg_chunks, Ends fwd, Ends rev, unsigned *err) {
  if (blockIdx.y == 0) sweep<N, kAdds>(in, nullptr, nullptr, seg_chunks, fwd, nullptr, nullptr, nullptr, err);
  else sweep<N, kAddsBack>(in, dy, nullptr, seg_chunks, rev, nullptr, nullptr, nullptr, err);
}
// The gradient's two sweeps, side by side: a sweep is a chain of tokens that
// leaves most of an SM idle.
template <int N>
__global__ void __launch_bounds__(256)
boundaries_kernel(const In<float> in, const float *__restrict__ dy, const float *__restrict__ dstate_out,
                  int seg_chunks, Ends fwd, Ends rev, float *__restrict__ states,
                  float *__restrict__ adjoints, float *dstate_in, unsigned *err) {
  if (blockIdx.y == 0)
    sweep<N, kStates>(in, nullptr, in.state_in, seg_chunks, fwd, nullptr, nullptr, states, err);
  else
    sweep<N, kAdjoint>(in, dy, dstate_out, seg_chunks, rev, nullptr, dstate_in, adjoints, err);
}

// One decode token of one (sequence, head, 64-column tile).  Bound by the
// state's HBM traffic, N x 64 fp32 read and written once; B and C are read
// by every head of a group and stay in the caches.  The decay is two floats:
// nothing but the state goes from token to token, so that the rounding of one
// float, token after token, would add up (2.8e-5 in 600 tokens of steps 1e-4 at
// A = -0.1).  The step is loaded in front of the state, so that its arithmetic
// is done when the state arrives, and the CTAs an SM are held to what hides the
// rest: 256 x 32 states of 128 x 128 165 us with four (bf16, whose bytes take 164
// at the copy rate; fp32 181), 210 with three.
template <typename T, int N>
__global__ void __launch_bounds__(256, N == 128 ? 4 : 6)
decode_kernel(const In<T> in, float *state, T *__restrict__ y) {
  __shared__ __align__(16) float4 part[16][16];
  const int tid = threadIdx.x, c4 = tid & 15, r = tid >> 4;  // columns 4 c4 .., rows r, r + 16, ..
  const int npt = in.P / 64;
  const int pt = blockIdx.x % npt, h = blockIdx.x / npt % in.H;
  const long long s = blockIdx.x / npt / in.H;
  const int g = h / (in.H / in.G);
  float *st = state + (s * in.H + h) * (long long)N * in.P + pt * 64 + c4 * 4;
  const T raw = in.raw[s * in.rs + h];
  const float A = in.A[h], bias = in.bias ? in.bias[h] : 0.0f;
  float4 v[N / 16];
#pragma unroll
  for (int i = 0; i < N / 16; ++i)
    v[i] = *reinterpret_cast<const float4 *>(st + (long long)(r + 16 * i) * in.P);
  const float dt = softplus(to_f32(raw) + bias);
  float a, al;
  exp_pair(dt * A, a, al);
  const float4 x = load4(in.x + s * in.xs + (long long)h * in.P + pt * 64 + c4 * 4);
  const T *bp = in.B + s * in.bs + g * N, *cp = in.C + s * in.cs + g * N;
  const uint64_t a2 = f2_pack(a, a), al2 = f2_pack(al, al), x01 = f2_pack(x.x, x.y), x23 = f2_pack(x.z, x.w);
  uint64_t acc01 = 0, acc23 = 0;
#pragma unroll
  for (int i = 0; i < N / 16; ++i) {
    const float b = dt * to_f32(bp[r + 16 * i]), c = to_f32(cp[r + 16 * i]);
    const uint64_t b2 = f2_pack(b, b), c2 = f2_pack(c, c);
    uint64_t v01 = f2_pack(v[i].x, v[i].y), v23 = f2_pack(v[i].z, v[i].w);
    v01 = f2_fma(a2, v01, f2_fma(al2, v01, f2_mul(b2, x01)));
    v23 = f2_fma(a2, v23, f2_fma(al2, v23, f2_mul(b2, x23)));
    acc01 = f2_fma(c2, v01, acc01);
    acc23 = f2_fma(c2, v23, acc23);
    f2_unpack(v01, v[i].x, v[i].y);
    f2_unpack(v23, v[i].z, v[i].w);
    *reinterpret_cast<float4 *>(st + (long long)(r + 16 * i) * in.P) = v[i];
  }
  float4 acc;
  f2_unpack(acc01, acc.x, acc.y);
  f2_unpack(acc23, acc.z, acc.w);
  part[r][c4] = acc;
  __syncthreads();
  if (tid < 64) {
    const float *f = reinterpret_cast<const float *>(part);
    float o = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) o += f[i * 64 + tid];
    const long long c = (long long)h * in.P + pt * 64 + tid;
    const float D = in.D ? in.D[h] : 0.0f;
    y[s * in.H * in.P + c] = T(fmaf(D, to_f32(in.x[s * in.xs + c]), o));
  }
}

// Gradient of one chunk of one head in matrix form, from the state H0 at its
// start and the adjoint Gn of the state at its end.  With c_t the inclusive
// sum of dt A inside the chunk, L_ij = exp(c_i - c_j) for i >= j:
//   S = C B^T, K = dy x^T, M = S L, W_ij = K_ij L_ij dt_j
//   dC_i = sum_j W_ij B_j + e^{c_i} H0 dy_i
//   dB_j = sum_i W_ij C_i + e^{c_n - c_j} dt_j Gn x_j
//   du_j = sum_i M_ij dy_i + e^{c_n - c_j} Gn^T B_j
//   dx = dt du + D dy,  ddt_t = A l_t + x_t . du_t
// where l_t, the gradient of the log decay of token t, adds up what crosses
// token t and nothing else, so that nothing has to cancel:
//   l_t = sum_{i >= t > j} S_ij W_ij + sum_{i >= t} e^{c_i} C_i . H0 dy_i
//         + sum_{j < t} e^{c_n - c_j} dt_j B_j . Gn x_j + e^{c_n} <Gn, H0>
// dB and dC go to per-head fp32 rows, added over a group's heads afterwards.
struct ChunkSmem {
  double c[kChunk];
  float lo[kChunk], hi[kChunk];  // c_t as a sum of two floats
  float dt[kChunk], sig[kChunk], gam[kChunk], del[kChunk];
  float r[kChunk], q[kChunk], xdu[kChunk], l[kChunk];
  float red[8], red2[8];
};

__device__ __forceinline__ float exp_gap(const ChunkSmem &m, int i, int j) {
  return expf((m.hi[i] - m.hi[j]) + (m.lo[i] - m.lo[j]));
}

// dt, its sigmoid and the decay sums of a chunk's n tokens, by one warp (two
// tokens a lane).  The sums are formed in 64 bits and kept as two floats:
// differences of neighbours stay exact where the sums themselves are large.
__device__ __forceinline__ void chunk_decays(const In<float> &in, long long row0, int n, int h,
                                             float A, float bias, ChunkSmem &m) {
  const int lane = threadIdx.x & 31;
  double a[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = 2 * lane + k;
    float dt = 0.0f, sg = 0.0f;
    if (t < n) {
      const float v = in.raw[(row0 + t) * in.rs + h] + bias;
      dt = softplus(v);
      sg = 1.0f / (1.0f + expf(-v));
    }
    m.dt[t] = dt;
    m.sig[t] = sg;
    // a token that forgets everything counts as exp(-1000) = 0: sums stay finite
    const double e = (double)dt * (double)A;
    a[k] = e < -1000.0 ? -1000.0 : e;
  }
  const double own = a[0] + a[1];
  double inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  const double ex = inc - own;
  const double total = __shfl_sync(0xffffffffu, inc, 31);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = 2 * lane + k;
    const double c = ex + (k ? own : a[0]);
    m.c[t] = c;
    m.hi[t] = (float)c;
    m.lo[t] = (float)(c - (double)(float)c);
    m.gam[t] = (float)exp(c);
    m.del[t] = (float)exp(total - c);
  }
}

template <int N, int P>
struct ChunkLayout {
  static constexpr int bn = N + 4, bp = P + 4, bl = kChunk + 1;
  static constexpr int B = 0, C = B + kChunk * bn, X = C + kChunk * bn, DY = X + kChunk * bp;
  static constexpr int M = DY + kChunk * bp, W = M + kChunk * bl, Z = W + kChunk * bl;
  // sixteen columns of a state at a time, rows 17 apart: reading a column of
  // it from global memory row by row took half of the kernel's time
  static constexpr int S = Z + kChunk * bl;
  static constexpr int floats = S + N * 17;
  static constexpr size_t bytes = floats * 4 + sizeof(ChunkSmem) + 16;
};

__device__ __forceinline__ float half_sum(float v) {  // over 16 neighbouring lanes
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Columns k0 .. k0 + 15 of a state [N][P] into rows of 17, by 256 threads.
template <int N, int P>
__device__ __forceinline__ void stage_columns(const float *__restrict__ state, int k0, float *s) {
  __syncthreads();  // the last ones have been read
  for (int i = threadIdx.x; i < N * 4; i += 256) {
    const float4 v = __ldg(reinterpret_cast<const float4 *>(state + (long long)(i / 4) * P + k0 + i % 4 * 4));
    float *d = s + (i / 4) * 17 + i % 4 * 4;
    d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
  }
  __syncthreads();
}

template <int N, int P>
__global__ void __launch_bounds__(256)
chunk_grad_kernel(const In<float> in, const float *__restrict__ dy, const float *__restrict__ states,
                  const float *__restrict__ adjoints, float *__restrict__ dx, float *__restrict__ draw,
                  float *__restrict__ dBh, float *__restrict__ dCh, float *__restrict__ part) {
  using L = ChunkLayout<N, P>;
  extern __shared__ __align__(16) float sm[];
  float *sB = sm + L::B, *sC = sm + L::C, *sX = sm + L::X, *sY = sm + L::DY;
  float *sM = sm + L::M, *sW = sm + L::W, *sZ = sm + L::Z, *sS = sm + L::S;
  ChunkSmem &m = *reinterpret_cast<ChunkSmem *>(
      (reinterpret_cast<uintptr_t>(sm + L::floats) + 7) & ~uintptr_t(7));
  const int tid = threadIdx.x, h = blockIdx.x % in.H, g = h / (in.H / in.G);
  const long long slot = blockIdx.x / in.H;
  const Tile t = find_tile(in.cu, in.n_seq, in.T_, kChunk, slot);
  float *po = part + (slot * in.H + h) * 4;
  const int n = t.seq < 0 ? 0 : (int)min((long long)kChunk, t.len - (long long)t.tile * kChunk);
  if (n <= 0) {
    if (tid < 3) po[tid] = 0.0f;
    return;
  }
  const long long row0 = t.start + (long long)t.tile * kChunk;
  const float A = in.A[h], D = in.D ? in.D[h] : 0.0f, bias = in.bias ? in.bias[h] : 0.0f;
  for (int i = tid; i < kChunk * N; i += 256) {
    const int r = i / N, c = i % N;
    sB[r * L::bn + c] = r < n ? in.B[(row0 + r) * in.bs + g * N + c] : 0.0f;
    sC[r * L::bn + c] = r < n ? in.C[(row0 + r) * in.cs + g * N + c] : 0.0f;
  }
  for (int i = tid; i < kChunk * P; i += 256) {
    const int r = i / P, c = i % P;
    sX[r * L::bp + c] = r < n ? in.x[(row0 + r) * in.xs + (long long)h * P + c] : 0.0f;
    sY[r * L::bp + c] = r < n ? dy[((row0 + r) * in.H + h) * P + c] : 0.0f;
  }
  if (tid < 32) chunk_decays(in, row0, n, h, A, bias, m);
  __syncthreads();

  const int ty = tid >> 4, tx = tid & 15;  // rows ty, ty + 16, ..; columns tx, tx + 16, ..
  {
    float S[4][4] = {}, K[4][4] = {};
    for (int k = 0; k < N; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) { a[i] = sC[(ty + 16 * i) * L::bn + k]; b[i] = sB[(tx + 16 * i) * L::bn + k]; }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][j] = fmaf(a[i], b[j], S[i][j]);
    }
    for (int k = 0; k < P; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) { a[i] = sY[(ty + 16 * i) * L::bp + k]; b[i] = sX[(tx + 16 * i) * L::bp + k]; }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) K[i][j] = fmaf(a[i], b[j], K[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = ty + 16 * i, c = tx + 16 * j;
        const float e = r >= c ? exp_gap(m, r, c) : 0.0f;
        const float w = K[i][j] * e * m.dt[c];
        sM[r * L::bl + c] = S[i][j] * e;
        sW[r * L::bl + c] = w;
        sZ[r * L::bl + c] = S[i][j] * w;
      }
  }
  const float *H0 = states + (slot * in.H + h) * (long long)N * P;
  const float *Gn = adjoints + (slot * in.H + h) * (long long)N * P;
  __syncthreads();

  // columns of Z summed from the last row up to each row
  if (tid < kChunk) {
    float s = 0.0f;
    for (int i = kChunk - 1; i >= 0; --i) {
      s += sZ[i * L::bl + tid];
      sZ[i * L::bl + tid] = s;
    }
  }
  // du, dx, and the row sums of them with x and dy
  float dD = 0.0f;
  {
    constexpr int J = P / 16;
    float a1[4][J] = {}, a2[4][J] = {};
    for (int k = 0; k < kChunk; ++k) {
      float b[J];
#pragma unroll
      for (int j = 0; j < J; ++j) b[j] = sY[k * L::bp + tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = sM[k * L::bl + ty + 16 * i];
#pragma unroll
        for (int j = 0; j < J; ++j) a1[i][j] = fmaf(a, b[j], a1[i][j]);
      }
    }
    for (int k = 0; k < N; ++k) {
      float b[J];
#pragma unroll
      for (int j = 0; j < J; ++j) b[j] = __ldg(Gn + (long long)k * P + tx + 16 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = sB[(ty + 16 * i) * L::bn + k];
#pragma unroll
        for (int j = 0; j < J; ++j) a2[i][j] = fmaf(a, b[j], a2[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
      float xdu = 0.0f, qq = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = tx + 16 * j;
        const float far = m.del[r] * a2[i][j], du = a1[i][j] + far;
        const float xv = sX[r * L::bp + c], dv = sY[r * L::bp + c];
        xdu = fmaf(xv, du, xdu);
        qq = fmaf(xv, far, qq);
        dD = fmaf(xv, dv, dD);
        if (r < n) dx[((row0 + r) * in.H + h) * P + c] = fmaf(m.dt[r], du, D * dv);
      }
      xdu = half_sum(xdu);
      qq = half_sum(qq);
      if (tx == 0) { m.xdu[r] = xdu; m.q[r] = m.dt[r] * qq; }
    }
  }
  // dC and the row sums of its part from H0 with C
  {
    constexpr int J = N / 16;
    float a1[4][J] = {}, a2[4][J] = {};
    for (int k = 0; k < kChunk; ++k) {
      float b[J];
#pragma unroll
      for (int j = 0; j < J; ++j) b[j] = sB[k * L::bn + tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = sW[(ty + 16 * i) * L::bl + k];
#pragma unroll
        for (int j = 0; j < J; ++j) a1[i][j] = fmaf(a, b[j], a1[i][j]);
      }
    }
    for (int k = 0; k < P; ++k) {
      if (k % 16 == 0) stage_columns<N, P>(H0, k, sS);
      float b[J];
#pragma unroll
      for (int j = 0; j < J; ++j) b[j] = sS[(tx + 16 * j) * 17 + k % 16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = sY[(ty + 16 * i) * L::bp + k];
#pragma unroll
        for (int j = 0; j < J; ++j) a2[i][j] = fmaf(a, b[j], a2[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
      float rr = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = tx + 16 * j;
        const float far = m.gam[r] * a2[i][j];
        rr = fmaf(sC[r * L::bn + c], far, rr);
        if (r < n) dCh[((row0 + r) * in.H + h) * N + c] = a1[i][j] + far;
      }
      rr = half_sum(rr);
      if (tx == 0) m.r[r] = rr;
    }
  }
  // dB
  {
    constexpr int J = N / 16;
    float a1[4][J] = {}, a2[4][J] = {};
    for (int k = 0; k < kChunk; ++k) {
      float b[J];
#pragma unroll
      for (int j = 0; j < J; ++j) b[j] = sC[k * L::bn + tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = sW[k * L::bl + ty + 16 * i];
#pragma unroll
        for (int j = 0; j < J; ++j) a1[i][j] = fmaf(a, b[j], a1[i][j]);
      }
    }
    for (int k = 0; k < P; ++k) {
      if (k % 16 == 0) stage_columns<N, P>(Gn, k, sS);
      float b[J];
#pragma unroll
      for (int j = 0; j < J; ++j) b[j] = sS[(tx + 16 * j) * 17 + k % 16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = sX[(ty + 16 * i) * L::bp + k];
#pragma unroll
        for (int j = 0; j < J; ++j) a2[i][j] = fmaf(a, b[j], a2[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (r < n)
          dBh[((row0 + r) * in.H + h) * N + tx + 16 * j] = fmaf(m.del[r] * m.dt[r], a2[i][j], a1[i][j]);
    }
  }
  float gh = 0.0f;
  for (int i = tid; i < N * P; i += 256) gh = fmaf(__ldg(H0 + i), __ldg(Gn + i), gh);
  gh = warp_sum(gh);
  dD = warp_sum(dD);
  if ((tid & 31) == 0) { m.red[tid >> 5] = gh; m.red2[tid >> 5] = dD; }
  __syncthreads();
  if (tid < kChunk) {  // l_t of token tid
    float l = 0.0f;
    for (int w = 0; w < 8; ++w) l += m.red[w];
    l *= m.gam[n - 1];
    float s = 0.0f;
    for (int j = 0; j < tid; ++j) s += sZ[tid * L::bl + j] + m.q[j];
    for (int i = tid; i < n; ++i) s += m.r[i];
    m.l[tid] = l + s;
  }
  __syncthreads();
  if (tid < 32) {
    float dA = 0.0f, db = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = tid + 32 * k;
      if (r < n) {
        const float d = fmaf(A, m.l[r], m.xdu[r]) * m.sig[r];
        draw[(row0 + r) * in.H + h] = d;
        dA = fmaf(m.dt[r], m.l[r], dA);
        db += d;
      }
    }
    dA = warp_sum(dA);
    db = warp_sum(db);
    if (tid == 0) {
      float d = 0.0f;
      for (int w = 0; w < 8; ++w) d += m.red2[w];
      po[0] = dA;
      po[1] = d;
      po[2] = db;
    }
  }
}

// dB, dC of a group: the sum of its heads' rows in head order.
template <typename T>
__global__ void __launch_bounds__(256)
head_sum_kernel(const float *__restrict__ dBh, const float *__restrict__ dCh, long long total,
                int R, int N, T *__restrict__ dB, T *__restrict__ dC) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (long long)gridDim.x * 256) {
    const long long row = i / N;  // (token, group)
    const int n = (int)(i - row * N);
    float b = 0.0f, c = 0.0f;
    for (int r = 0; r < R; ++r) {
      b += dBh[(row * R + r) * N + n];
      c += dCh[(row * R + r) * N + n];
    }
    dB[i] = T(b);
    dC[i] = T(c);
  }
}

// dA, dD, ddt_bias of a head: the chunks' parts added by 128 threads, then in order.
__global__ void __launch_bounds__(128)
head_param_kernel(const float *__restrict__ part, long long slots, int H, float *__restrict__ dA,
                  float *__restrict__ dD, float *__restrict__ dbias) {
  __shared__ float red[3][4];
  const int h = blockIdx.x;
  float v[3] = {0.0f, 0.0f, 0.0f};
  for (long long s = threadIdx.x; s < slots; s += 128)
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] += part[(s * H + h) * 4 + k];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    v[k] = warp_sum(v[k]);
    if ((threadIdx.x & 31) == 0) red[k][threadIdx.x >> 5] = v[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    const int k = threadIdx.x;
    const float s = (red[k][0] + red[k][1]) + (red[k][2] + red[k][3]);
    (k == 0 ? dA : k == 1 ? dD : dbias)[h] = s;
  }
}

}  // namespace scan
}  // namespace gdn
