// Host side of the selective state space scan: argument checks, workspaces
// and launches.
#include "gdn_host.cuh"
#include "gdn_layer.h"
#include "gdn_scan_grad.cuh"
#include "gdn_scan_mma.cuh"
#include "gdn_scan_simt.cuh"

namespace gdn {
namespace scan {

struct Call {
  const void *x, *raw, *B, *C;
  long long xs, rs, bs, cs;
  const float *A, *D, *bias, *state_in;
  const int *cu;
  int n_seq, T, H, P, G, N;
};

gdn_status check(const Call &c, gdn_dtype dt, bool token) {
  if (c.n_seq < 0 || c.T < 0 || c.H <= 0 || c.G <= 0 || c.P <= 0 || c.N <= 0 || c.H % c.G)
    return GDN_ERR_INVALID_ARG;
  if (!known_dtype(dt)) return GDN_ERR_UNSUPPORTED;
  if ((c.P != 64 && c.P != 128) || (c.N != 64 && c.N != 128)) return GDN_ERR_UNSUPPORTED;
  const long long slots = layer::slot_count(c.n_seq, c.T, kChunk, c.cu != nullptr);
  if (c.T > 0x7fffff00) return GDN_ERR_UNSUPPORTED;  // tiles are counted in 32-bit tokens
  if ((double)(token ? c.n_seq : slots) * c.H * (c.P / 64) > 2147483647.0) return GDN_ERR_UNSUPPORTED;
  const long long rows = c.cu ? c.T : (long long)c.n_seq * c.T;
  if (c.n_seq == 0) return GDN_OK;
  if (!c.A || !aligned_to(c.A, 4) || !aligned_to(c.D, 4) || !aligned_to(c.bias, 4) ||
      !aligned_to(c.state_in, 16) || !aligned_to(c.cu, 4))
    return GDN_ERR_INVALID_ARG;
  if (rows == 0) return GDN_OK;
  const size_t e = elem_bytes(dt);
  const long long v = 16 / (long long)e;
  if (!c.x || !c.raw || !c.B || !c.C) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(c.x, 16) || !aligned_to(c.B, 16) || !aligned_to(c.C, 16) || !aligned_to(c.raw, e))
    return GDN_ERR_INVALID_ARG;
  if (rows > 1 && (c.xs < (long long)c.H * c.P || c.bs < (long long)c.G * c.N ||
                   c.cs < (long long)c.G * c.N || c.rs < c.H || c.xs % v || c.bs % v || c.cs % v))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

template <typename T>
In<T> typed(const Call &c) {
  return In<T>{static_cast<const T *>(c.x), static_cast<const T *>(c.raw),
               static_cast<const T *>(c.B), static_cast<const T *>(c.C),
               c.xs, c.rs, c.bs, c.cs, c.A, c.D, c.bias, c.state_in, c.cu,
               c.n_seq, c.T, c.H, c.P, c.G};
}

unsigned units(const Call &c) { return (unsigned)(c.n_seq * c.H * (c.P / 64)); }

// Sequences are cut into runs of chunks where (sequence, head, 64 columns)
// units alone would leave SMs idle: a first launch forms what each run adds
// to a zero state, a second turns that into the state each run starts from.
// That is half of a prompt's work again, and twice a gradient's sweeps; there
// are as many runs as two CTAs on every SM, of four chunks at least (one
// sequence of 8191 tokens, 8 units: 61 us; 80 with half as many).  `enough`
// units go without.  Measured, us cut / not cut, one sequence of N = 128:
//   units                       8         32         56          72         96        112
//   bf16 prompt, 4096      41 / 282   90 / 283  171 / 285   205 / 285  256 / 289  333 / 290
//   fp32 prompt, 2048     201 / 743  278 / 747  507 / 754   641 / 794  834 / 911  1003 / 914
//   bf16 gradient, 4096   118 / 281  375 / 451  635 / 619   759 / 703  1007 / 959  1173 / 1054
//   fp32 gradient, 2048   324 / 823  1064 / 1454  1860 / 1940  2322 / 2190  3043 / 2736  3624 / 3045
// Shorter sequences lie closer together: bf16 prompts of 1024 tokens 59 / 76 at
// 56 units and 78 / 76 at 96, gradients 120 / 127 at 32 and 195 / 176 at 56, fp32
// calls of 512 tokens 5 % slower cut at 32.  The packed rule goes by the mean
// length: one long sequence among many of a chunk or two (a mean of four
// chunks at most), or in a call of enough units, is not cut.
struct Plan {
  int seg_chunks;   // chunks of a run
  bool split;
  long long slots;  // run slots of the call
  size_t state, decay, bytes;  // workspace parts
};
constexpr int kResident = 2 * 148, kEnough = 100, kEnoughGrad = 50;
Plan plan(int n_seq, int T, int H, int P, int N, bool packed, int enough) {
  Plan p = {};
  const long long units = (long long)n_seq * H * (P / 64);
  const long long chunks = (T + 63LL) / 64;
  const long long mean = packed && n_seq > 0 ? (chunks + n_seq - 1) / n_seq : chunks;
  long long seg = chunks > 0 ? chunks : 1;
  if (units > 0 && units < enough && mean > 4) {
    const long long want = (kResident + units - 1) / units;
    long long s = (mean + want - 1) / want;
    if (s < 4) s = 4;
    if (s < seg) {
      seg = s;
      p.split = true;
    }
  }
  p.seg_chunks = (int)seg;
  p.slots = layer::slot_count(n_seq, T, (int)(seg * 64), packed);
  if (p.split) {
    p.decay = (size_t)p.slots * H * N * P * 4;
    p.bytes = p.decay + ((size_t)p.slots * H * 4 + 15) / 16 * 16;
  }
  return p;
}

unsigned run_blocks(const Call &c, const Plan &p) { return (unsigned)(p.slots * c.H * (c.P / 64)); }

// What the runs add, then what they start from; rev.state: backwards too.
template <typename T, int N>
gdn_status run_starts(const Call &c, const Plan &p, const T *dy, const float *dstate_out, Ends fwd, Ends rev,
                      unsigned *err, cudaStream_t st) {
  const In<T> in = typed<T>(c);
  const dim3 grid(run_blocks(c, p), rev.state ? 2 : 1);
  if constexpr (sizeof(T) == 2) {
    constexpr int smem = (int)SweepSmem<N, kEnds>::bytes;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(ends_mma_kernel<N>, smem, done)) return GDN_ERR_CUDA;
    ends_mma_kernel<N><<<grid, kSweepThreads, smem, st>>>(in, dy, p.seg_chunks, fwd, rev, err);
  } else {
    adds_kernel<N><<<grid, 256, 0, st>>>(in, dy, p.seg_chunks, fwd, rev, err);
  }
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  const long long np = (long long)c.N * c.P;
  start_states_kernel<<<dim3((unsigned)(c.n_seq * c.H * (np / 1024)), grid.y), 256, 0, st>>>(
      c.cu, c.n_seq, c.T, c.H, np, c.state_in, dstate_out, p.seg_chunks, fwd, rev);
  return launched();
}
Ends ends_at(char *ws, size_t state, size_t decay) {
  return Ends{reinterpret_cast<float *>(ws + state), reinterpret_cast<float *>(ws + decay)};
}

template <typename T, int N>
gdn_status prefill_typed(const Call &c, char *ws, void *y, float *state_out, unsigned *err, cudaStream_t st) {
  const In<T> in = typed<T>(c);
  const Plan p = plan(c.n_seq, c.T, c.H, c.P, c.N, c.cu != nullptr, kEnough);
  Ends ends{nullptr, nullptr};
  if (p.split) {
    ends = ends_at(ws, p.state, p.decay);
    const gdn_status s = run_starts<T, N>(c, p, nullptr, nullptr, ends, Ends{nullptr, nullptr}, err, st);
    if (s != GDN_OK) return s;
  }
  if constexpr (sizeof(T) == 2) {
    constexpr int smem = (int)SweepSmem<N, kY>::bytes;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(scan_mma_kernel<N>, smem, done)) return GDN_ERR_CUDA;
    scan_mma_kernel<N><<<run_blocks(c, p), kSweepThreads, smem, st>>>(in, p.seg_chunks, ends,
                                                                      static_cast<T *>(y), state_out, err);
  } else {
    forward_kernel<N><<<run_blocks(c, p), 256, 0, st>>>(in, p.seg_chunks, ends, static_cast<T *>(y),
                                                           state_out, err);
  }
  return launched();
}

gdn_status prefill(const Call &c, gdn_dtype dt, char *ws, void *y, float *state_out, unsigned *err,
                   cudaStream_t st) {
  if (dt == GDN_DTYPE_BF16)
    return c.N == 128 ? prefill_typed<__nv_bfloat16, 128>(c, ws, y, state_out, err, st)
                      : prefill_typed<__nv_bfloat16, 64>(c, ws, y, state_out, err, st);
  return c.N == 128 ? prefill_typed<float, 128>(c, ws, y, state_out, err, st)
                    : prefill_typed<float, 64>(c, ws, y, state_out, err, st);
}

template <typename T>
gdn_status decode(const Call &c, float *state, void *y, cudaStream_t st) {
  const In<T> in = typed<T>(c);
  if (c.N == 128) decode_kernel<T, 128><<<units(c), 256, 0, st>>>(in, state, static_cast<T *>(y));
  else decode_kernel<T, 64><<<units(c), 256, 0, st>>>(in, state, static_cast<T *>(y));
  return launched();
}

// The gradient's workspace, every part a multiple of 16 bytes: the state at
// every chunk's start and its adjoint at every chunk's end (fp32, or three
// bf16 pieces), dB and dC of every head (fp32) or of every share of a group's
// heads (bf16, where there are several), the heads' parameters' parts of
// every chunk, and what runs of chunks hand over.
struct Workspace {
  Plan runs;
  long long slots, rows;
  int splits;
  size_t states, adjoints, dB, dC, part, fwd, fwd_decay, rev, rev_decay, bytes;
};

// CTAs that a group's heads are split over: each share forms C B^T again
// (half a head's work), so the split is the one with the least work in a
// row on one of the 148 SMs.  The whole gradient in us, P = 64, N = 128, with the
// split chosen here starred:
//   shares              1     2     3     4     8    16
//   8 chunks, R = 16   252   148   123    96    73   *62
//   16 chunks          254   152   125    98   *74    82
//   64 chunks          314  *214   244   217   233   248
//   128 chunks        *376   387   418   395   398   458
//   256 chunks, R = 32 1202  1222  1226 *1137  1194  1295
int head_splits(long long chunks_groups, int R) {
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= R; ++s) {
    if ((s - 1) * ((R + s - 1) / s) >= R) continue;  // an empty share
    const double waves = (double)((chunks_groups * s + 147) / 148);
    const double cost = waves * ((R + s - 1) / s + 0.5);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

Workspace workspace(int n_seq, int T, int H, int P, int G, int N, gdn_dtype dt, bool packed) {
  Workspace w = {};
  const bool mma = dt == GDN_DTYPE_BF16;
  w.slots = layer::slot_count(n_seq, T, kChunk, packed);
  w.rows = packed ? T : (long long)n_seq * T;
  w.splits = mma ? head_splits(w.slots * G, H / G) : H / G;
  const size_t states = (size_t)w.slots * H * N * P * (mma ? 2 * kPieces : 4);
  const size_t sums = mma && w.splits == 1 ? 0 : (size_t)w.rows * G * w.splits * N * 4;
  w.adjoints = states;
  w.dB = w.adjoints + states;
  w.dC = w.dB + sums;
  w.part = w.dC + sums;
  w.bytes = w.part + (size_t)w.slots * H * 16;
  w.runs = plan(n_seq, T, H, P, N, packed, kEnoughGrad);
  if (w.runs.split) {
    w.fwd = w.bytes;
    w.fwd_decay = w.fwd + w.runs.decay;
    w.rev = w.fwd + w.runs.bytes;
    w.rev_decay = w.rev + w.runs.decay;
    w.bytes = w.rev + w.runs.bytes;
  }
  return w;
}

struct Grads {
  const void *dy;
  const float *dstate_out;
  void *dx, *draw;
  float *dA;
  void *dB, *dC;
  float *dD, *dbias, *dstate_in;
};

template <typename T>
gdn_status sums(const Call &c, const Grads &g, const Workspace &w, char *ws, bool heads, cudaStream_t st) {
  const long long total = w.rows * c.G * c.N;
  if (heads && total > 0) {
    const long long want = (total + 255) / 256;
    head_sum_kernel<T><<<(unsigned)(want < 148 * 16 ? want : 148 * 16), 256, 0, st>>>(
        reinterpret_cast<float *>(ws + w.dB), reinterpret_cast<float *>(ws + w.dC), total, w.splits,
        c.N, static_cast<T *>(g.dB), static_cast<T *>(g.dC));
  }
  head_param_kernel<<<c.H, 128, 0, st>>>(reinterpret_cast<float *>(ws + w.part), w.slots, c.H, g.dA,
                                         g.dD, g.dbias);
  return launched();
}

template <int N, int P>
gdn_status backward_f32(const Call &c, const Grads &g, char *ws, unsigned *err, cudaStream_t st) {
  const In<float> in = typed<float>(c);
  const Workspace w = workspace(c.n_seq, c.T, c.H, c.P, c.G, c.N, GDN_DTYPE_F32, c.cu != nullptr);
  float *states = reinterpret_cast<float *>(ws + w.states);
  float *adjoints = reinterpret_cast<float *>(ws + w.adjoints);
  const float *dy = static_cast<const float *>(g.dy);
  Ends fwd{nullptr, nullptr}, rev{nullptr, nullptr};
  gdn_status s;
  if (w.runs.split) {
    fwd = ends_at(ws, w.fwd, w.fwd_decay);
    rev = ends_at(ws, w.rev, w.rev_decay);
    if ((s = run_starts<float, N>(c, w.runs, dy, g.dstate_out, fwd, rev, err, st)) != GDN_OK) return s;
  }
  boundaries_kernel<N><<<dim3(run_blocks(c, w.runs), 2), 256, 0, st>>>(
      in, dy, g.dstate_out, w.runs.seg_chunks, fwd, rev, states, adjoints, g.dstate_in, err);
  if ((s = launched()) != GDN_OK) return s;
  auto kern = chunk_grad_kernel<N, P>;
  constexpr size_t smem = ChunkLayout<N, P>::bytes;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kern, (int)smem, done)) return GDN_ERR_CUDA;
  kern<<<(unsigned)(w.slots * c.H), 256, smem, st>>>(
      in, dy, states, adjoints, static_cast<float *>(g.dx), static_cast<float *>(g.draw),
      reinterpret_cast<float *>(ws + w.dB), reinterpret_cast<float *>(ws + w.dC),
      reinterpret_cast<float *>(ws + w.part));
  return sums<float>(c, g, w, ws, true, st);
}

template <int N, int P>
gdn_status backward_mma(const Call &c, const Grads &g, char *ws, unsigned *err, cudaStream_t st) {
  using T = __nv_bfloat16;
  const In<T> in = typed<T>(c);
  const Workspace w = workspace(c.n_seq, c.T, c.H, c.P, c.G, c.N, GDN_DTYPE_BF16, c.cu != nullptr);
  const T *dy = static_cast<const T *>(g.dy);
  Ends fwd{nullptr, nullptr}, rev{nullptr, nullptr};
  uint32_t *states = reinterpret_cast<uint32_t *>(ws + w.states);
  uint32_t *adjoints = reinterpret_cast<uint32_t *>(ws + w.adjoints);
  gdn_status s;
  if (w.runs.split) {
    fwd = ends_at(ws, w.fwd, w.fwd_decay);
    rev = ends_at(ws, w.rev, w.rev_decay);
    if ((s = run_starts<T, N>(c, w.runs, dy, g.dstate_out, fwd, rev, err, st)) != GDN_OK) return s;
  }
  constexpr int sweep_smem = (int)SweepSmem<N, kChunks>::bytes;
  static std::atomic<uint64_t> sweeps_done{0}, chunks_done{0};
  if (!allow_smem(boundaries_mma_kernel<N>, sweep_smem, sweeps_done)) return GDN_ERR_CUDA;
  boundaries_mma_kernel<N><<<dim3(run_blocks(c, w.runs), 2), kSweepThreads, sweep_smem, st>>>(
      in, dy, g.dstate_out, w.runs.seg_chunks, fwd, rev, states, adjoints, g.dstate_in, err);
  if ((s = launched()) != GDN_OK) return s;
  auto kern = chunk_grad_mma_kernel<N, P>;
  constexpr int smem = (int)GradSmem<N, P>::bytes;
  if (!allow_smem(kern, smem, chunks_done)) return GDN_ERR_CUDA;
  const GroupOut out{static_cast<T *>(g.dB), static_cast<T *>(g.dC), reinterpret_cast<float *>(ws + w.dB),
                     reinterpret_cast<float *>(ws + w.dC)};
  kern<<<(unsigned)(w.slots * c.G * w.splits), kGradThreads, smem, st>>>(
      in, dy, reinterpret_cast<T *>(states), reinterpret_cast<T *>(adjoints), w.splits,
      static_cast<T *>(g.dx), static_cast<T *>(g.draw), out, reinterpret_cast<float *>(ws + w.part));
  if ((s = launched()) != GDN_OK) return s;
  return sums<T>(c, g, w, ws, w.splits > 1, st);
}

gdn_status backward(const Call &c, gdn_dtype dt, const Grads &g, char *ws, unsigned *err, cudaStream_t st) {
#define GDN_BWD(FN)                                                                      \
  (c.N == 128 ? (c.P == 128 ? FN<128, 128>(c, g, ws, err, st) : FN<128, 64>(c, g, ws, err, st)) \
              : (c.P == 128 ? FN<64, 128>(c, g, ws, err, st) : FN<64, 64>(c, g, ws, err, st)))
  return dt == GDN_DTYPE_BF16 ? GDN_BWD(backward_mma) : GDN_BWD(backward_f32);
#undef GDN_BWD
}

}  // namespace scan
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_scan_prefill_workspace_bytes(int n_seq, int T, int H, int P, int G, int N,
                                        gdn_dtype dtype, int packed) {
  const scan::Call c{nullptr, nullptr, nullptr, nullptr, 0, 0, 0, 0, nullptr, nullptr, nullptr,
                     nullptr, nullptr, 0, T, H, P, G, N};
  if (n_seq <= 0 || scan::check(c, dtype, false) != GDN_OK) return 0;
  return scan::plan(n_seq, T, H, P, N, packed != 0, scan::kEnough).bytes;
}

gdn_status gdn_scan_prefill(const void *x, int64_t x_stride, const void *dt_raw,
                            int64_t dt_stride, const float *A, const void *B, int64_t b_stride,
                            const void *C, int64_t c_stride, const float *D,
                            const float *dt_bias, const float *state_in,
                            const int32_t *cu_seqlens, int n_seq, int T, int H, int P, int G,
                            int N, gdn_dtype dtype, void *workspace, size_t workspace_bytes,
                            void *y, float *state_out, void *cuda_stream) {
  const scan::Call c{x, dt_raw, B, C, x_stride, dt_stride, b_stride, c_stride, A, D, dt_bias,
                     state_in, cu_seqlens, n_seq, T, H, P, G, N};
  gdn_status s = scan::check(c, dtype, false);
  if (s != GDN_OK || n_seq == 0) return s;
  if (!state_out || !aligned_to(state_out, 16) || (T > 0 && (!y || !aligned_to(y, 16))))
    return GDN_ERR_INVALID_ARG;
  const size_t need = gdn_scan_prefill_workspace_bytes(n_seq, T, H, P, G, N, dtype, cu_seqlens != nullptr);
  if (need && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need))
    return GDN_ERR_INVALID_ARG;
  unsigned *err = nullptr;
  if (cu_seqlens && (s = error_word(&err)) != GDN_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return scan::prefill(c, dtype, static_cast<char *>(workspace), y, state_out, err, st);
}

gdn_status gdn_scan_decode(const void *x, int64_t x_stride, const void *dt_raw,
                           int64_t dt_stride, const float *A, const void *B, int64_t b_stride,
                           const void *C, int64_t c_stride, const float *D,
                           const float *dt_bias, float *state_inout, int n_seq, int H, int P,
                           int G, int N, gdn_dtype dtype, void *y, void *cuda_stream) {
  const scan::Call c{x, dt_raw, B, C, x_stride, dt_stride, b_stride, c_stride, A, D, dt_bias,
                     nullptr, nullptr, n_seq, 1, H, P, G, N};
  gdn_status s = scan::check(c, dtype, true);
  if (s != GDN_OK || n_seq == 0) return s;
  if (!state_inout || !aligned_to(state_inout, 16) || !y || !aligned_to(y, 16))
    return GDN_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return dtype == GDN_DTYPE_F32 ? scan::decode<float>(c, state_inout, y, st)
                                : scan::decode<__nv_bfloat16>(c, state_inout, y, st);
}

size_t gdn_scan_backward_workspace_bytes(int n_seq, int T, int H, int P, int G, int N,
                                         gdn_dtype dtype, int packed) {
  const scan::Call c{nullptr, nullptr, nullptr, nullptr, 0, 0, 0, 0, nullptr, nullptr, nullptr,
                     nullptr, nullptr, 0, T, H, P, G, N};
  if (n_seq <= 0 || scan::check(c, dtype, false) != GDN_OK) return 0;
  return scan::workspace(n_seq, T, H, P, G, N, dtype, packed != 0).bytes;
}

gdn_status gdn_scan_backward(const void *x, int64_t x_stride, const void *dt_raw,
                             int64_t dt_stride, const float *A, const void *B, int64_t b_stride,
                             const void *C, int64_t c_stride, const float *D,
                             const float *dt_bias, const float *state_in,
                             const int32_t *cu_seqlens, int n_seq, int T, int H, int P, int G,
                             int N, gdn_dtype dtype, const void *dy, const float *dstate_out,
                             void *workspace, size_t workspace_bytes, void *dx, void *ddt,
                             float *dA, void *dB, void *dC, float *dD, float *ddt_bias,
                             float *dstate_in, void *cuda_stream) {
  const scan::Call c{x, dt_raw, B, C, x_stride, dt_stride, b_stride, c_stride, A, D, dt_bias,
                     state_in, cu_seqlens, n_seq, T, H, P, G, N};
  gdn_status s = scan::check(c, dtype, false);
  if (s != GDN_OK) return s;
  if (!dA || !dD || !ddt_bias || !aligned_to(dA, 4) || !aligned_to(dD, 4) || !aligned_to(ddt_bias, 4))
    return GDN_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (n_seq == 0) {
    for (float *p : {dA, dD, ddt_bias})
      if (cudaMemsetAsync(p, 0, (size_t)H * 4, st) != cudaSuccess) return GDN_ERR_CUDA;
    return GDN_OK;
  }
  const size_t e = elem_bytes(dtype);
  if (!dstate_in || !aligned_to(dstate_in, 16) || !aligned_to(dstate_out, 16))
    return GDN_ERR_INVALID_ARG;
  if (T > 0 && (!dy || !dx || !ddt || !dB || !dC || !aligned_to(dy, 16) || !aligned_to(dx, 16) ||
                !aligned_to(ddt, e) || !aligned_to(dB, 16) || !aligned_to(dC, 16)))
    return GDN_ERR_INVALID_ARG;
  const size_t need = gdn_scan_backward_workspace_bytes(n_seq, T, H, P, G, N, dtype, cu_seqlens != nullptr);
  if (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need) return GDN_ERR_INVALID_ARG;
  unsigned *err = nullptr;
  if (cu_seqlens && (s = error_word(&err)) != GDN_OK) return s;
  const scan::Grads g{dy, dstate_out, dx, ddt, dA, dB, dC, dD, ddt_bias, dstate_in};
  char *ws = static_cast<char *>(workspace);
  return scan::backward(c, dtype, g, ws, err, st);
}

}  // extern "C"
