// Selective state space scan of bf16 inputs on the tensor cores, 64 tokens
// (a chunk) at a time.  With c_t the inclusive sum of dt A inside the chunk:
//   M_ij = (C_i . B_j) e^{c_i - c_j} dt_j  (i >= j)
//   y = M x + e^{c_i} C_i S_0 + D x,   S_n = e^{c_n} S_0 + sum_j B_j (w_j x_j)^T,
//   w_j = e^{c_n - c_j} dt_j.
// A CTA of eight warps carries the state of one (sequence, head, 64 columns
// of P) through a run of chunks.  The state stays in registers as the
// accumulators of S^T (warp w: columns 16 (w mod 4) .. + 15 of P as rows, half
// w / 4 of N as columns), a layout that is at once the B operand of C S_0, so
// the state never passes through shared memory; the two halves' parts of
// C S_0 are exchanged instead.
//
// Precision: x, B, C are exact bf16 operands.  fp32 operands are split into
// bf16 pieces: two for M and S_0 as they enter y (2^-17 relative, far under
// y's own bf16 rounding), three for w x as it enters the state (2^-25).
// Everything is accumulated in fp32, and the state stays an fp32 quantity: what
// a chunk adds is summed by itself, and the decays of chunks and runs carry
// their roundings along.  Over 8192 to 16384 tokens of steps between 1e-5 and
// 1e-2 and A between -0.1 and -16 states were 1.6e-7 to 3e-7 off (2-norm).
//
// Why mma.sync: the products are small (64 x 64 x 128 and less, 3.3 million
// multiply-adds a chunk at N = 128 with the pieces), and at such sizes
// tcgen05 with both operands in shared memory was measured at 70 cycles for
// M = 128, N = 64, K = 16, against 128 at the legacy rate of 1024
// multiply-adds a clock; it would save the tensor pipe half its time but not
// the splits, exponentials and copies, which are four fifths of the
// instructions here, and would bring the state through TMEM and shared memory
// every chunk.  Measured on 64 packed sequences (131 thousand tokens, 16
// heads, P = 64): 0.78 ms, 6.6 thousand cycles a chunk and unit against 3.3
// thousand of tensor pipe and 3.4 thousand of instruction issue; bound by how
// little of the two overlaps with 16 warps an SM (128 registers each).
#pragma once

#include "gdn_scan_simt.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace scan {

__device__ __forceinline__ uint32_t smem_at(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
// d[16 x 8] += a[16 x 16] b[16 x 8]
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes from global memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// (a, b) as bf16 pairs: hi + lo (+ lo2), each the rounding of what is left.
__device__ __forceinline__ void rest_of(float &a, float &b, uint32_t piece) {
  float p, q;
  bf2_get(piece, p, q);
  f2_unpack(f2_fma(f2_pack(p, q), f2_pack(-1.0f, -1.0f), f2_pack(a, b)), a, b);
}
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = bf2_set(a, b);
  rest_of(a, b, hi);
  lo = bf2_set(a, b);
}
__device__ __forceinline__ void split3(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  hi = bf2_set(a, b);
  rest_of(a, b, hi);
  mid = bf2_set(a, b);
  rest_of(a, b, mid);
  lo = bf2_set(a, b);
}
// Tiles of 64 rows of COLS bf16 with 16 bytes behind each row: eight rows of
// one 16-byte column lie in different banks, and an address is a lane's own
// part plus a constant (exchanging column bits with the row's instead costs
// three instructions a load, a tenth of all that the sweeps execute).
template <int COLS>
constexpr uint32_t kRowBytes = COLS * 2 + 16;
template <int COLS>
constexpr uint32_t kTileBytes = 64 * kRowBytes<COLS>;
template <int COLS>
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int r, int ch) {
  return tile + (uint32_t)r * kRowBytes<COLS> + (uint32_t)ch * 16;
}
// The four 8 x 8 blocks of a 16 x 16 block at (r0, column ch0), rows first
// (an A operand as it lies, or with .trans a transposed one's columns) ...
template <int COLS>
__device__ __forceinline__ uint32_t block_rows(uint32_t tile, int r0, int ch0, int lane) {
  return tile_at<COLS>(tile, r0 + (lane & 15), ch0 + (lane >> 4));
}
// ... and columns first (two B operands of 8 columns as they lie).
template <int COLS>
__device__ __forceinline__ uint32_t block_cols(uint32_t tile, int r0, int ch0, int lane) {
  return tile_at<COLS>(tile, r0 + (lane & 7) + ((lane >> 4) << 3), ch0 + ((lane >> 3) & 1));
}

// n rows (of 64; the others zero) of COLS bf16 into a tile, by THREADS threads.
template <int COLS, int THREADS>
__device__ __forceinline__ void fetch_tile(uint32_t tile, const __nv_bfloat16 *src, long long stride,
                                           int n, int tid) {
  constexpr int kCh = COLS / 8;
#pragma unroll
  for (int i = tid; i < 64 * kCh; i += THREADS) {
    const int r = i / kCh, c = i % kCh;
    copy16(tile_at<COLS>(tile, r, c), src + (r < n ? r * stride : 0) + c * 8, r < n);
  }
}

// Decays of one chunk.  The sums are formed in 64 bits in units of log 2 and
// kept as two floats: differences of neighbours stay exact where the sums
// themselves are large.
struct alignas(16) Decays {  // two of them lie side by side and are read in pairs
  float hi[64], lo[64];   // c_t / ln 2
  float dt[64], sig[64];  // step, and the slope of its softplus
  float gam[64];          // e^{c_t}
  float del[64];          // e^{c_n - c_t}
  float w[64];            // del * dt
  float all;              // e^{c_n}: the decay of the state over the chunk
  float log;              // c_n
};
// 2^v with its subnormals (the decays of whole chunks reach them).
__device__ __forceinline__ float exp2_of(double v) {
  const float h = (float)v;
  const float l = (float)(v - (double)h);
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(h));
  return r * fmaf(l, 0.693147181f, 1.0f);
}
// The raw steps of a chunk, two tokens a lane, loaded well before they are used.
struct RawSteps {
  __nv_bfloat16 v[2];
};
__device__ __forceinline__ RawSteps raw_steps(const In<__nv_bfloat16> &in, long long row0, int n, int h) {
  const int t = 2 * (threadIdx.x & 31);
  RawSteps r;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    r.v[k] = t + k < n ? in.raw[(row0 + t + k) * in.rs + h] : __nv_bfloat16(0.0f);
  return r;
}
// By one warp; tokens past n have step 0 and decay 1.  CHAIN: `all` is a step
// of a chain of chunks, whose roundings `carry` takes along.
template <bool CHAIN>
__device__ __forceinline__ void decays_of(const RawSteps &raw, int n, float A, float bias, Decays &m,
                                          float &carry) {
  const int lane = threadIdx.x & 31;
  double a[2];
  float dt[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = 2 * lane + k;
    dt[k] = 0.0f;
    float sg = 0.0f;
    if (t < n) {
      const float v = to_f32(raw.v[k]) + bias;
      dt[k] = softplus(v);
      sg = 1.0f / (1.0f + expf(-v));
    }
    m.dt[t] = dt[k];
    m.sig[t] = sg;
    // a token that forgets everything counts as 2^-1500 = 0: sums stay finite
    const double e = (double)dt[k] * (double)A * 1.4426950408889634;
    a[k] = e < -1500.0 ? -1500.0 : e;
  }
  const double own = a[0] + a[1];
  double inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  const double total = __shfl_sync(0xffffffffu, inc, 31);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = 2 * lane + k;
    const double c = k ? inc : inc - a[1];
    const float hi = (float)c;
    m.hi[t] = hi;
    m.lo[t] = (float)(c - (double)hi);
    m.gam[t] = exp2_of(c);
    const float d = exp2_of(total - c);
    m.del[t] = d;
    m.w[t] = d * dt[k];
  }
  if (lane == 0) {
    if constexpr (CHAIN) {
      m.log = (float)(total * 0.6931471805599453);
      m.all = exp_step(m.log, carry);
    } else {
      m.all = exp2_of(total);
    }
  }
}

// What a sweep leaves behind.
enum Leave : int {
  kY = 0,      // y of every token and the last state
  kEnds = 1,   // the state that the run adds to zero, and its decay
  kChunks = 2  // the state at every chunk's start (backwards: end), in bf16 pieces
};
constexpr int kPieces = 3;  // of such a state: together 2^-25 relative

template <int N, int LEAVE>
struct SweepSmem {
  static constexpr bool Y = LEAVE == kY;
  static constexpr uint32_t C = 0, B = C + (Y ? kTileBytes<N> : 0), X = B + 2 * kTileBytes<N>;
  static constexpr uint32_t M = X + 2 * kTileBytes<64>;
  static constexpr uint32_t E = M + (Y ? 2 * kTileBytes<64> : 0);    // halves of C S_0 on their way
  static constexpr uint32_t O = E + (Y ? 8 * 16 * 32 * 4 : 0);    // a chunk's state on its way out
  static constexpr uint32_t D = O + (LEAVE == kChunks ? kPieces * kTileBytes<N> : 0);
  static constexpr uint32_t bytes = D + 2 * sizeof(Decays);
};
constexpr int kSweepThreads = 256;

// Two barriers a chunk: the tiles of B and x are double, C's is filled again
// as soon as M and C S_0 have been formed.  With four warps that hold all of
// N (168 registers, three CTAs an SM) packed batches ran the same (0.75 ms),
// one long sequence slower (0.11 ms against 0.08).  With sixteen that hold a
// quarter each, a CTA alone on its SM ran no faster either (4 x 4096 tokens x
// 16 heads of 128: 289 us against 279, before what a chunk adds was summed by
// itself; 287 now).  N = 128 spills 8 (prompt) and 68 bytes (boundaries) of the
// 128 registers that two CTAs an SM leave.
//
// REV: the adjoint G backwards over the chunks, G_0 = e^{c_n} G_n + sum_i
// e^{c_i} C_i dy_i^T, with C in B's place, dy in x's and e^{c_i} in w's.
template <int N, int LEAVE, bool REV>
__device__ __forceinline__ void sweep_run(const In<__nv_bfloat16> &in, const __nv_bfloat16 *__restrict__ dy,
                                          const float *first_state, int seg_chunks, Ends ends,
                                          __nv_bfloat16 *__restrict__ y, float *out_state,
                                          uint32_t *__restrict__ chunk_states, unsigned *err) {
  using S = SweepSmem<N, LEAVE>;
  constexpr int kT = N / 16;  // tiles of 8 columns in a warp's half of N
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sC = smem_at(smem) + S::C, sB0 = smem_at(smem) + S::B, sX0 = smem_at(smem) + S::X;
  const uint32_t sM = smem_at(smem) + S::M;
  Decays *dec = reinterpret_cast<Decays *>(smem + S::D);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pw = warp & 3, nh = warp >> 2;  // 16 columns of P, half of N
  const int g = lane >> 2, q = lane & 3;
  const int npt = in.P / 64;
  const int pt = blockIdx.x % npt, h = blockIdx.x / npt % in.H;
  long long slot = blockIdx.x / npt / in.H;
  const int grp = h / (in.H / in.G);
  if (in.cu && blockIdx.x == 0) check_seqlens(in.cu, in.n_seq, in.T_, err);
  // Packed sequences that are not cut into runs (one slot each, and one past
  // the last) go longest first: the short ones fill the tail.
  if (in.cu && seg_chunks * 64LL >= in.T_ && in.n_seq <= kSweepThreads && slot < in.n_seq)
    slot = seq_of_rank(in.cu, in.n_seq, (int)slot);
  const Tile t = find_tile(in.cu, in.n_seq, in.T_, seg_chunks * 64, slot);
  if (t.seq < 0) return;
  const long long row_end = t.start + t.len;
  const int chunks = (int)((t.len + 63) / 64);            // of the sequence
  const int segs = max(1, (chunks + seg_chunks - 1) / seg_chunks);
  const int c0 = t.tile * seg_chunks, c1 = min(chunks, c0 + seg_chunks);
  const bool last_seg = REV ? t.tile == 0 : t.tile == segs - 1;
  if (LEAVE == kEnds && last_seg) return;                  // nobody follows
  const float A = in.A[h], bias = in.bias ? in.bias[h] : 0.0f;

  // the state's (p, n) of this thread: rows 16 pw + g (+ 8) of P, columns
  // nh N / 2 + 8 i + 2 q (+ 1) of N
  float st[kT][4];
  const long long p0 = pt * 64 + pw * 16 + g;
  const int n0 = nh * (N / 2) + 2 * q;
  const long long np = (long long)N * in.P;
  auto at = [&](int i, int e) { return (n0 + 8 * i + (e & 1)) * (long long)in.P + (e >> 1) * 8; };
  {
    const float *src = LEAVE == kEnds ? nullptr
                       : ends.state   ? ends.state + (slot * in.H + h) * np + p0
                       : first_state  ? first_state + ((long long)t.seq * in.H + h) * np + p0
                                      : nullptr;
#pragma unroll
    for (int i = 0; i < kT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st[i][e] = src ? src[at(i, e)] : 0.0f;
  }

  const __nv_bfloat16 *Bp = REV ? in.C + grp * N : in.B + grp * N;
  const long long Bs = REV ? in.cs : in.bs;
  const __nv_bfloat16 *Xp = (REV ? dy : in.x) + (long long)h * in.P + pt * 64;
  const long long Xs = REV ? (long long)in.H * in.P : in.xs;
  auto chunk_at = [&](int k) { return REV ? c1 - 1 - k : c0 + k; };
  auto row_of = [&](int c) { return t.start + (long long)c * 64; };
  auto rows_in = [&](int c) { return (int)min(64LL, row_end - row_of(c)); };
  const int total = c1 - c0;
  float run_log = 0.0f, carry = 0.0f;

  if (total > 0) {
    const int c = chunk_at(0);
    if (LEAVE == kY)
      fetch_tile<N, kSweepThreads>(sC, in.C + grp * N + row_of(c) * in.cs, in.cs, rows_in(c), tid);
    fetch_tile<N, kSweepThreads>(sB0, Bp + row_of(c) * Bs, Bs, rows_in(c), tid);
    fetch_tile<64, kSweepThreads>(sX0, Xp + row_of(c) * Xs, Xs, rows_in(c), tid);
    copy_commit();
    if (warp == 7)
      decays_of<true>(raw_steps(in, row_of(c), rows_in(c), h), rows_in(c), A, bias, dec[0], carry);
  }
  const float Dh = LEAVE == kY && in.D ? in.D[h] : 0.0f;

#pragma unroll 1
  for (int k = 0; k < total; ++k) {
    const int c = chunk_at(k);
    const Decays &m = dec[k & 1];
    const uint32_t sB = sB0 + (k & 1) * kTileBytes<N>, sX = sX0 + (k & 1) * kTileBytes<64>;
    const bool more = k + 1 < total;
    const int cn = more ? chunk_at(k + 1) : c;  // the next chunk
    RawSteps raw;
    if (warp == 7 && more) raw = raw_steps(in, row_of(cn), rows_in(cn), h);
    copy_wait<0>();
    if (LEAVE == kChunks && tid < 64 * kPieces) sm100::bulk_wait_read_all();
    __syncthreads();  // this chunk is there, the last one's B, x and M are free
    if (more) {
      fetch_tile<N, kSweepThreads>(sB0 + ((k + 1) & 1) * kTileBytes<N>, Bp + row_of(cn) * Bs, Bs, rows_in(cn), tid);
      fetch_tile<64, kSweepThreads>(sX0 + ((k + 1) & 1) * kTileBytes<64>, Xp + row_of(cn) * Xs, Xs, rows_in(cn), tid);
      copy_commit();
    }

    if constexpr (LEAVE == kChunks) {  // rows p of N bf16, piece by piece
      // Through shared memory and one bulk copy a row: the accumulators'
      // layout would store 16 bytes of each 32-byte sector (114 us against
      // 89 for both sweeps of 2 x 4096 tokens x 16 heads).
      const uint32_t sO = smem_at(smem) + S::O;
#pragma unroll
      for (int i = 0; i < kT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t u[kPieces];
          split3(st[i][2 * e], st[i][2 * e + 1], u[0], u[1], u[2]);
          const uint32_t a = sO + (pw * 16 + g + 8 * e) * kRowBytes<N> + (n0 + 8 * i) * 2;
#pragma unroll
          for (int k = 0; k < kPieces; ++k)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(a + k * kTileBytes<N>), "r"(u[k]) : "memory");
        }
      sm100::fence_proxy_async();
      __syncthreads();
      if (tid < 64 * kPieces) {
        const long long slot64 = in.cu ? t.seq + t.start / 64 + c : (long long)t.seq * chunks + c;
        const int piece = tid >> 6, p = tid & 63;
        uint32_t *o = chunk_states + ((slot64 * in.H + h) * kPieces + piece) * (np / 2) + (pt * 64 + p) * (long long)(N / 2);
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(o),
                     "r"(sO + piece * kTileBytes<N> + p * kRowBytes<N>), "r"(N * 2)
                     : "memory");
        sm100::bulk_commit();
      }
    }

    float yv[4][2][4];  // rows 16 ((i + 2 nh) mod 4) + g (+ 8): 0 and 1 stay, 2 and 3 go
    if constexpr (LEAVE == kY) {
      // M = S e^{c_i - c_j} dt_j of one or two of the ten 16 x 16 blocks on
      // and below the diagonal, as bf16 pairs in shared memory
#pragma unroll 1
      for (int blk = warp; blk < 10; blk += 8) {
        const int br = blk < 1 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3, bc = blk - br * (br + 1) / 2;
        float s[2][2][4];  // two chains over N
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][j][e] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < N / 16; ++kk) {
          uint32_t a[4], b[4];
          ldsm4(block_rows<N>(sC, 16 * br, 2 * kk, lane), a);
          ldsm4(block_cols<N>(sB, 16 * bc, 2 * kk, lane), b);
          mma16816(s[kk & 1][0], a, b[0], b[1]);
          mma16816(s[kk & 1][1], a, b[2], b[3]);
        }
        const int r0 = 16 * br + g;
        const float h0 = m.hi[r0], l0 = m.lo[r0], h1 = m.hi[r0 + 8], l1 = m.lo[r0 + 8];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int cc = 16 * bc + 8 * j + 2 * q;
          const float2 hj = *reinterpret_cast<const float2 *>(&m.hi[cc]);
          const float2 lj = *reinterpret_cast<const float2 *>(&m.lo[cc]);
          const float2 dj = *reinterpret_cast<const float2 *>(&m.dt[cc]);
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = s[0][j][e] + s[1][j][e];
          v[0] = r0 >= cc ? v[0] * exp2_fast((h0 - hj.x) + (l0 - lj.x)) * dj.x : 0.0f;
          v[1] = r0 > cc ? v[1] * exp2_fast((h0 - hj.y) + (l0 - lj.y)) * dj.y : 0.0f;
          v[2] = r0 + 8 >= cc ? v[2] * exp2_fast((h1 - hj.x) + (l1 - lj.x)) * dj.x : 0.0f;
          v[3] = r0 + 8 > cc ? v[3] * exp2_fast((h1 - hj.y) + (l1 - lj.y)) * dj.y : 0.0f;
          uint32_t hi, lo;
          const uint32_t at0 = tile_at<64>(sM, r0, cc / 8) + q * 4;
          split2(v[0], v[1], hi, lo);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at0), "r"(hi) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at0 + kTileBytes<64>), "r"(lo) : "memory");
          split2(v[2], v[3], hi, lo);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at0 + 8 * kRowBytes<64>), "r"(hi) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at0 + 8 * kRowBytes<64> + kTileBytes<64>), "r"(lo) : "memory");
        }
      }
      if (warp == 7 && more) decays_of<true>(raw, rows_in(cn), A, bias, dec[(k + 1) & 1], carry);
      // C S_0 over this warp's half of N, the state's pieces straight from
      // the accumulators
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) yv[i][j][e] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < N / 32; ++kk) {
        uint32_t hb[2][2], lb[2][2];  // [8 columns of P][k half]
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            split2(st[2 * kk + u][2 * e], st[2 * kk + u][2 * e + 1], hb[e][u], lb[e][u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a[4];
          ldsm4(block_rows<N>(sC, 16 * ((i + 2 * nh) & 3), nh * (N / 16) + 2 * kk, lane), a);
#pragma unroll
          for (int e = 0; e < 2; ++e) mma16816(yv[i][e], a, hb[e][0], hb[e][1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) mma16816(yv[i][e], a, lb[e][0], lb[e][1]);
        }
      }
      float *ex = reinterpret_cast<float *>(smem + S::E);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) ex[(warp * 16 + i * 8 + j * 4 + e) * 32 + lane] = yv[2 + i][j][e];
      __syncthreads();  // M and the halves are there, C is free
      if (more) {
        fetch_tile<N, kSweepThreads>(sC, in.C + grp * N + row_of(cn) * in.cs, in.cs, rows_in(cn), tid);
        copy_commit();
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * (i + 2 * nh) + g;
        const float ga = m.gam[r], gb = m.gam[r + 8];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            yv[i][j][e] = (yv[i][j][e] + ex[((warp ^ 4) * 16 + i * 8 + j * 4 + e) * 32 + lane]) * (e < 2 ? ga : gb);
      }
    }

    if constexpr (LEAVE == kY) {  // y += M x, and its rows leave
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t x[4];  // (p, p + 8) x (j, j + 8) of x^T
        ldsm4t(block_cols<64>(sX, 16 * j, 2 * pw, lane), x);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (j > i + 2 * nh) continue;  // above the diagonal
#pragma unroll
          for (int piece = 0; piece < 2; ++piece) {
            uint32_t a[4];
            ldsm4(block_rows<64>(sM + piece * kTileBytes<64>, 16 * (i + 2 * nh), 2 * j, lane), a);
            mma16816(yv[i][0], a, x[0], x[2]);
            mma16816(yv[i][1], a, x[1], x[3]);
          }
        }
      }
      const int n = rows_in(c);
      __nv_bfloat16 *yo = y + (row_of(c) * in.H + h) * in.P + pt * 64 + pw * 16 + 2 * q;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 16 * (i + 2 * nh) + g + 8 * e;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t xr;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(xr) : "r"(tile_at<64>(sX, r, 2 * pw + j) + q * 4));
            float xa, xb;
            bf2_get(xr, xa, xb);
            if (r < n)
              *reinterpret_cast<uint32_t *>(yo + (long long)r * in.H * in.P + 8 * j) =
                  bf2_set(fmaf(Dh, xa, yv[i][j][2 * e]), fmaf(Dh, xb, yv[i][j][2 * e + 1]));
          }
        }
    }

    // What the chunk adds to the state is summed by itself: the tensor pipe
    // truncates a sum at its own magnitude, and twelve of those a chunk at the
    // state's took 3.4e-5 from states that remember most of 8192 tokens (now
    // 3e-7).  Behind y's stores, whose registers it takes; the barrier of the
    // warp keeps the compiler from drawing its loads up in front of them, which
    // spills (64 packed sequences, 125 thousand tokens, 16 heads of 64: 783 us
    // with it, 825 without, 778 with the sums on top of the state).
    __syncwarp();
    const float all = m.all;
    const uint64_t all2 = f2_pack(all, all);
    float add[kT][4];
#pragma unroll
    for (int i = 0; i < kT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) add[i][e] = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t x[4];
      ldsm4t(block_cols<64>(sX, 16 * j, 2 * pw, lane), x);
      const float *wv = REV ? m.gam : m.w;
      const float2 wa = *reinterpret_cast<const float2 *>(wv + 16 * j + 2 * q);
      const float2 wb = *reinterpret_cast<const float2 *>(wv + 16 * j + 8 + 2 * q);
      uint32_t u0[4], u1[4], u2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float lo, hi;
        bf2_get(x[e], lo, hi);
        const float2 w = e < 2 ? wa : wb;
        split3(lo * w.x, hi * w.y, u0[e], u1[e], u2[e]);
      }
#pragma unroll
      for (int i = 0; i < kT / 2; i += 2) {
        uint32_t b[2][4];  // (j, j + 8) x (n, n + 8)
        ldsm4t(block_rows<N>(sB, 16 * j, nh * (N / 16) + 2 * i, lane), b[0]);
        ldsm4t(block_rows<N>(sB, 16 * j, nh * (N / 16) + 2 * i + 2, lane), b[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mma16816(add[2 * (i + e)], u0, b[e][0], b[e][1]);
          mma16816(add[2 * (i + e) + 1], u0, b[e][2], b[e][3]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mma16816(add[2 * (i + e)], u1, b[e][0], b[e][1]);
          mma16816(add[2 * (i + e) + 1], u1, b[e][2], b[e][3]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mma16816(add[2 * (i + e)], u2, b[e][0], b[e][1]);
          mma16816(add[2 * (i + e) + 1], u2, b[e][2], b[e][3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kT; ++i) {
      f2_unpack(f2_fma(f2_pack(st[i][0], st[i][1]), all2, f2_pack(add[i][0], add[i][1])), st[i][0], st[i][1]);
      f2_unpack(f2_fma(f2_pack(st[i][2], st[i][3]), all2, f2_pack(add[i][2], add[i][3])), st[i][2], st[i][3]);
    }
    if (LEAVE == kEnds) run_log += m.log;
    if (more && LEAVE != kY && warp == 7) decays_of<true>(raw, rows_in(cn), A, bias, dec[(k + 1) & 1], carry);
  }

  if (LEAVE == kChunks && tid < 64 * kPieces) sm100::bulk_wait_all();
  float *dst = nullptr;
  if (LEAVE == kEnds) {
    dst = ends.state + (slot * in.H + h) * np + p0;
    if (tid == 0 && pt == 0) ends.log_decay[slot * in.H + h] = run_log;
  } else if (last_seg && out_state) {
    dst = out_state + ((long long)t.seq * in.H + h) * np + p0;
  }
  if (dst) {
#pragma unroll
    for (int i = 0; i < kT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[at(i, e)] = st[i][e];
  }
}

template <int N>
__global__ void __launch_bounds__(kSweepThreads, 2)
scan_mma_kernel(const In<__nv_bfloat16> in, int seg_chunks, Ends ends, __nv_bfloat16 *__restrict__ y,
                float *state_out, unsigned *err) {
  sweep_run<N, kY, false>(in, nullptr, in.state_in, seg_chunks, ends, y, state_out, nullptr, err);
}
template <int N>
__global__ void __launch_bounds__(kSweepThreads, 2)
ends_mma_kernel(const In<__nv_bfloat16> in, const __nv_bfloat16 *__restrict__ dy, int seg_chunks, Ends fwd,
                Ends rev, unsigned *err) {
  if (blockIdx.y == 0) sweep_run<N, kEnds, false>(in, nullptr, nullptr, seg_chunks, fwd, nullptr, nullptr, nullptr, err);
  else sweep_run<N, kEnds, true>(in, dy, nullptr, seg_chunks, rev, nullptr, nullptr, nullptr, err);
}
// The gradient's two sweeps, side by side.
template <int N>
__global__ void __launch_bounds__(kSweepThreads, 2)
boundaries_mma_kernel(const In<__nv_bfloat16> in, const __nv_bfloat16 *__restrict__ dy,
                      const float *__restrict__ dstate_out, int seg_chunks, Ends fwd, Ends rev,
                      uint32_t *__restrict__ states, uint32_t *__restrict__ adjoints, float *dstate_in,
                      unsigned *err) {
  if (blockIdx.y == 0)
    sweep_run<N, kChunks, false>(in, nullptr, in.state_in, seg_chunks, fwd, nullptr, nullptr, states, err);
  else
    sweep_run<N, kChunks, true>(in, dy, dstate_out, seg_chunks, rev, nullptr, dstate_in, adjoints, err);
}

}  // namespace scan
}  // namespace gdn
