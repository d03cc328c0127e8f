// Gradient of the scan's chunks for bf16 inputs on the tensor cores: the
// algebra of chunk_grad_kernel with mma.sync products of bf16 pieces.  dx takes
// a pair (2^-17 relative) for M.  dB and dC, which add up a group's heads, take
// three pieces of W, and a head's products are formed by themselves and added
// in fp32: with pairs, and the tensor pipe's truncating sums running on over
// 16 heads, the two differed from the rounded 64-bit gradient by 1.0e-4 to
// 1.4e-4 (2-norm) where a 32-bit form differs by 2.5e-5; now by 2.5e-5 to
// 4.6e-5, in no more time (386 us the call).  A third piece of M would take dx
// from 7.7e-5 to 3.9e-5 for 10 us.  What dA and ddt_bias add up over all tokens
// is kept to fp32's own rounding: Z stays fp32 and its factors are summed
// outside the tensor pipe, x_t . du_t is taken from Z's columns instead of du,
// and the states and adjoints come in three pieces (with two, dA was up to
// 8e-6 off; the third costs 45 us of the 229 below).
//
// A CTA of sixteen warps takes one chunk and a range of one group's heads.
// S = C B^T is formed once; dB and dC are summed over the heads in registers,
// so that neither leaves the SM before it is whole (with the heads split over
// several CTAs, their fp32 parts are added afterwards in order).
//
// 2 x 4096 tokens x 16 heads, N = 128, P = 64: 229 us, 27 thousand cycles a
// head and chunk for 6.6 of tensor pipe and 12.5 of shared-memory pipe (25 and
// 48 % busy); the rest is the latency of dependent stages between seven
// barriers.  Eight warps with twice the tile ran the same with states in two
// pieces (181 us against 188).  The 128 registers that sixteen warps leave spill
// 24 to 104 bytes, addresses and a head's scalars.
#pragma once

#include "gdn_scan_mma.cuh"

namespace gdn {
namespace scan {

template <int N, int P>
struct GradSmem {
  static constexpr uint32_t C = 0, B = C + kTileBytes<N>;
  static constexpr uint32_t X = B + kTileBytes<N>;         // P / 64 tiles of 64 x 64
  static constexpr uint32_t Y = X + P / 64 * kTileBytes<64>;
  static constexpr uint32_t H = Y + P / 64 * kTileBytes<64>;  // hi, lo: [64 p][N]
  static constexpr uint32_t G = H + 2 * kTileBytes<N>;
  static constexpr uint32_t M = G + 2 * kTileBytes<N>;     // hi, lo
  static constexpr uint32_t W = M + 2 * kTileBytes<64>;    // hi, mid, lo
  static constexpr uint32_t Z = W + 3 * kTileBytes<64>;    // fp32 [64][65]
  static constexpr uint32_t kZ = 64 * 65 * 4 > kTileBytes<N> ? 64 * 65 * 4 : kTileBytes<N>;
  static constexpr uint32_t V = (Z + kZ + 15) / 16 * 16;
  // the third pieces of H and G take the places of W and Z once those are read
  static constexpr uint32_t H3 = W, G3 = Z;
  static_assert(kTileBytes<N> <= 3 * kTileBytes<64>, "H's third piece fits into W");
  // row sums by warp column: r, q (4 each), Z block sums [4][64], Z's part of
  // l, l, gh and dD by warp
  struct Rows {
    float r[4][64], q[4][64], zb[4][64], lz[64], l[64], gh[16], dD[16];
  };
  static constexpr uint32_t D = V + (sizeof(Rows) + 15) / 16 * 16;
  static constexpr uint32_t bytes = D + 2 * sizeof(Decays);
  static_assert(bytes <= 227 * 1024, "a CTA's shared memory");
};

__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// d += a b with the products of one step in the tensor pipe and the sum in fp32:
// the pipe truncates a sum (towards zero, 2^-24 of it on average), and what Z
// is made of would lose that eight times over.
__device__ __forceinline__ void add_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  float t[4] = {0.f, 0.f, 0.f, 0.f};
  mma16816(t, a, b0, b1);
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] += t[e];
}

// dst: bf16 [tokens, G, N], or with parts fp32 [tokens, G, splits, N].
struct GroupOut {
  __nv_bfloat16 *b, *c;
  float *pb, *pc;
};

constexpr int kGradThreads = 512;

template <int N, int P>
__global__ void __launch_bounds__(kGradThreads, 1)
chunk_grad_mma_kernel(const In<__nv_bfloat16> in, const __nv_bfloat16 *__restrict__ dy,
                      const __nv_bfloat16 *__restrict__ states,
                      const __nv_bfloat16 *__restrict__ adjoints, int splits,
                      __nv_bfloat16 *__restrict__ dx, __nv_bfloat16 *__restrict__ draw, GroupOut out,
                      float *__restrict__ part) {
  using L = GradSmem<N, P>;
  constexpr int kPT = P / 64, kJ = N / 64;  // n16 blocks of a warp's share of N
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t base = smem_at(smem);
  const uint32_t sC = base + L::C, sB = base + L::B, sX = base + L::X, sY = base + L::Y;
  const uint32_t sH = base + L::H, sG = base + L::G, sM = base + L::M, sW = base + L::W;
  float *sZ = reinterpret_cast<float *>(smem + L::Z);
  typename L::Rows &rs = *reinterpret_cast<typename L::Rows *>(smem + L::V);
  Decays *dec = reinterpret_cast<Decays *>(smem + L::D);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int sp = blockIdx.x % splits, grp = blockIdx.x / splits % in.G;
  const long long slot = blockIdx.x / splits / in.G;
  const int R = in.H / in.G, per = (R + splits - 1) / splits;
  const int h0 = grp * R + min(R, sp * per), h1 = grp * R + min(R, (sp + 1) * per);
  const Tile t = find_tile(in.cu, in.n_seq, in.T_, 64, slot);
  const int n = t.seq < 0 ? 0 : (int)min(64LL, t.len - (long long)t.tile * 64);
  if (n <= 0) {
    for (int h = h0 + tid; h < h1; h += kGradThreads)
#pragma unroll
      for (int k = 0; k < 3; ++k) part[(slot * in.H + h) * 4 + k] = 0.0f;
    return;
  }
  const long long row0 = t.start + (long long)t.tile * 64;
  const long long np = (long long)N * in.P;
  float none = 0.0f;

  auto fetch_states = [&](int h, int pt) {
    const __nv_bfloat16 *s = states + (slot * in.H + h) * kPieces * np + (long long)pt * 64 * N;
    const __nv_bfloat16 *a = adjoints + (slot * in.H + h) * kPieces * np + (long long)pt * 64 * N;
    fetch_tile<N, kGradThreads>(sH, s, N, 64, tid);
    fetch_tile<N, kGradThreads>(sH + kTileBytes<N>, s + np, N, 64, tid);
    fetch_tile<N, kGradThreads>(sG, a, N, 64, tid);
    fetch_tile<N, kGradThreads>(sG + kTileBytes<N>, a + np, N, 64, tid);
  };
  auto fetch_third = [&](const __nv_bfloat16 *from, uint32_t to, int h, int pt) {
    fetch_tile<N, kGradThreads>(to, from + ((slot * in.H + h) * kPieces + 2) * np + (long long)pt * 64 * N, N, 64, tid);
  };
  auto fetch_head = [&](int h) {
#pragma unroll
    for (int pt = 0; pt < kPT; ++pt) {
      fetch_tile<64, kGradThreads>(sX + pt * kTileBytes<64>, in.x + row0 * in.xs + (long long)h * P + pt * 64, in.xs, n, tid);
      fetch_tile<64, kGradThreads>(sY + pt * kTileBytes<64>, dy + (row0 * in.H + h) * P + pt * 64, (long long)in.H * P, n, tid);
    }
    fetch_states(h, 0);
  };
  fetch_tile<N, kGradThreads>(sB, in.B + row0 * in.bs + grp * N, in.bs, n, tid);
  fetch_tile<N, kGradThreads>(sC, in.C + row0 * in.cs + grp * N, in.cs, n, tid);
  if (h0 < h1) {
    fetch_head(h0);
    if (warp == 0)
      decays_of<false>(raw_steps(in, row0, n, h0), n, in.A[h0], in.bias ? in.bias[h0] : 0.0f, dec[0], none);
  }
  copy_commit();

  // S for this warp's 16 rows and 16 columns, unless all lie above the diagonal
  const int sr = 16 * (warp >> 2), sc = 16 * (warp & 3);
  const bool lower = sc <= sr;
  const int gr = 16 * (warp >> 2), gc = (N / 4) * (warp & 3);  // rows, columns of dB and dC
  const int ur = gr, uc = 16 * (warp & 3);                     // of du
  float S[2][4], aB[2 * kJ][4], aC[2 * kJ][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[i][e] = 0.0f;
#pragma unroll
  for (int j = 0; j < 2 * kJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) aB[j][e] = aC[j][e] = 0.0f;

#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const Decays &m = dec[(h - h0) & 1];
    copy_wait<0>();
    __syncthreads();
    if (h == h0 && lower) {
#pragma unroll
      for (int kk = 0; kk < N / 16; ++kk) {
        uint32_t a[4], b[4];
        ldsm4(block_rows<N>(sC, sr, 2 * kk, lane), a);
        ldsm4(block_cols<N>(sB, sc, 2 * kk, lane), b);
        add_mma(S[0], a, b[0], b[1]);
        add_mma(S[1], a, b[2], b[3]);
      }
    }
    // K = dy x^T, then M, W and Z
    float dD = 0.0f;
    if (lower) {
      float K[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) K[i][e] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < P / 16; ++kk) {
        const uint32_t tx = sX + (kk / 4) * kTileBytes<64>, ty = sY + (kk / 4) * kTileBytes<64>;
        uint32_t a[4], b[4];
        ldsm4(block_rows<64>(ty, sr, 2 * (kk % 4), lane), a);
        ldsm4(block_cols<64>(tx, sc, 2 * (kk % 4), lane), b);
        add_mma(K[0], a, b[0], b[1]);
        add_mma(K[1], a, b[2], b[3]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = sr + g + 8 * e;
        const float hr = m.hi[r], lr = m.lo[r];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = sc + 8 * j + 2 * q;
          float mv[2], wv[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float k = K[j][2 * e + u], s = S[j][2 * e + u];
            const float d = r >= c + u ? exp2_fast((hr - m.hi[c + u]) + (lr - m.lo[c + u])) : 0.0f;
            if (r == c + u) dD += k;
            mv[u] = s * d;
            wv[u] = k * d * m.dt[c + u];
            sZ[r * 65 + c + u] = mv[u] * k;
          }
          uint32_t hi, mid, lo;
          const uint32_t at = tile_at<64>(0, r, c / 8) + q * 4;
          split2(mv[0], mv[1], hi, lo);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(sM + at), "r"(hi) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(sM + kTileBytes<64> + at), "r"(lo) : "memory");
          split3(wv[0], wv[1], hi, mid, lo);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(sW + at), "r"(hi) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(sW + kTileBytes<64> + at), "r"(mid) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(sW + 2 * kTileBytes<64> + at), "r"(lo) : "memory");
        }
      }
    } else {  // above the diagonal: Z alone is read there
      for (int i = lane; i < 16 * 16; i += 32) sZ[(sr + i / 16) * 65 + sc + i % 16] = 0.0f;
    }
    dD = warp_sum(dD);
    if (lane == 0) rs.dD[warp] = dD;
    float gh = 0.0f;
    __syncthreads();

    // Z summed from each 16-row block's last row up
    if (tid < 256) {
      const int c = tid & 63, b = tid >> 6;
      float s = 0.0f;
#pragma unroll
      for (int i = 15; i >= 0; --i) {
        s += sZ[(16 * b + i) * 65 + c];
        sZ[(16 * b + i) * 65 + c] = s;
      }
      rs.zb[b][c] = s;
    }
    // what needs no state: dC += W B (side 0), dB += W^T C (side 1)
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      float T[2 * kJ][4];
#pragma unroll
      for (int j = 0; j < 2 * kJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) T[j][e] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (side ? kk < gr / 16 : kk > gr / 16) continue;  // above the diagonal
        uint32_t b[kJ][4];
#pragma unroll
        for (int j = 0; j < kJ; ++j) ldsm4t(block_rows<N>(side ? sC : sB, 16 * kk, gc / 8 + 2 * j, lane), b[j]);
#pragma unroll
        for (int piece = 0; piece < 3; ++piece) {
          const uint32_t tW = sW + piece * kTileBytes<64>;
          uint32_t a[4];
          if (side) ldsm4t(block_cols<64>(tW, 16 * kk, gr / 8, lane), a);
          else ldsm4(block_rows<64>(tW, gr, 2 * kk, lane), a);
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            mma16816(T[2 * j], a, b[j][0], b[j][1]);
            mma16816(T[2 * j + 1], a, b[j][2], b[j][3]);
          }
        }
      }
      float(&acc)[2 * kJ][4] = side ? aB : aC;
#pragma unroll
      for (int j = 0; j < 2 * kJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] += T[j][e];
    }
    __syncthreads();  // Z's sums are there, W has been read
    fetch_third(states, base + L::H3, h, 0);
    copy_commit();
    if (tid < 256) {  // Z's part of l_t, four threads a token
      const int tt = tid >> 2, b = tid & 3;
      float s = 0.0f;
      for (int c = 16 * b; c < min(16 * b + 16, tt); ++c) {
        float v = sZ[tt * 65 + c];
        for (int k = tt / 16 + 1; k < 4; ++k) v += rs.zb[k][c];
        s = fmaf(m.dt[c], v, s);
      }
      s = quad_sum(s);
      if (b == 0) rs.lz[tt] = s;
    }
    float rsum[2] = {0.f, 0.f}, qsum[2] = {0.f, 0.f};
    const float Dh = in.D ? in.D[h] : 0.0f;
    // T = dy H0 (side 0) or x G (side 1) from `pieces` tiles at tS, the small
    // ones first, whose sums the pipe truncates at their own magnitude; its
    // scaled rows join dC or dB, their products with C or B the row sums
    auto with_state = [&](int side, uint32_t tA, uint32_t tS, int pieces) {
      const uint32_t tO = side ? sB : sC;
      float T[2 * kJ][4];
#pragma unroll
      for (int j = 0; j < 2 * kJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) T[j][e] = 0.0f;
#pragma unroll
      for (int piece = 1; piece >= 0; --piece) {
        if (piece >= pieces) continue;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t a[4];
          ldsm4(block_rows<64>(tA, gr, 2 * kk, lane), a);
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            uint32_t b[4];
            ldsm4t(block_rows<N>(tS + piece * kTileBytes<N>, 16 * kk, gc / 8 + 2 * j, lane), b);
            mma16816(T[2 * j], a, b[0], b[1]);
            mma16816(T[2 * j + 1], a, b[2], b[3]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = gr + g + 8 * e;
        const float f = side ? m.w[r] : m.gam[r];
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 2 * kJ; ++j) {
          uint32_t o;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(o) : "r"(tile_at<N>(tO, r, gc / 8 + j) + q * 4));
          float oa, ob;
          bf2_get(o, oa, ob);
          const float ta = T[j][2 * e], tb = T[j][2 * e + 1];
          s = fmaf(oa, ta, fmaf(ob, tb, s));
          float(&acc)[4] = side ? aB[j] : aC[j];
          acc[2 * e] = fmaf(f, ta, acc[2 * e]);
          acc[2 * e + 1] = fmaf(f, tb, acc[2 * e + 1]);
        }
        if (side) qsum[e] = fmaf(m.del[r], s, qsum[e]);
        else rsum[e] = fmaf(m.gam[r], s, rsum[e]);
      }
    };
#pragma unroll 1
    for (int pt = 0; pt < kPT; ++pt) {
      const uint32_t tX = sX + pt * kTileBytes<64>, tY = sY + pt * kTileBytes<64>;
      if (pt > 0) {
        __syncthreads();  // the first tile's states have been read
        fetch_states(h, pt);
        fetch_third(states, base + L::H3, h, pt);
        fetch_third(adjoints, base + L::G3, h, pt);
        copy_commit();
        copy_wait<0>();
        __syncthreads();
      }
      with_state(0, tY, sH, 2);
      if (pt == 0) {
        __syncthreads();  // Z has been read
        fetch_third(adjoints, base + L::G3, h, 0);
        copy_commit();
      }
      with_state(1, tX, sG, 2);
      // du = M^T dy + e^{c_n - c_j} B G^T and dx
      {
        float U[2][4], T[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) U[j][e] = T[j][e] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk < ur / 16) continue;  // above the diagonal
          uint32_t b[4];
          ldsm4t(block_rows<64>(tY, 16 * kk, uc / 8, lane), b);
#pragma unroll
          for (int piece = 0; piece < 2; ++piece) {
            uint32_t a[4];
            ldsm4t(block_cols<64>(sM + piece * kTileBytes<64>, 16 * kk, ur / 8, lane), a);
            mma16816(U[0], a, b[0], b[1]);
            mma16816(U[1], a, b[2], b[3]);
          }
        }
#pragma unroll
        for (int kk = 0; kk < N / 16; ++kk) {
          uint32_t a[4];
          ldsm4(block_rows<N>(sB, ur, 2 * kk, lane), a);
#pragma unroll
          for (int piece = 0; piece < 2; ++piece) {
            uint32_t b[4];
            ldsm4(block_cols<N>(sG + piece * kTileBytes<N>, uc, 2 * kk, lane), b);
            mma16816(T[0], a, b[0], b[1]);
            mma16816(T[1], a, b[2], b[3]);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = ur + g + 8 * e;
          const float d = m.del[r], dt = m.dt[r];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t yr;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(yr) : "r"(tile_at<64>(tY, r, uc / 8 + j) + q * 4));
            float ya, yb;
            bf2_get(yr, ya, yb);
            const float ua = fmaf(d, T[j][2 * e], U[j][2 * e]);
            const float ub = fmaf(d, T[j][2 * e + 1], U[j][2 * e + 1]);
            if (r < n)
              *reinterpret_cast<uint32_t *>(dx + ((row0 + r) * in.H + h) * P + pt * 64 + uc + 8 * j + 2 * q) =
                  bf2_set(fmaf(dt, ua, Dh * ya), fmaf(dt, ub, Dh * yb));
          }
        }
      }
      copy_wait<0>();
      __syncthreads();  // the third pieces are there
      with_state(0, tY, base + L::H3, 1);
      with_state(1, tX, base + L::G3, 1);
      // <G, H0>
      for (int i = tid; i < 64 * N / 4; i += kGradThreads) {  // four values of a row
        const uint32_t at = (uint32_t)(i / (N / 4)) * kRowBytes<N> + (uint32_t)(i % (N / 4)) * 8;
        float v[2][4] = {};
#pragma unroll
        for (int k = kPieces - 1; k >= 0; --k)
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const uint32_t from = k < 2 ? (side ? sG : sH) + k * kTileBytes<N> : base + (side ? L::G3 : L::H3);
            uint32_t a, b;
            asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "r"(from + at));
            float p[4];
            bf2_get(a, p[0], p[1]);
            bf2_get(b, p[2], p[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[side][e] += p[e];
          }
#pragma unroll
        for (int e = 0; e < 4; ++e) gh = fmaf(v[0][e], v[1][e], gh);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = gr + g + 8 * e;
      const float a = quad_sum(rsum[e]), b = quad_sum(qsum[e]);
      if (q == 0) {
        rs.r[warp & 3][r] = a;
        rs.q[warp & 3][r] = b;
      }
    }
    gh = warp_sum(gh);
    if (lane == 0) rs.gh[warp] = gh;
    __syncthreads();  // every tile of this head has been read
    if (h + 1 < h1) {
      fetch_head(h + 1);
      copy_commit();
      if (warp == 15)
        decays_of<false>(raw_steps(in, row0, n, h + 1), n, in.A[h + 1], in.bias ? in.bias[h + 1] : 0.0f,
                         dec[(h + 1 - h0) & 1], none);
    }
    // l_t, four threads a token
    if (tid < 256) {
      const int tt = tid >> 2, b = tid & 3;
      float s = 0.0f;
      for (int c = 16 * b; c < min(16 * b + 16, tt); ++c)
        s = fmaf(m.dt[c], (rs.q[0][c] + rs.q[1][c]) + (rs.q[2][c] + rs.q[3][c]), s);
      for (int c = max(16 * b, tt); c < 16 * b + 16; ++c)
        s += (rs.r[0][c] + rs.r[1][c]) + (rs.r[2][c] + rs.r[3][c]);
      s = quad_sum(s);
      if (b == 0) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < 16; ++w) v += rs.gh[w];
        rs.l[tt] = fmaf(m.all, v, s + rs.lz[tt]);
      }
    }
    __syncthreads();
    if (warp == 0) {
      const float A = in.A[h];
      float dA = 0.0f, db = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = lane + 32 * k;
        if (r < n) {
          // x . du: Z's column, and q
          const float x = ((rs.zb[0][r] + rs.zb[1][r]) + (rs.zb[2][r] + rs.zb[3][r])) +
                          ((rs.q[0][r] + rs.q[1][r]) + (rs.q[2][r] + rs.q[3][r]));
          const float d = fmaf(A, rs.l[r], x) * m.sig[r];
          draw[(row0 + r) * in.H + h] = __float2bfloat16_rn(d);
          dA = fmaf(m.dt[r], rs.l[r], dA);
          db += d;
        }
      }
      dA = warp_sum(dA);
      db = warp_sum(db);
      if (lane == 0) {
        float *po = part + (slot * in.H + h) * 4;
        float d = 0.0f;
#pragma unroll
        for (int w = 0; w < 16; ++w) d += rs.dD[w];
        po[0] = dA;
        po[1] = d;
        po[2] = db;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = gr + g + 8 * e;
    if (r >= n) continue;
    const long long row = (row0 + r) * in.G + grp;
#pragma unroll
    for (int j = 0; j < 2 * kJ; ++j) {
      const int c = gc + 8 * j + 2 * q;
      if (splits == 1) {
        *reinterpret_cast<uint32_t *>(out.b + row * N + c) = bf2_set(aB[j][2 * e], aB[j][2 * e + 1]);
        *reinterpret_cast<uint32_t *>(out.c + row * N + c) = bf2_set(aC[j][2 * e], aC[j][2 * e + 1]);
      } else {
        const long long at = (row * splits + sp) * N + c;
        *reinterpret_cast<float2 *>(out.pb + at) = make_float2(aB[j][2 * e], aB[j][2 * e + 1]);
        *reinterpret_cast<float2 *>(out.pc + at) = make_float2(aC[j][2 * e], aC[j][2 * e + 1]);
      }
    }
  }
}

}  // namespace scan
}  // namespace gdn
