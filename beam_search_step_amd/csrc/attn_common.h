// attn_common.h -- part of libbeamattn.so, included once by beamattn.hip.
//
// Shared device code of the attention kernels: matrix-instruction types, the
// layout of a 32-key step, online softmax, and the sums across waves.
#pragma once

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;  // of the kernels that take no NW
constexpr int kStep = 32;        // keys of one step of a wave
constexpr int kMaxSplits = 64;   // partial sums joined per query and head

// n / d for 0 <= n < 2^31 and a divisor of the launch: with 2^(s-32) < d <=
// 2^(s-31) and m = ceil(2^s / d), the error n * (m*d - 2^s) / (d * 2^s) is
// below 1/d.
struct FastDiv {
  uint32_t m;
  int s, d;
};
__device__ __forceinline__ int fast_div(FastDiv f, int n) {
  return (int)(((uint64_t)(uint32_t)n * f.m) >> f.s);
}

__device__ __forceinline__ float as_f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t as_u(float x) { return __float_as_uint(x); }
__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 x) { return __builtin_bit_cast(bf16x8, x); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {  // to nearest even
  bf16x2 r;
  r.x = (__bf16)lo;
  r.y = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, r);
}
// the high halves of two fp32 words: bf16 by truncation
__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(as_u(hi), as_u(lo), 0x07060302u);
}
__device__ __forceinline__ float trunc_bf16(float x) { return as_f(as_u(x) & 0xffff0000u); }

// Maximum and sum over the four lanes that share lane % 16.
__device__ __forceinline__ float quad_max(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(as_u(v), as_u(v), false, false);
  v = fmaxf(as_f(a[0]), as_f(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(as_u(v), as_u(v), false, false);
  return fmaxf(as_f(b[0]), as_f(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(as_u(v), as_u(v), false, false);
  v = as_f(a[0]) + as_f(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(as_u(v), as_u(v), false, false);
  return as_f(b[0]) + as_f(b[1]);
}

// What every streaming attention kernel knows of its queries and outputs.
struct QueryArgs {
  const void* q;
  int64_t q_stride;      // elements between query rows
  int heads, kv_heads, group, D;
  FastDiv by_group;
  float c;               // scale * log2(e): softmax in base 2
  void* out;             // [query rows][heads][D]
  float* pacc;           // [query rows * heads][ns][D] partial sums
  float* pml;            // [query rows * heads][ns][2] their maximum (base 2) and sum
  int ns;                // partials per query and head; 1: out is written at once
};

// The layout of one step. A wave takes 32 keys and 16 columns at a time, a
// column being one query of one head of the group. With lane = 16 g + c:
//   S^T = K Q^T   two 16-key tiles t; A: row c is key 16 t + c; B: column c;
//                 the result's row 4 g + r, column c is key 16 t + 4 g + r
//   O^T = V^T P^T the eight keys 16 t + 4 g + r of a lane are its eight
//                 contraction indices (any order serves a sum), so P^T, the
//                 right operand, is what the lane already holds; row c of the
//                 left operand's tile j is value VD c + j, so that a lane reads
//                 VD contiguous values of each of its eight keys
// and no value crosses a lane but a column's maximum and sum. Row 4 g + r of
// O^T's tile j is value VD (4 g + r) + j: a lane ends with 4 VD contiguous
// values of column c.
template <int NM>
struct Softmax {
  float m[NM];   // running maximum of a column, scaled to base 2; -inf: nothing seen
  float l[NM];   // this lane's part of the running sum
  __device__ void init() {
#pragma unroll
    for (int i = 0; i < NM; ++i) m[i] = -kInf, l[i] = 0.0f;
  }
  // scores to probabilities, in place; returns the factor of what was summed before
  __device__ float step(int i, float (&s)[8], float c) {
    float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])),
                      fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
    top = quad_max(top) * c;
    const float mn = fmaxf(m[i], top);
    const float ref = mn == -kInf ? 0.0f : mn;
    const float alpha = __builtin_amdgcn_exp2f(m[i] - ref);
    m[i] = mn;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, -ref));
    l[i] = fmaf(l[i], alpha, ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
    return alpha;
  }
};

// The sums of a workgroup's waves, joined in LDS in wave order, then the
// result or the workgroup's partial. One barrier: the waves write side by side.
// Nothing was seen, or only scores of -inf, where the sum is zero (a maximum of
// -inf does not say so: that of scores that are all NaN is -inf too, and their sum
// NaN). The result is zero then, whatever the values hold; a NaN that a key of no
// weight brought in is kept until it is known that others have some.
template <int DP, int NM, int NW>
struct JoinLds {
  float acc[NW][16 * NM][DP + 4];
  float m[NW][16 * NM], l[NW][16 * NM];
};

template <typename T>
__device__ __forceinline__ void store4(T* p, f32x4 v);
template <>
__device__ __forceinline__ void store4<float>(float* p, f32x4 v) {
  *reinterpret_cast<f32x4*>(p) = v;
}
template <>
__device__ __forceinline__ void store4<uint16_t>(uint16_t* p, f32x4 v) {
  u32x2 w = {pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
  *reinterpret_cast<u32x2*>(p) = w;
}

// Columns [col0, col0 + 16 NM) of `cols`; column / group is a query row behind
// row0, the rest a head behind head0. Every thread of the workgroup calls it.
template <int DP, int NM, int NW, typename TO>
__device__ __forceinline__ void join_and_store(const QueryArgs& a, JoinLds<DP, NM, NW>& lds,
                                               f32x4 (&acc)[NM][DP / 16], Softmax<NM>& sm,
                                               int col0, int cols, int64_t row0, int head0,
                                               int split) {
  constexpr int VD = DP / 16;
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    const float l = quad_sum(sm.l[i]);
    if (g == 0) {
      lds.m[wave][16 * i + c] = sm.m[i];
      lds.l[wave][16 * i + c] = l;
    }
  }
#pragma unroll
  for (int i = 0; i < NM; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float* p = &lds.acc[wave][16 * i + c][VD * (4 * g + r)];
#pragma unroll
      for (int j = 0; j < VD; j += 4)
        *reinterpret_cast<f32x4*>(p + j) =
            f32x4{acc[i][j][r], acc[i][j + 1][r], acc[i][j + 2][r], acc[i][j + 3][r]};
    }
  __syncthreads();
  for (int idx = tid; idx < 16 * NM * (DP / 4); idx += NW * 64) {
    const int x = idx / (DP / 4), d = (idx - x * (DP / 4)) * 4;
    const int col = col0 + x;
    if (col >= cols || d >= a.D) continue;
    float M = lds.m[0][x];
#pragma unroll
    for (int w = 1; w < NW; ++w) M = fmaxf(M, lds.m[w][x]);
    const float ref = M == -kInf ? 0.0f : M;
    float L = 0.0f;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = __builtin_amdgcn_exp2f(lds.m[w][x] - ref);
      L += f * lds.l[w][x];
      v += f * *reinterpret_cast<f32x4*>(&lds.acc[w][x][d]);
    }
    const int qr = fast_div(a.by_group, col);
    const int64_t u = (row0 + qr) * a.heads + head0 + (col - qr * a.group);
    if (a.ns == 1) {
      const float f = __builtin_amdgcn_rcpf(L);
      store4(reinterpret_cast<TO*>(a.out) + u * a.D + d, L == 0.0f ? f32x4{0, 0, 0, 0} : v * f);
    } else {
      if (d == 0) {
        float* p = a.pml + (u * a.ns + split) * 2;
        p[0] = M;
        p[1] = L;
      }
      store4(a.pacc + (u * a.ns + split) * a.D + d, v);
    }
  }
}

// Joins the partials of one query and head: out = sum_s 2^(m_s - M) acc_s /
// sum_s 2^(m_s - M) l_s, and zero where that is. LPU lanes take one query
// and head, four values each, eight partials in flight. A launch's latency bounds it:
// 32 rows of 32 heads of 128 and 7 partials are 3.9 us.
struct CombineArgs {
  const float* pacc;
  const float* pml;
  void* out;
  int64_t units;   // query rows * heads
  int ns, D;
};
template <typename TO, int LPU>
__global__ __launch_bounds__(kAttnThreads) void a_combine(CombineArgs a) {
  const int tid = threadIdx.x, sub = tid / LPU, d = (tid - sub * LPU) * 4;
  const int64_t u = (int64_t)blockIdx.x * (kAttnThreads / LPU) + sub;
  if (u >= a.units || d >= a.D) return;
  const float* ml = a.pml + u * a.ns * 2;
  const float* pa = a.pacc + u * a.ns * a.D + d;
  float M = -kInf, L = 0.0f;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < a.ns; s0 += 8) {
    f32x4 x[8];
    f32x2 y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int s = min(s0 + k, a.ns - 1);
      y[k] = *reinterpret_cast<const f32x2*>(ml + s * 2);
      x[k] = *reinterpret_cast<const f32x4*>(pa + (int64_t)s * a.D);
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, y[k].x);
    const float ref = top == -kInf ? 0.0f : top;
    const float f = __builtin_amdgcn_exp2f(M - ref);
    L *= f;
    v *= f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (s0 + k >= a.ns) continue;
      const float w = __builtin_amdgcn_exp2f(y[k].x - ref);
      L += w * y[k].y;
      v += w * x[k];
    }
    M = top;
  }
  const float f = __builtin_amdgcn_rcpf(L);
  store4(reinterpret_cast<TO*>(a.out) + u * a.D + d, L == 0.0f ? f32x4{0, 0, 0, 0} : v * f);
}

// ---------------------------------------------------------------------------
// bf16 matrix instructions: queries in NT bf16 terms, keys and values in one
// ---------------------------------------------------------------------------

// A bf16 query is one term. An fp32 query is cut into three terms of eight
// fraction bits each, by truncation, so that their sum is the query exactly and
// every product with a bf16 key is exact in fp32. Probabilities are cut the
// same way: two terms for bf16 outputs (2^-16, below the output's rounding),
// three for fp32.
template <int DP, int NM, int NT>
struct QueryBf16 {
  bf16x8 f[NM][DP / 32][NT];
  // value of contraction index e of step s in lane group g
  static __device__ int dim(int s, int g) { return 64 * (s >> 1) + 16 * g + 8 * (s & 1); }

  __device__ void load(const QueryArgs& a, int col0, int cols, int64_t row0, int head0) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const int col = min(col0 + 16 * i + c, cols - 1);
      const int qr = fast_div(a.by_group, col);
      const int64_t at = (row0 + qr) * a.q_stride + (int64_t)(head0 + col - qr * a.group) * a.D;
#pragma unroll
      for (int s = 0; s < DP / 32; ++s) {
        const int d = dim(s, g);
        const bool in = d < a.D;
        if constexpr (NT == 1) {
          u32x4 w = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(a.q) + at +
                                                    (in ? d : 0));
          if (!in) w = u32x4{0, 0, 0, 0};
          f[i][s][0] = as_bf16x8(w);
        } else {
          const float* p = reinterpret_cast<const float*>(a.q) + at + (in ? d : 0);
          const f32x4 x0 = *reinterpret_cast<const f32x4*>(p);
          const f32x4 x1 = *reinterpret_cast<const f32x4*>(p + 4);
          float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
          for (int k = 0; k < 8; ++k)  // a NaN may have all its bits in the half that is cut off
            x[k] = x[k] == x[k] ? x[k] : __builtin_nanf("");
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            u32x4 w;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = in ? high_halves(x[2 * k], x[2 * k + 1]) : 0;
            f[i][s][t] = as_bf16x8(w);
#pragma unroll
            for (int k = 0; k < 8; ++k)  // an infinity leaves no rest
              x[k] = fabsf(x[k]) < kInf ? x[k] - trunc_bf16(x[k]) : 0.0f;
          }
        }
      }
    }
  }
};

// P^T's operand from a lane's eight probabilities, in NP terms. Where values can be
// infinite (INF, two terms), no term of a probability above zero may be zero, since
// zero times infinity is NaN: the rest of one that the first term holds exactly is
// 2^-20 of it, a 32nd of what cutting the second term may lose.
constexpr float kRestUp = 1.0f + 0x1p-20f;
template <int NP, bool INF>
__device__ __forceinline__ void split_p(const float (&p)[8], bf16x8 (&f)[NP]) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = p[e];
#pragma unroll
  for (int t = 0; t < NP; ++t) {
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = NP == 1 ? pack_bf16(x[2 * k], x[2 * k + 1]) : high_halves(x[2 * k], x[2 * k + 1]);
    f[t] = as_bf16x8(w);
    if (t + 1 < NP) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = INF ? fmaf(x[e], kRestUp, -trunc_bf16(x[e])) : x[e] - trunc_bf16(x[e]);
    }
  }
}

// One step: load_k and load_v give the two key tiles and the value tiles, the
// second after the first is used up (registers); bm the step's 32 key bits (a
// zero bit: the key is not seen, its values are zero). With `causal`, lim[i] is
// the first key that column i does not see, less the step's first. INF: values may
// be infinite.
template <int DP, int NM, int NT, int NP, bool INF, typename LoadK, typename LoadV>
__device__ __forceinline__ void step_bf16(const QueryBf16<DP, NM, NT>& q, Softmax<NM>& sm,
                                          f32x4 (&acc)[NM][DP / 16], LoadK load_k, LoadV load_v,
                                          float c, uint32_t bm, bool causal,
                                          const int (&lim)[NM]) {
  const int g = (threadIdx.x & 63) >> 4;
  float p[NM][8];
  {
    bf16x8 kf[2][DP / 32];
    load_k(kf);
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      f32x4 st[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
      for (int s = 0; s < DP / 32; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          st[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[0][s], q.f[i][s][t], st[0], 0, 0, 0);
          st[1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[1][s], q.f[i][s][t], st[1], 0, 0, 0);
        }
#pragma unroll
      for (int e = 0; e < 8; ++e) p[i][e] = st[e >> 2][e & 3];
    }
  }
  uint32_t sees[NM];  // causal: which of its eight keys a lane's column sees
  if (bm != ~0u || causal) {
    const uint32_t mine = bm >> (4 * g);
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      sees[i] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int n = 16 * (e >> 2) + (e & 3);
        const bool seen = ((mine >> n) & 1) && (!causal || n + 4 * g < lim[i]);
        p[i][e] = seen ? p[i][e] : -kInf;
        sees[i] |= seen ? 1u << e : 0u;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    const float alpha = sm.step(i, p[i], c);
    if (__ballot(alpha != 1.0f)) {
#pragma unroll
      for (int j = 0; j < DP / 16; ++j) acc[i][j] *= alpha;
    }
  }
  bf16x8 vf[DP / 16];
  load_v(vf);
  // a non-finite value under a key that only some columns see is taken out of
  // the product, and put back as NaN for the columns that do see it
  if (causal) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < DP / 16; ++j) {
      const u32x4 w = __builtin_bit_cast(u32x4, vf[j]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        bad = bad || (w[k] & 0x7f80u) == 0x7f80u || (w[k] & 0x7f800000u) == 0x7f800000u;
    }
    if (__ballot(bad)) {
#pragma unroll
      for (int j = 0; j < DP / 16; ++j) {
        u32x4 w = __builtin_bit_cast(u32x4, vf[j]), ind;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool lo = (w[k] & 0x7f80u) == 0x7f80u, hi = (w[k] & 0x7f800000u) == 0x7f800000u;
          ind[k] = (lo ? 0x3f80u : 0u) | (hi ? 0x3f800000u : 0u);
          w[k] &= (lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u);
        }
        vf[j] = as_bf16x8(w);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          u32x4 one;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            one[k] = (((sees[i] >> (2 * k)) & 1) ? 0x3f80u : 0u) |
                     (((sees[i] >> (2 * k + 1)) & 1) ? 0x3f800000u : 0u);
          const f32x4 cnt = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              as_bf16x8(ind), as_bf16x8(one), f32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (cnt[r] > 0.0f) acc[i][j][r] = __builtin_nanf("");
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    bf16x8 pf[NP];
    split_p<NP, INF>(p[i], pf);
#pragma unroll
    for (int j = 0; j < DP / 16; ++j)
#pragma unroll
      for (int t = 0; t < NP; ++t)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[j], pf[t], acc[i][j], 0, 0, 0);
  }
}

// V^T's operand of tile j: element j of each of a lane's eight keys.
// rows[e][k] holds values 2k and 2k+1 of key e as bf16.
template <int VD>
__device__ __forceinline__ void gather_v(const uint32_t (&rows)[8][VD / 2], bf16x8 (&vf)[VD]) {
#pragma unroll
  for (int j = 0; j < VD; ++j) {
    const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = __builtin_amdgcn_perm(rows[2 * k + 1][j / 2], rows[2 * k][j / 2], sel);
    vf[j] = as_bf16x8(w);
  }
}

}  // namespace
