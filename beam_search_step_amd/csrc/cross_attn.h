// cross_attn.h -- part of libbeamattn.so, included once by beamattn.hip.
//
// Attention of an item's rows to its encoder's states: a2_cross (keys split
// over waves and workgroups).
#pragma once

namespace {

struct CrossArgs {
  QueryArgs q;
  const char* k;
  const char* v;
  int64_t batch_stride, head_stride;  // bytes
  int pos_stride;                     // bytes, below 2^26
  int n_rows, n_keys;
  const int* lens;                    // [B] or null
  const uint8_t* mask;                // [B][mask_stride] or null
  int64_t mask_stride;
  int splits, groups;
  int pairs;                          // items * kv heads
};

// The keys n0 .. n0 + 31 that an item sees, as bits.
__device__ __forceinline__ uint32_t seen_keys(const uint8_t* mrow, int len, int n0) {
  const int n = n0 + (threadIdx.x & 31);
  bool ok = n < len;
  if (mrow && ok) ok = mrow[n] != 0;
  return (uint32_t)__ballot(ok);
}

// bf16: the step as loaded. Key 16 t + c, values dim(s, g) ..; and values VD c
// .. of the lane's eight keys.
template <int DP>
struct RawBf16 {
  u32x4 k[2][DP / 32];
  uint32_t v[8][DP / 32];
  uint32_t bm;
};

template <int N>
__device__ __forceinline__ void load_dwords(const char* p, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    w[0] = x.x;
    w[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(p + 4 * i);
      w[i] = x.x;
      w[i + 1] = x.y;
      w[i + 2] = x.z;
      w[i + 3] = x.w;
    }
  }
}

template <int DP>
__device__ __forceinline__ void load_step(const CrossArgs& a, const char* kb, const char* vb,
                                          const uint8_t* mrow, int len, int n0,
                                          RawBf16<DP>& x) {
  constexpr int VD = DP / 16;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4, D = a.q.D;
  x.bm = seen_keys(mrow, len, n0);
  const char* kp = kb + (int64_t)n0 * a.pos_stride;
  const char* vp = vb + (int64_t)n0 * a.pos_stride;
  const int last = len - 1 - n0;  // keys past the length: the last one again
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int o = min(16 * t + c, last) * a.pos_stride;
#pragma unroll
    for (int s = 0; s < DP / 32; ++s) {
      const int d = QueryBf16<DP, 1, 1>::dim(s, g);
      x.k[t][s] = *reinterpret_cast<const u32x4*>(kp + (o + 2 * (d < D ? d : 0)));
    }
  }
  const int vd = VD * c < D ? VD * c : 0;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    load_dwords(vp + (min(16 * (e >> 2) + 4 * g + (e & 3), last) * a.pos_stride + 2 * vd), x.v[e]);
}

template <int DP>
__device__ __forceinline__ void widen_k(const RawBf16<DP>& x, int D,
                                        bf16x8 (&kf)[2][DP / 32]) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int s = 0; s < DP / 32; ++s) {
      const bool in = QueryBf16<DP, 1, 1>::dim(s, g) < D;
      kf[t][s] = as_bf16x8(in ? x.k[t][s] : u32x4{0, 0, 0, 0});
    }
}
template <int DP>
__device__ __forceinline__ void widen_v(const RawBf16<DP>& x, bf16x8 (&vf)[DP / 16]) {
  const int g = (threadIdx.x & 63) >> 4;
  if (x.bm == ~0u) {
    gather_v<DP / 16>(x.v, vf);
  } else {  // the values of a key that is not seen are zero
    const uint32_t mine = x.bm >> (4 * g);
    uint32_t rows[8][DP / 32];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool seen = (mine >> (16 * (e >> 2) + (e & 3))) & 1;
#pragma unroll
      for (int k = 0; k < DP / 32; ++k) rows[e][k] = seen ? x.v[e][k] : 0u;
    }
    gather_v<DP / 16>(rows, vf);
  }
}

// fp32: matrix instructions of four contraction indices. Value 16 s + 4 g + e
// is index g of instruction (s, e); key 16 t + 4 g + r is index g of
// instruction (t, r).
template <int DP>
struct RawF32 {
  f32x4 k[2][DP / 16];
  f32x4 v[8][DP / 64];
  uint32_t bm;
};

template <int DP>
__device__ __forceinline__ void load_step(const CrossArgs& a, const char* kb, const char* vb,
                                          const uint8_t* mrow, int len, int n0,
                                          RawF32<DP>& x) {
  constexpr int VD = DP / 16;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4, D = a.q.D;
  x.bm = seen_keys(mrow, len, n0);
  const char* kp = kb + (int64_t)n0 * a.pos_stride;
  const char* vp = vb + (int64_t)n0 * a.pos_stride;
  const int last = len - 1 - n0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int o = min(16 * t + c, last) * a.pos_stride;
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
      const int d = 16 * s + 4 * g;
      x.k[t][s] = *reinterpret_cast<const f32x4*>(kp + (o + 4 * (d < D ? d : 0)));
    }
  }
  const int vd = VD * c < D ? VD * c : 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int o = min(16 * (e >> 2) + 4 * g + (e & 3), last) * a.pos_stride + 4 * vd;
#pragma unroll
    for (int j = 0; j < VD / 4; ++j) x.v[e][j] = *reinterpret_cast<const f32x4*>(vp + (o + 16 * j));
  }
}

template <int DP, int NM>
struct QueryF32 {
  f32x4 f[NM][DP / 16];
  __device__ void load(const QueryArgs& a, int col0, int cols, int64_t row0, int head0) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const int col = min(col0 + 16 * i + c, cols - 1);
      const int qr = fast_div(a.by_group, col);
      const float* p = reinterpret_cast<const float*>(a.q) + (row0 + qr) * a.q_stride +
                       (int64_t)(head0 + col - qr * a.group) * a.D;
#pragma unroll
      for (int s = 0; s < DP / 16; ++s) {
        const int d = 16 * s + 4 * g;
        const f32x4 x = *reinterpret_cast<const f32x4*>(p + (d < a.D ? d : 0));
        f[i][s] = d < a.D ? x : f32x4{0, 0, 0, 0};
      }
    }
  }
};

template <int DP, int NM>
__device__ __forceinline__ void step_f32(const QueryF32<DP, NM>& q, Softmax<NM>& sm,
                                         f32x4 (&acc)[NM][DP / 16], RawF32<DP>& x, float c,
                                         int D) {
  const int g = (threadIdx.x & 63) >> 4;
  const uint32_t mine = x.bm >> (4 * g);
  if (x.bm != ~0u) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool seen = (mine >> (16 * (e >> 2) + (e & 3))) & 1;
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) x.v[e][j] = seen ? x.v[e][j] : f32x4{0, 0, 0, 0};
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int s = 0; s < DP / 16; ++s)
      if (16 * s >= D) x.k[t][s] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    f32x4 st[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int s = 0; s < DP / 16; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        st[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(x.k[0][s][e], q.f[i][s][e], st[0], 0, 0, 0);
        st[1] = __builtin_amdgcn_mfma_f32_16x16x4f32(x.k[1][s][e], q.f[i][s][e], st[1], 0, 0, 0);
      }
    float p[8] = {st[0].x, st[0].y, st[0].z, st[0].w, st[1].x, st[1].y, st[1].z, st[1].w};
    if (x.bm != ~0u) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        p[e] = (mine >> (16 * (e >> 2) + (e & 3))) & 1 ? p[e] : -kInf;
    }
    const float alpha = sm.step(i, p, c);
    if (__ballot(alpha != 1.0f)) {
#pragma unroll
      for (int j = 0; j < DP / 16; ++j) acc[i][j] *= alpha;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int j = 0; j < DP / 16; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x.v[e][j / 4][j % 4], p[e], acc[i][j],
                                                         0, 0, 0);
  }
}

// Workgroup idx of `units` x `groups`: the column groups of a unit read the same
// keys, so they follow each other on one XCD, whose L2 then holds them. Workgroups
// go round the eight XCDs; units past the last eight are dealt as they come. 56 fp32
// columns of 1403 keys, heads of 128: 88 us against 108. (Over the cache, whose keys are
// a quarter as wide, it measured nothing.)
__device__ __forceinline__ void unit_and_group(int idx, int units, int groups, int& unit,
                                               int& group) {
  unit = idx;
  group = 0;
  if (groups == 1) return;
  const int even = units & ~7, rest = units & 7;
  if (idx < even * groups) {
    const int j = idx >> 3;
    unit = j / groups;
    group = j - unit * groups;
    unit = unit * 8 + (idx & 7);
  } else {
    const int j = idx - even * groups;
    group = j / rest;
    unit = even + (j - group * rest);
  }
}

// Bound by bandwidth where keys are many and columns few: 16 items of 16 heads of 64,
// 1500 bf16 keys, 26.5 us, 3.7 TB/s; 1000 fp32 keys 39.7, 3.4 TB/s.
// Waves a SIMD that the registers have to leave (fp32 heads of 128, 48 items of 2
// heads, 4 rows and 4829 keys: two 108 us, one 120).
template <int DP, int NM, typename T>
constexpr int cross_waves() {
  return sizeof(T) == 4 ? (NM == 1 && DP == 128 ? 2 : 1)
                        : DP == 64 ? (NM == 1 ? 5 : 4) : DP == 128 ? 3 : 1;
}
template <int DP, int NM, int NW, typename T>
__global__ __launch_bounds__(NW * 64, (cross_waves<DP, NM, T>())) void a2_cross(CrossArgs a) {
  constexpr bool F32 = sizeof(T) == 4;
  __shared__ JoinLds<DP, NM, NW> lds;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int idx = blockIdx.x;
  int grp;
  unit_and_group(idx, a.pairs * a.splits, a.groups, idx, grp);
  const int sp = idx % a.splits;
  idx /= a.splits;
  const int h = idx % a.q.kv_heads, b = idx / a.q.kv_heads;
  const int cols = a.n_rows * a.q.group, col0 = grp * 16 * NM;
  const int64_t row0 = (int64_t)b * a.n_rows;
  const int head0 = h * a.q.group;
  const int len = a.lens ? min(max(a.lens[b], 0), a.n_keys) : a.n_keys;
  int per = (len + a.splits - 1) / a.splits;
  per = (per + NW * kStep - 1) / (NW * kStep) * (NW * kStep);
  const int begin = min((int64_t)sp * per, (int64_t)len), end = min(begin + per, len);
  const char* kb = a.k + b * a.batch_stride + h * a.head_stride;
  const char* vb = a.v + b * a.batch_stride + h * a.head_stride;
  const uint8_t* mrow = a.mask ? a.mask + b * a.mask_stride : nullptr;

  typename std::conditional<F32, QueryF32<DP, NM>, QueryBf16<DP, NM, 1>>::type q;
  Softmax<NM> sm;
  f32x4 acc[NM][DP / 16];
  q.load(a.q, col0, cols, row0, head0);
  sm.init();
#pragma unroll
  for (int i = 0; i < NM; ++i)
#pragma unroll
    for (int j = 0; j < DP / 16; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  int n0 = begin + wave * kStep;
  if (n0 < end) {
    typename std::conditional<F32, RawF32<DP>, RawBf16<DP>>::type cur;
    load_step<DP>(a, kb, vb, mrow, len, n0, cur);
    while (true) {
      const int n1 = n0 + NW * kStep;
      const bool more = n1 < end;
      if (cur.bm) {
        if constexpr (F32) {
          step_f32<DP, NM>(q, sm, acc, cur, a.q.c, a.q.D);
        } else {
          const int lim[NM] = {};
          step_bf16<DP, NM, 1, 2, true>(
              q, sm, acc, [&](bf16x8(&kf)[2][DP / 32]) { widen_k<DP>(cur, a.q.D, kf); },
              [&](bf16x8(&vf)[DP / 16]) { widen_v<DP>(cur, vf); }, a.q.c, cur.bm, false, lim);
        }
      }
      if (!more) break;
      load_step<DP>(a, kb, vb, mrow, len, n1, cur);
      n0 = n1;
    }
  }
  join_and_store<DP, NM, NW, T>(a.q, lds, acc, sm, col0, cols, row0, head0, sp);
}

}  // namespace
