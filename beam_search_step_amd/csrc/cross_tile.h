// cross_tile.h -- part of libbeamattn.so, included once by beamattn.hip.
//
// Attention of many rows to an encoder's states: a3_tile (bf16).
#pragma once

namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16;

// 128 columns (a column: one query of one head of the group) over all keys, or a
// split of them; every wave has 32 columns, and the workgroup's four share tiles
// of KT keys through LDS. With lane = 32 hh + x:
//   S^T = K Q^T   A: row x is key 32 t + x, values 16 s + 8 hh + e of step s; B:
//                 column x; the result's register 4 b + r, half hh is key 32 t +
//                 8 b + 4 hh + r
//   O^T = V^T P^T 16 keys at a time: index 8 hh + 4 b + r is key 16 kk + 8 b +
//                 4 hh + r, so that P^T is what the lane holds; A: row x of tile
//                 j is value VD x + j, the result's register 4 b + r value
//                 VD (8 b + 4 hh + r) + j
// K lies in LDS as its operands, the rows of step s and half hh permuted by
// x ^ (2 s + hh), so that neither the writes (16 chunks of a row at once) nor the
// reads (32 rows of a chunk) meet in a bank. V lies as its operands too: a thread
// turns 4 keys by 8 values into 8 values by 4 keys on the way in.
template <int DP>
struct TileLds {
  static constexpr int KT = 8192 / DP;   // keys of a tile: 16 KB of K and of V
  u32x4 k[2][1024];
  u32x2 v[2][2048];
};

template <int DP>
struct TileRegs {
  u32x4 k[4], v[4];
  uint64_t lo, hi;   // keys of the tile that are seen
};

template <int DP>
__device__ __forceinline__ void tile_load(const CrossArgs& a, const char* kb, const char* vb,
                                          const uint8_t* mrow, int len, int n0, TileRegs<DP>& x) {
  constexpr int CH = DP / 8, KT = TileLds<DP>::KT;
  const int tid = threadIdx.x, lane = tid & 63, D = a.q.D;
  const char* kp = kb + (int64_t)n0 * a.pos_stride;
  const char* vp = vb + (int64_t)n0 * a.pos_stride;
  const int last = len - 1 - n0;  // keys past the length: the last one again
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int idx = i * kAttnThreads + tid, key = idx / CH, d = idx % CH * 8;
    x.k[i] = *reinterpret_cast<const u32x4*>(kp + (min(key, last) * a.pos_stride + (d < D ? 2 * d : 0)));
    if (d >= D) x.k[i] = u32x4{0, 0, 0, 0};
  }
  const int d = tid % CH * 8, k0 = tid / CH * 4;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    x.v[r] = *reinterpret_cast<const u32x4*>(vp + (min(k0 + r, last) * a.pos_stride + (d < D ? 2 * d : 0)));
  x.lo = x.hi = ~(uint64_t)0;
  if (mrow || last < KT - 1) {
    bool ok = lane <= last, ok2 = lane + 64 <= last;
    if (mrow && ok) ok = mrow[n0 + lane] != 0;
    if (mrow && ok2 && KT > 64) ok2 = mrow[n0 + lane + 64] != 0;
    x.lo = __ballot(ok);
    x.hi = __ballot(ok2);
  }
}
template <int DP>
__device__ __forceinline__ bool tile_full(const TileRegs<DP>& x) {
  constexpr int KT = TileLds<DP>::KT;
  const uint64_t all = ~(uint64_t)0;
  return KT == 32 ? (uint32_t)x.lo == ~0u : x.lo == all && (KT == 64 || x.hi == all);
}

template <int DP>
__device__ __forceinline__ void tile_store(TileLds<DP>& lds, int buf, TileRegs<DP>& x) {
  constexpr int CH = DP / 8, VD = DP / 32;
  const int tid = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int idx = i * kAttnThreads + tid, key = idx / CH, c = idx % CH;
    lds.k[buf][((key >> 5) * (CH / 2) + (c >> 1)) * 64 + (c & 1) * 32 + ((key & 31) ^ c)] = x.k[i];
  }
  const int c = tid % CH, kg = tid / CH;
  if (!tile_full(x)) {  // the values of a key that is not seen are zero
    const uint64_t bits = kg < 16 ? x.lo >> (4 * kg) : x.hi >> (4 * (kg - 16));
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (!((bits >> r) & 1)) x.v[r] = u32x4{0, 0, 0, 0};
  }
  const int kk = kg >> 2, b = (kg >> 1) & 1, hh = kg & 1;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
    const u32x2 w = {__builtin_amdgcn_perm(x.v[1][j / 2], x.v[0][j / 2], sel),
                     __builtin_amdgcn_perm(x.v[3][j / 2], x.v[2][j / 2], sel)};
    const int d = 8 * c + j;
    lds.v[buf][((kk * VD + d % VD) * 64 + hh * 32 + d / VD) * 2 + b] = w;
  }
}

template <int DP>
__global__ __launch_bounds__(kAttnThreads, DP == 256 ? 1 : 2) void a3_tile(CrossArgs a) {
  constexpr int KT = TileLds<DP>::KT, NT = KT / 32, VD = DP / 32, NS = DP / 16;
  __shared__ TileLds<DP> lds;
  const int tid = threadIdx.x, lane = tid & 63, hh = lane >> 5, x = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // workgroups of one item and head follow each other on one XCD, whose L2 then
  // holds their keys
  const int pairs = a.pairs, xcd = blockIdx.x & 7;
  int idx = blockIdx.x >> 3;
  const int sp = idx % a.splits;
  idx /= a.splits;
  const int grp = idx % a.groups, pair = idx / a.groups * 8 + xcd;
  if (pair >= pairs) return;
  const int h = pair % a.q.kv_heads, b = pair / a.q.kv_heads;
  const int cols = a.n_rows * a.q.group;
  const int64_t row0 = (int64_t)b * a.n_rows;
  const int head0 = h * a.q.group;
  const int len = a.lens ? min(max(a.lens[b], 0), a.n_keys) : a.n_keys;
  int per = (len + a.splits - 1) / a.splits;
  per = (per + KT - 1) / KT * KT;
  const int begin = min((int64_t)sp * per, (int64_t)len), end = min(begin + per, len);
  const char* kb = a.k + b * a.batch_stride + h * a.head_stride;
  const char* vb = a.v + b * a.batch_stride + h * a.head_stride;
  const uint8_t* mrow = a.mask ? a.mask + b * a.mask_stride : nullptr;

  const int col = grp * 128 + wave * 32 + x, qc = min(col, cols - 1);
  const int qr = fast_div(a.q.by_group, qc);
  const int64_t unit = (row0 + qr) * a.q.heads + head0 + (qc - qr * a.q.group);
  bf16x8 q[NS];
  {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(a.q.q) + (row0 + qr) * a.q.q_stride +
                        (int64_t)(head0 + qc - qr * a.q.group) * a.q.D;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = 16 * s + 8 * hh;
      u32x4 w = *reinterpret_cast<const u32x4*>(p + (d < a.q.D ? d : 0));
      if (d >= a.q.D) w = u32x4{0, 0, 0, 0};
      q[s] = as_bf16x8(w);
    }
  }
  f32x16 acc[VD];
#pragma unroll
  for (int j = 0; j < VD; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[j][r] = 0.0f;
  float m = -kInf, l = 0.0f;
  const float c = a.q.c;
  bf16x2 ones;
  ones.x = ones.y = (__bf16)1.0f;

  TileRegs<DP> in;
  if (begin < end) {
    tile_load<DP>(a, kb, vb, mrow, len, begin, in);
    tile_store<DP>(lds, 0, in);
  }
  __syncthreads();
  int buf = 0;
  for (int n0 = begin; n0 < end; n0 += KT, buf ^= 1) {
    const bool full = tile_full(in);
    const uint64_t lo = in.lo, hi = in.hi;
    const bool more = n0 + KT < end;
    if (more) tile_load<DP>(a, kb, vb, mrow, len, n0 + KT, in);
    f32x16 st[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < 16; ++r) st[t][r] = 0.0f;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const u32x4 w = lds.k[buf][(t * NS + s) * 64 + hh * 32 + (x ^ (2 * s + hh))];
        st[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(w), q[s], st[t], 0, 0, 0);
      }
    }
    if (!full) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t bits = (uint32_t)((t < 2 ? lo : hi) >> (32 * (t & 1))) >> (4 * hh);
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (!((bits >> (8 * (r >> 2) + (r & 3))) & 1)) st[t][r] = -kInf;
      }
    }
    float top = st[0][0];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, st[t][r]);
    {
      auto sw = __builtin_amdgcn_permlane32_swap(as_u(top), as_u(top), false, false);
      top = fmaxf(as_f(sw[0]), as_f(sw[1])) * c;
    }
    const float mn = fmaxf(m, top);
    const float ref = mn == -kInf ? 0.0f : mn;
    if (__ballot(mn != m)) {
      const float alpha = __builtin_amdgcn_exp2f(m - ref);
      l *= alpha;
#pragma unroll
      for (int j = 0; j < VD; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[j][r] *= alpha;
    }
    m = mn;
    // the sum is of the rounded probabilities, those that the product uses
    bf16x8 pf[2 * NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        u32x4 w;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p0 = __builtin_amdgcn_exp2f(fmaf(st[t][8 * k2 + 2 * k], c, -ref));
          const float p1 = __builtin_amdgcn_exp2f(fmaf(st[t][8 * k2 + 2 * k + 1], c, -ref));
          bf16x2 pair;
          pair.x = (__bf16)p0;
          pair.y = (__bf16)p1;
          l = __builtin_amdgcn_fdot2_f32_bf16(pair, ones, l, false);
          w[k] = __builtin_bit_cast(uint32_t, pair);
        }
        pf[2 * t + k2] = as_bf16x8(w);
      }
#pragma unroll
    for (int kk = 0; kk < 2 * NT; ++kk)
#pragma unroll
      for (int j = 0; j < VD; ++j) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(
            &lds.v[buf][((kk * VD + j) * 64 + hh * 32 + x) * 2]);
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(w), pf[kk], acc[j], 0, 0, 0);
      }
    if (more) tile_store<DP>(lds, buf ^ 1, in);
    __syncthreads();
  }

  {
    auto sw = __builtin_amdgcn_permlane32_swap(as_u(l), as_u(l), false, false);
    l = as_f(sw[0]) + as_f(sw[1]);
  }
  if (col >= cols) return;
  const bool none = l == 0.0f;  // all-NaN scores leave m at -inf, but not l at zero
  const float f = none ? 0.0f : 1.0f / l;
  if (a.q.ns > 1 && hh == 0) {
    float* p = a.q.pml + (unit * a.q.ns + sp) * 2;
    p[0] = m;
    p[1] = l;
  }
#pragma unroll
  for (int bb = 0; bb < 4; ++bb)
#pragma unroll
    for (int i = 0; i < VD; ++i) {  // four values each: VD (8 bb + 4 hh) + 4 i ..
      const int d = VD * (8 * bb + 4 * hh) + 4 * i;
      if (d >= a.q.D) continue;
      f32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = acc[(4 * i + k) % VD][4 * bb + (4 * i + k) / VD];
      if (a.q.ns > 1) {
        if (!none) store4(a.q.pacc + (unit * a.q.ns + sp) * a.q.D + d, v);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = none ? 0.0f : v[k] * f;
        store4(reinterpret_cast<uint16_t*>(a.q.out) + unit * a.q.D + d, v);
      }
    }
}

}  // namespace
