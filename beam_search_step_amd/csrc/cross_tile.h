// cross_tile.h -- part of libbeamattn.so, included once by beamattn.hip.
//
// Attention of many rows to an encoder's states: a3_tile (bf16).
#pragma once

namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16;

// 32 NW columns (a column: one query of one head of the group) over all keys, or
// a split of them; every wave has 32 columns, and the workgroup's share tiles of KT
// keys through LDS. With lane = 32 hh + x:
//   S^T = K Q^T   A: row x is key 32 t + x, values 16 s + 8 hh + e of step s; B:
//                 column x; the result's register 4 b + r, half hh is key 32 t +
//                 8 b + 4 hh + r
//   O^T = V^T P^T 16 keys at a time: index 8 hh + 4 b + r is key 16 kk + 8 b +
//                 4 hh + r, so that P^T is what the lane holds; A: row x of tile
//                 j is value 32 j + x, read transposed from LDS; the result's
//                 register 4 b + r is value 32 j + 8 b + 4 hh + r
// The next tile's loads go straight to LDS while this one is used, so they take no
// registers, no instructions to turn V, and no writes. 8 items of 1024 rows over
// 2048 keys, 32 heads of 128: 431 us, 640 TFLOP/s, or 960 of matrix instructions, the
// second product being done in two terms. In one term (2^-8 of a probability instead
// of 2^-15) it is 320 us, but a query would then be answered less exactly beside many
// rows than beside few, where the other kernels keep two. Between two barriers the
// waves meet at the loads (32 KB at the 64 bytes a cycle that a CU takes in), the
// exponentials, and the barrier. Tried and no better: each 16 keys' exponentials right
// before their products, one term's products over all values before the other's; with one
// term, scores of the next tile during this one's exponentials, two tiles between
// barriers, priorities for the matrix phases.
template <int DP>
struct TileLds {
  static constexpr int KT = 8192 / DP;   // keys of a tile: 16 KB of K and of V
  u32x4 k[2][1024];
  u32x4 v[2][1024];
};

// Chunk c (eight values) of a key lies at c ^ swizzle of its row, so that the 16
// rows of one chunk that a read of K takes at once, and the 4 rows by 4 chunks of
// a read of V, lie in different banks.
template <int DP>
__device__ __forceinline__ int swizzle_k(int key) {
  return DP == 64 ? (key >> 1) & 7 : key & 15;
}
template <int DP>
__device__ __forceinline__ int swizzle_v(int key) {
  return DP == 64 ? 4 * ((key >> 1) & 1) : 4 * (key & 3);
}

struct SeenBits {
  uint64_t lo, hi;   // keys of a tile that are seen; bits past the tile are set
  __device__ bool all() const { return lo == ~(uint64_t)0 && hi == ~(uint64_t)0; }
};
template <int KT>
__device__ __forceinline__ SeenBits tile_bits(const uint8_t* mrow, int len, int n0) {
  SeenBits x = {~(uint64_t)0, ~(uint64_t)0};
  const int left = len - n0, lane = threadIdx.x & 63;
  if (mrow || left < KT) {
    bool a = lane < left, b = lane + 64 < left;
    if (mrow && a && lane < KT) a = mrow[n0 + lane] != 0;
    if (mrow && b && KT > 64) b = mrow[n0 + lane + 64] != 0;
    x.lo = __ballot(a || lane >= KT);
    x.hi = __ballot(b || KT <= 64);
  }
  return x;
}

// A tile's K or V straight into LDS: a load of a wave fills 64 chunks in a row,
// 16 bytes a lane, whole keys side by side. `off` is the lane's byte offset in a
// tile: the swizzles of keys 64 NW / CH apart are alike up to 16 chunks a key, with
// 32 there are two kinds.
template <int DP, int NW>
struct TileOffs {
  static constexpr int N = DP == 256 ? 2 : 1;
  int k[N], v[N];
  __device__ void init(int pos_stride, int D) {
    constexpr int CH = DP / 8;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int key = wave * (64 / CH) + lane / CH;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int ck = (lane % CH) ^ swizzle_k<DP>(key + i * (64 * NW / CH));
      const int cv = (lane % CH) ^ swizzle_v<DP>(key + i * (64 * NW / CH));
      k[i] = key * pos_stride + (8 * ck < D ? 16 * ck : 0);
      v[i] = key * pos_stride + (8 * cv < D ? 16 * cv : 0);
    }
  }
};
// the tile of keys n0 .., K at kp and V at vp; past the length: the last key again
template <int DP, int NW>
__device__ __forceinline__ void tile_load(const TileOffs<DP, NW>& off, const char* kp, const char* vp,
                                          int pos_stride, int len, int n0, u32x4* k, u32x4* v) {
  constexpr int CH = DP / 8, KT = TileLds<DP>::KT, N = TileOffs<DP, NW>::N, M = 16 / NW;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int last = len - 1 - n0;
#pragma unroll
  for (int i = 0; i < 2 * M; ++i) {
    const int ii = i % M, add = ii * (64 * NW / CH);
    const char* p = (i < M ? kp : vp) + (int64_t)add * pos_stride;
    int o = i < M ? off.k[ii % N] : off.v[ii % N];
    if (last < KT - 1) {
      const int key = wave * (64 / CH) + lane / CH;
      o += (min(key + add, last) - (key + add)) * pos_stride;
    }
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(p + o),
                                     (__attribute__((address_space(3))) void*)((i < M ? k : v) + (ii * NW + wave) * 64),
                                     16, 0, 0);
  }
}
// Waits for this wave's loads, and clears what a product must not meet: K past the
// head's values, the values of keys that are not seen.
template <int DP, int NW>
__device__ __forceinline__ void tile_ready(int D, SeenBits seen, u32x4* k, u32x4* v) {
  constexpr int CH = DP / 8;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if (D < DP) {
#pragma unroll
    for (int i = 0; i < 16 / NW; ++i) {
      const int key = (i * NW + wave) * (64 / CH) + lane / CH;
      if (8 * ((lane % CH) ^ swizzle_k<DP>(key)) >= D)
        k[(i * NW + wave) * 64 + lane] = u32x4{0, 0, 0, 0};
    }
  }
  if (!seen.all()) {
#pragma unroll
    for (int i = 0; i < 16 / NW; ++i) {
      const int key = (i * NW + wave) * (64 / CH) + lane / CH;
      if (!(((key < 64 ? seen.lo : seen.hi) >> (key & 63)) & 1))
        v[(i * NW + wave) * 64 + lane] = u32x4{0, 0, 0, 0};
    }
  }
}

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;
// 4 keys by 16 values, the lanes of a group of 16 holding 4 values each, four lanes
// to a key: lane i gets value i of the four keys.
__device__ __forceinline__ s16x4 read_transposed(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

template <int DP, int NW>
__global__ __launch_bounds__(NW * 64, DP == 256 ? 1 : 2) void a3_tile(CrossArgs a) {
  constexpr int KT = TileLds<DP>::KT, NT = KT / 32, VD = DP / 32, NS = DP / 16, CH = DP / 8;
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

  const int col = (grp * NW + wave) * 32 + x, qc = min(col, cols - 1);
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
  float m = -kInf, l = 0.0f, l1 = 0.0f;  // l, l1: sums of every other key
  const float c = a.q.c;

  // this lane's places in a tile: K's row x, chunk 2 s + hh; V's row 4 hh + y / 4 of
  // 16 kk + 8 b .., values 32 j + 16 (x / 16) + 4 (y % 4) .., y the lane in its 16
  const int y = lane & 15, vrow = 4 * hh + (y >> 2);
  const int vlane = vrow * DP * 2 + ((2 * (x >> 4) + ((y & 3) >> 1)) * 16 + (y & 1) * 8);
  const int ksw = swizzle_k<DP>(x), vsw = swizzle_v<DP>(vrow);

  TileOffs<DP, NW> off;
  off.init(a.pos_stride, a.q.D);
  kb += (int64_t)begin * a.pos_stride;
  vb += (int64_t)begin * a.pos_stride;
  SeenBits seen = {0, 0};
  if (begin < end) {
    seen = tile_bits<KT>(mrow, len, begin);
    tile_load<DP, NW>(off, kb, vb, a.pos_stride, len, begin, lds.k[0], lds.v[0]);
    tile_ready<DP, NW>(a.q.D, seen, lds.k[0], lds.v[0]);
  }
  __syncthreads();
  int buf = 0;
  for (int n0 = begin; n0 < end; n0 += KT, buf ^= 1) {
    const SeenBits now = seen;
    const bool more = n0 + KT < end;
    if (more) {
      seen = tile_bits<KT>(mrow, len, n0 + KT);
      kb += (int64_t)KT * a.pos_stride;
      vb += (int64_t)KT * a.pos_stride;
      tile_load<DP, NW>(off, kb, vb, a.pos_stride, len, n0 + KT, lds.k[buf ^ 1], lds.v[buf ^ 1]);
    }
    f32x16 st[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < 16; ++r) st[t][r] = 0.0f;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const u32x4 w = lds.k[buf][(32 * t + x) * CH + ((2 * s + hh) ^ ksw)];
        st[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(w), q[s], st[t], 0, 0, 0);
      }
    }
    if (!now.all()) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t bits = (uint32_t)((t < 2 ? now.lo : now.hi) >> (32 * (t & 1))) >> (4 * hh);
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
    // the point that scores are taken from follows the maximum only when it is
    // 2^8 behind: probabilities keep their relative rounding, and far from the
    // 2^127 that sums hold
    if (__ballot(top > m + 8.0f)) {
      const float mn = fmaxf(m, top);
      const float alpha = mn == -kInf ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
      l *= alpha;
      l1 *= alpha;
#pragma unroll
      for (int j = 0; j < VD; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[j][r] *= alpha;
      m = mn;
    }
    const float ref = m == -kInf ? 0.0f : m;
    // probabilities in two bf16 terms, as everywhere for bf16 outputs (2^-15); values
    // may be infinite, so the second is never zero (split_p)
    bf16x8 pf[2 * NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        u32x4 hi, lo;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p0 = __builtin_amdgcn_exp2f(fmaf(st[t][8 * k2 + 2 * k], c, -ref));
          const float p1 = __builtin_amdgcn_exp2f(fmaf(st[t][8 * k2 + 2 * k + 1], c, -ref));
          l += p0;
          l1 += p1;
          hi[k] = high_halves(p0, p1);
          lo[k] = high_halves(fmaf(p0, kRestUp, -trunc_bf16(p0)), fmaf(p1, kRestUp, -trunc_bf16(p1)));
        }
        pf[2 * t + k2][0] = as_bf16x8(hi);
        pf[2 * t + k2][1] = as_bf16x8(lo);
      }
#pragma unroll
    for (int kk = 0; kk < 2 * NT; ++kk)
#pragma unroll
      for (int j = 0; j < VD; ++j) {
        const char* p = reinterpret_cast<const char*>(lds.v[buf]) + vlane + ((4 * j) ^ vsw) * 16 +
                        16 * kk * DP * 2;
        const s16x4 lo = read_transposed(p), hi = read_transposed(p + 8 * DP * 2);
        const bf16x8 w = __builtin_bit_cast(
            bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, pf[kk][0], acc[j], 0, 0, 0);
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, pf[kk][1], acc[j], 0, 0, 0);
      }
    if (more) tile_ready<DP, NW>(a.q.D, seen, lds.k[buf ^ 1], lds.v[buf ^ 1]);
    __syncthreads();
  }

  {
    l += l1;
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
    for (int j = 0; j < VD; ++j) {
      const int d = 32 * j + 8 * bb + 4 * hh;
      if (d >= a.q.D) continue;
      f32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = acc[j][4 * bb + k];
      if (a.q.ns > 1) {
        store4(a.q.pacc + (unit * a.q.ns + sp) * a.q.D + d, v);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = none ? 0.0f : v[k] * f;
        store4(reinterpret_cast<uint16_t*>(a.q.out) + unit * a.q.D + d, v);
      }
    }
}

}  // namespace
