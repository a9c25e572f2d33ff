// cache_attn.h -- part of libbeamattn.so, included once by beamattn.hip.
//
// Attention over an 8-bit paged cache: a1_cache.
#pragma once

namespace {

// The keys of one kind of workgroup: an item's shared prompt, read once for all
// queries of the item's rows, or a row's own positions.
struct PagedSeg {
  const int* table;       // [units][table_stride]
  int64_t table_stride;
  const int* lens;        // [units]
  int mb;                 // entries of a table row
  int qrows;              // query rows of a unit
  int back;               // query i sees lens - back + i positions
  int splits, split0;     // workgroups along the keys, and their first partial
  int groups;             // groups of 16 columns
  int blocks;             // workgroups
};

struct CacheArgs {
  QueryArgs q;
  PagedSeg seg[2];
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  int64_t block_stride;
  int pos_stride;
  int n_blocks, bs;
  FastDiv by_bs;
};

// The bytes and scales of one step as loaded.
template <int DP>
struct RawKv {
  u32x4 k[2][DP / 64];          // key 16 t + c: bytes 64 s + 16 g ..
  uint32_t v[8][DP / 64];       // key 16 (e/4) + 4 g + e%4: bytes VD c ..
  float ks[2], vs[8];
  uint32_t bm;                  // keys seen
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    const u32x4 x = *reinterpret_cast<const u32x4*>(p);
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  }
}

// Loads the step of keys n0 .. n0 + 31. With UNI (block_size a multiple of 16)
// each 16-key tile lies in one block: its table entry is one scalar load and
// its addresses are a scalar base and a lane offset. Otherwise lane l looks key
// n0 + l % 32 up and the lanes that need it ask for it.
template <int DP, bool UNI>
__device__ __forceinline__ void load_step(const CacheArgs& a, const int* trow, int len, int n0,
                                          int h, RawKv<DP>& x) {
  constexpr int VD = DP / 16;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int D = a.q.D;
  const int vd = VD * c < D ? VD * c : 0;
  const int64_t hd = (int64_t)h * D;
  if constexpr (UNI) {
    x.bm = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int n = n0 + 16 * t;
      int id = -1, kb = 0;
      if (n < len) {
        kb = fast_div(a.by_bs, n);
        id = trow[kb];
      }
      const bool ok = (unsigned)id < (unsigned)a.n_blocks;
      const int bid = ok ? id : 0;
      const int left = ok ? min(len - n, 16) : 0;
      x.bm |= ((1u << left) - 1) << (16 * t);
      const int64_t base = bid * a.block_stride + (int64_t)(ok ? n - kb * a.bs : 0) * a.pos_stride + hd;
      const uint8_t* kp = a.k + base;
      const uint8_t* vp = a.v + base;
      const int last = max(left - 1, 0);  // rows past the length: the last one again
      const int kr = min(c, last) * a.pos_stride;
#pragma unroll
      for (int s = 0; s < DP / 64; ++s) {
        const int d = 64 * s + 16 * g;
        x.k[t][s] = *reinterpret_cast<const u32x4*>(kp + (kr + (d < D ? d : 0)));
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
        load_words(vp + (min(4 * g + r, last) * a.pos_stride + vd), x.v[4 * t + r]);
      const int64_t si = (int64_t)bid * a.q.kv_heads + h;
      x.ks[t] = a.ks[si];
      // without a block the scale is another's, perhaps NaN, which a zero would keep
      const float vs = ok ? a.vs[si] : 1.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) x.vs[4 * t + r] = vs;
    }
  } else {
    const int n = n0 + (lane & 31);
    int id = -1, kb = 0;
    if (n < len) {
      kb = fast_div(a.by_bs, n);
      id = trow[kb];
    }
    const bool ok = (unsigned)id < (unsigned)a.n_blocks;
    const int bid = ok ? id : 0;
    const int64_t off = bid * a.block_stride + (int64_t)(ok ? n - kb * a.bs : 0) * a.pos_stride + hd;
    const int64_t si = (int64_t)bid * a.q.kv_heads + h;
    const float ks = a.ks[si], vs = ok ? a.vs[si] : 1.0f;  // as above
    x.bm = (uint32_t)__ballot(ok);
    const int lo = (int)(uint32_t)off, hi = (int)(off >> 32);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int src = 16 * t + c;
      const int64_t o = ((int64_t)__shfl(hi, src) << 32) | (uint32_t)__shfl(lo, src);
      x.ks[t] = __shfl(ks, src);
#pragma unroll
      for (int s = 0; s < DP / 64; ++s) {
        const int d = 64 * s + 16 * g;
        x.k[t][s] = *reinterpret_cast<const u32x4*>(a.k + o + (d < D ? d : 0));
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int src = 16 * (e >> 2) + 4 * g + (e & 3);
      const int64_t o = ((int64_t)__shfl(hi, src) << 32) | (uint32_t)__shfl(lo, src);
      x.vs[e] = __shfl(vs, src);
      load_words(a.v + o + vd, x.v[e]);
    }
  }
}

// e4m3 times a power of two is exact in bf16 (scales are at least 2^-100).
template <int DP>
__device__ __forceinline__ void widen_k(const RawKv<DP>& x, int D, bf16x8 (&kf)[2][DP / 32]) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int s = 0; s < DP / 64; ++s) {
      const bool in = 64 * s + 16 * g < D;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        u32x4 w;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t b = in ? x.k[t][s][2 * hh + k] : 0u;
          w[2 * k] = __builtin_bit_cast(
              uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, x.ks[t], false));
          w[2 * k + 1] = __builtin_bit_cast(
              uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, x.ks[t], true));
        }
        kf[t][2 * s + hh] = as_bf16x8(w);
      }
    }
}
template <int DP>
__device__ __forceinline__ void widen_v(const RawKv<DP>& x, bf16x8 (&vf)[DP / 16]) {
  constexpr int VD = DP / 16;
  const int g = (threadIdx.x & 63) >> 4;
  const uint32_t mine = x.bm >> (4 * g);
  uint32_t rows[8][VD / 2];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // the values of a key that is not seen are zero
    const bool seen = (mine >> (16 * (e >> 2) + (e & 3))) & 1;
#pragma unroll
    for (int k = 0; k < DP / 64; ++k) {
      const uint32_t b = seen ? x.v[e][k] : 0u;
      rows[e][2 * k] = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, x.vs[e], false));
      rows[e][2 * k + 1] = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, x.vs[e], true));
    }
  }
  gather_v<VD>(rows, vf);
}

// Prompts of 16,000 to 48,000 tokens for 8 items of 4 beams, 32 heads on 8 of 128: 131
// us, 4.1 TB/s, bound by memory (a head whose bytes are 384 mod 1024 takes a third
// longer than the others); of 1000 tokens: 12.7, bound by the launch and the chain of
// lengths, table and keys.
// 16 columns a wave: two or four tiles of them read a key once for all, but leave no
// registers for a second wave (16 items, 16 beams of 4 heads a kv head, prompts of
// 1000 tokens: 20 us at 64 values a head, with two tiles 30; 33 at 128, with two 66).
// Waves a SIMD that the registers have to leave, as many as go without spilling:
// left to itself the compiler keeps sums in a second register file and one wave
// fewer (16 beams of 4 heads a kv head over prompts of 1000 tokens, 256 values a
// head: two waves 60 us, one 104; 128 fp32 values: three 45, two 59; the wide
// search's 4352 one-wave workgroups: five, all resident, 31, four 32).
template <int DP, int NW, int NT, bool UNI>
constexpr int cache_waves() {
  return DP == 64 ? (NT == 1 || NW == 1 ? 5 : 4)
                  : DP == 128 ? (NT == 1 || UNI ? 3 : 2) : NT == 1 ? 2 : 1;
}
template <int DP, int NW, int NT, bool UNI>
__global__ __launch_bounds__(NW * 64, (cache_waves<DP, NW, NT, UNI>())) void a1_cache(CacheArgs a) {
  using TO = typename std::conditional<NT == 1, uint16_t, float>::type;
  constexpr int NM = 1, NP = NT == 1 ? 2 : 3;
  __shared__ JoinLds<DP, NM, NW> lds;
  const int lane = threadIdx.x & 63, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int idx = blockIdx.x;
  const int which = idx >= a.seg[0].blocks ? 1 : 0;
  idx -= which ? a.seg[0].blocks : 0;
  const PagedSeg& s = a.seg[which];
  const int h = idx % a.q.kv_heads;
  idx /= a.q.kv_heads;
  const int sp = idx % s.splits;
  idx /= s.splits;
  const int grp = idx % s.groups;
  const int unit = idx / s.groups;
  const int cols = s.qrows * a.q.group, col0 = grp * 16 * NM;
  const int64_t row0 = (int64_t)unit * s.qrows;
  const int head0 = h * a.q.group;

  const int len = min(max(s.lens[unit], 0), s.mb * a.bs);
  // the keys of this split: a step of each wave, times a whole number
  int per = (len + s.splits - 1) / s.splits;
  per = (per + NW * kStep - 1) / (NW * kStep) * (NW * kStep);
  const int begin = min((int64_t)sp * per, (int64_t)len), end = min(begin + per, len);
  const int* trow = s.table + (int64_t)unit * s.table_stride;

  QueryBf16<DP, NM, NT> q;
  Softmax<NM> sm;
  f32x4 acc[NM][DP / 16];
  int first_unseen[NM];
  q.load(a.q, col0, cols, row0, head0);
  sm.init();
#pragma unroll
  for (int i = 0; i < NM; ++i) {
#pragma unroll
    for (int j = 0; j < DP / 16; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    const int col = min(col0 + 16 * i + c, cols - 1);
    first_unseen[i] = len - s.back + fast_div(a.q.by_group, col);
  }
  const int open = s.back ? len - s.back : len;  // keys below it are seen by every query

  int n0 = begin + wave * kStep;
  if (n0 < end) {
    RawKv<DP> cur;
    load_step<DP, UNI>(a, trow, len, n0, h, cur);
    while (true) {
      const int n1 = n0 + NW * kStep;
      const bool more = n1 < end;
      if (cur.bm) {
        int lim[NM];
#pragma unroll
        for (int i = 0; i < NM; ++i) lim[i] = first_unseen[i] - n0;
        step_bf16<DP, NM, NT, NP, false>(
            q, sm, acc, [&](bf16x8(&kf)[2][DP / 32]) { widen_k<DP>(cur, a.q.D, kf); },
            [&](bf16x8(&vf)[DP / 16]) { widen_v<DP>(cur, vf); }, a.q.c, cur.bm,
            s.back && n0 + kStep > open, lim);
      }
      if (!more) break;
      load_step<DP, UNI>(a, trow, len, n1, h, cur);
      n0 = n1;
    }
  }
  join_and_store<DP, NM, NW, TO>(a.q, lds, acc, sm, col0, cols, row0, head0, s.split0 + sp);
}

}  // namespace
