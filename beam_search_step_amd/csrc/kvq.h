// kvq.h -- part of libbeamattn.so, included once by beamattn.hip.
//
// The 8-bit paged cache: q1_write, q2_read, q3_scales.
#pragma once

namespace {

struct KvqPool {
  uint8_t* data[2];    // K, V
  float* scale[2];
  int n_blocks, heads, D;
  FastDiv by_bs;
  int64_t block_stride, pos_stride;
};

struct WriteArgs {
  KvqPool c;
  const void* x[2];    // K, V rows
  int64_t row_stride;  // elements
  const int* slots;
  int n;               // tokens
  int chunk;           // tokens of a workgroup
};

constexpr int kScaleLow = -100;  // the least scale exponent

__device__ __forceinline__ float two_to(int e) { return as_f((uint32_t)(e + 127) << 23); }

// The least e >= -100 with amax <= 448 * 2^e: amax = m 2^E, 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = as_u(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return two_to(max(e, kScaleLow));
}

// Four values as e4m3 bytes, to nearest even; non-finite ones as NaN. |x| is at
// most 448.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d) {
  uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
__device__ __forceinline__ float finite_or_nan(float x) {
  return fabsf(x) < kInf ? x : __builtin_nanf("");
}

// 8 values of a row
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
  Elem<float>::unpack(*reinterpret_cast<const uint4*>(p), x);
  Elem<float>::unpack(*reinterpret_cast<const uint4*>(p + 4), x + 4);
}
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t* p, float (&x)[8]) {
  Elem<uint16_t>::unpack(*reinterpret_cast<const uint4*>(p), x);
}

// Rounds and stores the rows of one run: tokens i0 .. i0 + run - 1 go to
// consecutive positions of one block, whose scale is theirs alone to set. A wave
// takes 64 / (D / 8) rows at a time, 8 values per lane; the rows of the first
// kHeld passes stay in registers between the maximum and the rounding. (K and V
// in one wave, half as many waves: 20.6 us against 15.5 for 8000 tokens of 8
// heads of 128.)
constexpr int kHeld = 4;
template <typename T>
__device__ __forceinline__ void write_run(const WriteArgs& a, int i0, int run, int slot, int h,
                                          int kv) {
  const KvqPool& c = a.c;
  const int lane = threadIdx.x & 63;
  const int lpr = c.D / 8, rpp = 64 / lpr;   // lanes per row, rows per pass
  const int lr = lane / lpr, d = (lane - lr * lpr) * 8;
  const bool on = lr < rpp;
  const int block = fast_div(c.by_bs, slot), off = slot - block * c.by_bs.d;
  uint8_t* base = c.data[kv] + block * c.block_stride + (int64_t)h * c.D + d;
  const T* src = reinterpret_cast<const T*>(a.x[kv]) + i0 * a.row_stride + (int64_t)h * c.D + d;
  float* sp = c.scale[kv] + (int64_t)block * c.heads + h;
  const float old = off > 0 ? *sp : 0.0f;
  float held[kHeld][8];
  uint32_t top = 0;  // of the magnitudes' bits: their order, non-finite ones on top
  auto take = [&](const float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, as_u(x[k]) & 0x7fffffffu);
  };
#pragma unroll
  for (int p = 0; p < kHeld; ++p) {
    const int r = p * rpp + lr;
    if (on && r < run) load8(src + r * a.row_stride, held[p]);
  }
#pragma unroll
  for (int p = 0; p < kHeld; ++p)
    if (on && p * rpp + lr < run) take(held[p]);
  for (int r = kHeld * rpp + lr; on && r < run; r += rpp) {
    float x[8];
    load8(src + r * a.row_stride, x);
    take(x);
  }
  const bool bad = __ballot(top >= 0x7f800000u) != 0;  // rare: once more without them
  if (bad) {
    top = 0;
    for (int r = lr; on && r < run; r += rpp) {
      float x[8];
      load8(src + r * a.row_stride, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t u = as_u(x[k]) & 0x7fffffffu;
        top = max(top, u < 0x7f800000u ? u : 0);
      }
    }
  }
  const float amax = wave_max_f(as_f(top));
  float s = scale_for(amax);
  if (off > 0 && old >= s) s = old;
  const float inv = 1.0f / s;  // a power of two: exact
  if (off > 0 && s != old) {   // the scale grows: the earlier positions are rounded to it
    const float f = old * inv;
    for (int r = lr; on && r < off; r += rpp) {
      uint8_t* q = base + r * c.pos_stride;
      const u32x2 w = *reinterpret_cast<const u32x2*>(q);
      u32x2 y;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f32x2 x0 = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], false);
        const f32x2 x1 = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], true);
        y[k] = to_e4m3(x0.x * f, x0.y * f, x1.x * f, x1.y * f);
      }
      *reinterpret_cast<u32x2*>(q) = y;
    }
  }
  if (lane == 0) *sp = s;
  auto put = [&](int r, const float (&x)[8]) {
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = (bad ? finite_or_nan(x[k]) : x[k]) * inv;
    *reinterpret_cast<u32x2*>(base + (off + r) * c.pos_stride) =
        u32x2{to_e4m3(y[0], y[1], y[2], y[3]), to_e4m3(y[4], y[5], y[6], y[7])};
  };
#pragma unroll
  for (int p = 0; p < kHeld; ++p) {
    const int r = p * rpp + lr;
    if (on && r < run) put(r, held[p]);
  }
  for (int r = kHeld * rpp + lr; on && r < run; r += rpp) {
    float x[8];
    load8(src + r * a.row_stride, x);
    put(r, x);
  }
}

// The block of the nearest token before t0 that has a slot, -1 if there is none.
__device__ __forceinline__ int block_before(const WriteArgs& a, int t0, int limit) {
  const int lane = threadIdx.x & 63;
  for (int e = t0 - 1; e >= 0; e -= 64) {
    const int slot = e - lane >= 0 ? a.slots[e - lane] : -1;
    const uint64_t ok = __ballot(slot >= 0 && slot < limit);
    if (ok) return fast_div(a.c.by_bs, __builtin_amdgcn_readlane(slot, __builtin_ctzll(ok)));
  }
  return -1;
}

// grid (token chunks, heads, K|V). The first token of a block in the list gives the
// block to a wave, which writes all its runs in list order, also those behind the
// chunk. The waves share the chunk's blocks. What bounds it is the chain slots,
// rows, maximum, store, once for each run, then its bytes: 8000 bf16 tokens of 8 heads
// of 128 are 16.3 us, 3.0 TB/s, fp32 ones 20.4 and 4.0.
template <typename T>
__global__ __launch_bounds__(kAttnThreads) void q1_write(WriteArgs a) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.y, kv = blockIdx.z, t0 = blockIdx.x * a.chunk;
  const int bs = a.c.by_bs.d;
  const int limit = a.c.n_blocks * bs;
  int slot = -1;
  const int before = t0 > 0 ? a.slots[t0 - 1] : -1;
  if (lane < a.chunk && t0 + lane < a.n) slot = a.slots[t0 + lane];
  const bool valid = slot >= 0 && slot < limit;
  const uint64_t have = __ballot(valid);
  if (!have) return;
  const int block = valid ? fast_div(a.c.by_bs, slot) : -2;
  const uint64_t below = have & (((uint64_t)1 << lane) - 1);
  int prev = __shfl(block, below ? 63 - __builtin_clzll(below) : 0);
  const int carry = before >= 0 && before < limit ? fast_div(a.c.by_bs, before)
                                                  : block_before(a, t0, limit);
  if (!below) prev = carry;
  // lanes whose slot follows the lane's before
  const int left = __shfl_up(slot, 1);
  const uint64_t follow = __ballot(valid && lane > 0 && left == slot - 1);
  uint64_t todo = __ballot(valid && prev != block);
  for (int k = 0; todo; ++k, todo &= todo - 1) {
    if (k % kAttnWaves != wave) continue;
    const int at = __builtin_ctzll(todo);
    const int blk = __builtin_amdgcn_readlane(block, at);
    int s0 = __builtin_amdgcn_readlane(slot, at), i0 = t0 + at;
    while (true) {
      const int most = min(bs - (s0 - blk * bs), a.n - i0);
      int run = 1;
      const int l = i0 - t0;
      if (l < a.chunk) {  // what the chunk shows of it
        const uint64_t ends = l < 63 ? ~(follow >> (l + 1)) : ~(uint64_t)0;
        run = min(1 + (int)__builtin_ctzll(ends), most);
      }
      if (l + run >= a.chunk) {  // and 64 slots at a time behind it
        while (run < most) {
          const int e = run + lane;
          const bool next = e < most && a.slots[i0 + e] == s0 + e;
          const uint64_t no = ~__ballot(next);
          const int got = no ? __builtin_ctzll(no) : 64;
          run += got;
          if (got < 64) break;
        }
      }
      write_run<T>(a, i0, run, s0, h, kv);
      // the next token with a slot: the same block's next run, or another's
      int found = -1;
      for (i0 += run; i0 < a.n; i0 += 64) {
        const int s = i0 + lane < a.n ? a.slots[i0 + lane] : -1;
        const uint64_t ok = __ballot(s >= 0 && s < limit);
        if (ok) {
          const int l = __builtin_ctzll(ok);
          found = __builtin_amdgcn_readlane(s, l);
          i0 += l;
          break;
        }
      }
      if (found < 0 || fast_div(a.c.by_bs, found) != blk) break;
      s0 = found;
      __threadfence_block();  // the next run reads what this one stored
    }
  }
}

struct ReadArgs {
  KvqPool c;
  void* y[2];
  const int* slots;
  int n;
};

// One thread per 8 values, K and V along the grid's y. Bandwidth: 8000 tokens of 8
// heads of 128 as bf16 are 10.6 us, 4.6 TB/s, as fp32 16.4 and 5.0.
template <typename T>
__global__ __launch_bounds__(kAttnThreads) void q2_read(ReadArgs a) {
  const KvqPool& c = a.c;
  const int per = c.heads * (c.D / 8);
  const int64_t idx = (int64_t)blockIdx.x * kAttnThreads + threadIdx.x;
  const int64_t i = idx / per;
  if (i >= a.n) return;
  const int e = (int)(idx - i * per) * 8, h = e / c.D, kv = blockIdx.y;
  const int slot = a.slots[i];
  float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (slot >= 0 && slot < c.n_blocks * c.by_bs.d) {
    const int block = fast_div(c.by_bs, slot), off = slot - block * c.by_bs.d;
    const u32x2 w = *reinterpret_cast<const u32x2*>(c.data[kv] + block * c.block_stride +
                                                    off * c.pos_stride + e);
    const float s = c.scale[kv][(int64_t)block * c.heads + h];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const f32x2 x0 = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], false);
      const f32x2 x1 = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], true);
      x[4 * k] = x0.x * s;
      x[4 * k + 1] = x0.y * s;
      x[4 * k + 2] = x1.x * s;
      x[4 * k + 3] = x1.y * s;
    }
  }
  T* y = reinterpret_cast<T*>(a.y[kv]) + idx * 8;
  store4(y, f32x4{x[0], x[1], x[2], x[3]});
  store4(y + 4, f32x4{x[4], x[5], x[6], x[7]});
}

// The scales of the step's copies on write: entry f of the list copied block
// cpy[3 f] to block cpy[3 f + 1]; every plane's row of scales follows. A launch's latency:
// 2.3 us a step for 32 layers of 8 items, 4 beams and 8 heads, beside 6.8 of the copies.
constexpr int kScalePlanes = 128;
struct ScaleArgs {
  float* plane[kScalePlanes];
  int n_planes, heads;
  const int* cpy;
  const int* ncpy;
  int parity, max_copies, n_blocks;
};
__global__ __launch_bounds__(kAttnThreads) void q3_scales(ScaleArgs a) {
  const int copies = min(a.ncpy[a.parity], a.max_copies);
  const int64_t all = (int64_t)copies * a.heads;
  float* p = a.plane[blockIdx.y];
  for (int64_t i = (int64_t)blockIdx.x * kAttnThreads + threadIdx.x; i < all;
       i += (int64_t)gridDim.x * kAttnThreads) {
    const int f = (int)(i / a.heads), h = (int)(i - (int64_t)f * a.heads);
    const int src = a.cpy[3 * f], dst = a.cpy[3 * f + 1];
    if ((unsigned)src < (unsigned)a.n_blocks && (unsigned)dst < (unsigned)a.n_blocks)
      p[(int64_t)dst * a.heads + h] = p[(int64_t)src * a.heads + h];
  }
}

}  // namespace
