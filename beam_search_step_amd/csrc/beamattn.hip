// beamattn.hip -- host runtime of libbeamattn.so (gfx950), and the one
// translation unit that includes its kernels.
//
// The operators that fill and read the caches around the beam step:
//
//   m1_map      (map_blocks.h)   block tables and slot maps from lengths
//   q1_write    (kvq.h)          K and V rows into an 8-bit paged cache
//   q2_read     (kvq.h)          the values it holds
//   q3_scales   (kvq.h)          scales of the blocks that a reorder copied
//   a1_cache    (cache_attn.h)   attention over that cache
//   a2_cross    (cross_attn.h)   attention to an encoder's states
//   a3_tile     (cross_tile.h)   the same for many rows, keys shared through LDS
//   a_combine   (attn_common.h)  joins the sums of keys that were split

#include <hip/hip_runtime.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <type_traits>

#include "beamattn.h"

#pragma clang fp contract(off)

#include "device_common.h"
#include "paged_dev.h"
#include "attn_common.h"
#include "map_blocks.h"
#include "kvq.h"
#include "cache_attn.h"
#include "cross_attn.h"
#include "cross_tile.h"

// ===========================================================================
// host runtime
// ===========================================================================

struct bs_cache_attn_state {
  bs_cache_attn_config cfg;
  hipStream_t stream;
  int device;
  int nw;              // waves of a workgroup
  int splits[2];       // workgroups along the keys: of a prompt, of a row
  float* block;        // the partial sums
  float* pml;
  float* pacc;
};

struct bs_cross_attn_state {
  bs_cross_attn_config cfg;
  hipStream_t stream;
  int device;
  int64_t units;       // partials that the workspace holds
  float* block;
  float* pml;
  float* pacc;
};

namespace {

int launch_status() { return hipGetLastError() == hipSuccess ? BS_OK : BS_EDEVICE; }

// The handle's device for the length of a call.
struct OnDevice {
  int before = -1;
  bool ok = true;
  explicit OnDevice(int device) {
    int now = -1;
    ok = hipGetDevice(&now) == hipSuccess;
    if (ok && now != device) {
      ok = hipSetDevice(device) == hipSuccess;
      before = now;
    }
  }
  ~OnDevice() {
    if (before >= 0) (void)hipSetDevice(before);
  }
};

FastDiv make_div(int d) {
  int sh = 0;
  while (((int64_t)1 << sh) < d) ++sh;
  FastDiv f;
  f.d = d;
  f.s = 31 + sh;
  f.m = (uint32_t)((((uint64_t)1 << f.s) + d - 1) / d);
  return f;
}

bool aligned(const void* p, int n) { return ((uintptr_t)p % n) == 0; }
bool dtype_ok(int t) { return t == BS_F32 || t == BS_BF16; }
int elem_size(int t) { return t == BS_F32 ? 4 : 2; }
bool head_dim_ok(int d) { return d >= 16 && d <= 256 && d % 16 == 0; }
// as a normal fp32 number, log2(e) times it too: a zero would make NaN of the -inf of
// a key that is not seen
bool scale_ok(double s) { return s >= 1e-37 && s < 1e30; }

constexpr int64_t kMaxPosStride = (int64_t)1 << 26;   // lane offsets of a step stay below 2^31
constexpr int64_t kTilePosStride = (int64_t)1 << 24;  // and those of a3_tile's 128 keys
constexpr int64_t kMaxTokens = 0x7fe00000;  // counters run up to 2^20 past the last token
constexpr int64_t kMaxGridX = 0xFFFFFFFFll / kAttnThreads;
bool grid_ok(int64_t groups, int threads) { return groups * threads <= 0xFFFFFFFFll; }

bool kvq_ok(const bs_kvq_desc* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return false;
  if (c->n_blocks < 1 || c->block_size < 1 || c->kv_heads < 1 || c->kv_heads > 65535) return false;
  if ((int64_t)c->n_blocks * c->block_size >= ((int64_t)1 << 31)) return false;
  if (!head_dim_ok(c->head_dim)) return false;
  const int64_t row = (int64_t)c->kv_heads * c->head_dim;
  if (c->pos_stride < row || c->pos_stride % 16 || c->pos_stride >= kMaxPosStride) return false;
  if (c->block_stride < (int64_t)(c->block_size - 1) * c->pos_stride + row ||
      c->block_stride % 16 || c->block_stride >= ((int64_t)1 << 40))
    return false;
  return aligned(c->k, 16) && aligned(c->v, 16) && aligned(c->k_scale, 4) && aligned(c->v_scale, 4);
}

KvqPool kvq_pool(const bs_kvq_desc* c) {
  KvqPool p;
  p.data[0] = (uint8_t*)c->k;
  p.data[1] = (uint8_t*)c->v;
  p.scale[0] = c->k_scale;
  p.scale[1] = c->v_scale;
  p.n_blocks = c->n_blocks;
  p.heads = c->kv_heads;
  p.D = c->head_dim;
  p.by_bs = make_div(c->block_size);
  p.block_stride = c->block_stride;
  p.pos_stride = c->pos_stride;
  return p;
}

// Workgroups along the keys: enough for kWantGroups in the launch, each with
// kMinKeys at least.
constexpr int kWantGroups = 768;
constexpr int kMinKeys = 256;
int choose_splits(int64_t groups, int64_t keys, int most) {
  int64_t s = (kWantGroups + groups - 1) / groups;
  // chunks of more than 2048 keys: a third more of them, so that the last
  // workgroups of ragged lengths are not late (8 prompts of 16,000 to 48,000
  // tokens: 131 us and 6 of the joining launch, against 134 and 5)
  if (keys > 2048 * s) s = (kWantGroups + kWantGroups / 3 + groups - 1) / groups;
  const int64_t by_keys = (keys + kMinKeys - 1) / kMinKeys;
  if (s > by_keys) s = by_keys;
  if (s > most) s = most;
  return s < 1 ? 1 : (int)s;
}

// Waves of a workgroup, for the kernels of one column tile. One where units are
// short and so many that a wave each fills the device (the wide search's 16 beams
// of 16 heads over 128 positions: 31 us, with four waves 34). Eight where there are
// units enough to go without partial sums and the launch that joins them: 64
// sequences of 8 heads and 500 keys, 16.0 us against 19.7; 1000-key fp32 sources of
// 16 by 16 heads, 39.7 against 40.2, 1500-key bf16 ones 26.5 against 26.4. Four else.
// Measured up to 2000 keys: far longer ragged ones would wait for their last workgroup.
int choose_waves(int64_t pairs, int64_t keys, bool one_kind) {
  if (pairs >= 2048 && keys <= 512) return 1;
  return one_kind && pairs >= 256 && keys > 256 ? 8 : 4;
}

int pad_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

// The most 16-column tiles of a wave of a2_cross. Two where keys are worth reading
// once for both and registers hold them without spilling: 32 columns of 14 items, 8 kv
// heads of 64 and 1403 bf16 keys are 15.1 us, one tile at a time 16.4; 4096 columns of 2
// items, 8 kv heads of 64 and 512 fp32 keys 108 us against 151.
template <int DP, typename T>
constexpr int cross_most() {
  return sizeof(T) == 2 ? (DP == 64 ? 2 : 1) : DP <= 128 ? 2 : 1;
}
// The tiles of a call, never more than that. fp32 heads of 128: 56 columns of 14 items
// and 1403 keys are 88 us one tile at a time and 119 with two, 4096 columns of 2 items and
// 512 keys 295 and 237
int cross_tiles(int64_t cols, int dp, int dtype) {
  if (cols <= 16 || (dtype == BS_F32 && dp == 128 && cols <= 64)) return 1;
  if (dtype == BS_F32)
    return dp == 64 ? cross_most<64, float>() : dp == 128 ? cross_most<128, float>()
                                                           : cross_most<256, float>();
  return dp == 64 ? cross_most<64, uint16_t>() : dp == 128 ? cross_most<128, uint16_t>()
                                                            : cross_most<256, uint16_t>();
}

QueryArgs query_args(const void* q, int64_t q_stride, int heads, int kv_heads, int D, double scale,
                     void* out) {
  QueryArgs a;
  a.q = q;
  a.q_stride = q_stride;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.D = D;
  a.by_group = make_div(a.group);
  a.c = (float)(scale * 1.4426950408889634074);
  a.out = out;
  a.pacc = a.pml = nullptr;
  a.ns = 1;
  return a;
}

int launch_combine(const QueryArgs& q, int64_t units, int dtype, hipStream_t s) {
  CombineArgs c;
  c.pacc = q.pacc;
  c.pml = q.pml;
  c.out = q.out;
  c.units = units;
  c.ns = q.ns;
  c.D = q.D;
  const int lpu = q.D <= 64 ? 16 : q.D <= 128 ? 32 : 64;  // four values a lane
  const int per = kAttnThreads / lpu;
  const dim3 grid((unsigned)((units + per - 1) / per)), blk(kAttnThreads);
  if (dtype == BS_F32) {
    if (lpu == 16) hipLaunchKernelGGL((a_combine<float, 16>), grid, blk, 0, s, c);
    else if (lpu == 32) hipLaunchKernelGGL((a_combine<float, 32>), grid, blk, 0, s, c);
    else hipLaunchKernelGGL((a_combine<float, 64>), grid, blk, 0, s, c);
  } else {
    if (lpu == 16) hipLaunchKernelGGL((a_combine<uint16_t, 16>), grid, blk, 0, s, c);
    else if (lpu == 32) hipLaunchKernelGGL((a_combine<uint16_t, 32>), grid, blk, 0, s, c);
    else hipLaunchKernelGGL((a_combine<uint16_t, 64>), grid, blk, 0, s, c);
  }
  return launch_status();
}

template <int DP, int NT>
void launch_cache_u(const CacheArgs& a, int nw, dim3 grid, hipStream_t s) {
  if (a.bs % 16) {
    hipLaunchKernelGGL((a1_cache<DP, 4, NT, false>), grid, dim3(256), 0, s, a);
    return;
  }
  if constexpr (DP < 256) {
    if (nw == 1) {
      hipLaunchKernelGGL((a1_cache<DP, 1, NT, true>), grid, dim3(64), 0, s, a);
      return;
    }
    if (nw == 8) {
      hipLaunchKernelGGL((a1_cache<DP, 8, NT, true>), grid, dim3(512), 0, s, a);
      return;
    }
  }
  hipLaunchKernelGGL((a1_cache<DP, 4, NT, true>), grid, dim3(256), 0, s, a);
}
void launch_cache(const CacheArgs& a, int dtype, int nw, dim3 grid, hipStream_t s) {
  const int dp = pad_dim(a.q.D);
  if (dtype == BS_BF16) {
    if (dp == 64) launch_cache_u<64, 1>(a, nw, grid, s);
    else if (dp == 128) launch_cache_u<128, 1>(a, nw, grid, s);
    else launch_cache_u<256, 1>(a, nw, grid, s);
  } else {
    if (dp == 64) launch_cache_u<64, 3>(a, nw, grid, s);
    else if (dp == 128) launch_cache_u<128, 3>(a, nw, grid, s);
    else launch_cache_u<256, 3>(a, nw, grid, s);
  }
}

template <int DP, int NM, typename T>
void launch_cross_w(const CrossArgs& a, int nw, dim3 grid, hipStream_t s) {
  if constexpr (NM == 1 && DP < 256) {
    if (nw == 1) {
      hipLaunchKernelGGL((a2_cross<DP, NM, 1, T>), grid, dim3(64), 0, s, a);
      return;
    }
    if (nw == 8) {
      hipLaunchKernelGGL((a2_cross<DP, NM, 8, T>), grid, dim3(512), 0, s, a);
      return;
    }
  }
  hipLaunchKernelGGL((a2_cross<DP, NM, 4, T>), grid, dim3(256), 0, s, a);
}
template <int DP, typename T>
void launch_cross_n(const CrossArgs& a, int nm, int nw, dim3 grid, hipStream_t s) {
  constexpr int MOST = cross_most<DP, T>();
  if constexpr (MOST >= 2)
    if (nm == 2) return launch_cross_w<DP, 2, T>(a, nw, grid, s);
  launch_cross_w<DP, 1, T>(a, nw, grid, s);
}
void launch_cross(const CrossArgs& a, int dtype, int nm, int nw, dim3 grid, hipStream_t s) {
  const int dp = pad_dim(a.q.D);
  if (dtype == BS_BF16) {
    if (dp == 64) launch_cross_n<64, uint16_t>(a, nm, nw, grid, s);
    else if (dp == 128) launch_cross_n<128, uint16_t>(a, nm, nw, grid, s);
    else launch_cross_n<256, uint16_t>(a, nm, nw, grid, s);
  } else {
    if (dp == 64) launch_cross_n<64, float>(a, nm, nw, grid, s);
    else if (dp == 128) launch_cross_n<128, float>(a, nm, nw, grid, s);
    else launch_cross_n<256, float>(a, nm, nw, grid, s);
  }
}

// bf16: more columns than this share keys through LDS (a3_tile). Of 14 items, 8 kv heads
// and 1403 keys, with the launch that joins split sums where there is one, streamed and
// tiled: 64 values 64 columns 24 and 25 us, 80 columns 27 and 26, 128 columns 32 and 29; 128
// values 32 columns 33 and 34, 40 columns 40 and 35; 256 values 40 columns 76 and 80, 56
// columns 93 and 85. Of 64 items and 600 keys: 64 values 64 columns 31 and 41, 128 columns
// 50 and 34; 128 values 32 columns 63 and 59, 64 columns 99 and 67.
int tile_cols(int dp) { return dp == 64 ? 64 : dp == 128 ? 32 : 48; }
// Waves of 32 columns in its workgroup. Eight, which bring a tile in for twice the
// columns, where they are a workgroup for every CU at least (8 x 1024 rows over 2048
// keys, 32 heads of 128: 431 us against 448); heads of 256 leave registers for four.
int tile_waves(int64_t pairs, int64_t cols, int dp) {
  return dp <= 128 && cols > 128 && pairs * ((cols + 255) / 256) >= 256 ? 8 : 4;
}
void launch_tile(const CrossArgs& a, int nw, dim3 grid, hipStream_t s) {
  const int dp = pad_dim(a.q.D);
  const dim3 blk(64 * nw);
  if (dp == 64) {
    if (nw == 8) hipLaunchKernelGGL((a3_tile<64, 8>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((a3_tile<64, 4>), grid, blk, 0, s, a);
  } else if (dp == 128) {
    if (nw == 8) hipLaunchKernelGGL((a3_tile<128, 8>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((a3_tile<128, 4>), grid, blk, 0, s, a);
  } else {
    hipLaunchKernelGGL((a3_tile<256, 4>), grid, blk, 0, s, a);
  }
}

// one allocation: the maxima and sums, then the partial sums
int alloc_partials(int64_t units, int D, float** block, float** pml, float** pacc) {
  const int64_t ml = (units * 2 + 63) / 64 * 64;
  if (hipMalloc((void**)block, (size_t)(ml + units * D) * 4) != hipSuccess) {
    (void)hipGetLastError();
    return BS_ENOMEM;
  }
  *pml = *block;
  *pacc = *block + ml;
  return BS_OK;
}

}  // namespace

extern "C" {

int bs_map_blocks(void* hip_stream, int32_t n, int32_t block_size, int32_t max_blocks,
                  const int32_t* starts, const int32_t* lens, const int32_t* free_blocks,
                  int32_t n_free, int32_t* table, int32_t* cu, int32_t* slots,
                  int32_t max_tokens, int32_t* used) {
  if (n < 1 || n > 65535 || block_size < 1 || max_blocks < 1 || n_free < 0 || max_tokens < 0)
    return BS_EINVAL;
  if ((int64_t)block_size * max_blocks > kMaxTokens || max_tokens > kMaxTokens) return BS_EINVAL;
  if (!lens || !table || !cu || !used || (max_tokens > 0 && !slots)) return BS_EINVAL;
  if (n_free > 0 && !free_blocks) return BS_EINVAL;
  MapArgs a;
  a.n = n;
  a.mb = max_blocks;
  a.n_free = n_free;
  a.max_tokens = max_tokens;
  a.by_bs = make_div(block_size);
  a.starts = starts;
  a.lens = lens;
  a.freel = free_blocks;
  a.table = table;
  a.cu = cu;
  a.slots = slots;
  a.used = used;
  // four requests or more to a workgroup, one to a wave at a time, of 512 tokens
  // or more each
  a.per = (n + 1023) / 1024;
  a.per = a.per < kAttnWaves ? kAttnWaves : a.per;
  a.chunks = (n + a.per - 1) / a.per;
  const int tails = max_tokens > 0 ? 1 : 0;
  a.shift = (block_size & (block_size - 1)) == 0 ? __builtin_ctz(block_size) : -1;
  const int64_t parts = max_tokens / ((int64_t)n * 512);
  const int most = 2048 / a.chunks;
  a.parts = parts < 1 ? 1 : parts > most ? most : (int)parts;
  hipLaunchKernelGGL(m1_map, dim3(a.chunks + tails, a.parts), dim3(kAttnThreads), 0,
                     (hipStream_t)hip_stream, a);
  return launch_status();
}

int bs_kvq_write(void* hip_stream, const bs_kvq_desc* cache, int32_t dtype, const void* k,
                 const void* v, int64_t row_stride, const int32_t* slots, int32_t n_tokens) {
  if (!kvq_ok(cache) || !dtype_ok(dtype) || n_tokens < 0 || n_tokens > kMaxTokens)
    return BS_EINVAL;
  if (n_tokens == 0) return BS_OK;
  if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16)) return BS_EINVAL;
  if (row_stride < (int64_t)cache->kv_heads * cache->head_dim ||
      (row_stride * elem_size(dtype)) % 16 || row_stride >= ((int64_t)1 << 40))
    return BS_EINVAL;
  WriteArgs a;
  a.c = kvq_pool(cache);
  a.x[0] = k;
  a.x[1] = v;
  a.row_stride = row_stride;
  a.slots = slots;
  a.n = n_tokens;
  // few tokens: a wave for each; many: chunks of 64
  a.chunk = (int64_t)n_tokens * cache->kv_heads <= 8192 ? kAttnWaves : 64;
  const dim3 grid((n_tokens + a.chunk - 1) / a.chunk, cache->kv_heads, 2);
  if (grid.x > kMaxGridX) return BS_EINVAL;
  if (dtype == BS_F32)
    hipLaunchKernelGGL(q1_write<float>, grid, dim3(kAttnThreads), 0, (hipStream_t)hip_stream, a);
  else
    hipLaunchKernelGGL(q1_write<uint16_t>, grid, dim3(kAttnThreads), 0, (hipStream_t)hip_stream,
                       a);
  return launch_status();
}

int bs_kvq_read(void* hip_stream, const bs_kvq_desc* cache, int32_t dtype, const int32_t* slots,
                int32_t n_slots, void* k, void* v) {
  if (!kvq_ok(cache) || !dtype_ok(dtype) || n_slots < 0) return BS_EINVAL;
  if (n_slots == 0) return BS_OK;
  if (!slots || !k || !v || !aligned(k, 16) || !aligned(v, 16)) return BS_EINVAL;
  const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
  const int64_t most = kMaxGridX / 2 * kAttnThreads / (row / 8);  // slots of a launch
  for (int64_t i = 0; i < n_slots; i += most) {
    ReadArgs a;
    a.c = kvq_pool(cache);
    a.y[0] = (char*)k + i * row * elem_size(dtype);
    a.y[1] = (char*)v + i * row * elem_size(dtype);
    a.slots = slots + i;
    a.n = (int)(n_slots - i < most ? n_slots - i : most);
    const dim3 grid((unsigned)((a.n * (row / 8) + kAttnThreads - 1) / kAttnThreads), 2);
    if (dtype == BS_F32)
      hipLaunchKernelGGL(q2_read<float>, grid, dim3(kAttnThreads), 0, (hipStream_t)hip_stream, a);
    else
      hipLaunchKernelGGL(q2_read<uint16_t>, grid, dim3(kAttnThreads), 0, (hipStream_t)hip_stream,
                         a);
    const int rc = launch_status();
    if (rc != BS_OK) return rc;
  }
  return BS_OK;
}

int bs_kvq_reorder(bs_kv_paged* p, const bs_kvq_desc* layers, int32_t n_layers, int32_t gen_len) {
  if (!p || !layers || n_layers < 1 || n_layers > (1 << 20)) return BS_EINVAL;
  const bs_kvq_desc& c = layers[0];
  for (int i = 0; i < n_layers; ++i) {
    const bs_kvq_desc& d = layers[i];
    if (!kvq_ok(&d) || d.block_size != p->bs || d.n_blocks < p->blocks) return BS_EINVAL;
    if (d.n_blocks != c.n_blocks || d.kv_heads != c.kv_heads || d.head_dim != c.head_dim ||
        d.block_stride != c.block_stride || d.pos_stride != c.pos_stride)
      return BS_EINVAL;
  }
  void** planes = (void**)malloc(sizeof(void*) * 2 * n_layers);
  if (!planes) return BS_ENOMEM;
  for (int i = 0; i < n_layers; ++i) {
    planes[2 * i] = layers[i].k;
    planes[2 * i + 1] = layers[i].v;
  }
  bs_kv_pool pool;
  pool.n_planes = 2 * n_layers;
  pool.pools = planes;
  pool.block_stride = c.block_stride;
  pool.pos_stride = c.pos_stride;
  pool.bytes_per_pos = (int64_t)c.kv_heads * c.head_dim;
  OnDevice on(p->device);
  int rc = on.ok ? bs_kv_paged_reorder(p, &pool, gen_len) : BS_EDEVICE;
  free(planes);
  if (rc != BS_OK) return rc;
  ScaleArgs a;
  a.heads = c.kv_heads;
  a.cpy = p->pg.cpy;
  a.ncpy = p->pg.ncpy;
  a.parity = gen_len & 1;
  a.max_copies = p->rows;
  a.n_blocks = c.n_blocks;
  const int64_t most = (int64_t)p->rows * c.kv_heads;
  const int x = (int)((most + kAttnThreads - 1) / kAttnThreads);
  for (int i0 = 0; i0 < n_layers; i0 += kScalePlanes / 2) {
    const int m = n_layers - i0 < kScalePlanes / 2 ? n_layers - i0 : kScalePlanes / 2;
    a.n_planes = 2 * m;
    for (int i = 0; i < m; ++i) {
      a.plane[2 * i] = layers[i0 + i].k_scale;
      a.plane[2 * i + 1] = layers[i0 + i].v_scale;
    }
    hipLaunchKernelGGL(q3_scales, dim3(x < 16 ? x : 16, a.n_planes), dim3(kAttnThreads), 0,
                       p->stream, a);
    rc = launch_status();
    if (rc != BS_OK) return rc;
  }
  return BS_OK;
}

int bs_cache_attn_create(const bs_cache_attn_config* cfg, void* hip_stream,
                         bs_cache_attn_state** out) {
  if (!out) return BS_EINVAL;
  *out = nullptr;
  if (!cfg) return BS_EINVAL;
  const bs_cache_attn_config& c = *cfg;
  if (c.batch < 1 || c.rows < 1 || c.q_len < 1 || c.q_len > 64 || c.batch > 65535 ||
      c.rows > 65535 || (int64_t)c.batch * c.rows * c.q_len > 65535)
    return BS_EINVAL;
  if (c.kv_heads < 1 || c.heads < 1 || c.heads > 65535 || c.heads % c.kv_heads) return BS_EINVAL;
  if (!head_dim_ok(c.head_dim) || !dtype_ok(c.dtype) || !scale_ok(c.scale)) return BS_EINVAL;
  if (c.block_size < 1 || c.max_blocks < 1 || c.max_prompt_blocks < 0 ||
      (int64_t)c.block_size * c.max_blocks >= ((int64_t)1 << 30) ||
      (int64_t)c.block_size * c.max_prompt_blocks >= ((int64_t)1 << 30))
    return BS_EINVAL;
  const int group = c.heads / c.kv_heads;
  const int64_t pg = ((int64_t)c.rows * c.q_len * group + 15) / 16;
  const int64_t rg = ((int64_t)c.q_len * group + 15) / 16;
  const int64_t pw = (int64_t)c.batch * c.kv_heads * pg;
  const int64_t rw = (int64_t)c.batch * c.rows * c.kv_heads * rg;
  const int64_t pk = (int64_t)c.max_prompt_blocks * c.block_size;
  const int64_t rk = (int64_t)c.max_blocks * c.block_size;
  const bool uniform = c.block_size % 16 == 0 && c.head_dim <= 128;
  const int nw = uniform ? choose_waves(rw, pk > rk ? pk : rk, !c.max_prompt_blocks) : 4;
  const int sp = !c.max_prompt_blocks ? 0 : nw == 4 ? choose_splits(pw, pk, kMaxSplits / 2) : 1;
  const int sr = nw == 4 ? choose_splits(rw, rk, kMaxSplits / 2) : 1;
  const int64_t units = (int64_t)c.batch * c.rows * c.q_len * c.heads;
  if (!grid_ok(pw * sp + rw * sr, 64 * nw) || units > kMaxGridX * 4) return BS_EINVAL;
  bs_cache_attn_state* h = (bs_cache_attn_state*)calloc(1, sizeof(bs_cache_attn_state));
  if (!h) return BS_ENOMEM;
  h->cfg = c;
  h->stream = (hipStream_t)hip_stream;
  h->nw = nw;
  h->splits[0] = sp;
  h->splits[1] = sr;
  if (hipGetDevice(&h->device) != hipSuccess) {
    free(h);
    return BS_EDEVICE;
  }
  if (sp + sr > 1) {
    const int rc = alloc_partials(units * (sp + sr), c.head_dim, &h->block, &h->pml, &h->pacc);
    if (rc != BS_OK) {
      free(h);
      return rc;
    }
  }
  *out = h;
  return BS_OK;
}

int bs_cache_attn(bs_cache_attn_state* h, const bs_kvq_desc* cache, const void* q,
                  int64_t q_stride, const int32_t* table, int32_t table_stride,
                  const int32_t* lens, const int32_t* prompt_table, const int32_t* prompt_lens,
                  void* out) {
  if (!h || !kvq_ok(cache) || !q || !table || !lens || !out) return BS_EINVAL;
  const bs_cache_attn_config& c = h->cfg;
  if (cache->block_size != c.block_size || cache->kv_heads != c.kv_heads ||
      cache->head_dim != c.head_dim || table_stride < c.max_blocks)
    return BS_EINVAL;
  if (q_stride < (int64_t)c.heads * c.head_dim || (q_stride * elem_size(c.dtype)) % 16 ||
      q_stride >= ((int64_t)1 << 40) || !aligned(q, 16) || !aligned(out, 16))
    return BS_EINVAL;
  if (!prompt_table != !prompt_lens || (prompt_table && !c.max_prompt_blocks)) return BS_EINVAL;
  OnDevice on(h->device);
  if (!on.ok) return BS_EDEVICE;
  CacheArgs a;
  a.q = query_args(q, q_stride, c.heads, c.kv_heads, c.head_dim, c.scale, out);
  a.k = (const uint8_t*)cache->k;
  a.v = (const uint8_t*)cache->v;
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.block_stride = cache->block_stride;
  a.pos_stride = (int)cache->pos_stride;
  a.n_blocks = cache->n_blocks;
  a.bs = cache->block_size;
  a.by_bs = make_div(cache->block_size);
  const int sp = prompt_table ? h->splits[0] : 0, sr = h->splits[1];
  PagedSeg& p = a.seg[0];
  p.table = prompt_table;
  p.table_stride = c.max_prompt_blocks;
  p.lens = prompt_lens;
  p.mb = c.max_prompt_blocks;
  p.qrows = c.rows * c.q_len;
  p.back = 0;
  p.splits = sp;
  p.split0 = 0;
  p.groups = (int)(((int64_t)p.qrows * a.q.group + 15) / 16);
  p.blocks = c.batch * c.kv_heads * p.groups * sp;
  PagedSeg& r = a.seg[1];
  r.table = table;
  r.table_stride = table_stride;
  r.lens = lens;
  r.mb = c.max_blocks;
  r.qrows = c.q_len;
  r.back = c.q_len - 1;
  r.splits = sr;
  r.split0 = sp;
  r.groups = (c.q_len * a.q.group + 15) / 16;
  r.blocks = c.batch * c.rows * c.kv_heads * r.groups * sr;
  a.q.ns = sp + sr;
  a.q.pml = h->pml;
  a.q.pacc = h->pacc;
  launch_cache(a, c.dtype, h->nw, dim3(p.blocks + r.blocks), h->stream);
  int rc = launch_status();
  if (rc == BS_OK && a.q.ns > 1)
    rc = launch_combine(a.q, (int64_t)c.batch * c.rows * c.q_len * c.heads, c.dtype, h->stream);
  return rc;
}

void bs_cache_attn_destroy(bs_cache_attn_state* h) {
  if (!h) return;
  OnDevice on(h->device);
  (void)hipStreamSynchronize(h->stream);
  if (h->block) (void)hipFree(h->block);
  free(h);
}

int bs_cross_attn_create(const bs_cross_attn_config* cfg, void* hip_stream,
                         bs_cross_attn_state** out) {
  if (!out) return BS_EINVAL;
  *out = nullptr;
  if (!cfg) return BS_EINVAL;
  const bs_cross_attn_config& c = *cfg;
  if (c.batch < 1 || c.max_rows < 1 || c.kv_heads < 1 || c.heads < 1 || c.heads % c.kv_heads)
    return BS_EINVAL;
  if ((int64_t)c.batch * c.kv_heads > 65535 || c.max_keys < 1 || c.max_keys >= (1 << 30))
    return BS_EINVAL;
  if (c.heads > 65535 || (int64_t)c.batch * c.max_rows >= ((int64_t)1 << 26) ||
      (int64_t)c.batch * c.max_rows * c.heads >= ((int64_t)1 << 26))
    return BS_EINVAL;
  if (!head_dim_ok(c.head_dim) || !dtype_ok(c.dtype) || !scale_ok(c.scale)) return BS_EINVAL;
  bs_cross_attn_state* h = (bs_cross_attn_state*)calloc(1, sizeof(bs_cross_attn_state));
  if (!h) return BS_ENOMEM;
  h->cfg = c;
  h->stream = (hipStream_t)hip_stream;
  if (hipGetDevice(&h->device) != hipSuccess) {
    free(h);
    return BS_EDEVICE;
  }
  // The partials that a call may use: every query and head in kMaxSplits, but at most
  // 98,304 of them (50 MB at 128 values). A call of more than half as many queries and
  // heads is not split, and one between gets the splits that fit, fewer than
  // choose_splits may ask for.
  const int64_t all = (int64_t)c.batch * c.max_rows * c.heads * kMaxSplits;
  const int64_t want = (int64_t)kWantGroups * 128;
  h->units = all < want ? all : want;
  const int rc = alloc_partials(h->units, c.head_dim, &h->block, &h->pml, &h->pacc);
  if (rc != BS_OK) {
    free(h);
    return rc;
  }
  *out = h;
  return BS_OK;
}

int bs_cross_attn(bs_cross_attn_state* h, const void* q, int64_t q_stride, int32_t n_rows,
                  const bs_cross_kv* kv, int32_t n_keys, const int32_t* lens,
                  const uint8_t* mask, int64_t mask_stride, void* out) {
  if (!h || !kv) return BS_EINVAL;
  const bs_cross_attn_config& c = h->cfg;
  if (n_rows < 0 || n_rows > c.max_rows || n_keys < 0 || n_keys > c.max_keys) return BS_EINVAL;
  if (n_rows == 0) return BS_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16)) return BS_EINVAL;
  if (n_keys > 0 && (!kv->k || !kv->v || !aligned(kv->k, 16) || !aligned(kv->v, 16)))
    return BS_EINVAL;
  if (mask && mask_stride < n_keys) return BS_EINVAL;
  const int es = elem_size(c.dtype);
  const int64_t big = (int64_t)1 << 40;
  if (q_stride < (int64_t)c.heads * c.head_dim || (q_stride * es) % 16 || q_stride >= big)
    return BS_EINVAL;
  const int64_t st[3] = {kv->batch_stride, kv->pos_stride, kv->head_stride};
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] >= big || (st[i] * es) % 16) return BS_EINVAL;
  if (kv->pos_stride * es >= kMaxPosStride) return BS_EINVAL;
  OnDevice on(h->device);
  if (!on.ok) return BS_EDEVICE;
  CrossArgs a;
  a.q = query_args(q, q_stride, c.heads, c.kv_heads, c.head_dim, c.scale, out);
  a.k = (const char*)kv->k;
  a.v = (const char*)kv->v;
  a.batch_stride = kv->batch_stride * es;
  a.head_stride = kv->head_stride * es;
  a.pos_stride = (int)(kv->pos_stride * es);
  a.n_rows = n_rows;
  a.n_keys = n_keys;
  a.lens = lens;
  a.mask = mask;
  a.mask_stride = mask_stride;
  const int64_t cols = (int64_t)n_rows * a.q.group;
  const int nm = cross_tiles(cols, pad_dim(c.head_dim), c.dtype);
  const bool tile = c.dtype == BS_BF16 && cols > tile_cols(pad_dim(c.head_dim)) &&
                    a.pos_stride < kTilePosStride;
  a.pairs = c.batch * c.kv_heads;
  const int tw = tile_waves(a.pairs, cols, pad_dim(c.head_dim));
  const int per = tile ? 32 * tw : 16 * nm;
  a.groups = (int)((cols + per - 1) / per);
  const int64_t units = (int64_t)c.batch * n_rows * c.heads;
  const int64_t wg = (int64_t)(tile ? (a.pairs + 7) / 8 * 8 : a.pairs) * a.groups;
  const int nw = nm == 1 && c.head_dim <= 128 && !tile ? choose_waves(wg, n_keys, true) : 4;
  a.splits = nw == 4 ? choose_splits(wg, n_keys, kMaxSplits) : 1;
  if (a.splits > 1 && units * a.splits > h->units) {
    a.splits = (int)(h->units / units);
    if (a.splits < 1) a.splits = 1;
  }
  if (!grid_ok(wg * a.splits, tile ? 64 * tw : 64 * nw)) return BS_EINVAL;
  a.q.ns = a.splits;
  a.q.pml = h->pml;
  a.q.pacc = h->pacc;
  const dim3 grid((unsigned)(wg * a.splits));
  if (tile)
    launch_tile(a, tw, grid, h->stream);
  else
    launch_cross(a, c.dtype, nm, nw, grid, h->stream);
  int rc = launch_status();
  if (rc == BS_OK && a.splits > 1) rc = launch_combine(a.q, units, c.dtype, h->stream);
  return rc;
}

void bs_cross_attn_destroy(bs_cross_attn_state* h) {
  if (!h) return;
  OnDevice on(h->device);
  (void)hipStreamSynchronize(h->stream);
  if (h->block) (void)hipFree(h->block);
  free(h);
}

}  // extern "C"
