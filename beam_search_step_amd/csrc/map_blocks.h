// map_blocks.h -- part of libbeamattn.so, included once by beamattn.hip.
//
// Block tables and slot maps from request lengths: m1_map.
#pragma once

namespace {

struct MapArgs {
  int n, mb, n_free, max_tokens;
  FastDiv by_bs;
  int shift;           // log2 of the block size, -1 where it is no power of two
  const int* starts;   // or null
  const int* lens;
  const int* freel;    // or null
  int* table;
  int* cu;
  int* slots;
  int* used;
  int per;             // requests of a workgroup, up to 64
  int chunks;          // workgroups along the requests; the one behind fills the slots' end
  int parts;           // workgroups along a request's tokens
};

struct MapReq {
  int start, len, have, want;
};
__device__ __forceinline__ MapReq map_request(const MapArgs& a, int start, int len) {
  MapReq r;
  r.start = max(start, 0);
  r.len = max(len, 0);
  const int end = r.start + r.len;
  // ceil(n / bs) as (n - 1) / bs + 1, -1 >> shift being -1
  if (a.shift >= 0) {
    r.have = min(((r.start - 1) >> a.shift) + 1, a.mb);
    r.want = max(min(((end - 1) >> a.shift) + 1, a.mb), r.have);
  } else {
    r.have = r.start > 0 ? min(fast_div(a.by_bs, r.start - 1) + 1, a.mb) : 0;
    r.want = end > 0 ? max(min(fast_div(a.by_bs, end - 1) + 1, a.mb), r.have) : r.have;
  }
  return r;
}

// Sums of the lengths and of the blocks taken over requests [0, to): uniform.
__device__ __forceinline__ void map_prefix(const MapArgs& a, int to, int& len, int& taken) {
  __shared__ int part[2][kAttnWaves];
  int l = 0, t = 0;
  for (int b0 = threadIdx.x; b0 < to; b0 += 8 * kAttnThreads) {  // eight in flight
    int st[8], ln[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int b = min(b0 + j * kAttnThreads, to - 1);
      ln[j] = a.lens[b];
      st[j] = a.starts ? a.starts[b] : 0;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (b0 + j * kAttnThreads >= to) continue;
      const MapReq r = map_request(a, st[j], ln[j]);
      l += r.len;
      t += r.want - r.have;
    }
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    l += __shfl_xor(l, s);
    t += __shfl_xor(t, s);
  }
  if ((threadIdx.x & 63) == 0) {
    part[0][threadIdx.x >> 6] = l;
    part[1][threadIdx.x >> 6] = t;
  }
  __syncthreads();
  len = part[0][0] + part[0][1] + part[0][2] + part[0][3];
  taken = part[1][0] + part[1][1] + part[1][2] + part[1][3];
  __syncthreads();
}

// Inclusive sum over the lanes of a wave: within rows of 16, then across them.
__device__ __forceinline__ int scan_add(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}

// id * bs + off, -1 where there is no block or no int32 holds it: with id at most
// 2^31 / bs the sum stays below 2^32.
__device__ __forceinline__ int slot_of(int id, int off, int bs, unsigned most_id) {
  const int s = (int)((unsigned)id * (unsigned)bs + (unsigned)off);
  return (unsigned)id <= most_id && s >= 0 ? s : -1;
}

// One launch: a workgroup sums the requests before its own; its waves then take
// its requests in turn, lane l holding request l, and write their table rows and
// slots. Few divisions, which is what it spent its time on: with one or two for
// each token and each request summed, 4096 requests of 1000 tokens took 18.4 us, now
// 12.0; 32 requests of one token 4.1, little more than a launch.
__global__ __launch_bounds__(kAttnThreads) void m1_map(MapArgs a) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int base, taken;
  if ((int)blockIdx.x >= a.chunks) {  // padding behind the last token
    map_prefix(a, a.n, base, taken);
    const int64_t step = (int64_t)gridDim.y * kAttnThreads;
    for (int64_t i = (int64_t)max(base, 0) + blockIdx.y * kAttnThreads + tid; i < a.max_tokens;
         i += step)
      a.slots[i] = -1;
    return;
  }
  const int b0 = blockIdx.x * a.per, mine = min(a.per, a.n - b0);
  const int part = blockIdx.y, bs = a.by_bs.d;
  const unsigned most_id = 0x80000000u / (unsigned)bs;
  MapReq r = {0, 0, 0, 0};
  if (lane < mine) r = map_request(a, a.starts ? a.starts[b0 + lane] : 0, a.lens[b0 + lane]);
  map_prefix(a, b0, base, taken);
  const int len_to = scan_add(r.len), took_to = scan_add(a.freel ? r.want - r.have : 0);
  if (part == 0 && wave == 0) {
    if (lane < mine) a.cu[b0 + lane] = base + len_to - r.len;
    if (lane == mine - 1 && b0 + mine == a.n) {
      a.cu[a.n] = base + len_to;
      a.used[0] = a.freel ? taken + took_to : 0;
    }
  }
  for (int i = wave; i < mine; i += kAttnWaves) {
    const int start = __builtin_amdgcn_readlane(r.start, i);
    const int len = __builtin_amdgcn_readlane(r.len, i);
    const int have = __builtin_amdgcn_readlane(r.have, i);
    const int want = __builtin_amdgcn_readlane(r.want, i);
    // table entry k is entry k + from of the list
    const int64_t from = (int64_t)taken + __builtin_amdgcn_readlane(took_to, i) -
                         (a.freel ? want - have : 0) - have;
    const int64_t first = (int64_t)base + __builtin_amdgcn_readlane(len_to, i) - len;
    int* row = a.table + (int64_t)(b0 + i) * a.mb;
    const int* list = a.freel ? a.freel + from : row;
    const int listed = a.freel ? (int)max(min(a.n_free - from, (int64_t)a.mb), (int64_t)0) : a.mb;
    // the table's first entries are loaded here and stored behind the slots
    const int to = a.freel ? min(want, listed) : 0, k0 = have + part * 64 + lane;
    const int entry = k0 < to ? list[k0] : -1;
    const int jmax = first < 0 ? 0 : (int)max(min((int64_t)len, a.max_tokens - first), (int64_t)0);
    int* out = a.slots + max(first, (int64_t)0);
    // a partly filled block first: its tokens' id is the table's
    int j0 = 0;
    if (a.freel && have > 0) {
      const int left = (int)min((int64_t)have * bs - start, (int64_t)jmax);
      if (left > 0) {
        const int id = row[have - 1];
        const int off = start - (have - 1) * bs;
        if (part == 0)
          for (int j = lane; j < left; j += 64) out[j] = slot_of(id, off + j, bs, most_id);
        j0 = left;
      }
    }
    // then block by block: a lane's position moves on by `step`
    const int step = a.parts * 64, step_k = fast_div(a.by_bs, step), step_off = step - step_k * bs;
    const int p0 = start + j0 + part * 64 + lane;
    int k = fast_div(a.by_bs, p0), off = p0 - k * bs;
    for (int j = j0 + part * 64 + lane; j < jmax; j += 8 * step) {  // eight in flight
      int id[8], o[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        id[x] = (unsigned)k < (unsigned)listed ? list[k] : -1;
        o[x] = off;
        off += step_off;
        const bool over = off >= bs;
        off -= over ? bs : 0;
        k += step_k + (over ? 1 : 0);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (j + x * step < jmax) out[j + x * step] = slot_of(id[x], o[x], bs, most_id);
    }
    if (a.freel) {
      if (k0 < a.mb) row[k0] = entry;
      for (int k = k0 + step; k < a.mb; k += step) row[k] = k < to ? list[k] : -1;
    }
  }
}

}  // namespace
