// map_blocks.h -- part of libbeamattn.so, included once by beamattn.hip.
//
// Block tables and slot maps from request lengths: m1_map.
#pragma once

namespace {

struct MapArgs {
  int n, mb, n_free, max_tokens;
  FastDiv by_bs;
  const int* starts;   // or null
  const int* lens;
  const int* freel;    // or null
  int* table;
  int* cu;
  int* slots;
  int* used;
  int per;             // requests of a workgroup
  int chunks;          // workgroups along the requests; those behind fill the slots' end
  int parts;           // workgroups along a request's tokens
};

struct MapReq {
  int start, len, have, want;
};
__device__ __forceinline__ MapReq map_request(const MapArgs& a, int b) {
  MapReq r;
  r.start = a.starts ? max(a.starts[b], 0) : 0;
  r.len = max(a.lens[b], 0);
  const int end = r.start + r.len;
  r.have = r.start > 0 ? min(fast_div(a.by_bs, r.start - 1) + 1, a.mb) : 0;
  r.want = end > 0 ? max(min(fast_div(a.by_bs, end - 1) + 1, a.mb), r.have) : r.have;
  return r;
}

// Sums of the lengths and of the blocks taken over requests [0, to): uniform.
__device__ __forceinline__ void map_prefix(const MapArgs& a, int to, int& len, int& taken) {
  __shared__ int part[2][kAttnWaves];
  int l = 0, t = 0;
  for (int b = threadIdx.x; b < to; b += kAttnThreads) {
    const MapReq r = map_request(a, b);
    l += r.len;
    t += r.want - r.have;
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

// One launch: a workgroup sums the requests before its own, then writes the
// table rows, sums and slots of its own, one after the other.
__global__ __launch_bounds__(kAttnThreads) void m1_map(MapArgs a) {
  const int tid = threadIdx.x;
  int base, taken;
  if ((int)blockIdx.x >= a.chunks) {  // padding behind the last token
    map_prefix(a, a.n, base, taken);
    const int step = (gridDim.x - a.chunks) * gridDim.y * kAttnThreads;
    int64_t i = (int64_t)max(base, 0) +
                ((blockIdx.x - a.chunks) * gridDim.y + blockIdx.y) * kAttnThreads + tid;
    for (; i < a.max_tokens; i += step) a.slots[i] = -1;
    return;
  }
  const int b0 = blockIdx.x * a.per, b1 = min(b0 + a.per, a.n);
  const int part = blockIdx.y;
  map_prefix(a, b0, base, taken);
  for (int b = b0; b < b1; ++b) {
    const MapReq r = map_request(a, b);
    const int64_t row = (int64_t)b * a.mb;
    if (a.freel) {
      for (int k = r.have + part * kAttnThreads + tid; k < a.mb; k += a.parts * kAttnThreads) {
        const int64_t f = (int64_t)taken + (k - r.have);
        a.table[row + k] = k < r.want && f < a.n_free ? a.freel[f] : -1;
      }
    }
    for (int i = part * kAttnThreads + tid; i < r.len; i += a.parts * kAttnThreads) {
      const int64_t at = (int64_t)base + i;
      if (at < 0 || at >= a.max_tokens) continue;
      const int p = r.start + i, k = fast_div(a.by_bs, p);
      int id = -1;
      if ((unsigned)k < (unsigned)a.mb) {
        if (k < r.have || !a.freel) {
          id = a.table[row + k];
        } else {
          const int64_t f = (int64_t)taken + (k - r.have);
          id = f < a.n_free ? a.freel[f] : -1;
        }
      }
      const int64_t slot = (int64_t)id * a.by_bs.d + (p - k * a.by_bs.d);
      a.slots[at] = id < 0 || slot > 0x7fffffff ? -1 : (int)slot;
    }
    if (part == 0 && tid == 0) a.cu[b] = base;
    base += r.len;
    if (a.freel) taken += r.want - r.have;
    if (part == 0 && tid == 0 && b == a.n - 1) {
      a.cu[a.n] = base;
      a.used[0] = a.freel ? taken : 0;
    }
  }
}

}  // namespace
