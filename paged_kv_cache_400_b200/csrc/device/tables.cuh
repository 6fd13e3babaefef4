// Block tables, lengths and slot maps of a step, built on the device from the
// requests' lengths, and the return of finished requests' blocks.
//
// The free blocks are a ring, taken from its head and given back at its tail
// in request and table order: the order in which the host block manager does
// the same ("如何通过PagedAttention实现LLM高性能推理：实战指南" §2.2 keeps the free
// blocks in a deque), so both hand out the same blocks.
//
// extend: request b of length L gets n new tokens. With c(x) = ceil(x / 16) it
// takes c(L + n) - c(L) blocks; an exclusive prefix sum over the requests says
// which of the ring's blocks are its own, another one where its tokens' slots
// begin. release: a prefix sum over c(L) of the finished requests.
//
// What is left after the sums is independent per output position p (a slot, or
// a returned block): find p's request, compute its entry. Every fresh block
// begins with one of the step's tokens, and the thread of that token also
// writes the block's table entry; so no position reads what another one wrote.
//
// Both calls are latency: a decode step of 256 requests moves 6 KB. So one
// launch does all: every CTA takes the sums over all requests for itself (up to
// kTablesCached, 8 bytes each, from L2 after the first CTA) and keeps them in
// shared memory, then does its share of the positions; the first CTA also
// writes lengths, query_start and the ring's state. A second launch comes in
// where that cannot be: lengths or state written over the inputs while other
// CTAs still read them, or more requests than shared memory holds (then the
// first launch, one CTA, leaves the sums in the workspace).
#pragma once

#include <algorithm>

#include "decode_common.cuh"

namespace pagedkv {

constexpr int kTablesCached = 4096;      // requests whose sums a CTA keeps in shared memory
// 512 threads with 2 requests, or positions, in flight each: a step of 256
// requests 3.4 us (4 in flight: 4.5, the code and the registers cost more than
// the latency; 1024 threads: 3.8), 1000 prompts 8.5 us. From 2048 requests on
// 1024 threads: 4096 released requests 10.0 us instead of 11.7.
constexpr int kTablesThreads = 512;
constexpr int kTablesMostThreads = 1024;
constexpr int kTablesPerThread = 2;
constexpr int32_t kTablesMost = 1 << 30;  // entries of a ring, slots
constexpr uint32_t kTablesCap = 0x7fffffffu;

struct TablesParams {
  int32_t* block_tables;    // [B][W]
  const int32_t* seq_lens;  // [B]
  const int32_t* asked;     // [B] extend: new tokens; release: non-zero = finished
  int32_t* ring;            // [F] block ids
  const int32_t* state;     // head, count
  int32_t* lens_out;        // [B]
  int32_t* query_start;     // [B + 1] (extend)
  int64_t* slots;           // [num_slots] (extend)
  int32_t* state_out;       // head, count, tokens granted, refused requests
  int32_t* ws_starts;       // [B + 1] workspace: first position of each request
  int32_t* ws_old;          // [B] workspace: old length
  int32_t* ws_first;        // [B] workspace: first of the request's ring entries, from the head
  int32_t* ws_ring;         // [2] workspace: head, count as used
  int32_t num_seqs;
  int32_t width;            // W
  int32_t ring_size;        // F
  int32_t num_blocks;
  int32_t num_slots;
  int32_t row_tokens;       // extend: 0 packed, else slots per request
};

// Sums are kept in 31 bits and stop at the cap, above every limit they are
// compared with; such a sum stays associative.
__device__ __forceinline__ uint32_t add_capped(uint32_t a, uint32_t b) { return min(a + b, kTablesCap); }

// Exclusive sums, in request order, of the CTA's kTablesPerThread values per
// thread: lane of warp w holds requests 32 (K w + k) + lane, k = 0 .. K - 1.
// `total` receives the sum of all.
template <int N>
__device__ __forceinline__ void cta_scan(uint32_t (&v)[N][kTablesPerThread], uint32_t (&total)[N],
                                         uint32_t (*sums)[32]) {
  const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  uint32_t own[N][kTablesPerThread];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int k = 0; k < kTablesPerThread; ++k) own[i][k] = v[i][k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < kTablesPerThread; ++k) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v[i][k], o);
        if (lane >= o) v[i][k] = add_capped(v[i][k], u);
      }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t run = 0;  // of the warp's earlier values
#pragma unroll
    for (int k = 0; k < kTablesPerThread; ++k) {
      const uint32_t all = __shfl_sync(0xffffffffu, v[i][k], 31);
      const uint32_t before = __shfl_up_sync(0xffffffffu, v[i][k], 1);
      v[i][k] = add_capped(run, lane ? before : 0u);
      run = add_capped(run, all);
    }
    if (lane == 0) sums[i][warp] = run;
  }
  __syncthreads();
  // every warp sums the warps' sums for itself
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t s = lane < warps ? sums[i][lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = add_capped(s, u);
    }
    total[i] = __shfl_sync(0xffffffffu, s, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, s, warp ? warp - 1 : 0);
#pragma unroll
    for (int k = 0; k < kTablesPerThread; ++k) v[i][k] = add_capped(v[i][k], warp ? before : 0u);
  }
  __syncthreads();  // sums may be written again
}

// The request that holds position p: the last b of lo .. hi with starts[b] <= p.
__device__ __forceinline__ int32_t request_of(const int32_t* starts, int32_t lo, int32_t hi, int32_t p) {
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (starts[mid] <= p) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Positions [p0, p1) by one CTA. starts, old and first: the request's sums, in
// shared memory or the workspace.
template <bool kExtend>
__device__ __forceinline__ void tables_positions(const TablesParams& t, int32_t p0, int32_t p1, int32_t head,
                                                 int32_t count, const int32_t* starts, const int32_t* old,
                                                 const int32_t* first) {
  const int32_t B = t.num_seqs;
  const int32_t total = starts[B];
  const bool packed = !kExtend || t.row_tokens == 0;
  int32_t lo = 0, hi = 0;
  if (packed && p0 < total) {
    lo = request_of(starts, 0, B - 1, p0);
    hi = request_of(starts, lo, B - 1, min(p1, total) - 1);
  }
  for (int32_t base = p0; base < p1; base += kTablesPerThread * blockDim.x) {
    int32_t b[kTablesPerThread], i[kTablesPerThread], id[kTablesPerThread];
    bool ok[kTablesPerThread];
#pragma unroll
    for (int k = 0; k < kTablesPerThread; ++k) {
      const int32_t p = base + k * (int32_t)blockDim.x + (int32_t)threadIdx.x;
      ok[k] = p < p1;
      b[k] = i[k] = 0;
      if (packed) {
        ok[k] &= p < total;
        if (ok[k]) {
          b[k] = request_of(starts, lo, hi, p);
          i[k] = p - starts[b[k]];
        }
      } else if (ok[k]) {
        const int32_t r = p / t.row_tokens;
        ok[k] = r < B;
        if (ok[k]) {
          b[k] = r;
          i[k] = p - r * t.row_tokens;
          ok[k] = i[k] < starts[r + 1] - starts[r];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kTablesPerThread; ++k) {
      id[k] = -1;
      if (!ok[k]) continue;
      if constexpr (kExtend) {
        const int32_t L = old[b[k]], pos = L + i[k], e = pos >> 4, had = (L + 15) >> 4;
        if (e < had) {
          id[k] = t.block_tables[(size_t)b[k] * t.width + e];
        } else {
          int32_t at = head + first[b[k]] + (e - had);  // below 2 * ring_size
          if (at >= t.ring_size) at -= t.ring_size;
          id[k] = t.ring[at];
        }
      } else {
        id[k] = t.block_tables[(size_t)b[k] * t.width + i[k]];
      }
    }
#pragma unroll
    for (int k = 0; k < kTablesPerThread; ++k) {
      const int32_t p = base + k * (int32_t)blockDim.x + (int32_t)threadIdx.x;
      const bool good = id[k] >= 0 && id[k] < t.num_blocks;
      if (ok[k] && !good) raise_device_error(PA_DEVERR_BLOCK);
      if constexpr (kExtend) {
        if (p >= p1) continue;
        int64_t slot = -1;
        if (ok[k]) {
          const int32_t L = old[b[k]], pos = L + i[k];
          // a fresh block begins with one of the step's tokens: its thread writes the entry
          if ((pos >> 4) >= ((L + 15) >> 4) && (pos & 15) == 0)
            t.block_tables[(size_t)b[k] * t.width + (pos >> 4)] = id[k];
          if (good) slot = (int64_t)id[k] * 16 + (pos & 15);
        }
        t.slots[p] = slot;
      } else if (ok[k]) {
        int64_t at = (int64_t)head + count + p;  // below 2 * ring_size
        if (at >= t.ring_size) at -= t.ring_size;
        t.ring[at] = id[k];
      }
    }
  }
}

// The sums over all requests, and what a launch is asked to do with them:
// kFill the positions, kOutputs lengths, query_start and state (by the first
// CTA), kKeep the sums into the workspace (one CTA, any number of requests),
// kMore let the call's second launch start. A call's last launch releases
// nothing early: what comes after it reads its lengths, tables and slots.
constexpr int kTablesFill = 1, kTablesOutputs = 2, kTablesKeep = 4, kTablesMore = 8;

template <bool kExtend>
__global__ void __launch_bounds__(kTablesMostThreads) tables_kernel(TablesParams t, int32_t positions, int32_t per_cta,
                                                                int32_t todo) {
  extern __shared__ int32_t cached[];  // starts [B + 1], old [B], first [B], unless kTablesKeep
  __shared__ uint32_t sums[2][32];
  __shared__ uint32_t taken;  // ring entries granted (release: given back)
  __shared__ int32_t refused;
  constexpr int K = kTablesPerThread;
  if (todo & kTablesMore) grid_dependents_launch();
  grid_dependency_wait();
  const bool keep = todo & kTablesKeep;
  const bool outputs = (todo & kTablesOutputs) && blockIdx.x == 0;
  int32_t* c_starts = keep ? t.ws_starts : cached;
  int32_t* c_old = keep ? t.ws_old : cached + t.num_seqs + 1;
  int32_t* c_first = keep ? t.ws_first : cached + 2 * t.num_seqs + 1;
  const int32_t tid = threadIdx.x, lane = tid & 31;
  // lengths and requests of a pass; the first one's arrive together with the ring's state
  int32_t L[K], n[K];
  auto load = [&](int32_t b0) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int32_t b = b0 + (tid >> 5) * 32 * K + 32 * k + lane;
      L[k] = b < t.num_seqs ? t.seq_lens[b] : 0;
      n[k] = b < t.num_seqs ? t.asked[b] : 0;
    }
  };
  load(0);
  const int32_t head_in = t.state[0], count_in = t.state[1];
  int32_t head = head_in, count = count_in;
  const bool usable = head >= 0 && head < t.ring_size && count >= 0 && count <= t.ring_size;
  if (!usable) {
    if (tid == 0) raise_device_error(PA_DEVERR_BLOCK);
    head = 0;
    count = kExtend ? 0 : t.ring_size;  // nothing to take, no room to give back
  }
  if (tid == 0) {
    taken = 0;
    refused = 0;
    c_starts[0] = 0;
    if (outputs && kExtend) t.query_start[0] = 0;
  }
  const uint32_t block_limit = kExtend ? (uint32_t)count : (uint32_t)(t.ring_size - count);
  const uint32_t token_limit = kExtend && t.row_tokens == 0 ? (uint32_t)t.num_slots : kTablesCap;
  const int64_t room = (int64_t)t.width * 16;
  uint32_t blocks0 = 0, tokens0 = 0, granted0 = 0;  // sums over the earlier passes' requests
  bool clean = true;                                // nothing refused so far
  for (int32_t b0 = 0; b0 < t.num_seqs; b0 += K * (int32_t)blockDim.x) {
    if (b0 > 0) load(b0);
    uint32_t v[2][K], take[K], sum[2];
    bool bad[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (kExtend) {
        bad[k] = L[k] < 0 || n[k] < 0 || (int64_t)L[k] + n[k] > room || (t.row_tokens > 0 && n[k] > t.row_tokens);
        if (bad[k]) n[k] = 0;
        take[k] = bad[k] ? 0u : (uint32_t)((((int64_t)L[k] + n[k] + 15) >> 4) - (((int64_t)L[k] + 15) >> 4));
      } else {
        n[k] = n[k] != 0;
        bad[k] = n[k] && (L[k] < 0 || L[k] > room);
        if (bad[k]) n[k] = 0;
        take[k] = n[k] ? (uint32_t)(((int64_t)L[k] + 15) >> 4) : 0u;
      }
      if (bad[k]) raise_device_error(PA_DEVERR_SEQLEN);
      v[0][k] = take[k];
      v[1][k] = (uint32_t)n[k];
    }
    cta_scan<2>(v, sum, sums);
    bool ok[K];
    uint32_t g[1][K], granted[1];
    bool any_refused = false;
    uint32_t top = 0;
    int32_t lost = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[0][k] = add_capped(blocks0, v[0][k]);
      const uint32_t blocks = add_capped(v[0][k], take[k]);                 // up to and with this request
      const uint32_t tokens = add_capped(add_capped(tokens0, v[1][k]), (uint32_t)n[k]);
      ok[k] = ((kExtend ? take[k] == 0 : n[k] == 0) || (blocks <= block_limit && blocks < kTablesCap)) &&
              (!kExtend || n[k] == 0 || tokens <= token_limit);
      any_refused |= !ok[k];
      if (bad[k] || !ok[k]) ++lost;
      if (ok[k] && take[k]) top = max(top, blocks);
      g[0][k] = ok[k] ? (kExtend ? (uint32_t)n[k] : take[k]) : 0u;
    }
    // positions: tokens granted (extend), blocks given back (release)
    uint32_t own[K];
#pragma unroll
    for (int k = 0; k < K; ++k) own[k] = g[0][k];
    clean = !__syncthreads_or(any_refused) && clean;
    if (clean) {
#pragma unroll
      for (int k = 0; k < K; ++k) g[0][k] = kExtend ? v[1][k] : v[0][k] - blocks0;
      granted[0] = kExtend ? sum[1] : sum[0];
    } else {
      cta_scan<1>(g, granted, sums);
    }
    if (top) atomicMax(&taken, top);
    if (lost) atomicAdd(&refused, lost);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int32_t b = b0 + (tid >> 5) * 32 * K + 32 * k + lane;
      if (b >= t.num_seqs) continue;
      const int32_t end = (int32_t)(granted0 + g[0][k] + own[k]);
      c_starts[b + 1] = end;
      if constexpr (kExtend) {
        c_old[b] = L[k];
        c_first[b] = (int32_t)v[0][k];
      }
      if (outputs) {
        t.lens_out[b] = kExtend ? (ok[k] ? L[k] + n[k] : L[k]) : (n[k] && ok[k] ? 0 : L[k]);
        if constexpr (kExtend) t.query_start[b + 1] = end;
      }
    }
    blocks0 = add_capped(blocks0, sum[0]);
    tokens0 = add_capped(tokens0, sum[1]);
    granted0 += granted[0];
  }
  __syncthreads();
  if (tid == 0) {
    const int32_t moved = (int32_t)taken;
    if (keep) {
      t.ws_ring[0] = head;
      t.ws_ring[1] = count;
    }
    if (outputs) {
      int32_t h = head;
      if (kExtend && (h += moved) >= t.ring_size) h -= t.ring_size;
      t.state_out[0] = usable ? h : head_in;
      t.state_out[1] = !usable ? count_in : kExtend ? count - moved : count + moved;
      t.state_out[2] = kExtend ? (int32_t)granted0 : 0;
      t.state_out[3] = refused;
    }
  }
  if (todo & kTablesFill) {
    const int64_t p0 = (int64_t)blockIdx.x * per_cta;
    const int32_t end = kExtend ? positions : min(positions, (int32_t)granted0);
    const int32_t p1 = (int32_t)min(p0 + per_cta, (int64_t)end);
    if (p0 < p1) tables_positions<kExtend>(t, (int32_t)p0, p1, head, count, c_starts, c_old, c_first);
  }
}

// The positions from the workspace's sums, after a launch with kTablesKeep.
template <bool kExtend>
__global__ void __launch_bounds__(kTablesMostThreads) tables_fill_kernel(TablesParams t, int32_t positions,
                                                                     int32_t per_cta) {
  grid_dependency_wait();
  const int64_t p0 = (int64_t)blockIdx.x * per_cta;
  const int32_t end = kExtend ? positions : min(positions, t.ws_starts[t.num_seqs]);
  const int32_t p1 = (int32_t)min(p0 + per_cta, (int64_t)end);
  if (p0 < p1)
    tables_positions<kExtend>(t, (int32_t)p0, p1, t.ws_ring[0], t.ws_ring[1], t.ws_starts, t.ws_old, t.ws_first);
}

inline size_t tables_workspace_bytes(int32_t num_seqs) { return ((size_t)3 * num_seqs + 3) * sizeof(int32_t); }

// positions: slots (extend), or an upper bound of the blocks given back.
template <bool kExtend>
inline cudaError_t launch_tables(TablesParams t, void* workspace, int64_t positions, cudaStream_t st) {
  int32_t* ws = reinterpret_cast<int32_t*>(workspace);
  t.ws_ring = ws;
  t.ws_starts = ws + 2;
  t.ws_old = t.ws_starts + t.num_seqs + 1;
  t.ws_first = t.ws_old + t.num_seqs;
  const int32_t n = (int32_t)positions;
  // a position per thread, and more on at most one CTA per SM: each takes the sums for itself
  const int32_t threads = t.num_seqs > 2048 ? kTablesMostThreads : kTablesThreads;
  const int32_t ctas = std::max(1, std::min((n + threads - 1) / threads, device_sm_count()));
  const int32_t per_cta = (n + ctas - 1) / ctas;
  const bool cached = t.num_seqs <= kTablesCached;
  const size_t smem = cached ? (size_t)(kExtend ? 3 : 1) * (t.num_seqs + 1) * sizeof(int32_t) : 0;
  static PerDevice<int32_t> smem_set;
  cudaError_t e = set_smem_once(smem_set, tables_kernel<kExtend>, 3 * (kTablesCached + 1) * (int32_t)sizeof(int32_t));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  const bool in_place = t.lens_out == t.seq_lens || t.state_out == t.state;
  if (cached && (ctas == 1 || !in_place))
    return cudaLaunchKernelEx(&cfg, tables_kernel<kExtend>, t, n, per_cta, kTablesFill | kTablesOutputs);
  if (cached) {
    e = cudaLaunchKernelEx(&cfg, tables_kernel<kExtend>, t, n, per_cta, kTablesFill | kTablesMore);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(1);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tables_kernel<kExtend>, t, n, per_cta, kTablesOutputs);
  }
  cfg.gridDim = dim3(1);
  e = cudaLaunchKernelEx(&cfg, tables_kernel<kExtend>, t, n, per_cta,
                         kTablesOutputs | kTablesKeep | kTablesMore);
  if (e != cudaSuccess || n == 0) return e;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tables_fill_kernel<kExtend>, t, n, per_cta);
}

}  // namespace pagedkv
