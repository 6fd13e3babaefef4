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
// Both calls are latency: a decode step of 256 requests moves 6 KB. One CTA
// does the sums (its carries would be the only thing to pass between CTAs) and,
// up to kTablesOneCta positions, the positions too, from shared memory; above
// that a second, wide grid takes the positions, launched as a programmatic
// dependent, so that its start overlaps the sums.
#pragma once

#include "decode_common.cuh"

namespace pagedkv {

constexpr int kTablesThreads = 1024;
constexpr int kTablesCached = 2048;    // requests whose starts a CTA keeps in shared memory
constexpr int kTablesOneCta = 8192;    // positions one CTA does on its own

struct TablesParams {
  int32_t* block_tables;    // [B][W]
  const int32_t* seq_lens;  // [B]
  const int32_t* asked;     // [B] extend: new tokens; release: non-zero = finished
  int32_t* ring;            // [F] block ids
  const int32_t* state;     // head, count
  int32_t* lens_out;        // [B]
  int32_t* query_start;     // [B + 1] (extend)
  int64_t* slots;           // [num_slots] (extend)
  int32_t* state_out;       // head, count, tokens | blocks, refused requests
  int32_t* starts;          // [B + 1] first position of each request (query_start, or workspace)
  int32_t* old_lens;        // [B] workspace
  int32_t* first;           // [B] workspace: first of the request's ring entries, from the head
  int32_t* scratch;         // [2] workspace: head, count as read
  int32_t num_seqs;
  int32_t width;            // W
  int32_t ring_size;        // F
  int32_t num_blocks;
  int32_t num_slots;
  int32_t row_tokens;       // extend: 0 packed, else slots per request
};

// Inclusive sums of x over the CTA's threads, in thread order; `total` = the
// last. Two values at once: a barrier costs more than the arithmetic.
__device__ __forceinline__ void cta_scan2(int64_t& x, int64_t& y, int64_t& tx, int64_t& ty, int64_t (*sums)[32]) {
  const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += a;
      y += b;
    }
  }
  if (lane == 31) {
    sums[0][warp] = x;
    sums[1][warp] = y;
  }
  __syncthreads();
  // every warp scans the warps' sums for itself
  int64_t a = lane < (int32_t)(blockDim.x >> 5) ? sums[0][lane] : 0, b = lane < (int32_t)(blockDim.x >> 5) ? sums[1][lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, a, o), w = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += u;
      b += w;
    }
  }
  tx = __shfl_sync(0xffffffffu, a, 31);
  ty = __shfl_sync(0xffffffffu, b, 31);
  const int64_t px = __shfl_sync(0xffffffffu, a, warp ? warp - 1 : 0), py = __shfl_sync(0xffffffffu, b, warp ? warp - 1 : 0);
  if (warp) {
    x += px;
    y += py;
  }
  __syncthreads();  // sums may be written again
}

// The request that holds position p: the last b with starts[b] <= p.
__device__ __forceinline__ int32_t request_of(const int32_t* starts, int32_t num_seqs, int32_t p) {
  int32_t lo = 0, hi = num_seqs - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (starts[mid] <= p) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Position p of the step (see above). starts, old_lens and first may be the
// global arrays or a CTA's copies of them.
template <bool kExtend>
__device__ __forceinline__ void tables_position(const TablesParams& t, int32_t p, int32_t total, int32_t head,
                                                int32_t count, const int32_t* starts, const int32_t* old_lens,
                                                const int32_t* first) {
  if constexpr (!kExtend) {
    if (p >= total) return;
    const int32_t b = request_of(starts, t.num_seqs, p);
    const int32_t id = t.block_tables[(size_t)b * t.width + (p - starts[b])];
    if (id < 0 || id >= t.num_blocks) raise_device_error(PA_DEVERR_BLOCK);
    t.ring[((int64_t)head + count + p) % t.ring_size] = id;
    return;
  }
  int32_t b, i;
  bool token;
  if (t.row_tokens > 0) {
    b = p / t.row_tokens;
    i = p - b * t.row_tokens;
    token = b < t.num_seqs && i < starts[b + 1] - starts[b];
  } else {
    token = p < total;
    b = token ? request_of(starts, t.num_seqs, p) : 0;
    i = token ? p - starts[b] : 0;
  }
  int64_t slot = -1;
  if (token) {
    const int32_t L = old_lens[b];
    const int32_t pos = L + i;
    const int32_t e = pos >> 4, had = (L + 15) >> 4;
    int32_t* entry = t.block_tables + (size_t)b * t.width + e;
    int32_t id;
    if (e < had) {
      id = *entry;
    } else {
      id = t.ring[((int64_t)head + first[b] + (e - had)) % t.ring_size];
      if ((pos & 15) == 0) *entry = id;
    }
    if (id >= 0 && id < t.num_blocks) slot = (int64_t)id * 16 + (pos & 15);
    else raise_device_error(PA_DEVERR_BLOCK);
  }
  t.slots[p] = slot;
}

// The sums, one CTA; with kPositions also the positions (at most kTablesCached
// requests).
template <bool kExtend, bool kPositions>
__global__ void __launch_bounds__(kTablesThreads) tables_scan_kernel(TablesParams t, int32_t positions) {
  __shared__ int64_t sums[2][32];
  __shared__ int32_t c_starts[kPositions ? kTablesCached + 1 : 1];
  __shared__ int32_t c_old[kPositions && kExtend ? kTablesCached : 1];
  __shared__ int32_t c_first[kPositions && kExtend ? kTablesCached : 1];
  __shared__ unsigned long long taken;  // ring entries granted (release: given back)
  __shared__ int32_t refused;
  grid_dependents_launch();
  const int32_t tid = threadIdx.x;
  const int32_t head_in = t.state[0], count_in = t.state[1];
  int32_t head = head_in, count = count_in;
  bool usable = true;
  if (head < 0 || head >= t.ring_size || count < 0 || count > t.ring_size) {
    if (tid == 0) raise_device_error(PA_DEVERR_BLOCK);
    usable = false;
    head = 0;
    count = kExtend ? 0 : t.ring_size;  // nothing to take, no room to give back
  }
  if (tid == 0) {
    taken = 0;
    refused = 0;
  }
  __syncthreads();
  int64_t blocks0 = 0, tokens0 = 0, granted0 = 0;  // sums over the earlier passes' requests
  bool clean = true;                               // nothing refused so far
  for (int32_t b0 = 0; b0 < t.num_seqs; b0 += kTablesThreads) {
    const int32_t b = b0 + tid;
    int32_t L = 0, n = 0;
    int64_t take = 0;
    bool bad = false;
    if (b < t.num_seqs) {
      L = t.seq_lens[b];
      n = t.asked[b];
      const int64_t room = (int64_t)t.width * 16;
      if constexpr (kExtend) {
        bad = L < 0 || n < 0 || (int64_t)L + n > room || (t.row_tokens > 0 && n > t.row_tokens);
        if (bad) n = 0;
        else take = (((int64_t)L + n + 15) >> 4) - (((int64_t)L + 15) >> 4);
      } else {
        n = n != 0;
        bad = n && (L < 0 || L > room);
        if (bad) n = 0;
        if (n) take = ((int64_t)L + 15) >> 4;
      }
      if (bad) raise_device_error(PA_DEVERR_SEQLEN);
    }
    int64_t x = take, y = n, tx, ty;
    cta_scan2(x, y, tx, ty, sums);
    const int64_t blocks = blocks0 + x, tokens = tokens0 + y;  // inclusive
    bool ok;
    if constexpr (kExtend) ok = (take == 0 || blocks <= count) && (t.row_tokens > 0 || n == 0 || tokens <= t.num_slots);
    else ok = blocks <= (int64_t)t.ring_size - count;
    const int32_t got = ok ? n : 0;
    if (b < t.num_seqs && (bad || (n && !ok))) atomicAdd(&refused, 1);
    if (ok && take > 0 && b < t.num_seqs) atomicMax(&taken, (unsigned long long)blocks);
    // positions: tokens granted (extend), blocks given back (release)
    int64_t g = kExtend ? got : (ok ? take : 0), gt;
    clean = !__syncthreads_or(!ok) && clean;
    if (clean) {
      g = kExtend ? y : x;
      gt = kExtend ? ty : tx;
    } else {
      int64_t z = 0, tz;
      cta_scan2(g, z, gt, tz, sums);
    }
    if (b < t.num_seqs) {
      const int32_t end = (int32_t)(granted0 + g);
      t.lens_out[b] = kExtend ? L + got : (n && ok ? 0 : L);
      t.starts[b + 1] = end;
      if constexpr (kPositions) c_starts[b + 1] = end;
      if constexpr (kExtend) {
        const int32_t f = (int32_t)(blocks - take);
        if constexpr (kPositions) {
          c_old[b] = L;
          c_first[b] = f;
        } else {
          t.old_lens[b] = L;
          t.first[b] = f;
        }
      }
    }
    blocks0 += tx;
    tokens0 += ty;
    granted0 += gt;
  }
  __syncthreads();
  const int32_t total = (int32_t)granted0;
  if (tid == 0) {
    const int32_t moved = (int32_t)taken;
    t.starts[0] = 0;
    if constexpr (kPositions) {
      c_starts[0] = 0;
    } else {
      t.scratch[0] = head;
      t.scratch[1] = count;
    }
    t.state_out[0] = !usable ? head_in : kExtend ? (int32_t)(((int64_t)head + moved) % t.ring_size) : head;
    t.state_out[1] = !usable ? count_in : kExtend ? count - moved : count + moved;
    t.state_out[2] = total;
    t.state_out[3] = refused;
  }
  if constexpr (kPositions) {
    __syncthreads();
    const int32_t end = kExtend ? positions : min(positions, total);
    for (int32_t p = tid; p < end; p += kTablesThreads)
      tables_position<kExtend>(t, p, total, head, count, c_starts, c_old, c_first);
  }
}

// The positions, after tables_scan_kernel<kExtend, false>.
template <bool kExtend>
__global__ void __launch_bounds__(256) tables_fill_kernel(TablesParams t, int32_t positions) {
  __shared__ int32_t c_starts[kTablesCached + 1];
  grid_dependency_wait();
  const bool cached = t.num_seqs <= kTablesCached;
  if (cached) {
    for (int32_t i = threadIdx.x; i <= t.num_seqs; i += blockDim.x) c_starts[i] = __ldcg(t.starts + i);
    __syncthreads();
  }
  const int32_t* starts = cached ? c_starts : t.starts;
  const int32_t total = starts[t.num_seqs];
  const int32_t head = t.scratch[0], count = t.scratch[1];
  const int32_t end = kExtend ? positions : min(positions, total);
  for (int64_t p = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; p < end; p += (int64_t)gridDim.x * blockDim.x)
    tables_position<kExtend>(t, (int32_t)p, total, head, count, starts, t.old_lens, t.first);
}

inline size_t tables_workspace_bytes(int32_t num_seqs) { return ((size_t)3 * num_seqs + 3) * sizeof(int32_t); }

// positions: slots (extend), or an upper bound of the blocks given back.
template <bool kExtend>
inline cudaError_t launch_tables(TablesParams t, void* workspace, int64_t positions, cudaStream_t st) {
  int32_t* ws = reinterpret_cast<int32_t*>(workspace);
  t.scratch = ws;
  t.old_lens = ws + 2;
  t.first = t.old_lens + t.num_seqs;
  t.starts = kExtend ? t.query_start : t.first + t.num_seqs;
  const int32_t n = (int32_t)positions;
  if (n <= kTablesOneCta && t.num_seqs <= kTablesCached) {
    tables_scan_kernel<kExtend, true><<<1, kTablesThreads, 0, st>>>(t, n);
    return cudaGetLastError();
  }
  tables_scan_kernel<kExtend, false><<<1, kTablesThreads, 0, st>>>(t, n);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || n == 0) return e;
  cudaLaunchConfig_t cfg = {};
  const int64_t ctas = (positions + 1023) / 1024, most = (int64_t)8 * device_sm_count();
  cfg.gridDim = dim3((unsigned)(ctas < most ? ctas : most));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tables_fill_kernel<kExtend>, t, n);
}

}  // namespace pagedkv
