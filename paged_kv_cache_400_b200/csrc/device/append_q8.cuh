// Cache append into an 8-bit pool: each new K/V row coded into its slot, with
// one scale per (block, K|V, head) tile.
//
// With A the largest finite magnitude of a tile's new rows (0 below 2^-100),
// the tile's scale s becomes first(A) when its row 0 is among them, grown(s, A)
// otherwise (q8_common.cuh), rows it keeps are coded again where s grew, and a
// new element is stored as the code nearest to x * (1 / s).
//
// One warp owns a tile, so a scale and the rows under it change together and
// nothing is summed or ordered across warps. A block's tokens may lie anywhere
// in slot_mapping, in any order, and a row named twice takes the later token.
// So each CTA looks at the whole list for its own few entries: their blocks go
// into a hash table in shared memory, and every entry of the list that names
// one of them either says that an earlier CTA leads the block, or is noted as
// the latest token of its row. The blocks left over are the CTA's, and its warps
// share their (block, K|V, head) tiles.
//
// Bound by its bytes (reads T * Hkv * D elements twice over for K and V, writes
// half or a quarter as many) for many tokens, by latency for few. The scale and
// all new rows of a tile are in flight together, 16 bytes a lane, and stay in
// registers between the maximum and the codes: up to 124 a thread (held to 80, for
// half as many warps again, 64 prompt tokens took 7.4 us in place of 4.3). The
// looks at the list are T entries for each CTA, so a CTA takes more entries where
// the list is long: 8192 prompt tokens of 8 heads, e4m3, 17.4 us (2.9 TB/s);
// a decode step of 256 requests 6.3 us.
#pragma once

#include <algorithm>

#include "q8_common.cuh"

namespace pagedkv {

constexpr int kAppendQ8Warps = 8;
constexpr int kAppendQ8CtasPerSm = 2;
constexpr int kAppendQ8Run = 256;                  // most entries of a CTA, one per thread
constexpr float kQ8Tiny = 7.888609052210118e-31f;  // 2^-100: below it a tile counts as zeros (1 / s stays finite)

// Largest magnitude of words of elements, on their bit patterns (which order
// as the magnitudes do): per word, and as the fp32 pattern of the larger half.
template <typename T> struct Bits;
template <> struct Bits<float> {
  __device__ __forceinline__ static uint32_t max_abs(uint32_t m, uint32_t w) { return max(m, w & 0x7fffffffu); }
  __device__ __forceinline__ static uint32_t widest(uint32_t m) { return m; }
  __device__ __forceinline__ static float get(const uint32_t* w, int c) { return __uint_as_float(w[c]); }
  // the pattern of a, or of the largest finite value below it
  __device__ __forceinline__ static uint32_t finite(float a) { return min(__float_as_uint(a), 0x7f7fffffu); }
  // NaN -> 0, an infinity -> `most` with its sign
  __device__ __forceinline__ static uint32_t replace_odd(uint32_t w, uint32_t most) {
    const uint32_t a = w & 0x7fffffffu;
    return a < 0x7f800000u ? w : a > 0x7f800000u ? 0u : (w & 0x80000000u) | most;
  }
};
template <> struct Bits<__nv_bfloat16> {
  __device__ __forceinline__ static uint32_t max_abs(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
  __device__ __forceinline__ static uint32_t widest(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
  __device__ __forceinline__ static float get(const uint32_t* w, int c) {
    return __uint_as_float(c & 1 ? w[c / 2] & 0xffff0000u : w[c / 2] << 16);
  }
  // to nearest: 2^-9 off at most, which the codes' own rounding takes up
  __device__ __forceinline__ static uint32_t finite(float a) {
    return min((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(a)), 0x7f7fu);
  }
  __device__ __forceinline__ static uint32_t replace_odd(uint32_t w, uint32_t most) {
    uint32_t out = 0;
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      const uint32_t x = (w >> h) & 0xffffu, a = x & 0x7fffu;
      out |= (a < 0x7f80u ? x : a > 0x7f80u ? 0u : (x & 0x8000u) | most) << h;
    }
    return out;
  }
};

// A CTA's shared memory. Hash table of its blocks, of a power of two of slots, at
// least four times its entries; then by entry (a block goes by the entry that
// put it into the table): the latest token of each row, whether the block is led
// elsewhere, and the list of the blocks that are the CTA's.
constexpr int32_t kAppendQ8Empty = INT32_MIN;
struct AppendQ8Shared {
  int32_t rows[kAppendQ8Run][16];
  int32_t key[4 * kAppendQ8Run];
  int32_t owner[4 * kAppendQ8Run];
  int32_t elsewhere[kAppendQ8Run];
  int2 lead[kAppendQ8Run];  // entry, block
  int32_t num_lead;
};

// CTA (x, y): the blocks first named by entries [run * x, + run), planes
// [group * y, + group) of the 2 * num_kv_heads (K of every head, then V).
template <typename T, int D, typename Code>
__global__ void __launch_bounds__(kAppendQ8Warps * 32, kAppendQ8CtasPerSm)
append_q8_kernel(const T* __restrict__ k, const T* __restrict__ v, uint8_t* __restrict__ pool,
                 const int64_t* __restrict__ slots, int32_t num_tokens, int32_t num_kv_heads, int64_t num_slots,
                 Q8Layout lay, int32_t run, int32_t group) {
  constexpr uint32_t kAll = 0xffffffffu;
  constexpr int E = 16 / sizeof(T);     // elements per lane and step
  constexpr int kLanes = D / E;         // lanes of a row
  constexpr int kRows = 32 / kLanes;    // rows of a step
  constexpr int kSteps = 16 / kRows;
  constexpr int C = kSteps < 8 ? kSteps : 8;  // steps held in registers (of 16, fp32 rows of 128, half at a time)
  using Codes = Vec<uint8_t, E>;
  union Words {  // 16 bytes of a row
    uint4 q;
    uint32_t w[4];
    __device__ __forceinline__ float get(int c) const { return Bits<T>::get(w, c); }
  };
  __shared__ AppendQ8Shared sh;
  int32_t table = 32;
  while (table < 4 * run) table *= 2;
  const int32_t tid = threadIdx.x;
  const int32_t warp = tid >> 5;
  const int32_t lane = tid & 31;
  const int32_t t0 = blockIdx.x * run;
  auto hash = [&](int32_t b) -> int32_t { return (int32_t)((uint32_t)b * 2654435761u >> 16) & (table - 1); };

  // the CTA's entries, and the first looks at the list, in flight together
  constexpr int kLook = 8;
  int64_t seen[kLook];
  auto look = [&](int32_t base) {
#pragma unroll
    for (int i = 0; i < kLook; ++i) {
      const int64_t t = (int64_t)base + i * (kAppendQ8Warps * 32) + tid;
      seen[i] = t < num_tokens ? __ldg(slots + t) : -1;
    }
  };
  const bool mine = tid < run && tid < num_tokens - t0;
  const int64_t my_slot = mine ? __ldg(slots + t0 + tid) : -1;
  look(0);
  for (int32_t i = tid; i < table; i += kAppendQ8Warps * 32) sh.key[i] = kAppendQ8Empty;
  for (int32_t i = tid; i < run * 16; i += kAppendQ8Warps * 32) (&sh.rows[0][0])[i] = -1;
  sh.elsewhere[tid] = 0;
  if (tid == 0) sh.num_lead = 0;
  __syncthreads();
  int32_t my_at = -1;  // this entry's place in the table, where it stands for its block
  if (my_slot >= num_slots && blockIdx.y == 0) raise_device_error(PA_DEVERR_SLOT);
  if (my_slot >= 0 && my_slot < num_slots) {
    const int32_t b = (int32_t)(my_slot >> 4);
    int32_t at = hash(b);
    for (;;) {
      const int32_t was = atomicCAS(sh.key + at, kAppendQ8Empty, b);
      if (was == kAppendQ8Empty) {
        sh.owner[at] = tid;
        my_at = at;
      }
      if (was == kAppendQ8Empty || was == b) break;
      at = (at + 1) & (table - 1);
    }
  }
  __syncthreads();
  for (int32_t base = 0;;) {
    int32_t has[kLook];
#pragma unroll
    for (int i = 0; i < kLook; ++i) has[i] = sh.key[hash((int32_t)(seen[i] >> 4))];
#pragma unroll
    for (int i = 0; i < kLook; ++i) {
      if (has[i] == kAppendQ8Empty) continue;
      const int64_t s = seen[i];
      const int32_t b = (int32_t)(s >> 4);
      int32_t at = hash(b);
      while (has[i] != b && has[i] != kAppendQ8Empty) {
        at = (at + 1) & (table - 1);
        has[i] = sh.key[at];
      }
      if (has[i] == b && s >= 0 && s < num_slots) {
        const int32_t t = base + i * (kAppendQ8Warps * 32) + tid;
        const int32_t o = sh.owner[at];
        if (t < t0) sh.elsewhere[o] = 1;
        else atomicMax(&sh.rows[o][(int32_t)(s & 15)], t);
      }
    }
    if (num_tokens - base <= kLook * kAppendQ8Warps * 32) break;
    base += kLook * kAppendQ8Warps * 32;
    look(base);
  }
  __syncthreads();
  if (my_at >= 0 && !sh.elsewhere[tid]) sh.lead[atomicAdd(&sh.num_lead, 1)] = make_int2(tid, sh.key[my_at]);
  __syncthreads();

  const int32_t my_row = lane / kLanes;
  const int32_t my_col = (lane % kLanes) * E;
  const int32_t planes = min(group, 2 * num_kv_heads - (int32_t)blockIdx.y * group);
  const int32_t tiles = sh.num_lead * planes;
  const uint32_t stride = (uint32_t)num_kv_heads * D * sizeof(T);  // bytes of a token
  for (int32_t i = warp; i < tiles; i += kAppendQ8Warps) {
    const int32_t plane = blockIdx.y * group + i % planes;
    const int32_t kv = plane >= num_kv_heads, h = plane - kv * num_kv_heads;
    const uint8_t* src = reinterpret_cast<const uint8_t*>((kv ? v : k) + h * D + my_col);
    const int2 at = sh.lead[i / planes];
    const int32_t blk = at.y;
    const int32_t* row_src = sh.rows[at.x];
    uint8_t* tile = pool + (size_t)blk * lay.block_bytes + ((size_t)kv * num_kv_heads + h) * 16 * D;
    float* scale_at = reinterpret_cast<float*>(pool + q8_scale_at(lay, blk, kv, h, num_kv_heads));
    const float s_old = *scale_at;
    const bool fresh = row_src[0] >= 0;

    // rows of steps c0 .. c0 + C - 1
    Words x[C];
    uint32_t written = 0;  // bit i: this lane's row of step i is new
    auto load = [&](int c0) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int32_t t = row_src[(c0 + i) * kRows + my_row];
        x[i].q = make_uint4(0, 0, 0, 0);
        if (t >= 0) {
          written |= 1u << (c0 + i);
          x[i].q = __ldg(reinterpret_cast<const uint4*>(src + (uint64_t)(uint32_t)t * stride));
        }
      }
    };
    // largest magnitude, on the bit patterns
    uint32_t top = 0;
#pragma unroll
    for (int c0 = 0; c0 < kSteps; c0 += C) {
      load(c0);
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) top = Bits<T>::max_abs(top, x[i].w[c]);
    }
    top = __reduce_max_sync(kAll, Bits<T>::widest(top));
    const bool odd = top >= 0x7f800000u;  // a NaN or an infinity among the rows
    if (odd) {
      top = 0;
#pragma unroll 1
      for (int c0 = 0; c0 < kSteps; c0 += C) {
        load(c0);
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int c = 0; c < E; ++c) {
            const uint32_t a = __float_as_uint(fabsf(x[i].get(c)));
            if (a < 0x7f800000u) top = max(top, a);
          }
      }
      top = __reduce_max_sync(kAll, top);
      if (lane == 0) raise_device_error(PA_DEVERR_NONFINITE);
    }
    float amax = __uint_as_float(top);
    if (amax < kQ8Tiny) amax = 0.f;
    const float s_new = fresh ? __fmul_rn(amax, Code::kInvMax) : Code::grown(s_old, amax);
    const float inv = s_new > 0.f ? __fdiv_rn(1.f, s_new) : 0.f;

    if (!fresh && s_new > s_old) {
      // rows that stay: coded again at the grown scale
      const float ratio = __fdiv_rn(s_old, s_new);
#pragma unroll 1
      for (int c0 = 0; c0 < kSteps; c0 += 4) {
        Codes c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((written >> (c0 + i)) & 1u))
            c[i] = *reinterpret_cast<const Codes*>(tile + ((c0 + i) * kRows + my_row) * D + my_col);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((written >> (c0 + i)) & 1u) continue;
#pragma unroll
          for (int e = 0; e < E; ++e) c[i].v[e] = (uint8_t)Code::encode(__fmul_rn(Code::decode(c[i].v[e]), ratio));
          *reinterpret_cast<Codes*>(tile + ((c0 + i) * kRows + my_row) * D + my_col) = c[i];
        }
      }
    }
#pragma unroll
    for (int c0 = 0; c0 < kSteps; c0 += C) {
      if (kSteps > C) {
        load(c0);  // a second time, from L1
      } else {
        // the values are unpacked again: kept since the maximum they would take
        // twice the registers of the rows
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) asm volatile("" : "+r"(x[i].w[c]));
      }
      if (odd) {
        // NaN -> 0, an infinity -> what the largest code of its sign stands for
        const uint32_t most = Bits<T>::finite(__fmul_rn(Code::kMax, s_new));
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[i].w[c] = Bits<T>::replace_odd(x[i].w[c], most);
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        if (!((written >> (c0 + i)) & 1u)) continue;
        Vec<uint32_t, E / 4> c;
#pragma unroll
        for (int e = 0; e < E; e += 4)
          c.v[e / 4] = Code::encode4(__fmul_rn(x[i].get(e), inv), __fmul_rn(x[i].get(e + 1), inv),
                                     __fmul_rn(x[i].get(e + 2), inv), __fmul_rn(x[i].get(e + 3), inv));
        *reinterpret_cast<Vec<uint32_t, E / 4>*>(tile + ((c0 + i) * kRows + my_row) * D + my_col) = c;
      }
    }
    if (lane == 0 && (fresh || s_new != s_old)) *scale_at = s_new;
  }
}

template <typename T, int D, typename Code>
inline cudaError_t launch_append_q8(const void* k, const void* v, void* pool, const int64_t* slots,
                                    int32_t num_tokens, int32_t num_kv_heads, int32_t num_blocks, cudaStream_t st) {
  // Eight planes a CTA, one for each warp, and as few entries as leave all CTAs
  // resident at once (8 heads: 2048 prompt tokens 8.5 us by 16 entries, 11.1 by 4,
  // 12.5 by 64; 8192 tokens 17.5 us by 64, 27.3 by 16; a step of 256 requests 6.3 us
  // by 2, 6.9 by 1, 8.2 by 4). Lists too long for that get more planes into a CTA,
  // for fewer looks at the list (131072 tokens 245 us, 371 with eight planes).
  const int64_t planes = (int64_t)2 * num_kv_heads, resident = (int64_t)kAppendQ8CtasPerSm * device_sm_count();
  int64_t group = std::min<int64_t>(planes, kAppendQ8Warps);
  int32_t run = 1;
  auto chunks = [&]() { return ((int64_t)num_tokens + run - 1) / run; };
  auto groups = [&]() { return (planes + group - 1) / group; };
  while (run < kAppendQ8Run && chunks() * groups() > resident) run *= 2;
  while (group < planes && chunks() * groups() > 2 * resident) group = std::min(2 * group, planes);
  const dim3 grid((unsigned)chunks(), (unsigned)groups());
  append_q8_kernel<T, D, Code><<<grid, kAppendQ8Warps * 32, 0, st>>>(
      reinterpret_cast<const T*>(k), reinterpret_cast<const T*>(v), reinterpret_cast<uint8_t*>(pool), slots,
      num_tokens, num_kv_heads, (int64_t)num_blocks * 16, q8_layout(num_kv_heads, D), run, (int32_t)group);
  return cudaGetLastError();
}

}  // namespace pagedkv
