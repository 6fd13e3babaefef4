// Cache append into an 8-bit pool: each new K/V row coded into its slot, with
// one scale per (block, K|V, head) tile.
//
// With A the largest finite magnitude of a tile's new rows (0 below 2^-100),
// the tile's scale s becomes first(A) when its row 0 is among them, grown(s, A)
// otherwise (q8_common.cuh), rows it keeps are coded again where s grew, and a
// new element is stored as the code nearest to x * (1 / s).
//
// One warp owns a tile, so a scale and the rows under it change together and
// nothing is summed or ordered across warps: the warp of a block's first token
// in slot_mapping (its leader: none of the 31 entries before it names the block)
// gathers the block's other tokens behind it, as long as each lies within 31
// entries of the one before; these lead nothing. A row named twice takes the
// later token. A block that comes back after a longer gap has a second leader,
// which writes at the same time: requests that share a prefix and are admitted
// in one step name its whole blocks with the same values, so both start the
// tile afresh and store the same bytes.
//
// Bound by its bytes (reads T * Hkv * D elements twice over for K and V, writes
// half or a quarter as many) for many tokens, by latency for few. A warp looks
// at a run of entries at once, with the entries before and behind them, and
// then serves their leaders: the scale and all new rows of a tile are in flight
// together, 16 bytes a lane, and stay in registers between the maximum and the
// codes.
#pragma once

#include "q8_common.cuh"

namespace pagedkv {

constexpr int kAppendQ8Warps = 4;
constexpr int kAppendQ8Run = 16;                   // most entries a warp looks at
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

// Warp (4 x + w, head y, kv z) serves the leaders among entries
// [run * (4 x + w), + run).
template <typename T, int D, typename Code>
__global__ void __launch_bounds__(kAppendQ8Warps * 32, 6)
append_q8_kernel(const T* __restrict__ k, const T* __restrict__ v, uint8_t* __restrict__ pool,
                 const int64_t* __restrict__ slots, int32_t num_tokens, int32_t num_kv_heads, int64_t num_slots,
                 Q8Layout lay, int32_t run) {
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
  __shared__ int32_t row_src[kAppendQ8Warps][16];
  const int32_t warp = threadIdx.x >> 5;
  const int32_t lane = threadIdx.x & 31;
  const int32_t h = blockIdx.y;
  const int32_t kv = blockIdx.z;
  const bool reports = h == 0 && kv == 0;
  const T* src = kv ? v : k;
  const int32_t t0 = (blockIdx.x * kAppendQ8Warps + warp) * run;
  if (t0 >= num_tokens) return;
  // entry t's slot, -1 for padding, a bad slot or an entry outside the list
  auto slot_of = [&](int64_t t) -> int64_t { return t >= 0 && t < num_tokens ? __ldg(slots + t) : -1; };
  const int64_t raw0 = slot_of((int64_t)t0 + lane), raw_prev = slot_of((int64_t)t0 - 32 + lane);
  const int64_t raw1 = slot_of((int64_t)t0 + 32 + lane), raw2 = slot_of((int64_t)t0 + 64 + lane);
  auto block_of = [&](int64_t s) -> int32_t { return s >= 0 && s < num_slots ? (int32_t)(s >> 4) : -1; };
  const int32_t b0 = block_of(raw0), b_prev = block_of(raw_prev);
  if (reports && lane < run && raw0 >= num_slots) raise_device_error(PA_DEVERR_SLOT);

  // leaders: the run's first entry of a block that none of the 31 entries before it names
  const uint32_t same0 = __match_any_sync(kAll, b0);
  uint32_t todo = __ballot_sync(kAll, b0 >= 0 && lane < run && (same0 & ((1u << lane) - 1u)) == 0);
  const int32_t my_row = lane / kLanes;
  const int32_t my_col = (lane % kLanes) * E;
  while (todo) {
    const int32_t first = __ffs(todo) - 1;
    todo &= todo - 1;
    const int32_t blk = __shfl_sync(kAll, b0, first);
    if (__any_sync(kAll, b_prev == blk && lane > first)) continue;  // an earlier entry leads
    uint8_t* tile = pool + (size_t)blk * lay.block_bytes + ((size_t)kv * num_kv_heads + h) * 16 * D;
    float* scale_at = reinterpret_cast<float*>(pool + q8_scale_at(lay, blk, kv, h, num_kv_heads));
    const float s_old = *scale_at;

    // row -> its latest entry, counted from t0 (-1: not written now), 32 entries at a time
    __syncwarp();
    if (lane < 16) row_src[warp][lane] = -1;
    __syncwarp();
    int64_t raw = raw0;
    uint32_t in = __ballot_sync(kAll, b0 == blk);
    for (int32_t w = 0;;) {
      const bool member = (in >> lane) & 1u;
      const int32_t r = member ? (int32_t)(raw & 15) : 32 + lane;
      const uint32_t same = __match_any_sync(kAll, r);
      if (member && (same >> lane) == 1u) row_src[warp][r] = 32 * w + lane;
      __syncwarp();
      const int32_t last = 31 - __clz(in);  // of this window
      ++w;
      raw = w == 1 ? raw1 : w == 2 ? raw2 : slot_of((int64_t)t0 + 32 * w + lane);
      in = __ballot_sync(kAll, block_of(raw) == blk);
      if (in == 0 || __ffs(in) + 31 - last > 31) break;
    }
    const bool fresh = row_src[warp][0] >= 0;

    // rows of steps c0 .. c0 + C - 1
    Words x[C];
    uint32_t written = 0;  // bit i: this lane's row of step i is new
    auto load = [&](int c0) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int32_t e = row_src[warp][(c0 + i) * kRows + my_row];
        x[i].q = make_uint4(0, 0, 0, 0);
        if (e >= 0) {
          written |= 1u << (c0 + i);
          x[i].q = __ldg(reinterpret_cast<const uint4*>(src + ((size_t)(t0 + e) * num_kv_heads + h) * D + my_col));
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
  // One entry per warp while all warps are resident at once (24 per SM; a decode
  // step: every token leads a tile of its own: 256 tokens of 8 heads 5.6 us by
  // two entries a warp, 6.3 by one); with more, a warp takes a run of entries,
  // of which a prompt's tokens make one or two tiles.
  const int64_t tiles = (int64_t)num_tokens * num_kv_heads * 2;
  int32_t run = 1;
  while (run < kAppendQ8Run && tiles / run > (int64_t)(run == 1 ? 24 : 64) * device_sm_count()) run *= 2;
  const int64_t per_cta = (int64_t)run * kAppendQ8Warps;
  const dim3 grid((unsigned)((num_tokens + per_cta - 1) / per_cta), (unsigned)num_kv_heads, 2);
  append_q8_kernel<T, D, Code><<<grid, kAppendQ8Warps * 32, 0, st>>>(
      reinterpret_cast<const T*>(k), reinterpret_cast<const T*>(v), reinterpret_cast<uint8_t*>(pool), slots,
      num_tokens, num_kv_heads, (int64_t)num_blocks * 16, q8_layout(num_kv_heads, D), run);
  return cudaGetLastError();
}

}  // namespace pagedkv
