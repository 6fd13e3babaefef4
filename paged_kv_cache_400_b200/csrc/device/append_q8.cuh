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
// in slot_mapping (its leader) gathers the block's other tokens from the 31
// entries behind it, and the warps of those other tokens leave at once. A row
// named twice takes the later token.
//
// Bound by its bytes (reads T * Hkv * D elements twice over for K and V, writes
// half or a quarter as many) for many tokens, by latency for few: a step of one
// token per request gives every token a warp per (K|V, head), and all of a
// tile's rows are loaded before the first is used.
#pragma once

#include "q8_common.cuh"

namespace pagedkv {

constexpr int kAppendQ8Warps = 4;
constexpr int kAppendWindow = 32;  // a block's tokens lie within this many entries
constexpr float kQ8Tiny = 7.888609052210118e-31f;  // 2^-100: below it a tile counts as zeros (1 / s stays finite)

// Warp (4 x + w, head y, kv z) serves the leaders among tokens
// [per_warp * (4 x + w), + per_warp).
template <typename T, int D, typename Code>
__global__ void __launch_bounds__(kAppendQ8Warps * 32)
append_q8_kernel(const T* __restrict__ k, const T* __restrict__ v, uint8_t* __restrict__ pool,
                 const int64_t* __restrict__ slots, int32_t num_tokens, int32_t num_kv_heads, int64_t num_slots,
                 Q8Layout lay, int32_t per_warp) {
  constexpr int PER = D / 32;  // elements of a row per lane
  using In = Vec<T, PER>;
  using Codes = Vec<uint8_t, PER>;
  __shared__ __align__(16) uint8_t row_src[kAppendQ8Warps][16];
  const int32_t warp = threadIdx.x >> 5;
  const int32_t lane = threadIdx.x & 31;
  const int32_t h = blockIdx.y;
  const int32_t kv = blockIdx.z;
  const T* src = kv ? v : k;
  // block of entry t, -1 for padding, an entry outside the list or a bad slot
  auto block_of = [&](int64_t t, int64_t& s) -> int64_t {
    s = t >= 0 && t < num_tokens ? __ldg(slots + t) : -1;
    return s >= 0 && s < num_slots ? s >> 4 : -1;
  };
  const int64_t t_first = ((int64_t)blockIdx.x * kAppendQ8Warps + warp) * per_warp;
  const int64_t t_end = min(t_first + per_warp, (int64_t)num_tokens);
  for (int64_t t = t_first; t < t_end; ++t) {
    int64_t s, s_prev, s_next;
    const int64_t blk_here = block_of(t + lane, s);              // entries t .. t + 31
    const int64_t blk_prev = block_of(t - 31 + lane, s_prev);    // entries t - 31 .. t (lane 31: t itself)
    const int64_t blk_next = block_of(t + 32 + lane, s_next);    // entries t + 32 .. t + 63
    const int64_t blk = __shfl_sync(0xffffffffu, blk_here, 0);
    if (blk < 0) {
      if (lane == 0 && s >= num_slots && h == 0 && kv == 0) raise_device_error(PA_DEVERR_SLOT);
      continue;
    }
    if (__any_sync(0xffffffffu, lane < 31 && blk_prev == blk)) continue;  // an earlier entry leads
    // tokens of the block behind the window are not written
    if (__any_sync(0xffffffffu, lane < 31 && blk_next == blk) && lane == 0 && h == 0 && kv == 0)
      raise_device_error(PA_DEVERR_SLOT);

    uint8_t* tile = pool + (size_t)blk * lay.block_bytes + ((size_t)kv * num_kv_heads + h) * 16 * D;
    float* scale_at = reinterpret_cast<float*>(pool + q8_scale_at(lay, blk, kv, h, num_kv_heads));
    const float s_old = *scale_at;

    // row -> entry of the window (0xff: not written now)
    const bool member = blk_here == blk;
    if (lane < 16) row_src[warp][lane] = 0xff;
    __syncwarp();
    const uint32_t same = __match_any_sync(0xffffffffu, member ? (int32_t)(s & 15) : 16 + lane);
    if (member && (same >> lane) == 1u) row_src[warp][s & 15] = (uint8_t)lane;  // the latest of its row
    __syncwarp();
    const uint4 rs = *reinterpret_cast<const uint4*>(row_src[warp]);
    const uint32_t rsw[4] = {rs.x, rs.y, rs.z, rs.w};
    __syncwarp();

    In x[16];
    float amax = 0.f;
    bool odd = false;  // a non-finite element
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const uint32_t e = (rsw[r >> 2] >> (8 * (r & 3))) & 0xffu;
      if (e != 0xffu)
        x[r] = *reinterpret_cast<const In*>(src + ((size_t)(t + e) * num_kv_heads + h) * D + lane * PER);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if (((rsw[r >> 2] >> (8 * (r & 3))) & 0xffu) == 0xffu) continue;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float a = fabsf(Elem<T>::to_f32(x[r].v[i]));
        if (a <= FLT_MAX) amax = fmaxf(amax, a);
        else odd = true;
      }
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if (__any_sync(0xffffffffu, odd) && lane == 0) raise_device_error(PA_DEVERR_NONFINITE);
    if (amax < kQ8Tiny) amax = 0.f;
    const bool fresh = (rsw[0] & 0xffu) != 0xffu;
    const float s_new = fresh ? __fmul_rn(amax, Code::kInvMax) : Code::grown(s_old, amax);
    const float inv = s_new > 0.f ? __fdiv_rn(1.f, s_new) : 0.f;

    if (!fresh && s_new > s_old) {
      // rows that stay: coded again at the grown scale
      const float ratio = __fdiv_rn(s_old, s_new);
      Codes c[16];
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (((rsw[r >> 2] >> (8 * (r & 3))) & 0xffu) == 0xffu)
          c[r] = *reinterpret_cast<const Codes*>(tile + r * D + lane * PER);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (((rsw[r >> 2] >> (8 * (r & 3))) & 0xffu) != 0xffu) continue;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          c[r].v[i] = (uint8_t)Code::encode(__fmul_rn(Code::decode(c[r].v[i]), ratio));
        *reinterpret_cast<Codes*>(tile + r * D + lane * PER) = c[r];
      }
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if (((rsw[r >> 2] >> (8 * (r & 3))) & 0xffu) == 0xffu) continue;
      Codes c;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        float y = Elem<T>::to_f32(x[r].v[i]);
        if (!(fabsf(y) <= FLT_MAX)) y = y != y ? 0.f : copysignf(FLT_MAX, y);  // NaN -> 0, inf -> the largest code
        c.v[i] = (uint8_t)Code::encode(__fmul_rn(y, inv));
      }
      *reinterpret_cast<Codes*>(tile + r * D + lane * PER) = c;
    }
    if (lane == 0 && (fresh || s_new != s_old)) *scale_at = s_new;
  }
}

template <typename T, int D, typename Code>
inline cudaError_t launch_append_q8(const void* k, const void* v, void* pool, const int64_t* slots,
                                    int32_t num_tokens, int32_t num_kv_heads, int32_t num_blocks, cudaStream_t st) {
  // One token per warp while that keeps the warps to a few per SM (a decode
  // step: every token leads a tile of its own); with more, a warp goes through
  // up to 16 entries, of which a prompt's tokens make one or two tiles.
  const int64_t tiles = (int64_t)num_tokens * num_kv_heads * 2;
  int32_t per_warp = 1;
  while (per_warp < 16 && tiles / per_warp > (int64_t)64 * device_sm_count()) per_warp *= 2;
  const int64_t per_cta = (int64_t)per_warp * kAppendQ8Warps;
  const dim3 grid((unsigned)((num_tokens + per_cta - 1) / per_cta), (unsigned)num_kv_heads, 2);
  append_q8_kernel<T, D, Code><<<grid, kAppendQ8Warps * 32, 0, st>>>(
      reinterpret_cast<const T*>(k), reinterpret_cast<const T*>(v), reinterpret_cast<uint8_t*>(pool), slots,
      num_tokens, num_kv_heads, (int64_t)num_blocks * 16, q8_layout(num_kv_heads, D), per_warp);
  return cudaGetLastError();
}

}  // namespace pagedkv
