// Split-KV paged decode over an 8-bit pool (int8 or e4m3 codes, one fp32 scale
// per (block, K|V, head) tile), head_dim 64 or 128, up to 16 query heads per KV
// head, bf16 or fp32 queries and outputs.
//
//     s_t = scale * k_b * <q, c^K_t>,   out = sum_t softmax(s)_t v_b c^V_t
//
// for token t of block b with codes c and tile scales k_b, v_b. Codes are exact
// in fp16, so the matrix instructions work on the codes themselves and the
// scales stay in fp32 beside them: k_b on a block's 16 scores, v_b on its
// probabilities before those are rounded to fp16.
//
// Bound by the pool bytes read once: 2 * D bytes per token and KV head, half of
// a bf16 pool's, so there is half the time for the same arithmetic. Hence:
//  * S^T = K Q^T and O^T = V^T P^T: the codes are the A operand of m16n8k16 (16
//    tokens, or 16 head dims, by 16), the query heads its N. A group of up to 8
//    heads fills one N tile; with the heads as M instead half of each
//    instruction, and of every softmax register, would be padding.
//  * One ldmatrix word holds 4 codes of one token (K) or of 2 head dims x 2
//    tokens (V, transposed in 16-bit units). Unpacked in place these are the A
//    fragments of a K axis (K) or M axis (V) in another order, and that order is
//    undone where it is free: in the query fragments and in the output's rows.
//    int8: two byte permutes put codes + 128 under the exponent of 1024, one
//    fp16x2 subtraction leaves them exact (5 instructions per 4 codes); e4m3:
//    the hardware conversion.
//  * The reference a head's exponentials are taken against rises only when a
//    score exceeds it by more than 2^8, which one warp vote finds out; the
//    shuffles of a true running maximum are left out of the common block.
//
// Two references per head: m for the sum l = sum 2^(x - m), and n for what is
// fed to the tensor core, P = 2^(x + log2 v_b - n + 7), whose largest value lies
// in [2^7, 2^15] whatever the V scales are: fp16 holds P to 2^-11 relative down
// to 2^-21 of the head's largest, and to 2^-32 of that largest below.
//
// fp32 queries: q (scaled per head by a power of two) and P are split into two
// fp16 terms each (22 significand bits), each term its own MMA.
//
// Staging, work list and partitions are those of decode_staged.cuh: a ring of
// TMA boxes per warp (here one box of K and V per block), one CTA per
// (partition, KV head, sequence) or, from kWorkListPartitions on, resident CTAs
// that take them from the plan's list; partition_merge_kernel joins them.
#pragma once

#include <type_traits>

#include "decode_staged.cuh"
#include "q8_common.cuh"

namespace pagedkv {

constexpr int kQ8Warps = 4;
constexpr int kQ8RingBytes = 16384;  // per warp: 4 blocks of head_dim 128, 8 of 64
constexpr int kQ8Smem = kQ8Warps * kQ8RingBytes + 1024;
constexpr float kQ8Raise = 8.0f;     // a reference rises past this excess (log2)
constexpr float kQ8Lift = 7.0f;      // P is held 2^7 higher than its reference says: at most 2^15 in fp16
constexpr float kQ8NoRef = -1e30f;   // reference n before any V scale was seen (finite: n - n stays 0)

template <int D>
struct Q8Tile {
  static constexpr int kLines = 16 * D / 128;        // 128-byte lines of a K or V tile
  static constexpr int kBytes = 16 * D;              // a K or V tile
  static constexpr int kStage = 2 * kBytes;
  static constexpr int kStages = kQ8RingBytes / kStage;
  // Byte offset of 16-byte chunk c of token t in a tile, 128-byte swizzle: the
  // chunk's place in its line is XORed with the line's index, so the 8 rows of
  // an ldmatrix fall in 8 different bank groups for both head sizes.
  __device__ __forceinline__ static uint32_t chunk(int t, int c) {
    if constexpr (D == 128) return (uint32_t)(t * 128 + ((c ^ (t & 7)) << 4));
    const int line = t >> 1;
    return (uint32_t)(line * 128 + ((((t & 1) * 4 + c) ^ (line & 7)) << 4));
  }
};

struct Q8Shared {
  uint64_t bars[kQ8Warps][8];
  float red_m[kQ8Warps][16];
  float red_l[kQ8Warps][16];
  int32_t next_item;
  int32_t abort;
};

// Four codes of one word -> two fp16 pairs: (b0, b1), (b2, b3) of the bytes.
__device__ __forceinline__ void q8_unpack(CodeInt8, uint32_t w, bool interleaved, uint32_t& p, uint32_t& q) {
  const uint32_t u = w ^ 0x80808080u;  // code + 128
  const uint32_t a = __byte_perm(u, 0x64646464u, interleaved ? 0x4240 : 0x4140);
  const uint32_t b = __byte_perm(u, 0x64646464u, interleaved ? 0x4341 : 0x4342);
  const uint32_t bias = 0x64806480u;   // 1024 + 128
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p) : "r"(a), "r"(bias));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(q) : "r"(b), "r"(bias));
}
__device__ __forceinline__ void q8_unpack(CodeE4m3, uint32_t w, bool interleaved, uint32_t& p, uint32_t& q) {
  if (interleaved) w = __byte_perm(w, 0, 0x3120);  // (b0, b2), (b1, b3)
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(p), "=r"(q)
      : "r"(w));
}

// D = A * B + D, A 16x16 fp16 (row), B 16x8 fp16 (col), D 16x8 fp32.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements held across the warp.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// The fp16 pair closest to what (hi-part pair) leaves of (lo, hi).
__device__ __forceinline__ uint32_t pack_f16x2_rest(float lo, float hi, uint32_t head) {
  const __half2 h = *reinterpret_cast<const __half2*>(&head);
  return pack_f16x2(lo - __low2float(h), hi - __high2float(h));
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Attention over partition `part` of sequence b for KV head g (all G query
// heads, NT = ceil(G / 8) tiles of 8). `phase` as in decode_partition.
template <typename T, int D, int NT, typename Code>
__device__ __forceinline__ void decode_q8_partition(const CUtensorMap& tmap, const DecodeParams& p,
                                                    const Q8Layout& lay, uint8_t* smem, Q8Shared& sh, int32_t part,
                                                    int32_t g, int32_t b, int32_t L, uint32_t& phase) {
  using Tile = Q8Tile<D>;
  constexpr int S = Tile::kStages;
  constexpr int KK = D / 16;                              // k-steps of QK, row tiles of PV
  constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;           // fp16 terms of q and P
  constexpr int kRow = D + 8;                             // floats per row of the merge buffer
  static_assert(kQ8Warps * 8 * NT * kRow * 4 <= kQ8Warps * kQ8RingBytes, "the merge buffer reuses the stages");
  const int32_t warp = threadIdx.x >> 5;
  const int32_t lane = threadIdx.x & 31;
  const int32_t gid = lane >> 2;
  const int32_t tig = lane & 3;
  const int32_t G = p.group;
  const int32_t H = p.num_heads;

  const int32_t PT = p.partition_tokens;
  const int32_t nparts = (L + PT - 1) / PT;
  const int32_t t0 = part * PT;
  const int32_t t1 = min(t0 + PT, L);
  const int32_t nb = (t1 - t0 + 15) >> 4;
  const int32_t my = nb > warp ? (nb - warp + kQ8Warps - 1) / kQ8Warps : 0;
  uint8_t* wsm = smem + warp * kQ8RingBytes;
  const uint32_t wsm_addr = smem_addr(wsm);
  const int32_t* table = p.block_tables + (size_t)b * p.max_blocks + (t0 >> 4);

  // lane i holds the id of the warp's i-th block and, once they arrive, its scales
  const int32_t my_blk = lane < my ? __ldg(table + warp + lane * kQ8Warps) : -1;
  const bool my_ok = my_blk >= 0 && my_blk < p.num_blocks;
  if (lane < my && !my_ok) raise_device_error(PA_DEVERR_BLOCK);
  const uint32_t ok_mask = __ballot_sync(0xffffffffu, my_ok);

  auto issue = [&](int32_t i) {
    const int32_t s = i % S;
    const int32_t blk = __shfl_sync(0xffffffffu, my_blk, i);
    if (lane == 0) {
      uint64_t* bar = &sh.bars[warp][s];
      if ((ok_mask >> i) & 1u) {
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(bar, Tile::kStage);
        tma_load_5d(wsm + s * Tile::kStage, &tmap, bar, 0, 0, g, 0, blk);
      } else {
        mbar_arrive(bar);
      }
    }
  };
  const int32_t npre = my < S ? my : S;
  for (int32_t i = 0; i < npre; ++i) issue(i);

  float my_ks = 0.f, my_lv = 0.f;  // K scale; log2 of the V scale
  if (my_ok) {
    const uint8_t* pool = reinterpret_cast<const uint8_t*>(p.pool);
    my_ks = __ldg(reinterpret_cast<const float*>(pool + q8_scale_at(lay, my_blk, 0, g, p.num_kv_heads)));
    my_lv = log2f(__ldg(reinterpret_cast<const float*>(pool + q8_scale_at(lay, my_blk, 1, g, p.num_kv_heads))));
  }

  // Query fragments: B of S^T = K Q^T, head 8 nt + gid, dims 16 kk + 4 tig + (0, 1 | 2, 3),
  // scaled per head so that its largest magnitude lies in [2^14, 2^15).
  uint32_t qb[TERMS][NT][KK][2];
  float sfac[NT][2];  // scale * log2 e / that power of two, heads 8 nt + 2 tig (+ 1)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int32_t head = 8 * nt + gid;
    float x[KK][4];
    float a = 0.f;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      if (head < G) {
        load_f32<T, 4>(reinterpret_cast<const T*>(p.q) + ((size_t)b * H + (size_t)g * G + head) * D + 16 * kk + 4 * tig,
                       x[kk]);
      } else {
        x[kk][0] = x[kk][1] = x[kk][2] = x[kk][3] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) a = fmaxf(a, fabsf(x[kk][i]));
    }
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    // exponent of a, kept where both powers of two below are normal
    const int32_t e = max((int32_t)(__float_as_uint(a) >> 23) - 127, -100);
    const float up = __uint_as_float((uint32_t)(127 + 14 - min(e, 127)) << 23);
    const float down = p.scale_log2 * __uint_as_float((uint32_t)max(127 - 14 + min(e, 127), 1) << 23);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float lo = x[kk][2 * j] * up, hi = x[kk][2 * j + 1] * up;
        qb[0][nt][kk][j] = pack_f16x2(lo, hi);
        if constexpr (TERMS == 2) qb[1][nt][kk][j] = pack_f16x2_rest(lo, hi, qb[0][nt][kk][j]);
      }
    }
    sfac[nt][0] = __shfl_sync(0xffffffffu, down, 8 * tig);
    sfac[nt][1] = __shfl_sync(0xffffffffu, down, 8 * tig + 4);
  }

  float o[KK][NT][4];
  float m[NT][2], n[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m[nt][j] = -INFINITY;
      n[nt][j] = kQ8NoRef;
      l[nt][j] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < KK; ++c) o[c][nt][0] = o[c][nt][1] = o[c][nt][2] = o[c][nt][3] = 0.f;
  }

  for (int32_t i = 0; i < my; ++i) {
    const int32_t s = i % S;
    const bool arrived = mbar_wait_bounded(&sh.bars[warp][s], (phase >> s) & 1u, kWaitLimitNs);
    if (__any_sync(0xffffffffu, !arrived)) {
      // as in decode_partition: report, let the copies in flight land, drop this warp's state
      if (lane == 0) raise_device_error(PA_DEVERR_TIMEOUT);
      const int32_t issued = min(i + S, my);
      for (int32_t k = i; k < issued; ++k) {
        const int32_t sk = k % S;
        mbar_wait_bounded(&sh.bars[warp][sk], (phase >> sk) & 1u, kWaitLimitNs);
        phase ^= 1u << sk;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int c = 0; c < KK; ++c) o[c][nt][0] = o[c][nt][1] = o[c][nt][2] = o[c][nt][3] = 0.f;
      }
      if (lane == 0) sh.abort = 1;
      break;
    }
    phase ^= 1u << s;
    const int32_t nvalid = min(16, t1 - (t0 + (warp + i * kQ8Warps) * 16));
    const bool valid = (ok_mask >> i) & 1u;
    uint8_t* stg = wsm + s * Tile::kStage;
    const uint32_t st = wsm_addr + s * Tile::kStage;
    const float ks = __shfl_sync(0xffffffffu, my_ks, i);
    const float lv = __shfl_sync(0xffffffffu, my_lv, i);
    if constexpr (std::is_same<Code, CodeE4m3>::value) {
      // rows behind the sequence end may hold NaN codes, which a zero
      // probability does not silence: their V rows become zero
      if (valid && nvalid < 16) {
        for (int32_t e = lane; e < (16 - nvalid) * (D / 16); e += 32)
          *reinterpret_cast<uint4*>(stg + Tile::kBytes + Tile::chunk(nvalid + e / (D / 16), e % (D / 16))) =
              make_uint4(0, 0, 0, 0);
        __syncwarp();
      }
    }

    // S^T: rows = tokens (gid, gid + 8), columns = heads (2 tig, 2 tig + 1)
    float sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
    const int32_t tok = (lane & 7) + (((lane >> 3) & 1) << 3);
    if (valid) {
      float sc2[NT][4];  // odd k-steps: two shorter chains of dependent MMAs
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc2[nt][0] = sc2[nt][1] = sc2[nt][2] = sc2[nt][3] = 0.f;
#pragma unroll
      for (int c = 0; c < KK; c += 2) {
        uint32_t r[4];
        ldsm_x4(st + Tile::chunk(tok, c + (lane >> 4)), r[0], r[1], r[2], r[3]);
        uint32_t a0[4], a1[4];
        q8_unpack(Code{}, r[0], false, a0[0], a0[2]);
        q8_unpack(Code{}, r[1], false, a0[1], a0[3]);
        q8_unpack(Code{}, r[2], false, a1[0], a1[2]);
        q8_unpack(Code{}, r[3], false, a1[1], a1[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int term = 0; term < TERMS; ++term) {
            mma_f16_16816(sc[nt], a0, qb[term][nt][c][0], qb[term][nt][c][1]);
            mma_f16_16816(sc2[nt], a1, qb[term][nt][c + 1][0], qb[term][nt][c + 1][1]);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] += sc2[nt][e];
    }
    bool exceeds = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int32_t row = gid + (e >> 1) * 8;
        const float x = row < nvalid ? sc[nt][e] * (sfac[nt][e & 1] * ks) : -INFINITY;
        sc[nt][e] = x;
        exceeds |= x > m[nt][e & 1] + kQ8Raise || x + lv > n[nt][e & 1] + kQ8Raise;
      }
    }
    if (__any_sync(0xffffffffu, exceeds)) {
      // both references to the largest score so far
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float bm = fmaxf(sc[nt][j], sc[nt][j + 2]);
          bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
          bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
          bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
          const float mn = fmaxf(m[nt][j], bm), nn = fmaxf(n[nt][j], bm + lv);
          const float am = ex2_ftz(m[nt][j] - mn), an = ex2_ftz(n[nt][j] - nn);
          m[nt][j] = mn;
          n[nt][j] = nn;
          l[nt][j] *= am;
#pragma unroll
          for (int c = 0; c < KK; ++c) {
            o[c][nt][j] *= an;
            o[c][nt][j + 2] *= an;
          }
        }
      }
    }
    uint32_t pb[TERMS][NT][2];  // B of O^T = V^T P^T: head gid, tokens 2 tig (+ 1), + 8
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pv[e] = ex2_ftz(sc[nt][e] + (lv + kQ8Lift - n[nt][e & 1]));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        l[nt][j] += ex2_ftz(sc[nt][j] - m[nt][j]) + ex2_ftz(sc[nt][j + 2] - m[nt][j]);
      const uint32_t w0 = pack_f16x2(pv[0], pv[1]), w1 = pack_f16x2(pv[2], pv[3]);
      pb[0][nt][0] = transpose_8x8(w0);
      pb[0][nt][1] = transpose_8x8(w1);
      if constexpr (TERMS == 2) {
        pb[1][nt][0] = transpose_8x8(pack_f16x2_rest(pv[0], pv[1], w0));
        pb[1][nt][1] = transpose_8x8(pack_f16x2_rest(pv[2], pv[3], w1));
      }
    }
    if (valid) {
#pragma unroll
      for (int c = 0; c < KK; c += 2) {
        uint32_t r[4];
        ldsm_x4_trans(st + Tile::kBytes + Tile::chunk(tok, c + (lane >> 4)), r[0], r[1], r[2], r[3]);
        uint32_t a0[4], a1[4];
        q8_unpack(Code{}, r[0], true, a0[0], a0[1]);
        q8_unpack(Code{}, r[1], true, a0[2], a0[3]);
        q8_unpack(Code{}, r[2], true, a1[0], a1[1]);
        q8_unpack(Code{}, r[3], true, a1[2], a1[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int term = 0; term < TERMS; ++term) {
            mma_f16_16816(o[c][nt], a0, pb[term][nt][0], pb[term][nt][1]);
            mma_f16_16816(o[c + 1][nt], a1, pb[term][nt][0], pb[term][nt][1]);
          }
        }
      }
    }
    __syncwarp();
    if (i + S < my) issue(i + S);
  }

  // ---- merge of the four warps' states -----------------------------------------
  __syncthreads();  // every warp has consumed all its stages
  float* so = reinterpret_cast<float*>(smem);  // [4 warps][8 NT heads][kRow]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float ls = l[nt][j];
      ls += __shfl_xor_sync(0xffffffffu, ls, 4);
      ls += __shfl_xor_sync(0xffffffffu, ls, 8);
      ls += __shfl_xor_sync(0xffffffffu, ls, 16);
      const int32_t head = 8 * nt + 2 * tig + j;
      if (gid == 0) {
        sh.red_m[warp][head] = m[nt][j];
        sh.red_l[warp][head] = ls;
      }
      // the accumulators in units of 2^m, like l (a warp without blocks holds zeros)
      const float f = m[nt][j] > -INFINITY ? exp2f(n[nt][j] - kQ8Lift - m[nt][j]) : 0.f;
      float* row = so + (warp * 8 * NT + head) * kRow + 2 * gid;
#pragma unroll
      for (int c = 0; c < KK; ++c)
        *reinterpret_cast<float2*>(row + 16 * c) = make_float2(o[c][nt][j] * f, o[c][nt][j + 2] * f);
    }
  }
  __syncthreads();

  T* out = reinterpret_cast<T*>(p.out);
  for (int32_t i = threadIdx.x; i < G * D; i += blockDim.x) {
    const int32_t h = i / D;
    const int32_t d = i % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) M = fmaxf(M, sh.red_m[w][h]);
    float Ls = 0.f, A = 0.f;
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) {
      const float e = exp2f(sh.red_m[w][h] - M);  // 0 for a warp that had no block
      Ls = fmaf(sh.red_l[w][h], e, Ls);
      A = fmaf(so[(w * 8 * NT + h) * kRow + d], e, A);
    }
    const size_t bh = (size_t)b * H + (size_t)g * G + h;
    if (nparts == 1) {
      out[bh * D + d] = Elem<T>::from_f32(A / Ls);
    } else {
      p.ws_acc[(bh * p.max_partitions + part) * D + d] = A;
      if (d == 0) {
        p.ws_ml[(bh * p.max_partitions + part) * 2] = M;
        p.ws_ml[(bh * p.max_partitions + part) * 2 + 1] = Ls;
      }
    }
  }
}

template <typename T, int D, int NT, typename Code>
__global__ void __launch_bounds__(kQ8Warps * 32)
decode_q8_kernel(const __grid_constant__ CUtensorMap tmap, DecodeParams p, Q8Layout lay) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Q8Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int32_t warp = threadIdx.x >> 5;
  const int32_t lane = threadIdx.x & 31;
  grid_dependents_launch();
  int32_t grid_len = 0;
  if (p.work_items == nullptr) {
    const int32_t part = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    grid_len = checked_len(p, b, part == 0 && g == 0 && threadIdx.x == 0);
    if (grid_len == 0) {
      if (part == 0) {
        T* out = reinterpret_cast<T*>(p.out);
        for (int32_t i = threadIdx.x; i < p.group * D; i += blockDim.x)
          out[((size_t)b * p.num_heads + (size_t)g * p.group) * D + i] = Elem<T>::from_f32(0.f);
      }
      return;
    }
    if (part >= (grid_len + p.partition_tokens - 1) / p.partition_tokens) return;
  }
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < Q8Tile<D>::kStages; ++s) mbar_init(&sh.bars[warp][s], 1);
    fence_barrier_init();
    if (warp == 0) prefetch_tensormap(&tmap);
  }
  __syncwarp();
  uint32_t phase = 0;
  if (p.work_items == nullptr) {
    decode_q8_partition<T, D, NT, Code>(tmap, p, lay, smem, sh, blockIdx.x, blockIdx.y, blockIdx.z, grid_len, phase);
    return;
  }
  grid_dependency_wait();  // the plan kernel's item list is complete
  const int32_t total = __ldcg(p.work_header) * p.num_kv_heads;
  if (threadIdx.x == 0) {
    sh.next_item = atomicAdd(p.work_header + 1, 1);
    sh.abort = 0;
  }
  __syncthreads();
  int32_t item = sh.next_item;
  while (item < total && !sh.abort) {
    int32_t next = 0;
    if (threadIdx.x == 0) next = atomicAdd(p.work_header + 1, 1);  // in flight during the item
    const uint32_t bp = (uint32_t)__ldcg(p.work_items + item / p.num_kv_heads);
    const int32_t g = item % p.num_kv_heads;
    const int32_t b = (int32_t)(bp >> 16);
    decode_q8_partition<T, D, NT, Code>(tmap, p, lay, smem, sh, (int32_t)(bp & 0xffffu), g, b,
                                        checked_len(p, b, false), phase);
    fence_proxy_async_smem();  // the item's shared-memory reads precede the next item's TMA writes
    if (threadIdx.x == 0) sh.next_item = next;
    __syncthreads();
    item = sh.next_item;
  }
}

// ---- host side ---------------------------------------------------------------

// Tensor map of an 8-bit pool's codes: (byte of a 128-byte line, line of the
// tile, kv head, K|V, block); box = the K and V tiles of one (block, head).
inline pa_status encode_q8_map(const void* pool, int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks,
                               CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t tile = (cuuint64_t)16 * head_dim;
  const cuuint64_t hkv = (cuuint64_t)num_kv_heads;
  const cuuint64_t dims[5] = {128, tile / 128, hkv, 2, (cuuint64_t)num_blocks};
  const cuuint64_t strides[4] = {128, tile, hkv * tile, (cuuint64_t)q8_layout(num_kv_heads, head_dim).block_bytes};
  const cuuint32_t box[5] = {128, (cuuint32_t)(tile / 128), 1, 2, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(pool), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return PA_OK;
}

template <typename T, int D, int NT, typename Code>
inline pa_status launch_decode_q8(const DecodeParams& p, cudaStream_t st) {
  CUtensorMap map;
  pa_status s = encode_q8_map(p.pool, p.num_kv_heads, D, p.num_blocks, &map);
  if (s != PA_OK) return s;
  auto kernel = decode_q8_kernel<T, D, NT, Code>;
  static PerDevice<int32_t> occupancy;  // resident CTAs per SM, with the shared-memory limit set once per device
  int32_t per_sm = 1;
  cudaError_t e = occupancy.get(&per_sm, [&](int32_t* v) {
    int32_t n = 0;
    cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kQ8Smem);
    if (r == cudaSuccess) r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kQ8Warps * 32, kQ8Smem);
    *v = n > 0 ? n : 1;
    return r;
  });
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_decode_q8: %s", cudaGetErrorString(e));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kQ8Warps * 32);
  cfg.dynamicSmemBytes = kQ8Smem;
  cfg.stream = st;
  if (p.work_items == nullptr) {
    cfg.gridDim = dim3(p.max_partitions, p.num_kv_heads, p.num_seqs);
  } else {
    cudaLaunchConfig_t plan = {};
    plan.gridDim = dim3(1);
    plan.blockDim = dim3(kPlanThreads);
    plan.stream = st;
    plan.attrs = attr;
    plan.numAttrs = 1;
    e = cudaLaunchKernelEx(&plan, decode_plan_kernel<(int32_t)(D * sizeof(T) / 16)>, p);
    if (e != cudaSuccess)
      return fail(PA_ERR_CUDA, "pa_decode_q8 (plan): launch failed: %s", cudaGetErrorString(e));
    const int64_t most = (int64_t)p.num_seqs * p.max_partitions * p.num_kv_heads;
    const int64_t resident = (int64_t)per_sm * device_sm_count();
    cfg.gridDim = dim3((unsigned)(most < resident ? most : resident));
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  e = cudaLaunchKernelEx(&cfg, kernel, map, p, q8_layout(p.num_kv_heads, D));
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_decode_q8: launch failed: %s", cudaGetErrorString(e));
  if (p.max_partitions <= 1) return PA_OK;
  e = launch_partition_merge<T, D, true>(p, st);
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_decode_q8 (merge): launch failed: %s", cudaGetErrorString(e));
  return PA_OK;
}

template <typename T, int D>
inline pa_status launch_decode_q8_code(const DecodeParams& p, int32_t dtype, cudaStream_t st) {
  if (dtype == PA_Q8_INT8)
    return p.group <= 8 ? launch_decode_q8<T, D, 1, CodeInt8>(p, st) : launch_decode_q8<T, D, 2, CodeInt8>(p, st);
  return p.group <= 8 ? launch_decode_q8<T, D, 1, CodeE4m3>(p, st) : launch_decode_q8<T, D, 2, CodeE4m3>(p, st);
}

}  // namespace pagedkv
