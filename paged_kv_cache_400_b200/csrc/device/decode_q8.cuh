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
//    e4m3: the hardware conversion. int8, fp32 queries: two byte permutes put
//    code + 128 under the exponent of 1024, one subtraction leaves the code.
//    int8, bf16 queries: the subtraction is put off; the bytes code + 128 stand
//    in fp16's subnormals, u 2^-24, and 128 times the sum of the queries, or of
//    the probabilities (one more MMA, against ones), comes off the fp32 sums.
//    The sums then err by up to 255 parts in 2^24 of a code for each term, where
//    the probabilities' rounding is 2^-11; a block takes 64 instructions less.
//  * The reference a head's exponentials are taken against rises only when an
//    exponent exceeds it by more than 8, which one warp vote finds out; the
//    shuffles of a true running maximum are left out of the common block.
//
// What the tensor core is fed is P = 2^(x + log2 v_b - n + 7) with x the score
// and n the reference of the head: its largest value lies in [2^7, 2^15]
// whatever the V scales are, so fp16 holds P to 2^-11 relative down to 2^-21 of
// the head's largest, and to 2^-32 of that largest below. n is kept as the sum
// of a score m and a log2 v_b, r: where scores are so large that fp32 spaces
// them by more than a fraction, x - m is formed first, from rounded x, so that
// the largest exponent is still what it should be. The same fp32 values of P,
// before they are rounded, give the sum l += P / v_b. A block whose V scale is 0
// adds nothing to the output, so it stays out of n, which would sink the others'
// P in fp16: its scores go into a sum of their own, with a reference of its own,
// that joins l where the warps' states are joined.
//
// fp32 queries: q (scaled per head by a power of two) and P are split into two
// fp16 terms each (22 significand bits), each term its own MMA.
//
// Staging and work list are those of decode_staged.cuh: a ring of TMA boxes per
// warp, here one box of K and V per block; one CTA per (partition, KV head,
// sequence), or resident CTAs that take them from the plan kernel's list, or a
// warp per (sequence, KV head); a merge kernel joins the partitions.
//
// Measured: 256 requests of lognormal lengths (32 heads over 8, int8) 121 to 128 us
// by machine, 5.6 to 5.9 TB/s of the pool's bytes; 64 requests with 32 KV heads,
// e4m3, 99 to 113 us, 5.6 to 6.4 TB/s, up to what a copy reaches. What is left in
// the first is the launches of plan and merge (8 us) and the ends of the items.
#pragma once

#include <algorithm>
#include <type_traits>

#include "decode_staged.cuh"
#include "q8_common.cuh"

namespace pagedkv {

constexpr int kQ8Warps = 4;
constexpr int kQ8Stages = 4;         // blocks in flight per warp
constexpr float kQ8Raise = 8.0f;     // the reference rises past this excess (log2)
constexpr float kQ8Lift = 7.0f;      // P is held 2^7 higher than its reference says: at most 2^15 in fp16
constexpr float kQ8Far = 1024.0f;    // scores (log2) from which fp32 leaves exponents less than 13 bits
constexpr float kQ8NoRef = -3e38f;   // reference before any score was seen (finite: n - n stays 0)

template <int D>
struct Q8Tile {
  static constexpr int kLines = 16 * D / 128;        // 128-byte lines of a K or V tile
  static constexpr int kBytes = 16 * D;              // a K or V tile
  static constexpr int kStage = 2 * kBytes;
  static constexpr int kStages = kQ8Stages;
  static constexpr int kRing = kStages * kStage;     // per warp
  static constexpr int kSmem = kQ8Warps * kRing + 1024;
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
  uint64_t bars[kQ8Warps][kQ8Stages];
  float red_m[kQ8Warps][16];
  float red_l[kQ8Warps][16];
  float2 zero[kQ8Warps][16];  // by head: reference and sum of the warp's blocks of V scale 0
  int32_t next_item;
  int32_t abort;
};

// The same word as four fp16 subnormals (code + 128) 2^-24.
__device__ __forceinline__ void q8_unpack_biased(uint32_t w, bool interleaved, uint32_t& p, uint32_t& q) {
  const uint32_t u = w ^ 0x80808080u;
  p = __byte_perm(u, 0, interleaved ? 0x4240 : 0x4140);
  q = __byte_perm(u, 0, interleaved ? 0x4341 : 0x4342);
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

// The fp16 pair closest to what (hi-part pair) leaves of (lo, hi).
__device__ __forceinline__ uint32_t pack_f16x2_rest(float lo, float hi, uint32_t head) {
  const __half2 h = *reinterpret_cast<const __half2*>(&head);
  return pack_f16x2(lo - __low2float(h), hi - __high2float(h));
}

// Read through L2 (written by another SM just before).
__device__ __forceinline__ Vec<float, 4> load_cg(const Vec<float, 4>* a) {
  const float4 x = __ldcg(reinterpret_cast<const float4*>(a));
  return {{x.x, x.y, x.z, x.w}};
}
__device__ __forceinline__ Vec<float, 2> load_cg(const Vec<float, 2>* a) {
  const float2 x = __ldcg(reinterpret_cast<const float2*>(a));
  return {{x.x, x.y}};
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Lane i's table entry of partition `part`: the id of block rank + i * W, where
// the table has such an entry. It does not depend on the sequence's length, so
// the two can be asked for together.
__device__ __forceinline__ int32_t q8_table_entry(const DecodeParams& p, int32_t part, int32_t b, int32_t rank,
                                                  int32_t W) {
  const int64_t e = (int64_t)part * (p.partition_tokens >> 4) + rank + (int64_t)(threadIdx.x & 31) * W;
  return e < p.max_blocks ? __ldg(p.block_tables + (size_t)b * p.max_blocks + e) : -1;
}

// Attention over partition `part` of sequence b for KV head g (all G query
// heads, NT = ceil(G / 8) tiles of 8), by W warps: a CTA (4), or one warp on its
// own (then part 0, the whole sequence). entry: q8_table_entry's; `phase` as in
// decode_partition.
template <typename T, int D, int NT, typename Code, int W>
__device__ __forceinline__ void decode_q8_partition(const CUtensorMap& tmap, const DecodeParams& p,
                                                    const Q8Layout& lay, uint8_t* smem, int32_t ring_bytes,
                                                    Q8Shared& sh, int32_t part, int32_t g, int32_t b, int32_t L,
                                                    int32_t entry, uint32_t& phase) {
  using Tile = Q8Tile<D>;
  constexpr int S = Tile::kStages;
  constexpr int KK = D / 16;                              // k-steps of QK, row tiles of PV
  constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;           // fp16 terms of q and P
  constexpr bool kBias = std::is_same<Code, CodeInt8>::value && TERMS == 1;  // codes as (c + 128) 2^-24
  constexpr float kUnit = kBias ? 16777216.f : 1.f;       // what an operand of the MMAs has to be multiplied by
  auto unpack = [](uint32_t w, bool interleaved, uint32_t& lo, uint32_t& hi) {
    if constexpr (kBias) q8_unpack_biased(w, interleaved, lo, hi);
    else q8_unpack(Code{}, w, interleaved, lo, hi);
  };
  constexpr int kRow = D + 8;                             // floats per row of the merge buffer
  static_assert(8 * NT * kRow * 4 <= Tile::kRing, "the merge buffer reuses the stages");
  const int32_t warp = threadIdx.x >> 5;
  const int32_t rank = W == 1 ? 0 : warp;  // of the W warps: owns blocks rank, rank + W, ...
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
  const int32_t my = nb > rank ? (nb - rank + W - 1) / W : 0;
  uint8_t* wsm = smem + warp * ring_bytes;
  const uint32_t wsm_addr = smem_addr(wsm);

  // the queries' words, in flight while the block ids and the first blocks arrive
  using QWord = Vec<T, 4>;
  QWord qw[NT][KK];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      const int32_t head = 8 * nt + gid;
#pragma unroll
      for (int i = 0; i < 4; ++i) qw[nt][kk].v[i] = Elem<T>::from_f32(0.f);
      if (head < G)
        qw[nt][kk] = *reinterpret_cast<const QWord*>(reinterpret_cast<const T*>(p.q) +
                                                     ((size_t)b * H + (size_t)g * G + head) * D + 16 * kk + 4 * tig);
    }

  // lane i holds the id of the warp's i-th block and, once they arrive, its
  // scales: k_b, log2 v_b and 1 / v_b
  const int32_t my_blk = lane < my ? entry : -1;
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

  float my_ks = 0.f, my_lv = -INFINITY, my_rv = 0.f;
  bool has_v = false;
  if (my_ok) {
    const uint8_t* pool = reinterpret_cast<const uint8_t*>(p.pool);
    my_ks = __ldg(reinterpret_cast<const float*>(pool + q8_scale_at(lay, my_blk, 0, g, p.num_kv_heads)));
    const float vs = __ldg(reinterpret_cast<const float*>(pool + q8_scale_at(lay, my_blk, 1, g, p.num_kv_heads)));
    has_v = vs > 0.f;
    if (has_v) {
      my_lv = log2f(vs);
      my_rv = 1.f / vs;
    }
  }
  const uint32_t v_mask = __ballot_sync(0xffffffffu, has_v);

  // Query fragments: B of S^T = K Q^T, head 8 nt + gid, dims 16 kk + 4 tig + (0, 1 | 2, 3),
  // scaled per head so that its largest magnitude lies in [2^14, 2^15).
  uint32_t qb[TERMS][NT][KK][2];
  float sfac[NT][2];  // scale * log2 e * unit / that power of two, heads 8 nt + 2 tig (+ 1)
  float qsum[NT][2];  // 128 / unit * the sum of the scaled query (kBias)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float x[KK][4];
    float a = 0.f;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[kk][i] = Elem<T>::to_f32(qw[nt][kk].v[i]);
        a = fmaxf(a, fabsf(x[kk][i]));
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
    sfac[nt][0] = __shfl_sync(0xffffffffu, down, 8 * tig) * kUnit;
    sfac[nt][1] = __shfl_sync(0xffffffffu, down, 8 * tig + 4) * kUnit;
    if constexpr (kBias) {
      float sum = 0.f;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 x2 = __half22float2(*reinterpret_cast<const __half2*>(&qb[0][nt][kk][j]));
          sum += x2.x + x2.y;
        }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      qsum[nt][0] = __shfl_sync(0xffffffffu, sum, 8 * tig) * (128.f / kUnit);
      qsum[nt][1] = __shfl_sync(0xffffffffu, sum, 8 * tig + 4) * (128.f / kUnit);
    } else {
      qsum[nt][0] = qsum[nt][1] = 0.f;
    }
  }

  float o[KK][NT][4];
  float ps[NT][4];                     // kBias: the sums of the P that o is made of
  // reference m + r and sum, heads 8 nt + 2 tig (+ 1); o and l in units of 2^(m + r - lift)
  float m[NT][2], r[NT][2], l[NT][2];
  bool far = false;                    // some |m| > kQ8Far (the same in the whole warp)
  auto clear = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kQ8NoRef;
      r[nt][0] = r[nt][1] = l[nt][0] = l[nt][1] = 0.f;
      ps[nt][0] = ps[nt][1] = ps[nt][2] = ps[nt][3] = 0.f;
#pragma unroll
      for (int c = 0; c < KK; ++c) o[c][nt][0] = o[c][nt][1] = o[c][nt][2] = o[c][nt][3] = 0.f;
    }
  };
  clear();
  if (lane < 16) sh.zero[warp][lane] = make_float2(kQ8NoRef, 0.f);
  __syncwarp();
  const int32_t row = lane & 15;  // of this lane's ldmatrix address
  const uint32_t row_addr = wsm_addr + Tile::chunk(row, lane >> 4);

  // S^T of the block at `at`: rows = tokens (gid, gid + 8), columns = heads (2 tig, 2 tig + 1)
  auto scores = [&](uint32_t at, float (&sc)[NT][4]) {
    float sc2[NT][4];  // odd k-steps: two shorter chains of dependent MMAs
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[nt][e] = sc2[nt][e] = 0.f;
#pragma unroll
    for (int c = 0; c < KK; c += 2) {
      uint32_t w[4];
      ldsm_x4(at ^ (c << 4), w[0], w[1], w[2], w[3]);
      uint32_t a0[4], a1[4];
      unpack(w[0], false, a0[0], a0[2]);
      unpack(w[1], false, a0[1], a0[3]);
      unpack(w[2], false, a1[0], a1[2]);
      unpack(w[3], false, a1[1], a1[3]);
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
  };

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
      clear();
      if (lane == 0) sh.abort = 1;
      break;
    }
    phase ^= 1u << s;
    const int32_t nvalid = min(16, t1 - (t0 + (rank + i * W) * 16));
    const float ks = __shfl_sync(0xffffffffu, my_ks, i);
    const float lv = __shfl_sync(0xffffffffu, my_lv, i);
    const float rv = __shfl_sync(0xffffffffu, my_rv, i);
    const bool no_v = !((v_mask >> i) & 1u);  // lv is -inf: all of P is 0
    if (nvalid < 16 || no_v) {
      // What must not count becomes zero codes: both tiles of a block that was
      // not loaded, the V tile under a zero scale, and the V rows behind the
      // sequence's end (they may hold NaN codes, which a zero probability does
      // not silence).
      uint8_t* stg = wsm + s * Tile::kStage;
      const bool loaded = (ok_mask >> i) & 1u;
      const int32_t from = no_v ? 0 : nvalid;
      for (int32_t e = lane; e < Tile::kStage / 16; e += 32) {
        const int32_t kv = e / (Tile::kBytes / 16), t = e / (D / 16) % 16, c = e % (D / 16);
        if (!loaded || (kv == 1 && t >= from))
          *reinterpret_cast<uint4*>(stg + kv * Tile::kBytes + Tile::chunk(t, c)) = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
      if (no_v) {
        float zs[NT][4];
        scores(row_addr + s * Tile::kStage, zs);
        // the block's share of the sum, in the units of l: 2^(reference - lift)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float2* z = &sh.zero[warp][8 * nt + 2 * tig + j];
            const float f = sfac[nt][j] * ks;
            const float y0 = gid < nvalid ? __fmul_rn(zs[nt][j] - qsum[nt][j], f) : -INFINITY;
            const float y1 = gid + 8 < nvalid ? __fmul_rn(zs[nt][j + 2] - qsum[nt][j], f) : -INFINITY;
            float zm = fmaxf(fmaxf(y0, y1), z->x);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) zm = fmaxf(zm, __shfl_xor_sync(0xffffffffu, zm, off));
            float zl = (ex2_ftz(y0 - zm) + ex2_ftz(y1 - zm)) * 128.f;
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) zl += __shfl_xor_sync(0xffffffffu, zl, off);
            zl = fmaf(z->y, ex2_ftz(z->x - zm), zl);
            __syncwarp();
            if (gid == 0) *z = make_float2(zm, zl);
          }
        }
        __syncwarp();
      }
    }

    const uint32_t at = row_addr + s * Tile::kStage;
    float sc[NT][4];
    scores(at, sc);
    // the exponents x + log2 v_b - (m + r) + lift
    float x[NT][4];
    auto exponents = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f = sfac[nt][j] * ks, c = lv + kQ8Lift - r[nt][j];
          if (!far) {
            const float c2 = kBias ? fmaf(-qsum[nt][j], f, c - m[nt][j]) : c - m[nt][j];
            x[nt][j] = fmaf(sc[nt][j], f, c2);
            x[nt][j + 2] = fmaf(sc[nt][j + 2], f, c2);
          } else {
            x[nt][j] = (__fmul_rn(sc[nt][j] - qsum[nt][j], f) - m[nt][j]) + c;
            x[nt][j + 2] = (__fmul_rn(sc[nt][j + 2] - qsum[nt][j], f) - m[nt][j]) + c;
          }
        }
      }
      if (nvalid < 16) {  // rows behind the end
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (gid + (e >> 1) * 8 >= nvalid) x[nt][e] = -INFINITY;
      }
    };
    exponents();
    float top = x[0][0];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, x[nt][e]);
    if (__any_sync(0xffffffffu, top > kQ8Lift + kQ8Raise)) {
      // the reference to the largest x + log2 v_b so far
      bool now_far = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float bm = m[nt][j], br = r[nt][j];
#pragma unroll
          for (int e = j; e < 4; e += 2) {
            const float y = __fmul_rn(sc[nt][e] - qsum[nt][j], sfac[nt][j] * ks);
            if (gid + (e >> 1) * 8 < nvalid && y + lv > bm + br) {
              bm = y;
              br = lv;
            }
          }
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, bm, off), orr = __shfl_xor_sync(0xffffffffu, br, off);
            // one order for both lanes of a pair, so that all end with the same reference
            if (om + orr > bm + br || (om + orr == bm + br && om > bm)) {
              bm = om;
              br = orr;
            }
          }
          const float a = ex2_ftz((m[nt][j] - bm) + (r[nt][j] - br));
          m[nt][j] = bm;
          r[nt][j] = br;
          now_far |= fabsf(bm) > kQ8Far && bm != kQ8NoRef;
          l[nt][j] *= a;
          ps[nt][j] *= a;
          ps[nt][j + 2] *= a;
#pragma unroll
          for (int c = 0; c < KK; ++c) {
            o[c][nt][j] *= a;
            o[c][nt][j + 2] *= a;
          }
        }
      }
      far = __any_sync(0xffffffffu, now_far);
      exponents();
    }
    uint32_t pb[TERMS][NT][2];  // B of O^T = V^T P^T: head gid, tokens 2 tig (+ 1), + 8
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pv[e] = ex2_ftz(x[nt][e]);
#pragma unroll
      for (int j = 0; j < 2; ++j) l[nt][j] = fmaf(pv[j] + pv[j + 2], rv, l[nt][j]);
      const uint32_t w0 = pack_f16x2(pv[0], pv[1]), w1 = pack_f16x2(pv[2], pv[3]);
      pb[0][nt][0] = transpose_8x8(w0);
      pb[0][nt][1] = transpose_8x8(w1);
      if constexpr (TERMS == 2) {
        pb[1][nt][0] = transpose_8x8(pack_f16x2_rest(pv[0], pv[1], w0));
        pb[1][nt][1] = transpose_8x8(pack_f16x2_rest(pv[2], pv[3], w1));
      }
      if constexpr (kBias) {
        constexpr uint32_t one = 0x3c003c00u;
        const uint32_t ones[4] = {one, one, one, one};
        mma_f16_16816(ps[nt], ones, pb[0][nt][0], pb[0][nt][1]);
      }
    }
#pragma unroll
    for (int c = 0; c < KK; c += 2) {
      uint32_t w[4];
      ldsm_x4_trans((at ^ (c << 4)) + Tile::kBytes, w[0], w[1], w[2], w[3]);
      uint32_t a0[4], a1[4];
      unpack(w[0], true, a0[0], a0[1]);
      unpack(w[1], true, a0[2], a0[3]);
      unpack(w[2], true, a1[0], a1[1]);
      unpack(w[3], true, a1[2], a1[3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
          mma_f16_16816(o[c][nt], a0, pb[term][nt][0], pb[term][nt][1]);
          mma_f16_16816(o[c + 1][nt], a1, pb[term][nt][0], pb[term][nt][1]);
        }
      }
    }
    __syncwarp();
    if (i + S < my) issue(i + S);
  }
  if constexpr (kBias) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < KK; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][nt][e] = fmaf(o[c][nt][e], kUnit, -128.f * ps[nt][e]);
  }

  if constexpr (W == 1) {
    // a head's sum lies in the 8 lanes of its column; dims 16 c + 2 gid (+ 1) here
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float ls = l[nt][j];
        ls += __shfl_xor_sync(0xffffffffu, ls, 4);
        ls += __shfl_xor_sync(0xffffffffu, ls, 8);
        ls += __shfl_xor_sync(0xffffffffu, ls, 16);
        const int32_t head = 8 * nt + 2 * tig + j;
        const float n = m[nt][j] + r[nt][j];
        const float2 z = sh.zero[warp][head];
        const float M = fmaxf(n, z.x), f = exp2f(n - M);
        const float inv = f / fmaf(ls, f, z.y * exp2f(z.x - M));
        if (head < G) {
          T* out = reinterpret_cast<T*>(p.out) + ((size_t)b * H + (size_t)g * G + head) * D + 2 * gid;
#pragma unroll
          for (int c = 0; c < KK; ++c)
            *reinterpret_cast<Vec<T, 2>*>(out + 16 * c) = {Elem<T>::from_f32(o[c][nt][j] * inv),
                                                           Elem<T>::from_f32(o[c][nt][j + 2] * inv)};
        }
      }
    }
    return;
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
        sh.red_m[warp][head] = m[nt][j] + r[nt][j];
        sh.red_l[warp][head] = ls;
      }
      float* row = so + (warp * 8 * NT + head) * kRow + 2 * gid;
#pragma unroll
      for (int c = 0; c < KK; ++c)
        *reinterpret_cast<float2*>(row + 16 * c) = make_float2(o[c][nt][j], o[c][nt][j + 2]);
    }
  }
  __syncthreads();

  // each head's weights of the four warps, divided by the sum where this is the output
  if (threadIdx.x < G) {
    const int32_t h = threadIdx.x;
    float M = kQ8NoRef;
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) M = fmaxf(M, fmaxf(sh.red_m[w][h], sh.zero[w][h].x));
    float e[kQ8Warps], Ls = 0.f;
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) {
      e[w] = exp2f(sh.red_m[w][h] - M);  // 0 for a warp that had no block
      Ls = fmaf(sh.red_l[w][h], e[w], Ls);
      const float2 z = sh.zero[w][h];
      Ls = fmaf(z.y, exp2f(z.x - M), Ls);
    }
    const float f = nparts == 1 ? 1.f / Ls : 1.f;
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) sh.red_m[w][h] = e[w] * f;
    if (nparts > 1)
      reinterpret_cast<float2*>(p.ws_ml)[((size_t)b * H + (size_t)g * G + h) * p.max_partitions + part] =
          make_float2(M, Ls);
  }
  __syncthreads();
  T* out = reinterpret_cast<T*>(p.out);
  for (int32_t i = threadIdx.x; i < G * (D / 4); i += blockDim.x) {
    const int32_t h = i / (D / 4), d = i % (D / 4) * 4;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(so + (w * 8 * NT + h) * kRow + d);
      const float e = sh.red_m[w][h];
      A.x = fmaf(x.x, e, A.x);
      A.y = fmaf(x.y, e, A.y);
      A.z = fmaf(x.z, e, A.z);
      A.w = fmaf(x.w, e, A.w);
    }
    const size_t bh = (size_t)b * H + (size_t)g * G + h;
    if (nparts == 1)
      *reinterpret_cast<Vec<T, 4>*>(out + bh * D + d) = {Elem<T>::from_f32(A.x), Elem<T>::from_f32(A.y),
                                                         Elem<T>::from_f32(A.z), Elem<T>::from_f32(A.w)};
    else
      *reinterpret_cast<float4*>(p.ws_acc + (bh * p.max_partitions + part) * D + d) = A;
  }
}

template <typename T, int D, int NT, typename Code>
__global__ void __launch_bounds__(kQ8Warps * 32, NT == 2 && sizeof(T) == 2 && D == 128 ? 3 : 1)
decode_q8_kernel(const __grid_constant__ CUtensorMap tmap, DecodeParams p, Q8Layout lay) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Q8Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int32_t warp = threadIdx.x >> 5;
  const int32_t lane = threadIdx.x & 31;
  grid_dependents_launch();
  int32_t grid_len = 0, entry = -1;
  if (p.work_items == nullptr) {
    const int32_t part = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    entry = q8_table_entry(p, part, b, warp, kQ8Warps);
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
    decode_q8_partition<T, D, NT, Code, kQ8Warps>(tmap, p, lay, smem, Q8Tile<D>::kRing, sh, blockIdx.x, blockIdx.y,
                                                  blockIdx.z, grid_len, entry, phase);
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
    const int32_t b = (int32_t)(bp >> 16), part = (int32_t)(bp & 0xffffu);
    entry = q8_table_entry(p, part, b, warp, kQ8Warps);
    decode_q8_partition<T, D, NT, Code, kQ8Warps>(tmap, p, lay, smem, Q8Tile<D>::kRing, sh, part, g, b,
                                                  checked_len(p, b, false), entry, phase);
    fence_proxy_async_smem();  // the item's shared-memory reads precede the next item's TMA writes
    if (threadIdx.x == 0) sh.next_item = next;
    __syncthreads();
    item = sh.next_item;
  }
}

// A warp per (sequence, KV head), for sequences of at most kQ8WarpTokens.
constexpr int kQ8WarpTokens = 32 * 16;  // a lane holds one block id

template <typename T, int D, int NT, typename Code>
__global__ void __launch_bounds__(kQ8Warps * 32, NT == 2 && sizeof(T) == 2 && D == 128 ? 3 : 1)
decode_q8_warp_kernel(const __grid_constant__ CUtensorMap tmap, DecodeParams p, Q8Layout lay, int32_t ring_bytes) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Q8Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int32_t warp = threadIdx.x >> 5;
  const int32_t lane = threadIdx.x & 31;
  grid_dependents_launch();
  const int64_t item = (int64_t)blockIdx.x * kQ8Warps + warp;
  if (item >= (int64_t)p.num_seqs * p.num_kv_heads) return;
  const int32_t b = (int32_t)(item / p.num_kv_heads), g = (int32_t)(item % p.num_kv_heads);
  const int32_t entry = q8_table_entry(p, 0, b, 0, 1);
  const int32_t L = checked_len(p, b, g == 0 && lane == 0);
  if (L == 0) {
    T* out = reinterpret_cast<T*>(p.out) + ((size_t)b * p.num_heads + (size_t)g * p.group) * D;
    for (int32_t i = lane; i < p.group * D; i += 32) out[i] = Elem<T>::from_f32(0.f);
    return;
  }
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < Q8Tile<D>::kStages; ++s) mbar_init(&sh.bars[warp][s], 1);
    fence_barrier_init();
  }
  __syncwarp();
  uint32_t phase = 0;
  decode_q8_partition<T, D, NT, Code, 1>(tmap, p, lay, smem, ring_bytes, sh, 0, g, b, L, entry, phase);
}

// Merge of the partition states of one sequence. kSplit (many partitions): a
// CTA of 8 warps per head, which share its partitions and join through shared
// memory. Otherwise: a CTA of 4 warps per KV head, a warp takes a head at a
// time. Bound by the latency of a few dependent L2 reads: a warp has 8
// partitions' accumulators in flight. Every CTA waits for the partition kernel
// before it reads anything, the lengths too, and also where it has nothing to
// merge (see partition_merge_kernel).
template <bool kSplit>
constexpr int kQ8MergeWarps = kSplit ? 8 : 4;

template <typename T, int D, bool kSplit>
__global__ void __launch_bounds__(kQ8MergeWarps<kSplit> * 32) decode_q8_merge_kernel(DecodeParams p) {
  constexpr int kWarps = kQ8MergeWarps<kSplit>;
  constexpr int E = D / 32;  // output elements per lane
  using Acc = Vec<float, E>;
  __shared__ float sh_ml[kWarps][2];
  __shared__ Acc sh_acc[kSplit ? kWarps : 1][32];
  const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t b = blockIdx.y;
  grid_dependency_wait();
  const int32_t L = checked_len(p, b, false);
  const int32_t nparts = (L + p.partition_tokens - 1) / p.partition_tokens;
  if (nparts <= 1) return;  // finished by the partition kernel
  const int32_t heads = kSplit ? 1 : p.group;
  for (int32_t h = kSplit ? 0 : warp; h < heads; h += kSplit ? 1 : kWarps) {
    const size_t bh = (size_t)b * p.num_heads + (size_t)blockIdx.x * heads + h;
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + bh * p.max_partitions;
    const Acc* acc = reinterpret_cast<const Acc*>(p.ws_acc) + bh * p.max_partitions * 32 + lane;
    // chunks of partitions, this warp's first and the stride to its next
    constexpr int32_t kChunk = kSplit ? 16 : 32;
    const int32_t c0 = kSplit ? warp * kChunk : 0, step = kSplit ? kWarps * kChunk : kChunk;
    float M = kQ8NoRef, l = 0.f;
    Acc a;
#pragma unroll
    for (int e = 0; e < E; ++e) a.v[e] = 0.f;
    for (int32_t q0 = c0; q0 < nparts; q0 += step) {
      const int32_t cnt = min(kChunk, nparts - q0);
      // the first accumulators are asked for together with the references
      Acc x[8];
      auto load = [&](int32_t q) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (q + j < cnt) x[j] = load_cg(acc + (size_t)(q0 + q + j) * 32);
      };
      const float2 s = lane < cnt ? __ldcg(ml + q0 + lane) : make_float2(kQ8NoRef, 0.f);
      load(0);
      float m = s.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = fmaxf(m, M);
      const float w = exp2f(s.x - m), old = exp2f(M - m);
      M = m;
      l = fmaf(l, old, warp_sum(s.y * w));
#pragma unroll
      for (int e = 0; e < E; ++e) a.v[e] *= old;
      for (int32_t q = 0; q < cnt; q += 8) {
        if (q > 0) load(q);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float wj = __shfl_sync(0xffffffffu, w, (q + j) & 31);
          if (q + j < cnt) {
#pragma unroll
            for (int e = 0; e < E; ++e) a.v[e] = fmaf(x[j].v[e], wj, a.v[e]);
          }
        }
      }
    }
    if constexpr (kSplit) {
      sh_acc[warp][lane] = a;
      if (lane == 0) {
        sh_ml[warp][0] = M;
        sh_ml[warp][1] = l;
      }
      __syncthreads();
      if (warp > 0) return;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float m = fmaxf(M, sh_ml[w][0]);
        const float f0 = exp2f(M - m), f1 = exp2f(sh_ml[w][0] - m);
        M = m;
        l = fmaf(l, f0, sh_ml[w][1] * f1);
#pragma unroll
        for (int e = 0; e < E; ++e) a.v[e] = fmaf(a.v[e], f0, sh_acc[w][lane].v[e] * f1);
      }
    }
    const float inv = 1.f / l;
    Vec<T, E> y;
#pragma unroll
    for (int e = 0; e < E; ++e) y.v[e] = Elem<T>::from_f32(a.v[e] * inv);
    reinterpret_cast<Vec<T, E>*>(p.out)[bh * 32 + lane] = y;
  }
}

// ---- host side ---------------------------------------------------------------

template <typename T, int D, bool kSplit>
inline cudaError_t launch_decode_q8_merge(const DecodeParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSplit ? p.num_heads : p.num_kv_heads, p.num_seqs);
  cfg.blockDim = dim3(kQ8MergeWarps<kSplit> * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_q8_merge_kernel<T, D, kSplit>, p);
}

// CTAs of a decode kernel that an SM holds, with the kernel's shared-memory limit
// set; asked of the device once.
template <typename T, int D, int NT, typename Code>
inline cudaError_t q8_ctas_per_sm(int32_t* per_sm) {
  static PerDevice<int32_t> occupancy;
  return occupancy.get(per_sm, [](int32_t* v) {
    auto kernel = decode_q8_kernel<T, D, NT, Code>;
    int32_t n = 0;
    cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Q8Tile<D>::kSmem);
    if (r == cudaSuccess)
      r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kQ8Warps * 32, Q8Tile<D>::kSmem);
    *v = n > 0 ? n : 1;
    return r;
  });
}

// CTAs that are resident at once on the current device; a B200's where no device
// can be asked (sizing a workspace on a host without a GPU). What fits is decided
// by shared memory for head_dim 128 and up to 8 heads a group (3), by registers
// elsewhere (64: 4; 9 to 16 heads: 2 or 3).
template <typename T, int D, int NT, typename Code>
inline int32_t q8_resident_of() {
  int32_t n = 0;
  if (q8_ctas_per_sm<T, D, NT, Code>(&n) != cudaSuccess) {
    cudaGetLastError();  // clear the error of a failed query
    constexpr bool bf16 = sizeof(T) == 2, e4m3 = std::is_same<Code, CodeE4m3>::value;
    n = NT == 1 ? (D == 64 ? 4 : 3) : bf16 && (D == 128 || e4m3) ? 3 : 2;
  }
  return n * device_sm_count();
}
inline int32_t q8_resident(int32_t head_dim, int32_t group, int32_t dtype, int32_t io_dtype) {
  auto of = [&](auto io, auto code) {
    using T = decltype(io);
    using Code = decltype(code);
    if (head_dim == 64) return group <= 8 ? q8_resident_of<T, 64, 1, Code>() : q8_resident_of<T, 64, 2, Code>();
    return group <= 8 ? q8_resident_of<T, 128, 1, Code>() : q8_resident_of<T, 128, 2, Code>();
  };
  auto of_code = [&](auto code) { return io_dtype == PA_BF16 ? of(__nv_bfloat16{}, code) : of(float{}, code); };
  return dtype == PA_Q8_INT8 ? of_code(CodeInt8{}) : of_code(CodeE4m3{});
}
// A warp per (sequence, KV head) where sequences are short and pairs many: 200
// sequences x 8 heads of up to 137 tokens take 10.5 us by warps and 23.8 us by
// CTAs. With fewer than three pairs per SM the warps are too few to fill it (82
// x 8 heads of 90 tokens, 4.4 per SM: 10.4 and 14.1 us).
inline bool q8_by_warp(int64_t pairs, int32_t max_seq_len) {
  return max_seq_len <= kQ8WarpTokens && pairs >= (int64_t)3 * device_sm_count();
}
// CTAs from which the work list pays: four rounds of them for head_dim 64, whose
// items are shorter beside the list's launch, three for 128 (64: 64 x 8 heads,
// 3.5 rounds, lognormal up to 8192 34.1 us without the list and its partitions,
// 38.2 with them, all of 8192 105 and 113, uniform 76 and 73. 128: 48 x 8, 3.5
// rounds, 41.9 and 41.2, 142 and 142, 94 and 88).
inline int64_t q8_list_from(int32_t head_dim, int64_t resident) { return (head_dim == 64 ? 4 : 3) * resident; }
// Tokens of a partition, a multiple of 16, at most 2048: when every sequence
// has the longest length, the resident CTAs take one partition each, or as many
// as 2048 tokens make necessary (one request of 131071 tokens and 8 heads: two
// rounds of 1184 tokens, 54 us; three rounds 60 us). Up to 256 tokens, four
// blocks a warp, a partition is the sequence: the launch that merges costs more
// (230 tokens: 5.9 us, in two partitions 6.3 us). Two rounds throughout were
// slower on batches of even lengths (6 x 8 heads of 2928 tokens: 15.0 us by one
// round, 19.1 by two) and faster on ragged ones (28 x 2 of up to 10517: 23.0 and
// 18.7 us). Batches of up to ten rounds of 2048 tokens, taken from the list,
// get 1024: their lengths are ragged as a rule, and the longest items would end
// alone (64 x 8 heads, lognormal up to 8192: 42.8 us, by 2048 tokens 51.7; all of
// 8192: 174.5 and 174.8). Beyond ten rounds 2048 are enough and cheaper (256 x 8:
// 121 us, by 1024 tokens 130), and sequences that fit one partition are not cut
// (64 x 32 of up to 2048: 99 and 106 us).
inline int32_t q8_partition_tokens(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int64_t resident,
                                   int32_t max_seq_len) {
  const int64_t pairs = std::max<int64_t>((int64_t)num_seqs * num_kv_heads, 1);
  if (q8_by_warp(pairs, max_seq_len)) return kQ8WarpTokens;  // one partition
  const int64_t least = ((int64_t)max_seq_len + 2047) / 2048;  // partitions a sequence needs
  const int64_t rounds = std::max<int64_t>((least * pairs + resident - 1) / resident, 1);
  const int64_t parts = std::max<int64_t>(rounds * resident / pairs, 1);
  const int64_t tokens = (((int64_t)max_seq_len + parts - 1) / parts + 15) / 16 * 16;
  const int64_t smallest = max_seq_len <= 256 ? 256 : 128;
  const bool some_rounds = pairs * least > q8_list_from(head_dim, resident) && pairs * least <= 10 * resident;
  const int64_t most = least > 1 && some_rounds ? 1024 : 2048;
  return (int32_t)std::min<int64_t>(std::max<int64_t>(tokens, smallest), most);
}
// The plan kernel's list from more than so many rounds of CTAs on: it saves the
// empty CTAs of ragged batches and starts the longest partitions first, but is a
// launch more (182 x 2 heads of 4608 tokens, 2.5 rounds: 80.3 us without, 84.5
// with it).
inline bool q8_use_list(int64_t pairs, int32_t partitions, int32_t head_dim, int64_t resident) {
  return partitions >= 2 && pairs * partitions > q8_list_from(head_dim, resident);
}

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
  if (q8_by_warp((int64_t)p.num_seqs * p.num_kv_heads, p.max_seq_len)) {
    auto warp_kernel = decode_q8_warp_kernel<T, D, NT, Code>;
    static PerDevice<int32_t> smem_set;
    cudaError_t e = set_smem_once(smem_set, warp_kernel, Q8Tile<D>::kSmem);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_decode_q8: %s", cudaGetErrorString(e));
    // no more stages than a sequence has blocks: short ones leave room for more CTAs
    const int32_t stages = std::min<int32_t>(Q8Tile<D>::kStages, (p.max_seq_len + 15) / 16);
    const int32_t ring = std::max<int32_t>(stages, 1) * Q8Tile<D>::kStage;
    const int64_t items = (int64_t)p.num_seqs * p.num_kv_heads;
    warp_kernel<<<(unsigned)((items + kQ8Warps - 1) / kQ8Warps), kQ8Warps * 32, kQ8Warps * ring + 1024, st>>>(
        map, p, q8_layout(p.num_kv_heads, D), ring);
    e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_decode_q8: launch failed: %s", cudaGetErrorString(e));
    return PA_OK;
  }
  auto kernel = decode_q8_kernel<T, D, NT, Code>;
  int32_t per_sm = 1;
  cudaError_t e = q8_ctas_per_sm<T, D, NT, Code>(&per_sm);
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_decode_q8: %s", cudaGetErrorString(e));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kQ8Warps * 32);
  cfg.dynamicSmemBytes = Q8Tile<D>::kSmem;
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
  // one CTA per head where its warps have partitions to share
  e = p.max_partitions > 8 ? launch_decode_q8_merge<T, D, true>(p, st) : launch_decode_q8_merge<T, D, false>(p, st);
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
