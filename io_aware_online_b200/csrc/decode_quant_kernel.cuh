// decode_quant_kernel.cuh -- attention of a few query rows per sequence against an 8-bit
// (paged) KV cache, sm_100a.
//
//   x_ij = c( scale * q_i . k_j ) - slope |i + off - j|,   k_j = kcode_j * kscale_j
//   O_i  = sum_j softmax(x_i)_j v_j,                       v_j = vcode_j * vscale_j
//
// Bound by HBM: 2 (D + 4) bytes per (key, KV head), each read once for every query row of
// its KV head.  Half the bytes of a 16-bit cache leave half the time per key, so the
// products run on the warps' matrix instructions (m16n8k16, fp16 operands, fp32 sums); the
// codes of both formats are exact in fp16, and so are bf16 queries once a row is scaled by
// a power of two, so the scores carry no rounding but that of their fp32 sums.
//
// Work.  A pair is one (sequence, KV head, group of up to 8 NT query rows); its keys are cut
// into tiles of 64.  The tiles of all pairs form one line, sequence by sequence, which is cut
// into equal shares, one per WARP of the grid: warps differ by at most one tile however ragged
// the batch is, and no two warps ever have to meet.  A share ends inside a pair as a rule, so a
// warp has at most two pieces of pairs that it shares with a neighbour: it writes (O, max, sum)
// of such a piece to its own two slots of the workspace and a second launch joins the pieces;
// pairs that lie in one share are written at once.  Neighbouring shares go to different SMs, so
// that a few tiles spread over the machine.  Every warp finds its share from cache_seqlens, by
// itself, so nothing has to be set up or cleared before the launch and no barrier is met.
//   (Measured, B=64, 1K..32K keys, 8 KV heads, d=128, E4M3: shares per CTA with the warps joining
//   through shared memory took 445 us, and 20 us where the cache holds 8 x 1000 keys: the joins'
//   barriers stall every warp of a CTA at every piece.)
//
// A warp has one K and one V buffer and brings its tiles itself, by TMA and bulk copies: the
// next K tile (with both scale rows) as soon as the scores are taken, the next V tile after
// P V.  Nobody waits for an empty buffer.  (One producer warp per CTA spent ~1200 clocks per
// tile on finding and bringing it and bounded every shape: 594 us.)
//   Scores: S^T[16 keys x 8 rows] = K[16 x 16] Q^T[16 x 8].  A lane reads 16 neighbouring
//     head-dim codes of two keys at a time; which head-dim elements and keys sit at which
//     index of the product is free as long as both operands agree, and the order is chosen so
//     that every 16-byte read of a quarter warp touches all banks once (d=128).
//   P V: O^T[16 head-dim x 8 rows] = V^T[16 x 16 keys] P^T[16 x 8].  A lane reads 16
//     head-dim codes of four keys and pairs the bytes of two keys with a byte permute, which
//     transposes them; P^T comes from the score layout by an 8 x 8 transpose in registers.
//   P carries v's scale, so that it fits fp16 relative to the largest p vscale that its query row
//     has met: p vscale / ref * 2^14, ref a power of two above that product (full precision down to
//     2^-28 of the largest, steps of 2^-38 of it below).  O is rescaled when a product reaches ref, as
//     it is when the running max grows.  (Relative to the largest vscale alone, a key of a large
//     scale that weighs nothing, or that only another row sees, took the others' precision.)
//     Rounding P to fp16 (2^-11 relative) is an eighth of a bf16 output's own rounding but as much
//     as an fp16 output's: for those the remainder is a second operand on the same V registers
//     (2^-22), half as many products more.  (For bf16 outputs too it would cost 0-8% at d=128, 7%
//     at d=64 and 11-15% with 16 rows, for an error of 1.66e-3 in place of 1.67e-3.)
//
// Measured (B=64, 1K..32K keys, 8 KV heads, 4 query heads each, bf16, graph replays on several boxes,
// of the copy rate; 2.32 GB at d=128: 353 us).  Rows of all heads together, the default order: d=128
// E4M3 440-447 us (79-80%), int8 414-445 (79-85%), since a tile is then 64 pieces of 128 bytes, 1 KB
// apart; d=64 240 (76%) and 220-240 (76-82%).  Rows of a head together: d=128 357-392 us (90-99%; 396
// back to back for seconds, where the SM clock gives way at the power limit) and 367-384 (92-96%),
// d=64 198-208 (88-92%) and 220-224 (81-83%): there, and with 16 query rows (460-466 and 520-530 us,
// 76% and 67%), the issue of instructions and the logic pipe (58-63% busy) bound it.  fp16 outputs,
// with the second part of P: d=128 E4M3 351-362, d=64 int8 240-254, 16 rows int8 578-589.  More rows
// read a cache again for every 16 (64 sequences of 1K..8K keys, E4M3: 16 rows 150 us, 32 276, 64 545;
// the bytes alone 95).  Few keys (8 x 1000): 11.9 us, all latency: the share 2.5 us, the first
// tile's way 1.5, one tile's chain 3, the join 4.
#pragma once

#include <climits>

#include "quant_device.cuh"

namespace fa {

constexpr int kDqTok = 64;        // keys per tile
template <int D, int NT>
struct DqCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kWarps = decode_quant_warps(D, 8 * NT);
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTileBytes = kDqTok * D;             // one K (or V) tile
  static constexpr int kScaleOff = 2 * kWarps * kTileBytes; // K and V scales of each warp's tile
  static constexpr int kScaleBytes = 2 * kDqTok * 4;
  // With 16 rows the query operands do not fit a lane's registers beside O and the scores:
  // each lane keeps its own in shared memory.
  static constexpr bool kQShared = NT == 2;
  static constexpr int kQOff = kScaleOff + kWarps * kScaleBytes;
  static constexpr int kQBytes = kQShared ? NT * (D / 16) * 32 * 8 : 0;  // per warp
  static constexpr int kBarOff = kQOff + kWarps * kQBytes;          // K full, V full of each warp
  static constexpr int kSmemBytes = kBarOff + 2 * kWarps * 8;
  static constexpr int kSmemAlloc = kSmemBytes + 1024;
};

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// D += A B, one m16n8k16 product of fp16 with fp32 sums.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held by a warp (lane l: row l / 4, columns
// 2 (l mod 4) and the next).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The four codes of a word as two pairs of fp16, exactly: bytes 0 and 2, and bytes 1 and 3.
// E4M3 comes out times 2^-8: its exponent field, put under fp16's, is off by that (for its
// subnormals too).  The conversion instruction takes fewer issue slots and less power but its
// unit is slow: with it alone, a tile's 256 conversions (d=128) took ~1024 clocks of an SM, more
// than the tile's share of HBM time (730).  So E4M3's K goes through it and V through these
// operations: B=64, 1K..32K keys, d=128, back to back for seconds (at the power limit, where
// the SM clock falls to 1.6 GHz) 385 us, against 427 us with K through them too and 413 us
// with half of K; d=64 unthrottled 269, 284 and 274 us.
template <bool E4M3>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& even, uint32_t& odd) {
  if constexpr (E4M3) {
    even = ((w & 0x007f007fu) << 7) | ((w << 8) & 0x80008000u);
    odd = ((w & 0x7f007f00u) >> 1) | (w & 0x80008000u);
  } else {
    // byte ^ 0x80 = code + 128; under the exponent of 1024 it reads as 1024 + 128 + code
    const uint32_t a = (w & 0x00ff00ffu) ^ 0x64806480u, b = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
    const __half2 k = __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), k);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), k);
    even = *reinterpret_cast<const uint32_t*>(&x);
    odd = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// The same by the conversion instruction, bytes 0 and 1, and bytes 2 and 3, unscaled.
__device__ __forceinline__ void codes_cvt(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// The bounded wait of a warp that meets no other (the other warps of the CTA run on).
__device__ __forceinline__ bool dq_wait(const DecodeQuantParams& p, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > p.timeout_ns) {
      atomicOr(p.status, kDevWaitTimeout);
      return false;
    }
  }
  return true;
}

// a / b, by a 32-bit division where both fit (a 64-bit one takes several times as long).
__device__ __forceinline__ int64_t dq_div(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__device__ __forceinline__ uint32_t dq_pack(bool bf16, float lo, float hi) {
  return bf16 ? pack2<true>(lo, hi) : pack2<false>(lo, hi);
}

// Attended keys of sequence b: length and the tiles [lo, lo + n) that hold every key any of
// its query rows may see (n is 1 for a sequence that sees none, which still has to be written).
struct DqSeq {
  int L, off, key_lo, key_hi, t_lo, n;
};

__device__ __forceinline__ DqSeq dq_seq(const DecodeQuantParams& p, int b, bool report) {
  DqSeq s;
  s.L = p.cache_seqlens != nullptr ? p.cache_seqlens[b] : p.c.rows;
  const int cap = p.c.block_table != nullptr ? p.c.max_blocks * p.c.rows : p.c.rows;
  if (s.L < 0 || s.L > cap) {  // a length that the cache cannot hold: clamped and reported
    if (report) atomicOr(p.status, kDevBadLength);
    s.L = min(max(s.L, 0), cap);
  }
  s.off = s.L - p.Sq;
  int lo = 0, hi = s.L;
  if (p.wl >= 0) lo = max(lo, s.off - p.wl);
  const int right = p.causal ? 0 : p.wr;
  // (no sum here leaves 32 bits: a window side is cut to the cache's capacity by the host)
  if (right >= 0) hi = min(hi, p.Sq + s.off + right);
  s.key_lo = lo;
  s.key_hi = max(hi, lo);
  s.t_lo = lo / kDqTok;
  s.n = hi > lo ? (hi + kDqTok - 1) / kDqTok - s.t_lo : 0;
  s.n = max(s.n, 1);
  return s;
}

// A walk along a warp's share of the line of tiles.
struct DqWalk {
  DqSeq sq;
  int b, hk, grp;     // sequence, KV head and group of query rows: the pair
  int at;             // tile within the pair
  int n;              // the tile's place in the share
  int row, block;     // where its rows start: row of the block (or slab), block (or sequence)
};

// Moves `by` tiles on; behind the share's `count` tiles only `n` is kept.
__device__ __forceinline__ void dq_advance(const DecodeQuantParams& p, DqWalk& w, int by, int count) {
  w.n += by;
  if (w.n >= count) return;
  w.at += by;
  while (w.at >= w.sq.n) {
    w.at -= w.sq.n;
    if (++w.grp == p.groups) {
      w.grp = 0;
      if (++w.hk == p.Hkv) {
        w.hk = 0;
        w.b = min(w.b + 1, p.B - 1);
        w.sq = dq_seq(p, w.b, false);
      }
    }
  }
}

// Finds the walk's tile in the cache.  A warp does so one tile before it brings it, so that the
// table's entry has arrived by then.
__device__ __forceinline__ void dq_locate(const DecodeQuantParams& p, DqWalk& w) {
  const int tile = w.sq.t_lo + w.at;
  if (p.c.block_table == nullptr) {
    w.row = tile * kDqTok;
    w.block = w.b;
    return;
  }
  // tile / tiles of a page, by the reciprocal 2^32 / tiles rounded down: at most one too small
  int page = static_cast<int>(__umulhi(static_cast<uint32_t>(tile), p.page_rcp));
  int in = tile - page * p.page_tiles;
  if (in >= p.page_tiles) {
    in -= p.page_tiles;
    ++page;
  }
  w.row = in * kDqTok;
  // (the one tile of a sequence without keys may lie behind the table; it is not loaded)
  w.block = p.c.block_table[static_cast<int64_t>(w.b) * p.c.max_blocks + min(page, p.c.max_blocks - 1)];
}

// Brings the walk's K tile and scale rows (V = false), or its V tile, into this warp's buffer.
// Called by the whole warp; the buffer's contents have been used by every lane.
template <int D, int NT, bool V>
__device__ __forceinline__ void dq_fill(const DecodeQuantParams& p, const CUtensorMap* map,
                                        const DqWalk& w, uint8_t* buf, float* sc, uint64_t* full) {
  using Cfg = DqCfg<D, NT>;
  const int lane = threadIdx.x % 32;
  if (w.sq.key_hi <= w.sq.key_lo) return;  // a sequence without keys: nothing to bring
  int block = w.block;
  if (p.c.block_table != nullptr && (block < 0 || block >= p.c.num_blocks)) {
    if (lane == 0) atomicOr(p.status, kDevBadBlock);
    block = 0;  // a block of the pool; the status word reports the fault
  }
  if (lane == 0) {
    if (V) {
      mbar_arrive_expect_tx(full, Cfg::kTileBytes);
      tma_load_4d(buf, map, full, 0, w.hk, w.row, block);
    } else {
      // rows behind the slab's end: zeros for the codes, nothing for the scales
      const uint32_t sb = p.bulk_scales ? static_cast<uint32_t>(min(kDqTok, p.c.rows - w.row)) * 4u : 0u;
      mbar_arrive_expect_tx(full, Cfg::kTileBytes + 2 * sb);
      tma_load_4d(buf, map, full, 0, w.hk, w.row, block);
      if (sb != 0) {
        const int64_t so = (static_cast<int64_t>(block) * p.Hkv + w.hk) * p.c.rows + w.row;
        bulk_load(sc, p.c.ks + so, sb, full);
        bulk_load(sc + kDqTok, p.c.vs + so, sb, full);
      }
    }
  }
  if (!V && !p.bulk_scales) {  // rows of scales that do not start on 16 bytes: word by word
    const int64_t so = (static_cast<int64_t>(block) * p.Hkv + w.hk) * p.c.rows + w.row;
    const int key0 = (w.sq.t_lo + w.at) * kDqTok;
#pragma unroll
    for (int r = lane; r < kDqTok; r += 32) {
      if (key0 + r < w.sq.key_hi) {
        cp_async4(sc + r, p.c.ks + so + r);
        cp_async4(sc + kDqTok + r, p.c.vs + so + r);
      }
    }
    cp_async_arrive(full);
  }
}

// The query rows of a lane's score columns: factors, bounds and position.
template <int NT>
struct DqRows {
  float rf[NT][2], slope[NT][2];  // score factor and ALiBi slope (base 2)
  int lo[NT][2], hi[NT][2], pos[NT][2];
};

// Products -> base-2 scores of a tile: scale, softcap, ALiBi and (unless every row sees all
// of the tile) the mask; their max per row, and the value scales.
template <bool WHOLE, bool EXTRA, int NT>
__device__ __forceinline__ void dq_scores(const DecodeQuantParams& p, const DqRows<NT>& rows,
                                          const DqSeq& sq, int key0, int perm, const float* sks,
                                          const float* svs, float2 (&x)[4][NT][2], float (&vs)[4][2],
                                          float (&mx)[NT][2]) {
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int h2 = 0; h2 < 2; ++h2) {
      const int r = 16 * mt + perm + 8 * h2, key = key0 + r;
      const float ks = sks[r];
      const bool in = WHOLE || (key >= sq.key_lo && key < sq.key_hi);
      vs[mt][h2] = in ? svs[r] : 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 f = mul2(make_float2(ks, ks), make_float2(rows.rf[nt][0], rows.rf[nt][1]));
        float2 v = mul2(x[mt][nt][h2], f);
        if (EXTRA) {
          if (p.has_softcap) {
            v.x = fmaf(-2.f * p.softcap_log2, rcp(ex2(v.x) + 1.f), p.softcap_log2);
            v.y = fmaf(-2.f * p.softcap_log2, rcp(ex2(v.y) + 1.f), p.softcap_log2);
          }
          if (p.alibi != nullptr) {
            v.x = fmaf(-rows.slope[nt][0], fabsf(static_cast<float>(rows.pos[nt][0] - key)), v.x);
            v.y = fmaf(-rows.slope[nt][1], fabsf(static_cast<float>(rows.pos[nt][1] - key)), v.y);
          }
        }
        if (!WHOLE) {
          v.x = in && key >= rows.lo[nt][0] && key <= rows.hi[nt][0] ? v.x : -INFINITY;
          v.y = in && key >= rows.lo[nt][1] && key <= rows.hi[nt][1] ? v.y : -INFINITY;
        }
        x[mt][nt][h2] = v;
        if (h2 == 1) {  // two keys at a time
          mx[nt][0] = max3f(mx[nt][0], x[mt][nt][0].x, v.x);
          mx[nt][1] = max3f(mx[nt][1], x[mt][nt][0].y, v.y);
        }
      }
    }
}

// Scores -> probabilities times their values' scales; the probabilities' sums, and the largest
// product of each row.
template <bool WHOLE, int NT>
__device__ __forceinline__ void dq_weights(float2 (&x)[4][NT][2], const float (&vs)[4][2],
                                           const float2 (&m_neg)[NT], float2 (&l_run)[NT], float (&wm)[NT][2]) {
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        const float2 v = x[mt][nt][h2];
        const float2 d = add2(v, m_neg[nt]);
        const float2 pr = make_float2(ex2(d.x), ex2(d.y));
        l_run[nt] = add2(l_run[nt], pr);
        float2 w = mul2(pr, both(vs[mt][h2]));
        if (!WHOLE) {  // a masked key's scale may be anything
          w.x = v.x == -INFINITY ? 0.f : w.x;
          w.y = v.y == -INFINITY ? 0.f : w.y;
        }
        x[mt][nt][h2] = w;
      }
      wm[nt][0] = max3f(wm[nt][0], x[mt][nt][0].x, x[mt][nt][1].x);
      wm[nt][1] = max3f(wm[nt][1], x[mt][nt][0].y, x[mt][nt][1].y);
    }
}

__device__ __forceinline__ float dq_pow2(int field) { return __uint_as_float(static_cast<uint32_t>(field) << 23); }

// The reference of a row's products is the power of two above the largest of them, `top`, kept as
// inv = 2^14 / ref.  (At least 2^-112, so that inv and its inverse are normal numbers.)
constexpr int kDqInvMax = 268 - 15;  // exponent field of inv for the smallest reference

// Multiplies O by al and moves it from the reference behind inv to that of `top`.
template <int KS>
__device__ __forceinline__ void dq_rebase(float top, float al, int h, float& inv, float (&acc)[KS][4]) {
  const int now = 268 - static_cast<int>(min(max((__float_as_uint(top) >> 23) + 1u, 15u), 253u));
  // (beyond 2^127 only where al is 0, below 2^-126 only where nothing of O is left)
  const int field = 127 + now - static_cast<int>(__float_as_uint(inv) >> 23);
  const float f = al * dq_pow2(min(max(field, 0), 254));
  inv = dq_pow2(now);
#pragma unroll
  for (int k = 0; k < KS; ++k) acc[k][h] *= f, acc[k][2 + h] *= f;
}

// P V over the tile, from the products of probabilities and scales.  SPLIT: what rounding them to
// fp16 leaves is a second operand, so that they carry 22 bits.
template <int D, bool E4M3, int NT, bool SPLIT, bool WHOLE>
__device__ __forceinline__ void dq_values(const DqSeq& sq, int key0, const uint8_t* sV, int t4, int vchunk,
                                          const float2 (&w)[4][NT][2], const float2 (&inv)[NT],
                                          float (&acc)[NT][D / 16][4]) {
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
    for (int h2 = 0; h2 < 2; ++h2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 pv = mul2(w[mt][nt][h2], inv[nt]);
        const uint32_t hi = pack2<false>(pv.x, pv.y);
        pb[nt][h2] = transpose8(hi);
        if constexpr (SPLIT) {
          const float2 r = unpack2<false>(hi);
          pl[nt][h2] = transpose8(pack2<false>(pv.x - r.x, pv.y - r.y));
        }
      }
    }
    // P V over these 16 keys: this lane's keys are t4, t4 + 4, t4 + 8, t4 + 12
    uint32_t vw[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * mt + t4 + 4 * i;
      if constexpr (D == 128) {
        const uint4 v = *reinterpret_cast<const uint4*>(sV + r * 128 + ((vchunk ^ (r & 7)) << 4));
        vw[i][0] = v.x, vw[i][1] = v.y, vw[i][2] = v.z, vw[i][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(
            sV + r * 64 + ((((vchunk >> 1) ^ ((r >> 1) & 3)) << 4) | ((vchunk & 1) << 3)));
        vw[i][0] = v.x, vw[i][1] = v.y;
      }
      if (!WHOLE) {  // codes behind the last key may be anything, an E4M3 NaN among it
        const bool in = key0 + r >= sq.key_lo && key0 + r < sq.key_hi;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) vw[i][c] = in ? vw[i][c] : 0u;
      }
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // bytes of two keys side by side: one pair of fp16 is two keys of one element
        const uint32_t sel = h == 0 ? 0x5410 : 0x7632;
        uint32_t a0, a1, a2, a3;
        codes_f16<E4M3>(__byte_perm(vw[0][c], vw[1][c], sel), a0, a1);
        codes_f16<E4M3>(__byte_perm(vw[2][c], vw[3][c], sel), a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(acc[nt][2 * c + h], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
          if constexpr (SPLIT) mma_f16(acc[nt][2 * c + h], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
        }
      }
  }
}

// One piece's result: O of a pair's query rows (m, l, acc as in the kernel), written as final
// rows or as partial ones.
template <int D, int NT, bool BF16>
__device__ __forceinline__ void dq_write(const DecodeQuantParams& p, const DqWalk& wk, bool direct,
                                         int64_t slot, int g, int t4, int vchunk, float per_inv,
                                         const float2 (&inv)[NT], const float (&m_run)[NT][2], const float2 (&l_run)[NT],
                                         const float (&acc)[NT][D / 16][4]) {
  constexpr float kLn2 = 0.6931471805599453f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = h == 0 ? l_run[nt].x : l_run[nt].y;
#pragma unroll
      for (int o = 4; o < 32; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
      const int rr = nt * 8 + 2 * t4 + h, r = wk.grp * 8 * NT + rr;
      if (r >= p.R) continue;
      const float m = m_run[nt][h], unit = per_inv / (h == 0 ? inv[nt].x : inv[nt].y);
      if (direct) {
        // no allowed key: l is 0 and the row is 0 with LSE -inf; a NaN stays one
        const float f = l == 0.f ? 0.f : unit / l;
        const int gq = r / p.Sq, i = r % p.Sq, hq = wk.hk * p.G + gq;
        uint16_t* dst = static_cast<uint16_t*>(p.out) +
                        ((static_cast<int64_t>(wk.b) * p.Sq + i) * p.H + hq) * D + vchunk * (D / 8);
#pragma unroll
        for (int c = 0; c < D / 32; c += 2) {
          uint4 v;
          v.x = pack2<BF16>(acc[nt][2 * c][h] * f, acc[nt][2 * c][2 + h] * f);
          v.y = pack2<BF16>(acc[nt][2 * c + 1][h] * f, acc[nt][2 * c + 1][2 + h] * f);
          v.z = pack2<BF16>(acc[nt][2 * c + 2][h] * f, acc[nt][2 * c + 2][2 + h] * f);
          v.w = pack2<BF16>(acc[nt][2 * c + 3][h] * f, acc[nt][2 * c + 3][2 + h] * f);
          *reinterpret_cast<uint4*>(dst + 4 * c) = v;
        }
        if (g == 0 && p.lse != nullptr)
          p.lse[(static_cast<int64_t>(wk.b) * p.H + hq) * p.Sq + i] =
              l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        float* ws = p.ws_parts + (slot * 8 * NT + rr) * (D + 4);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          *reinterpret_cast<float4*>(ws + vchunk * (D / 8) + 4 * c) =
              make_float4(acc[nt][2 * c][h] * unit, acc[nt][2 * c][2 + h] * unit,
                          acc[nt][2 * c + 1][h] * unit, acc[nt][2 * c + 1][2 + h] * unit);
        if (g == 0) {
          ws[D] = m;
          ws[D + 1] = l;
        }
      }
    }
}

template <int D, bool E4M3, int NT, bool EXTRA, bool BF16>
__global__ void __launch_bounds__(DqCfg<D, NT>::kThreads, 1)
    decode_quant_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const DecodeQuantParams p) {
  using Cfg = DqCfg<D, NT>;
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kUnit = E4M3 ? 256.f : 1.f;  // acc * kUnit / inv is in units of v
  constexpr int KS = D / 16;      // k-steps of the scores, and 16-row blocks of O^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // the join may be brought to the SMs now; it waits for this grid's end by itself
  asm volatile("griddepcontrol.launch_dependents;");
  uint64_t* fullK = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff) + 2 * warp;
  uint64_t* fullV = fullK + 1;
  if (lane == 0) {
    mbar_init(fullK, p.bulk_scales ? 1 : 1 + 32);  // the copies; each lane's scale words
    mbar_init(fullV, 1);
    fence_mbar_init();
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
  }
  // every lane waits on both barriers and, where the scales come word by word, arrives on the first:
  // shuffles alone would not order that behind their initialisation
  __syncwarp();

  // ---- this warp's share of the line of tiles.  (The host has made sure that 31 bits count it.)
  const int pairs = p.Hkv * p.groups;  // pairs of one sequence
  const int share_id = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
  int total = 0;
  for (int b = lane; b < p.B; b += 32) total += dq_seq(p, b, share_id == 0).n * pairs;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) total += __shfl_xor_sync(0xffffffffu, total, o);
  // the first `more` shares have one tile more than the rest
  const int share = static_cast<int>(static_cast<unsigned>(total) / static_cast<unsigned>(p.shares));
  const int more = total - share * p.shares;
  const int line0 = share_id * share + min(share_id, more);
  const int count = share + (share_id < more);  // tiles of this share
  if (count == 0) return;
  // its first sequence: 32 at a time, each lane the end of its own on the line
  DqWalk wk;  // the piece at hand
  wk.n = 0;
  for (int base = 0, before = 0;; base += 32) {
    if (base >= p.B) return;  // (only if the lengths changed since they were added up)
    DqSeq sq = {};
    int end = 0;
    if (base + lane < p.B) {
      sq = dq_seq(p, base + lane, false);
      end = sq.n * pairs;
    }
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    end += before;
    const unsigned past = __ballot_sync(0xffffffffu, end > line0);
    if (past != 0u) {
      const int i = __ffs(past) - 1;
      wk.b = base + i;
      wk.sq.L = __shfl_sync(0xffffffffu, sq.L, i);
      wk.sq.off = __shfl_sync(0xffffffffu, sq.off, i);
      wk.sq.key_lo = __shfl_sync(0xffffffffu, sq.key_lo, i);
      wk.sq.key_hi = __shfl_sync(0xffffffffu, sq.key_hi, i);
      wk.sq.t_lo = __shfl_sync(0xffffffffu, sq.t_lo, i);
      wk.sq.n = __shfl_sync(0xffffffffu, sq.n, i);
      const int in = line0 - (__shfl_sync(0xffffffffu, end, i) - wk.sq.n * pairs);
      const int pair = static_cast<int>(static_cast<unsigned>(in) / static_cast<unsigned>(wk.sq.n));
      wk.at = in - pair * wk.sq.n;
      wk.hk = p.groups == 1 ? pair : pair / p.groups;
      wk.grp = pair - wk.hk * p.groups;
      break;
    }
    before = __shfl_sync(0xffffffffu, end, 31);
  }
  // this warp's buffers, and the next tile that it brings
  uint8_t* bufK = smem + 2 * warp * Cfg::kTileBytes;
  uint8_t* bufV = bufK + Cfg::kTileBytes;
  float* sks = reinterpret_cast<float*>(smem + Cfg::kScaleOff + warp * Cfg::kScaleBytes);
  float* svs = sks + kDqTok;
  DqWalk fw = wk;
  int filled_k, filled_v;  // tiles brought so far
  dq_locate(p, fw);
  dq_fill<D, NT, false>(p, &tmK, fw, bufK, sks, fullK);
  dq_fill<D, NT, true>(p, &tmV, fw, bufV, sks, fullV);
  filled_k = filled_v = fw.sq.key_hi > fw.sq.key_lo;
  dq_advance(p, fw, 1, count);
  if (fw.n < count) dq_locate(p, fw);

  const int g = lane / 4, t4 = lane % 4;
  // Index g of a product of 16 keys is key perm(g) (rows 0-7) and perm(g) + 8.
  const int perm = (g >> 1) + 4 * (g & 1);
  const int vchunk = D == 128 ? (((g & 1) << 2) | (g >> 1)) : g;  // this lane's head-dim part in P V
  const bool causal_or_right = p.causal || p.wr >= 0;
  const int right = p.causal ? 0 : p.wr;
  uint32_t phase = 0;  // of this warp's buffers
  bool ok = true;
  while (wk.n < count) {
    const DqSeq& sq = wk.sq;
    const int hk = wk.hk;
    const int cnt = min(sq.n - wk.at, count - wk.n);  // tiles of the piece
    const int r0 = wk.grp * Cfg::kRows;  // first query row of the pair (row r: head r / Sq, query r % Sq)

    // ---- query rows as the B operand: lane (g, t4) holds row g of each block of 8, the head-dim
    // elements of its 16-byte code chunks
    uint32_t qf[Cfg::kQShared ? 1 : NT][KS][2];
    uint2* qs = reinterpret_cast<uint2*>(smem + Cfg::kQOff + warp * Cfg::kQBytes) + lane;
    DqRows<NT> rows;  // rows 2 t4 and 2 t4 + 1 of each block
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + nt * 8 + g;
      const bool live = r < p.R;
      uint32_t raw[KS][2];
      {
        const int gq = live ? r / p.Sq : 0, i = live ? r % p.Sq : 0;
        const uint16_t* row = static_cast<const uint16_t*>(p.q) +
                              ((static_cast<int64_t>(wk.b) * p.Sq + i) * p.H + hk * p.G + gq) * D;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (live) v = __ldg(reinterpret_cast<const uint4*>(row + (t4 + 4 * c) * 16) + h);
            raw[c * 4 + 2 * h][0] = v.x, raw[c * 4 + 2 * h][1] = v.y;
            raw[c * 4 + 2 * h + 1][0] = v.z, raw[c * 4 + 2 * h + 1][1] = v.w;
          }
        }
      }
      // the row times a power of two that brings its largest magnitude to 2^6 .. 2^7: exact in
      // fp16 down to 2^-20 of the largest, and off by at most 2^-32 of the largest below
      float back;
      {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          m = __vmaxu2(m, raw[k][0] & 0x7fff7fffu);
          m = __vmaxu2(m, raw[k][1] & 0x7fff7fffu);
        }
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = max(m & 0xffffu, m >> 16);
        const float big = unpack2<BF16>(m).x;
        // 2^(133 - e), exponent field 260 - e, kept within 7 .. 253 with its inverse (an
        // infinity or a NaN in the row stays one)
        const int f = min(max(260 - static_cast<int>(__float_as_uint(big) >> 23), 7), 253);
        const float up = __uint_as_float(static_cast<uint32_t>(f) << 23);
        back = __uint_as_float(static_cast<uint32_t>(254 - f) << 23);
        // elements 4 k .. 4 k + 3 in the pairs that the codes come in
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const float2 x = unpack2<BF16>(raw[k][0]);
          const float2 y = unpack2<BF16>(raw[k][1]);
          const uint32_t q0 = E4M3 ? pack2<false>(x.x * up, x.y * up) : pack2<false>(x.x * up, y.x * up);
          const uint32_t q1 = E4M3 ? pack2<false>(y.x * up, y.y * up) : pack2<false>(x.y * up, y.y * up);
          if constexpr (Cfg::kQShared)
            qs[(nt * KS + k) * 32] = make_uint2(q0, q1);
          else
            qf[nt][k][0] = q0, qf[nt][k][1] = q1;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int rr = r0 + nt * 8 + 2 * t4 + h;
        const bool lv = rr < p.R;
        const int gq = lv ? rr / p.Sq : 0, i = lv ? rr % p.Sq : 0;
        const float fac = EXTRA && p.has_softcap ? p.tanh_k : p.scale_log2;
        rows.rf[nt][h] = fac * __shfl_sync(0xffffffffu, back, 4 * (2 * t4 + h));
        rows.slope[nt][h] = EXTRA && p.alibi != nullptr ? p.alibi[hk * p.G + gq] * kLog2e : 0.f;
        const int at = i + sq.off;
        rows.pos[nt][h] = at;
        rows.lo[nt][h] = lv && p.wl >= 0 ? at - p.wl : INT_MIN;
        rows.hi[nt][h] = lv && causal_or_right ? min(at + right, sq.L - 1) : sq.L - 1;
      }
    }
    // keys that every row of the sequence sees: tiles inside need no mask
    const int all_lo = p.wl >= 0 ? max(sq.off + p.Sq - 1 - p.wl, 0) : 0;
    const int all_hi = causal_or_right ? min(sq.off + right, sq.L - 1) : sq.L - 1;

    float m_run[NT][2], acc[NT][KS][4];
    float2 l_run[NT];
    float top[NT][2];  // the largest product of a probability and a value scale met so far
    float2 inv[NT];    // 2^14 by the power of two above it
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m_run[nt][0] = m_run[nt][1] = -INFINITY;
      top[nt][0] = top[nt][1] = 0.f;
      inv[nt] = both(dq_pow2(kDqInvMax));
      l_run[nt] = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][k][e] = 0.f;
    }

    const bool seen = sq.key_hi > sq.key_lo;
    for (int t = 0; t < cnt; ++t) {
      const bool follows = fw.n < count;  // another tile of this warp's
      if (seen) {
        ok = dq_wait(p, fullK, phase);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        // ---- products of 64 keys: x[mt][nt][h2] = key 16 mt + perm + 8 h2, rows 2 t4 and 2 t4 + 1
        float c4[4][NT][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) c4[mt][nt][e] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t wa[4][4], wb[4][4];
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            const int ra = 16 * mt + perm, rb = ra + 8;
            const int at_a = D == 128 ? ra * 128 + (((t4 + 4 * c) ^ (ra & 7)) << 4)
                                      : ra * 64 + ((t4 ^ ((ra >> 1) & 3)) << 4);
            const int at_b = D == 128 ? rb * 128 + (((t4 + 4 * c) ^ (rb & 7)) << 4)
                                      : rb * 64 + ((t4 ^ ((rb >> 1) & 3)) << 4);
            const uint4 ka = *reinterpret_cast<const uint4*>(bufK + at_a);
            const uint4 kb = *reinterpret_cast<const uint4*>(bufK + at_b);
            wa[mt][0] = ka.x, wa[mt][1] = ka.y, wa[mt][2] = ka.z, wa[mt][3] = ka.w;
            wb[mt][0] = kb.x, wb[mt][1] = kb.y, wb[mt][2] = kb.z, wb[mt][3] = kb.w;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t qb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (Cfg::kQShared) {
                const uint2 v = qs[(nt * KS + c * 4 + i) * 32];
                qb[nt][0] = v.x, qb[nt][1] = v.y;
              } else {
                qb[nt][0] = qf[nt][c * 4 + i][0], qb[nt][1] = qf[nt][c * 4 + i][1];
              }
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {  // four independent chains of sums
              uint32_t a0, a1, a2, a3;
              if constexpr (E4M3) {
                codes_cvt(wa[mt][i], a0, a2);
                codes_cvt(wb[mt][i], a1, a3);
              } else {
                codes_f16<false>(wa[mt][i], a0, a2);
                codes_f16<false>(wb[mt][i], a1, a3);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(c4[mt][nt], a0, a1, a2, a3, qb[nt][0], qb[nt][1]);
            }
          }
        }
        float2 x[4][NT][2];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            x[mt][nt][0] = make_float2(c4[mt][nt][0], c4[mt][nt][1]);
            x[mt][nt][1] = make_float2(c4[mt][nt][2], c4[mt][nt][3]);
          }
        // ---- base-2 scores, the tile's max per row
        const int key0 = (sq.t_lo + wk.at + t) * kDqTok;
        const bool whole = key0 >= all_lo && key0 + kDqTok - 1 <= all_hi;
        float vs[4][2];  // value scales of this lane's keys
        float mx[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
        if (whole)
          dq_scores<true, EXTRA, NT>(p, rows, sq, key0, perm, sks, svs, x, vs, mx);
        else
          dq_scores<false, EXTRA, NT>(p, rows, sq, key0, perm, sks, svs, x, vs, mx);
        // the K tile and the scales are used: bring the next ones
        __syncwarp();
        if (follows) {
          dq_fill<D, NT, false>(p, &tmK, fw, bufK, sks, fullK);
          filled_k += fw.sq.key_hi > fw.sq.key_lo;
        }
#pragma unroll
        for (int o = 4; o < 32; o *= 2)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mx[nt][h] = fmaxf(mx[nt][h], __shfl_xor_sync(0xffffffffu, mx[nt][h], o));
        // ---- grown max: the sums, O and the products' reference move with it
        bool grown = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) grown |= mx[nt][h] > m_run[nt][h];
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float m_new = fmaxf(m_run[nt][h], mx[nt][h]);
              const float al = m_new == -INFINITY ? 1.f : ex2(m_run[nt][h] - m_new);
              m_run[nt][h] = m_new;
              (h == 0 ? l_run[nt].x : l_run[nt].y) *= al;
              top[nt][h] *= al;
              dq_rebase<KS>(top[nt][h], al, h, h == 0 ? inv[nt].x : inv[nt].y, acc[nt]);
            }
        }
        float2 m_neg[NT];  // minus the max (0 while a row has met no key)
        float wm[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          m_neg[nt] = make_float2(m_run[nt][0] == -INFINITY ? 0.f : -m_run[nt][0],
                                  m_run[nt][1] == -INFINITY ? 0.f : -m_run[nt][1]);
          wm[nt][0] = wm[nt][1] = 0.f;
        }
        if (whole)
          dq_weights<true, NT>(x, vs, m_neg, l_run, wm);
        else
          dq_weights<false, NT>(x, vs, m_neg, l_run, wm);
        // ---- a product that reaches the reference: it moves above the tile's largest
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          over |= wm[nt][0] * inv[nt].x >= 16384.f || wm[nt][1] * inv[nt].y >= 16384.f;
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int o = 4; o < 32; o *= 2)
                wm[nt][h] = fmaxf(wm[nt][h], __shfl_xor_sync(0xffffffffu, wm[nt][h], o));
              top[nt][h] = fmaxf(top[nt][h], wm[nt][h]);
              dq_rebase<KS>(top[nt][h], 1.f, h, h == 0 ? inv[nt].x : inv[nt].y, acc[nt]);
            }
        }
        ok = dq_wait(p, fullV, phase);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        phase ^= 1;
        if (whole)
          dq_values<D, E4M3, NT, !BF16, true>(sq, key0, bufV, t4, vchunk, x, inv, acc);
        else
          dq_values<D, E4M3, NT, !BF16, false>(sq, key0, bufV, t4, vchunk, x, inv, acc);
        __syncwarp();
      } else if (follows) {  // no keys: nothing was brought, the buffers are free
        dq_fill<D, NT, false>(p, &tmK, fw, bufK, sks, fullK);
        filled_k += fw.sq.key_hi > fw.sq.key_lo;
      }
      if (follows) {
        dq_fill<D, NT, true>(p, &tmV, fw, bufV, sks, fullV);
        filled_v += fw.sq.key_hi > fw.sq.key_lo;
        dq_advance(p, fw, 1, count);
        if (fw.n < count) dq_locate(p, fw);
      }
    }
    if (!ok) {
      // a wait gave up: let this warp's copies land before the shared memory goes away
      cp_async_wait_all();
      const uint64_t t0 = globaltimer_ns();
      while (!(mbar_try_wait(fullK, (filled_k - 1) & 1) && mbar_try_wait(fullV, (filled_v - 1) & 1)))
        if (globaltimer_ns() - t0 > p.timeout_ns) break;
      return;
    }
    const bool direct = wk.at == 0 && cnt == sq.n;  // the whole pair lies in this share
    const int64_t slot = 2 * static_cast<int64_t>(share_id) + (wk.n == 0 ? 0 : 1);
    dq_write<D, NT, BF16>(p, wk, direct, slot, g, t4, vchunk, kUnit, inv, m_run, l_run, acc);
    // the warp that begins a pair notes which slots hold its pieces
    if (wk.at == 0 && lane == 0) {
      const int64_t pair = static_cast<int64_t>(wk.b) * pairs + wk.hk * p.groups + wk.grp;
      // the share that ends it, and how many pieces follow the first
      const int end = line0 + wk.n + sq.n - 1, longer = more * (share + 1);
      const int last = end < longer ? static_cast<int>(static_cast<unsigned>(end) / static_cast<unsigned>(share + 1))
                                    : more + static_cast<int>(static_cast<unsigned>(end - longer) / static_cast<unsigned>(share));
      p.ws_notes[pair] = make_int2(static_cast<int>(slot), last - share_id);
    }
    dq_advance(p, wk, cnt, count);
  }
}

// Joins the pieces of the pairs that span several shares.  Slot `note.x` holds the first piece;
// the following shares' pieces are their first ones (even slots).  W warps per query row take
// every W-th piece each.
constexpr int kDqJoinThreads = 256;

template <int D, int NT, int W>
__global__ void __launch_bounds__(kDqJoinThreads) decode_quant_join_kernel(const DecodeQuantParams p) {
  constexpr float kLn2 = 0.6931471805599453f;
  constexpr int kRows = 8 * NT, V = D / 32;  // V columns per lane
  __shared__ float part[W > 1 ? kDqJoinThreads / 32 : 1][D + 2];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, wj = warp % W;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * (kDqJoinThreads / 32) + warp) / W;
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv * p.R;
  const int64_t pr = dq_div(row, p.R);  // (sequence, KV head)
  const int r = static_cast<int>(row - pr * p.R);
  const int b = static_cast<int>(dq_div(pr, p.Hkv)), hk = static_cast<int>(pr - static_cast<int64_t>(b) * p.Hkv);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are written
  if (row >= rows) return;  // (all W warps of a row)
  const int2 note = p.ws_notes[pr * p.groups + r / kRows];
  if (note.y == 0) return;  // written by the warp that had all of it
  // A warp whose wait ran out leaves its notes unwritten (and the status word set): nothing outside
  // the slots is read.
  if (note.x < 0 || note.y < 0 || note.y > p.shares || note.x / 2 + note.y >= p.shares) return;
  const int64_t step = static_cast<int64_t>(2) * kRows * (D + 4);
  const float* first = p.ws_parts + (static_cast<int64_t>(note.x) * kRows + r % kRows) * (D + 4);
  const float* rest = first - (note.x & 1) * static_cast<int64_t>(kRows) * (D + 4);  // even slots
  // one pass with a running max: eight pieces are read at once, then taken in
  float M = -INFINITY, l = 0.f, o[V];
#pragma unroll
  for (int c = 0; c < V; ++c) o[c] = 0.f;
  auto take = [&](float m, float lp, const float (&v)[V]) {
    const float n = fmaxf(M, m);
    // a piece without an allowed key adds nothing; one with a NaN makes the row NaN
    const float f = m == -INFINITY ? (lp == lp ? 0.f : lp) : ex2(m - n);
    const float g = M == -INFINITY ? (l == l ? 0.f : l) : ex2(M - n);
    l = fmaf(lp, f, l * g);
#pragma unroll
    for (int c = 0; c < V; ++c) o[c] = fmaf(v[c], f, o[c] * g);
    M = n;
  };
  constexpr int U = 8;
  for (int i0 = wj; i0 <= note.y; i0 += U * W) {
    float m[U], lp[U], v[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * W;
      m[u] = -INFINITY, lp[u] = 0.f;
#pragma unroll
      for (int c = 0; c < V; ++c) v[u][c] = 0.f;
      if (i <= note.y) {
        const float* src = i == 0 ? first : rest + i * step;
        const float2 ml = *reinterpret_cast<const float2*>(src + D);
        m[u] = ml.x, lp[u] = ml.y;
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src + lane * 4);
          v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src + lane * 2);
          v[u][0] = x.x, v[u][1] = x.y;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) take(m[u], lp[u], v[u]);
  }
  if constexpr (W > 1) {  // a CTA has the W warps of whole rows; they all get here together
#pragma unroll
    for (int c = 0; c < V; ++c) part[warp][lane * V + c] = o[c];
    if (lane == 0) part[warp][D] = M, part[warp][D + 1] = l;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / W), "r"(32 * W) : "memory");
    if (wj != 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      float v[V];
#pragma unroll
      for (int c = 0; c < V; ++c) v[c] = part[warp + w][lane * V + c];
      take(part[warp + w][D], part[warp + w][D + 1], v);
    }
  }
  const float inv_l = l == 0.f ? 0.f : 1.f / l;
  const int gq = r / p.Sq, i2 = r % p.Sq, h = hk * p.G + gq;
  uint16_t* dst = static_cast<uint16_t*>(p.out) +
                  ((static_cast<int64_t>(b) * p.Sq + i2) * p.H + h) * D + lane * V;
  if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(dq_pack(p.bf16, o[0] * inv_l, o[1] * inv_l),
                                                dq_pack(p.bf16, o[2] * inv_l, o[3] * inv_l));
  } else {
    *reinterpret_cast<uint32_t*>(dst) = dq_pack(p.bf16, o[0] * inv_l, o[1] * inv_l);
  }
  if (lane == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(b) * p.H + h) * p.Sq + i2] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

}  // namespace fa
