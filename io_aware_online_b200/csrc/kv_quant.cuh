// kv_quant.cuh -- the 8-bit KV cache: where a row lies, and how it is quantised.
//
// A row is one (token, KV head): D values.  With m = max |x| over the row and `top` the
// format's largest value (448 for E4M3, 127 for int8),
//
//   scale = m / top,   code = round(x * top / m),   value = code * scale.
//
// One scale per row needs no calibration pass, and one large row (or one large head) costs
// no other row precision.  The codes are the correctly rounded ones: fp32 holds far more bits
// than separate any quotient of two 16-bit floats from a rounding border it does not lie on.
#pragma once

#include "quant_device.cuh"

namespace fa {

// Row `pos` of sequence b: the element offset of its head 0 in the code arrays and the
// offset of its head 0 in the scale arrays (heads are `rows` apart there).
struct CacheRow {
  int64_t code;
  int64_t scale;
};

// 0, or the FA_DEV_* bit of a position the cache does not hold.
__device__ __forceinline__ unsigned locate_row(const QuantCache& c, int b, int64_t pos,
                                               CacheRow* out) {
  int64_t blk = b, row = pos;
  if (c.block_table != nullptr) {
    if (pos < 0 || pos >= static_cast<int64_t>(c.max_blocks) * c.rows) return kDevBadLength;
    const unsigned page = divide(static_cast<unsigned>(pos), c.div_rows);  // (pos is below 2^30)
    blk = c.block_table[static_cast<int64_t>(b) * c.max_blocks + page];
    if (blk < 0 || blk >= c.num_blocks) return kDevBadBlock;
    row = static_cast<unsigned>(pos) - page * c.div_rows.d;
  } else if (pos < 0 || pos >= c.rows) {
    return kDevBadLength;
  }
  out->code = blk * c.st_block + row * c.st_row;
  out->scale = blk * c.Hkv * c.rows + row;
  return 0u;
}

// The sequence that owns packed row r: the last b with cu[b] <= r (cu[0] is 0).  Each lane for
// itself; the table's upper levels are shared by all rows and stay in L1.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int r) {
  int lo = 0, n = B;
  while (n > 1) {
    const int half = n / 2;
    if (cu[lo + half] <= r) {
      lo += half;
      n -= half;
    } else {
      n = half;
    }
  }
  return lo;
}

// ---- quantising one row, held by LPR neighbouring lanes as packed 16-bit pairs

template <bool BF16>
__device__ __forceinline__ uint32_t abs2(uint32_t x) {
  uint32_t y;
  if constexpr (BF16)
    asm("abs.bf16x2 %0, %1;" : "=r"(y) : "r"(x));
  else
    asm("abs.f16x2 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The larger of two pairs, NaN if either is one.
template <bool BF16>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t y;
  if constexpr (BF16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// Largest magnitude of the row as 16-bit float bits: for |x| their order as whole
// numbers is the order of the values, with infinity and then NaN above them.
template <bool BF16, int NW, int LPR>
__device__ __forceinline__ uint32_t row_max_bits(const uint32_t (&w)[NW]) {
  uint32_t m = abs2<BF16>(w[0]);
#pragma unroll
  for (int i = 1; i < NW; ++i) m = max2_nan<BF16>(m, abs2<BF16>(w[i]));
#pragma unroll
  for (int o = 1; o < LPR; o *= 2) m = max2_nan<BF16>(m, __shfl_xor_sync(0xffffffffu, m, o));
  return max(m & 0xffffu, m >> 16);
}

struct RowQuant {
  float scale;    // what a code is worth
  float hi, lo;   // top / m in two parts: hi + lo is it to 2^-40 (2^-28 where lo is subnormal)
};

// The factors of a row; w, a lane's part of it, is put right where the row has no scale or a
// largest value whose reciprocal leaves fp32.
template <bool BF16, bool E4M3, int NW>
__device__ __forceinline__ RowQuant row_quant(uint32_t max_bits, uint32_t (&w)[NW]) {
  constexpr float kTop = E4M3 ? 448.f : 127.f;
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  // bf16 below 2^-99: the scale nears fp32's subnormals and top / m leaves it, so the scale is
  // had by a division, and the row is quantised times 2^60 (exact)
  constexpr uint32_t kTiny = BF16 ? 28u << 7 : 1u;
  RowQuant r;
  const bool none = max_bits == 0 || max_bits >= kInf, tiny = max_bits < kTiny;
  float m = unpack2<BF16>(max_bits).x;
  // m / top rounded correctly: the product with the rounded reciprocal and one residual step (the
  // division by a constant of Brisebarre, Muller and Raina; tested over every mantissa)
  constexpr float kRcpTop = 1.f / kTop;
  const float s = m * kRcpTop;
  r.scale = fmaf(fmaf(-s, kTop, m), kRcpTop, s);
  if (none || tiny) {
    // an all-zero row stands for zeros; a row with an infinity or a NaN has no scale and
    // reads back as NaN throughout.  Their codes are 0.
    if (none) {
      r.scale = max_bits == 0 ? 0.f : __uint_as_float(0x7fc00000u);
      m = 1.f;
    } else {
      r.scale = __fdiv_rn(m, kTop);
      m *= 0x1p60f;
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const float2 x = unpack2<BF16>(w[i]);
      w[i] = none ? 0u : pack2<BF16>(x.x * 0x1p60f, x.y * 0x1p60f);
    }
  }
  // m brought near 1 by a power of two, so that the reciprocal stays in the normal range
  const uint32_t e = min(__float_as_uint(m) >> 23, 253u);
  const float f = __uint_as_float((254u - e) << 23);
  const float n = m * f;
  // hi is below top / m (the reciprocal is good to 2^-23), so that lo is positive and a -0 keeps
  // its sign; the remainder is exact
  const float c = rcp(n), hi = c * (kTop * (1.f - 0x1p-20f));
  r.lo = fmaf(-hi, n, kTop) * c * f;
  r.hi = hi * f;
  return r;
}

// x * top / m rounded to fp32, for a pair: the exact sum of x * hi and a product that is off by
// less than 2^-27 of it.  Where the quotient lies on a rounding border, which fp32 holds, the sum
// is rounded to just that; a quotient beside a border is at least 2^-19 of it away (for int8:
// 254 X and (2 k + 1) M 2^e are different whole numbers below 2^19).  Exact codes for two
// operations a pair: an IEEE division costs several times these.
__device__ __forceinline__ float2 quotient(float2 x, const RowQuant& r) {
  return fma2(x, both(r.hi), mul2(x, both(r.lo)));
}

// Eight packed values -> eight codes, lowest index in the lowest byte.
template <bool BF16, bool E4M3>
__device__ __forceinline__ uint2 quantise8(const uint32_t* w, const RowQuant& r) {
  uint32_t c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float2 a = quotient(unpack2<BF16>(w[2 * i]), r), b = quotient(unpack2<BF16>(w[2 * i + 1]), r);
    if constexpr (E4M3) {
      c[i] = pack4_e4m3(a.x, a.y, b.x, b.y);
    } else {
      // adding 1.5 * 2^23 rounds to a whole number (ties to even) and leaves its two's
      // complement in the low byte
      constexpr float kRound = 12582912.f;
      a = add2(a, both(kRound));
      b = add2(b, both(kRound));
      const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
      const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
      c[i] = __byte_perm(lo, hi, 0x5410);
    }
  }
  return make_uint2(c[0], c[1]);
}

}  // namespace fa
