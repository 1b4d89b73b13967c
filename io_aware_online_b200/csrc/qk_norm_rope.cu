// qk_norm_rope.cu -- the input side of attention: RMS norm of every query and key head and
// the position rotation in one pass, its gradient, and the same pass ending in an 8-bit KV
// cache (keys normalised, rotated and quantised, values quantised).
//
//   n = x * rsqrt(mean(x^2) + eps) * w                   over the head dim
//   (a, b) -> (a cos - b sin, b cos + a sin)             over the first `rot` elements
//
// Pure streaming, bound by HBM: each row is read once and written once, and a token's cos
// and sin row once per group of heads.  A row of D 16-bit values belongs to D / 16
// neighbouring lanes, two 16-byte vectors each.  The two vectors of a lane are chosen so that
// both halves of every rotated pair lie in one lane: the rotation then needs no exchange, and
// the norm only the sum over the row's lanes.  A group is 32 / (D / 16) rows of one token (1 KB);
// the grid is one wave (several for long calls without a cache), and each warp walks a stretch of
// neighbouring groups, two at a time.
// What bounds such a pass is how much of it is in flight: a warp copies the next groups (and a
// new token's angles) into a ring in shared memory while it works on one, so that the loads do
// not have to fit its registers.  What the groups of 32 tokens need besides their rows (their
// sequences, places in the cache, positions) is worked out by the 32 lanes at once.
//   (Measured, 4 x 4096 tokens of 32 + 8 heads, d=128, bf16: four groups per warp held in
//   registers took 91 us at 16 resident warps per SM; the ring in one wave 72, in waves of 12 steps
//   60.5 us, 87% of the copy rate; 4 x 16384 tokens 217 us, 97%.  What bounds it now is the issue of
//   instructions beside HBM: 55% of the slots, ~196 per group.)
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "kv_quant.cuh"

namespace fa {

namespace {

constexpr int kRowsThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

// Which two 16-byte vectors (8 elements each) of a row lane j of its group holds: for the
// rotated part vector j and the one half of `rot` further on, for the rest two neighbours.
struct LaneVecs {
  int c0, c1;
  bool turn;  // both lie in the rotated part
};

__device__ __forceinline__ LaneVecs lane_vecs(int j, int rot) {
  const int pairs = rot / 16;
  if (j < pairs) return {j, j + pairs, true};
  const int c = 2 * pairs + 2 * (j - pairs);
  return {c, c + 1, false};
}

// The 8 cosines and sines of a lane.  Pairs half of `rot` apart: element e of vector c0 turns
// with element e of c1, angle 8 j + e.  Adjacent pairs: angles 4 c0 .. and 4 c1 ...
struct LaneAngles {
  float2 c[4], s[4];
};

__device__ __forceinline__ void load_pairs(const float* p, float2& a, float2& b) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  a = make_float2(v.x, v.y);
  b = make_float2(v.z, v.w);
}

// The lane's angles from a token's cos and sin rows in shared memory (rot / 2 floats each).
__device__ __forceinline__ void read_angles(const float* cs, int rot, const LaneVecs& lv, bool inter,
                                            LaneAngles& a) {
  if (!lv.turn) return;
  const int i0 = inter ? 4 * lv.c0 : 8 * lv.c0;
  const int i1 = inter ? 4 * lv.c1 : 8 * lv.c0 + 4;
  load_pairs(cs + i0, a.c[0], a.c[1]);
  load_pairs(cs + i1, a.c[2], a.c[3]);
  load_pairs(cs + rot / 2 + i0, a.s[0], a.s[1]);
  load_pairs(cs + rot / 2 + i1, a.s[2], a.s[3]);
}

// Rotates the lane's 16 values (x[0..3] of vector c0, x[4..7] of c1, in pairs).
template <bool BACK>
__device__ __forceinline__ void turn(float2 (&x)[8], const LaneAngles& a, bool inter) {
  if (inter) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = i % 2 == 0 ? a.c[i / 2].x : a.c[i / 2].y;
      const float s = (BACK ? -1.f : 1.f) * (i % 2 == 0 ? a.s[i / 2].x : a.s[i / 2].y);
      x[i] = fma2(make_float2(x[i].y, x[i].x), make_float2(-s, s), mul2(x[i], both(c)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 neg = make_float2(-a.s[i].x, -a.s[i].y);
      const float2 u = x[i], v = x[i + 4];
      x[i] = fma2(v, BACK ? a.s[i] : neg, mul2(u, a.c[i]));
      x[i + 4] = fma2(u, BACK ? neg : a.s[i], mul2(v, a.c[i]));
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void load_weights(const void* w, bool fp32, const LaneVecs& lv,
                                             float2 (&out)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = h == 0 ? lv.c0 : lv.c1;
    if (w == nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[4 * h + i] = both(1.f);
    } else if (fp32) {
      load_pairs(static_cast<const float*>(w) + 8 * c, out[4 * h], out[4 * h + 1]);
      load_pairs(static_cast<const float*>(w) + 8 * c + 4, out[4 * h + 2], out[4 * h + 3]);
    } else {
      const uint4 v = __ldg(static_cast<const uint4*>(w) + c);
      out[4 * h] = unpack2<BF16>(v.x), out[4 * h + 1] = unpack2<BF16>(v.y);
      out[4 * h + 2] = unpack2<BF16>(v.z), out[4 * h + 3] = unpack2<BF16>(v.w);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void unpack16(const uint32_t (&w)[8], float2 (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = unpack2<BF16>(w[i]);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o *= 2) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// rsqrt(mean(x^2) + eps) of the row.
template <int D>
__device__ __forceinline__ float inv_rms(const float2 (&x)[8], float eps) {
  float2 ss = mul2(x[0], x[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) ss = fma2(x[e], x[e], ss);
  return rsqrtf(row_sum<D / 16>(ss.x + ss.y) * (1.f / D) + eps);
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int src) {
  const int lo = __shfl_sync(kFull, static_cast<int>(v), src);
  const int hi = __shfl_sync(kFull, static_cast<int>(v >> 32), src);
  return static_cast<int64_t>(static_cast<uint32_t>(lo)) | (static_cast<int64_t>(hi) << 32);
}

// A lane's vectors of a row: at p, and `next` bytes further on.
__device__ __forceinline__ void read_row(const uint8_t* p, int next, uint32_t (&w)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + next);
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

// A token's cos and sin rows into shared memory, 16 bytes a lane.
__device__ __forceinline__ void copy_angles(uint32_t dst, const float* cos, const float* sin, int64_t at,
                                            int rot) {
  const int lane = threadIdx.x % 32, n = rot / 8;  // 16-byte vectors per row
  if (lane < 2 * n) {
    const float* src = lane < n ? cos + at + 4 * lane : sin + at + 4 * (lane - n);
    cp_async16(dst + 16 * lane, src, 16);
  }
}

__device__ __forceinline__ void store_row(uint8_t* p, int next, const uint32_t (&w)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p + next) = make_uint4(w[4], w[5], w[6], w[7]);
}

// A place in a stretch of groups: a token and the first head of its group at hand.
struct GroupWalk {
  int tok, head;
  __device__ __forceinline__ void start(unsigned x, const FastDiv& div, int rpw) {
    tok = static_cast<int>(divide(x, div));
    head = static_cast<int>(x - static_cast<unsigned>(tok) * div.d) * rpw;
  }
  __device__ __forceinline__ void next(int heads, int rpw) {
    head += rpw;
    if (head >= heads) {
      head = 0;
      ++tok;
    }
  }
};

// The element offset of a position's row of the cos and sin tables.
__device__ __forceinline__ int64_t angle_row(int64_t pos, int max_pos, int rot,
                                             unsigned int* status) {
  if (pos < 0 || pos >= max_pos) {
    atomicOr(status, kDevBadPosition);
    pos = pos < 0 ? 0 : max_pos - 1;
  }
  return pos * (rot / 2);
}

constexpr int kRing = 4;                          // steps in a warp's ring
constexpr int kGroupBytes = 1024;                 // 32 / (D / 16) rows of D 16-bit values

// ROPE false: only k and v, as they are, into a cache.  That needs 80 registers, so that 24 warps
// fit an SM: 4 x 8192 tokens 39 us, 45 with 16 warps; 61K ragged tokens 43.5 and 52 (four blocks
// and a ring of three: 39 and 47).  With norm and rotation 24 warps spill and are slower (4 x 4096
// tokens 66 us against 60.5), and so are 20, in blocks whose warps the four schedulers share
// unevenly (68-70) or in one block (73).
template <bool ROPE>
struct RowsCfg {
  // a step's slot: two groups, and a token's cos and sin rows
  static constexpr int kSlotBytes = 2 * kGroupBytes + (ROPE ? 512 : 0);
  static constexpr int kBlocksPerSm = ROPE ? 2 : 3;
  static constexpr int kSmem = kRowsThreads / 32 * kRing * kSlotBytes;
};

template <int D, bool BF16, int MODE, bool ROPE>
__global__ void __launch_bounds__(kRowsThreads, RowsCfg<ROPE>::kBlocksPerSm) rows_kernel(const RowsParams p) {
  constexpr int kSlotBytes = RowsCfg<ROPE>::kSlotBytes;
  constexpr int LPR = D / 16;        // lanes per row
  constexpr int RPW = 32 / LPR;      // rows of a group
  extern __shared__ __align__(128) uint8_t ring_mem[];
  const int lane = threadIdx.x % 32, j = lane % LPR;
  uint8_t* ring = ring_mem + threadIdx.x / 32 * (kRing * kSlotBytes);
  int gw = blockIdx.x * (kRowsThreads / 32) + threadIdx.x / 32;
  const bool is_q = ROPE && gw < p.warps_q;
  if (!is_q) gw -= p.warps_q;
  // A step is two groups: the next two of a token's q (or, without a cache, k) heads, or the same
  // heads of k and of v, which go to the same place of the cache.
  const bool kv = MODE != kRowsPlain && !is_q;
  const int heads = is_q ? p.H : p.Hkv, step = kv ? RPW : 2 * RPW;
  const FastDiv div = is_q ? p.div_q : p.div_k;
  const unsigned steps = static_cast<unsigned>(p.tokens) * div.d;
  const unsigned x0 = static_cast<unsigned>(gw) * p.per;
  if (x0 >= steps) return;
  const int count = static_cast<int>(min(steps - x0, static_cast<unsigned>(p.per)));
  const uint8_t* src[2] = {static_cast<const uint8_t*>(is_q ? p.q : p.k),
                           static_cast<const uint8_t*>(kv ? p.v : is_q ? p.q : p.k)};
  const int64_t* st = is_q ? p.q_s : p.k_s;
  const int64_t* st1 = kv ? p.v_s : st;
  const int64_t* so = is_q ? p.qo_s : p.ko_s;
  const bool rotate = ROPE && p.cos != nullptr, norm = ROPE && p.norm;
  const LaneVecs lv = lane_vecs(j, p.rot);

  // ---- what lane i knows about token base + i: its sequence b and row s in it
  auto place = [&](int tok, int& b, int& s) {
    if (p.cu != nullptr) {
      b = find_sequence(p.cu, p.B, tok);
      const int begin = p.cu[b];
      s = tok - begin;
      return tok >= begin && tok < p.cu[p.B];  // rows outside every sequence stay as they are
    }
    b = static_cast<int>(divide(tok, p.div_s));
    s = tok - b * p.S;
    return true;
  };
  // a lane's first vector of a group in shared memory, and the second's distance (there, in q, k
  // and v and in the outputs alike)
  const int row = lane / LPR, at0 = row * (2 * D) + 16 * lv.c0, next = 16 * (lv.c1 - lv.c0);
  const uint32_t ring_u32 = smem_u32(ring);

  // ---- ahead: copies of the next steps
  GroupWalk aw;
  aw.start(x0, div, step);
  int a_left = count, a_base = aw.tok - 32;
  uint32_t a_slot = 0;  // bytes
  const uint8_t* a_ptr[2] = {nullptr, nullptr};
  int64_t my_src[2] = {0, 0}, my_ang = 0;
  bool a_new = true;
  auto ahead = [&]() {
    if (a_left > 0) {
      --a_left;
      if (a_new) {
        if (aw.tok - a_base >= 32) {  // the next 32 tokens
          a_base = aw.tok;
          const int tok = min(a_base + lane, p.tokens - 1);
          int b = 0, s = tok;
          if (p.cu == nullptr) place(tok, b, s);
          my_src[0] = b * st[0] + s * st[1];
          my_src[1] = b * st1[0] + s * st1[1];
          if (rotate) {
            // (of tokens of this stretch only: another warp reports its own)
            const bool mine = static_cast<unsigned>(tok) * div.d < x0 + count;
            int64_t at;
            bool live = true;
            if (p.positions != nullptr) {
              at = p.positions[tok];
              if (p.cu != nullptr) live = tok < p.cu[p.B];
            } else {
              live = place(tok, b, s);
              at = (MODE != kRowsPlain ? p.cache_seqlens[b] : 0) + static_cast<int64_t>(s);
            }
            my_ang = mine && live ? angle_row(at, p.max_pos, p.rot, p.status) : 0;
          }
        }
        const int h = aw.head + row;
        a_ptr[0] = src[0] + 2 * (shfl64(my_src[0], aw.tok - a_base) + h * st[2]) + 16 * lv.c0;
        if (kv) a_ptr[1] = src[1] + 2 * (shfl64(my_src[1], aw.tok - a_base) + h * st1[2]) + 16 * lv.c0;
        if (rotate)
          copy_angles(ring_u32 + a_slot + 2 * kGroupBytes, p.cos, p.sin, shfl64(my_ang, aw.tok - a_base), p.rot);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // (a head behind the last reads nothing; its address is not used)
        const int bytes = aw.head + (kv ? 0 : i * RPW) + row < heads ? 16 : 0;
        const uint8_t* from = kv ? a_ptr[i] : a_ptr[0] + i * (2 * RPW) * st[2];
        if (bytes == 0) from = src[0];
        cp_async16(ring_u32 + a_slot + i * kGroupBytes + at0, from, bytes);
        cp_async16(ring_u32 + a_slot + i * kGroupBytes + at0 + next, from + next, bytes);
      }
      a_ptr[0] += 2 * step * st[2];
      if (kv) a_ptr[1] += 2 * step * st1[2];
      const int tok = aw.tok;
      aw.next(heads, step);
      a_new = aw.tok != tok;
      a_slot = a_slot + kSlotBytes == kRing * kSlotBytes ? 0 : a_slot + kSlotBytes;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) ahead();

  float2 wt[8];
  if (norm) load_weights<BF16>(is_q ? p.wq : p.wk, p.w_fp32, lv, wt);
  LaneAngles ang;
  GroupWalk cw;
  cw.start(x0, div, step);
  int c_base = cw.tok - 32, c_slot = 0;
  uint8_t* c_out = nullptr;     // this lane's part of its output row (16-bit output)
  int64_t c_code = 0, c_scale = 0;  // or the offsets of its code row and of its scale
  int64_t my_out = 0, my_scale = 0;
  bool c_new = true, c_live = true, my_live = true;
  for (int n = 0; n < count; ++n) {
    cp_async_wait<kRing - 2>();
    __syncwarp();  // every lane's copies of this step are there, and the last step is used
    ahead();
    const uint8_t* slot = ring + c_slot;
    c_slot = c_slot + kSlotBytes == kRing * kSlotBytes ? 0 : c_slot + kSlotBytes;
    if (c_new) {
      if (cw.tok - c_base >= 32) {  // where the rows of the next 32 tokens go
        c_base = cw.tok;
        const int tok = min(c_base + lane, p.tokens - 1);
        int b, s;
        my_live = place(tok, b, s);
        if (!kv) {
          my_out = p.cu != nullptr ? tok * so[1] : b * so[0] + s * so[1];
        } else if (my_live) {
          CacheRow at = {0, 0};
          const unsigned bad = locate_row(p.c, b, p.cache_seqlens[b] + static_cast<int64_t>(s), &at);
          if (bad != 0u && static_cast<unsigned>(tok) * div.d < x0 + count) atomicOr(p.status, bad);
          my_live = bad == 0u;
          my_out = at.code;
          my_scale = at.scale;
        }
      }
      const int64_t out = shfl64(my_out, cw.tok - c_base);
      c_live = __shfl_sync(kFull, my_live, cw.tok - c_base);
      const int h = cw.head + row;
      if (!kv) {
        c_out = static_cast<uint8_t*>(is_q ? p.q_out : p.k_out) + 2 * (out + h * so[2]) + 16 * lv.c0;
      } else {
        c_code = out + h * p.c.st_head + 8 * lv.c0;
        c_scale = shfl64(my_scale, cw.tok - c_base) + static_cast<int64_t>(h) * p.c.rows;
      }
      if (rotate)
        read_angles(reinterpret_cast<const float*>(slot + 2 * kGroupBytes), p.rot, lv, p.interleaved, ang);
    }
    const int head = cw.head, tok = cw.tok;
    cw.next(heads, step);
    c_new = cw.tok != tok;

#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int first = kv ? head : head + i * RPW;
      if (first >= heads) break;  // warp-uniform: a token's last step may have one group
      const bool store = first + row < heads && c_live;
      uint32_t w[8];
      read_row(slot + i * kGroupBytes + at0, next, w);
      if (!(kv && i == 1) && (norm || rotate)) {
        float2 v[8];
        unpack16<BF16>(w, v);
        if (norm) {
          const float2 r = both(inv_rms<D>(v, p.eps));
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = mul2(mul2(v[e], r), wt[e]);
        }
        if (rotate && lv.turn) turn<false>(v, ang, p.interleaved);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = pack2<BF16>(v[e].x, v[e].y);
      }
      if (!kv) {
        if (store) store_row(c_out + i * (2 * RPW) * so[2], next, w);
      } else if constexpr (MODE != kRowsPlain) {
        // the 16-bit rows (the keys already rounded, as a call of its own would leave them).
        // (Append alone: 4 x 8192 tokens of 8 heads, d=128, bf16 to E4M3, 39 us, 79% of the copy
        // rate; 61K ragged tokens, d=64, fp16 to int8, 43.5 us, 82%; bound by HBM and the issue of
        // instructions together)
        const RowQuant rq = row_quant<BF16, MODE == kRowsE4M3>(row_max_bits<BF16, 8, LPR>(w), w);
        const uint2 lo = quantise8<BF16, MODE == kRowsE4M3>(w, rq);
        const uint2 hi = quantise8<BF16, MODE == kRowsE4M3>(w + 4, rq);
        if (store) {
          uint8_t* dst = static_cast<uint8_t*>(i == 0 ? p.c.k : p.c.v) + c_code;
          *reinterpret_cast<uint2*>(dst) = lo;
          *reinterpret_cast<uint2*>(dst + next / 2) = hi;
          if (j == 0) (i == 0 ? p.c.ks : p.c.vs)[c_scale] = rq.scale;
        }
      }
    }
    if (!kv) {
      c_out += 2 * step * so[2];
    } else {
      c_code += step * p.c.st_head;
      c_scale += static_cast<int64_t>(step) * p.c.rows;
    }
  }
}

// Lets the current device's copy of a kernel have `bytes` of dynamic shared memory; `ready` has
// a bit for each device where it may already.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (ready.load() >> dev & 1u)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready.fetch_or(1ull << dev);
  return e;
}

// Steps per warp for `most` warps, so that the two kinds' stretches (each a whole number of
// warps) fit them.
int steps_per_warp(int64_t steps, int64_t most) {
  most = std::max<int64_t>(most - 1, 1);
  return static_cast<int>((steps + most - 1) / most);
}

template <int D, bool BF16, int MODE, bool ROPE>
cudaError_t launch_rows_inst(RowsParams p, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 16), WARPS = kRowsThreads / 32;
  constexpr int STEP = 2 * RPW, STEP_K = MODE == kRowsPlain ? STEP : RPW;  // heads of a step
  p.div_q = fast_div((p.H + STEP - 1) / STEP);
  p.div_k = fast_div((p.Hkv + STEP_K - 1) / STEP_K);
  p.div_s = fast_div(std::max(p.S, 1));
  const int64_t nq = p.q != nullptr ? static_cast<int64_t>(p.tokens) * p.div_q.d : 0;
  const int64_t nk = static_cast<int64_t>(p.tokens) * p.div_k.d;
  p.per = steps_per_warp(nq + nk, static_cast<int64_t>(p.sm_count) * RowsCfg<ROPE>::kBlocksPerSm * WARPS);
  // Long stretches leave the end to the slowest SM: from 24 steps a warp on, several waves of 12
  // (4 x 4096 tokens, 32 + 8 heads, d=128: 35 steps in one wave 72 us, 12 in three 60.5; at 18
  // steps, d=64, two waves are no faster).  Not for the cache, where a warp first looks its
  // tokens' places up (4 x 8192 tokens: one wave and three are equally fast).
  if (MODE == kRowsPlain && p.per >= 24) p.per = 12;
  p.warps_q = static_cast<int>((nq + p.per - 1) / p.per);
  const int64_t warps = p.warps_q + (nk + p.per - 1) / p.per;
  const int blocks = static_cast<int>((warps + WARPS - 1) / WARPS);
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(rows_kernel<D, BF16, MODE, ROPE>, RowsCfg<ROPE>::kSmem, ready);
  if (e != cudaSuccess) return e;
  rows_kernel<D, BF16, MODE, ROPE><<<blocks, kRowsThreads, RowsCfg<ROPE>::kSmem, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ gradient
//
//   g = R^T dy,  n = x r,  r = rsqrt(mean(x^2) + eps)
//   dw = sum over tokens and heads of g n
//   dx = r (g w - n mean(g w n))
//
// x and dy are read once and dx written once, with the ring of the forward pass (a slot holds
// both).  A lane sums dw over its rows in registers, a block over its warps in shared memory,
// and a second small launch over the blocks.  The order of the sums depends on the sizes and
// the SM count alone, so the same call gives the same bits.
//   (Measured, 2 x 6001 tokens of 32 + 8 heads, d=128, bf16: 69-72 us with the second launch, 80-82%
//   of the copy rate (a call 76 us); without the ring, two groups per warp in registers, 97 us.  Several waves, each
//   block with its own partial sums, are slower.  59% of the issue slots; the second launch brought
//   to the SMs early, as the attention's join is, gains nothing: the registers are all taken.)
constexpr int kBwdThreads = 256;

constexpr int kBwdRing = 4;
constexpr int kBwdSlotBytes = 2 * kGroupBytes + 512;
constexpr int kBwdSmem = kBwdThreads / 32 * kBwdRing * kBwdSlotBytes;

template <int D, bool BF16>
__global__ void __launch_bounds__(kBwdThreads, kRowsBwdBlocksPerSm)
    rows_bwd_kernel(const RowsBwdParams p) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  constexpr int WARPS = kBwdThreads / 32;
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ float part[WARPS][D];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, j = lane % LPR;
  uint8_t* ring = ring_mem + warp * (kBwdRing * kBwdSlotBytes);
  const int gw0 = blockIdx.x * WARPS + warp;
  const int t = gw0 < p.warps_q ? 0 : 1;  // q or k
  const int gw = t == 0 ? gw0 : gw0 - p.warps_q;
  const int heads = p.heads[t];
  const FastDiv div = p.div[t];
  const unsigned groups = static_cast<unsigned>(p.tokens) * div.d;
  const unsigned x0 = min(static_cast<unsigned>(gw) * static_cast<unsigned>(p.per), groups);
  const int count = static_cast<int>(min(groups - x0, static_cast<unsigned>(p.per)));
  const LaneVecs lv = lane_vecs(j, p.rot);
  const bool rotate = p.cos != nullptr;
  const int64_t x_b = p.x_s[t][0], x_s = p.x_s[t][1], x_h = p.x_s[t][2];
  const int64_t g_b = p.dy_s[t][0], g_s = p.dy_s[t][1], g_h = p.dy_s[t][2];
  const int64_t d_b = p.dx_s[t][0], d_s = p.dx_s[t][1], d_h = p.dx_s[t][2];

  const int row = lane / LPR, at0 = row * (2 * D) + 16 * lv.c0, next = 16 * (lv.c1 - lv.c0);
  const uint32_t ring_u32 = smem_u32(ring);
  GroupWalk aw;
  aw.start(x0, div, RPW);
  int a_left = count, a_base = aw.tok - 32;
  uint32_t a_slot = 0;  // bytes
  const uint8_t *a_x = nullptr, *a_g = nullptr;
  int64_t my_ang = 0;
  bool a_new = true;
  auto ahead = [&]() {
    if (a_left > 0) {
      --a_left;
      if (a_new) {
        const int b = static_cast<int>(divide(aw.tok, p.div_s)), s = aw.tok - b * p.S;
        const int h = aw.head + row;
        a_x = static_cast<const uint8_t*>(p.x[t]) + 2 * (b * x_b + s * x_s + h * x_h) + 16 * lv.c0;
        a_g = static_cast<const uint8_t*>(p.dy[t]) + 2 * (b * g_b + s * g_s + h * g_h) + 16 * lv.c0;
        if (rotate) {
          if (aw.tok - a_base >= 32) {  // the angles of the next 32 tokens
            a_base = aw.tok;
            const int tok = min(a_base + lane, p.tokens - 1);
            const int pos = p.positions != nullptr ? p.positions[tok]
                                                   : tok - static_cast<int>(divide(tok, p.div_s)) * p.S;
            // (of tokens of this stretch only: another warp reports its own)
            my_ang = static_cast<unsigned>(tok) * div.d < x0 + count
                         ? angle_row(pos, p.max_pos, p.rot, p.status) : 0;
          }
          copy_angles(ring_u32 + a_slot + 2 * kGroupBytes, p.cos, p.sin, shfl64(my_ang, aw.tok - a_base), p.rot);
        }
      }
      const int bytes = aw.head + row < heads ? 16 : 0;
      const uint8_t* from = bytes != 0 ? a_g : static_cast<const uint8_t*>(p.dy[t]);
      cp_async16(ring_u32 + a_slot + at0, from, bytes);
      cp_async16(ring_u32 + a_slot + at0 + next, from + next, bytes);
      if (p.norm) {
        from = bytes != 0 ? a_x : static_cast<const uint8_t*>(p.x[t]);
        cp_async16(ring_u32 + a_slot + kGroupBytes + at0, from, bytes);
        cp_async16(ring_u32 + a_slot + kGroupBytes + at0 + next, from + next, bytes);
      }
      a_g += 2 * RPW * g_h;
      a_x += 2 * RPW * x_h;
      const int tok = aw.tok;
      aw.next(heads, RPW);
      a_new = aw.tok != tok;
      a_slot = a_slot + kBwdSlotBytes == kBwdRing * kBwdSlotBytes ? 0 : a_slot + kBwdSlotBytes;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kBwdRing - 1; ++i) ahead();

  float2 wt[8], acc[8];
  load_weights<BF16>(p.norm ? p.w[t] : nullptr, p.w_fp32, lv, wt);
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = both(0.f);
  LaneAngles ang;
  GroupWalk cw;
  cw.start(x0, div, RPW);
  int c_slot = 0;
  uint8_t* c_ptr = nullptr;
  bool c_new = true;
  for (int n = 0; n < count; ++n) {
    cp_async_wait<kBwdRing - 2>();
    __syncwarp();  // every lane's copies of this group are there, and the last group is used
    ahead();
    const uint8_t* slot = ring + c_slot;
    c_slot = c_slot + kBwdSlotBytes == kBwdRing * kBwdSlotBytes ? 0 : c_slot + kBwdSlotBytes;
    if (c_new) {
      const int b = static_cast<int>(divide(cw.tok, p.div_s)), s = cw.tok - b * p.S;
      c_ptr = static_cast<uint8_t*>(p.dx[t]) + 2 * (b * d_b + s * d_s + (cw.head + row) * d_h) + 16 * lv.c0;
      if (rotate)
        read_angles(reinterpret_cast<const float*>(slot + 2 * kGroupBytes), p.rot, lv, p.interleaved, ang);
    }
    const bool store = cw.head + row < heads;
    const int tok = cw.tok;
    cw.next(heads, RPW);
    c_new = cw.tok != tok;
    uint32_t w[8];
    float2 g[8];
    read_row(slot + at0, next, w);
    unpack16<BF16>(w, g);
    if (rotate && lv.turn) turn<true>(g, ang, p.interleaved);
    if (p.norm) {
      float2 v[8];
      read_row(slot + kGroupBytes + at0, next, w);
      unpack16<BF16>(w, v);
      // (heads behind the last are zeros here: with eps 0 their r would be infinite, and what they add
      // to dw a NaN)
      const float rms = inv_rms<D>(v, p.eps), r = store ? rms : 0.f;
      float2 dot = both(0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = mul2(v[e], both(r));
        acc[e] = fma2(g[e], v[e], acc[e]);
        g[e] = mul2(g[e], wt[e]);
        dot = fma2(g[e], v[e], dot);
      }
      const float mean = row_sum<LPR>(dot.x + dot.y) * (1.f / D);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = mul2(fma2(v[e], both(-mean), g[e]), both(r));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = pack2<BF16>(g[e].x, g[e].y);
    if (store) store_row(c_ptr, next, w);
    c_ptr += 2 * RPW * d_h;
  }

  // ---- dw of this block's warps, those of q and those of k
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float v = e % 2 == 0 ? acc[e / 2].x : acc[e / 2].y;
#pragma unroll
    for (int o = LPR; o < 32; o *= 2) v += __shfl_xor_sync(kFull, v, o);
    if (lane < LPR) part[warp][8 * (e < 8 ? lv.c0 : lv.c1) + e % 8] = v;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kBwdThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
      if ((blockIdx.x * WARPS + w < p.warps_q) == (c < D)) v += part[w][c % D];
    if (p.dw[c / D] != nullptr) p.ws[static_cast<int64_t>(blockIdx.x) * 2 * D + c] = v;
  }
}

// dw[t][col] = sum over the blocks of ws[block][t][col].  A block per 32 columns: each of its 32
// warps takes every 32nd partial, then the first adds up the warps' sums.
constexpr int kDwWarps = 32;

__global__ void __launch_bounds__(kDwWarps * 32) rows_bwd_dw_kernel(const RowsBwdParams p, int D) {
  __shared__ float part[kDwWarps][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int per = D / 32;
  const int t = blockIdx.x / per, col = blockIdx.x % per * 32 + lane;
  float* dw = p.dw[t];
  if (dw == nullptr) return;  // block-uniform
  float v = 0.f;
  for (int b = warp; b < p.blocks; b += kDwWarps) v += p.ws[(static_cast<int64_t>(b) * 2 + t) * D + col];
  part[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < kDwWarps; ++w) v += part[w][lane];
    dw[col] = v;
  }
}

template <int D, bool BF16>
cudaError_t launch_rows_bwd_inst(RowsBwdParams p, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 16);
  int64_t g[2];
  for (int t = 0; t < 2; ++t) {
    p.div[t] = fast_div((p.heads[t] + RPW - 1) / RPW);
    g[t] = static_cast<int64_t>(p.tokens) * p.div[t].d;
  }
  p.div_s = fast_div(p.S);
  p.per = steps_per_warp(g[0] + g[1], static_cast<int64_t>(p.blocks) * (kBwdThreads / 32));
  p.warps_q = static_cast<int>((g[0] + p.per - 1) / p.per);
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(rows_bwd_kernel<D, BF16>, kBwdSmem, ready);
  if (e != cudaSuccess) return e;
  rows_bwd_kernel<D, BF16><<<p.blocks, kBwdThreads, kBwdSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || (p.dw[0] == nullptr && p.dw[1] == nullptr)) return e;
  rows_bwd_dw_kernel<<<2 * (D / 32), kDwWarps * 32, 0, stream>>>(p, D);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ reading the cache back
//
// A warp takes a stretch of packed rows (tokens), each Hkv rows of K and of V; the places of 32
// tokens are looked up by the 32 lanes at once.  A row of D codes belongs to D / 16 lanes, 16
// bytes in and 32 bytes out each.  (Measured, of the copy rate: 4 x 8192 tokens of 8 heads, d=128,
// E4M3, 37 us, 83%; 16 ragged sequences, 61K tokens, d=64, int8, 53 us, 73%; half of the issue
// slots at that.)
constexpr int kReadThreads = 256;
constexpr int kReadBlocksPerSm = 6;

template <bool E4M3>
__device__ __forceinline__ void codes4(uint32_t w, float2& lo, float2& hi) {
  if constexpr (E4M3) {
    lo = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(w & 0xffffu, __NV_E4M3)));
    hi = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(w >> 16, __NV_E4M3)));
  } else {
    // byte ^ 0x80 = code + 128, as the low byte of 2^23 + 128 + code
    const uint32_t u = w ^ 0x80808080u;
    const float2 k = both(-8388736.f);  // -(2^23 + 128)
    lo = add2(make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)),
                          __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441))), k);
    hi = add2(make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)),
                          __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443))), k);
  }
}

template <int D, bool E4M3, bool BF16>
__global__ void __launch_bounds__(kReadThreads, kReadBlocksPerSm) read_quant_kernel(const ReadParams p) {
  constexpr int LPR = D / 16, RPW = 32 / LPR, UNROLL = 2;
  const int lane = threadIdx.x % 32, j = lane % LPR;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * (kReadThreads / 32) + threadIdx.x / 32;
  const int64_t first = gw * p.per;
  const int end = static_cast<int>(min(static_cast<int64_t>(p.total), first + p.per));
  const int rows = 2 * p.c.Hkv;  // K heads, then V heads
  int64_t my_code = 0, my_scale = 0;
  int my_state = 0, base = static_cast<int>(min(first, static_cast<int64_t>(end))) - 32;
  for (int tok = base + 32; tok < end; ++tok) {
    if (tok - base >= 32) {  // the next 32 tokens
      base = tok;
      const int r = min(base + lane, end - 1);
      const int b = find_sequence(p.cu, p.B, r);
      const int begin = p.cu[b];
      my_state = 0;  // outside every sequence: left as it is
      if (r >= begin && r < p.cu[p.B]) {
        CacheRow at = {0, 0};
        const int64_t pos = static_cast<int64_t>(r - begin) + (p.start != nullptr ? p.start[b] : 0);
        const unsigned bad = locate_row(p.c, b, pos, &at);
        if (bad != 0u) atomicOr(p.status, bad);
        my_state = bad != 0u ? 1 : 2;  // a row the cache does not hold reads as zeros
        my_code = at.code;
        my_scale = at.scale;
      }
    }
    const int state = __shfl_sync(kFull, my_state, tok - base);
    if (state == 0) continue;  // warp-uniform
    const int64_t code0 = shfl64(my_code, tok - base) + 16 * j, scale0 = shfl64(my_scale, tok - base);
    const int64_t out0 = static_cast<int64_t>(tok) * p.c.Hkv * D + 16 * j;
    for (int r0 = lane / LPR; r0 - lane / LPR < rows; r0 += UNROLL * RPW) {
      uint4 code[UNROLL];
      float scale[UNROLL];
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        const int x = r0 + i * RPW;
        const bool is_v = x >= p.c.Hkv;
        const int h = is_v ? x - p.c.Hkv : x;
        code[i] = make_uint4(0u, 0u, 0u, 0u);
        scale[i] = 0.f;
        if (x < rows && state == 2) {
          const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.c.v : p.c.k) + code0 + h * p.c.st_head;
          code[i] = *reinterpret_cast<const uint4*>(src);
          scale[i] = (is_v ? p.c.vs : p.c.ks)[scale0 + static_cast<int64_t>(h) * p.c.rows];
        }
      }
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        const int x = r0 + i * RPW;
        const bool is_v = x >= p.c.Hkv;
        const int h = is_v ? x - p.c.Hkv : x;
        const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 lo, hi;
          codes4<E4M3>(w[e], lo, hi);
          lo = mul2(lo, both(scale[i]));
          hi = mul2(hi, both(scale[i]));
          o[2 * e] = pack2<BF16>(lo.x, lo.y);
          o[2 * e + 1] = pack2<BF16>(hi.x, hi.y);
        }
        if (x >= rows) continue;
        uint16_t* dst = static_cast<uint16_t*>(is_v ? p.v_out : p.k_out) + out0 + h * D;
        if (p.wide) {
          store32(dst, o);
        } else {
          store_row(reinterpret_cast<uint8_t*>(dst), 16, o);
        }
      }
    }
  }
}

template <int D, bool E4M3, bool BF16>
cudaError_t launch_read_inst(ReadParams p, cudaStream_t stream) {
  constexpr int WARPS = kReadThreads / 32;
  const int64_t most = static_cast<int64_t>(p.sm_count) * kReadBlocksPerSm * WARPS;
  // few tokens a warp, so that the SMs even out over several waves, but at least 1.5 KB of codes
  // for each look-up of places (4 x 8192 tokens of 8 heads: d=128, one token 37 us, two 39, five
  // in one wave 44; d=64, one token 57 us, two 52.5, three 51)
  const int few = (1536 + 2 * p.c.Hkv * D - 1) / (2 * p.c.Hkv * D);
  p.per = static_cast<int>(std::min<int64_t>((p.total + most - 1) / most, few));
  const int64_t warps = (static_cast<int64_t>(p.total) + p.per - 1) / p.per;
  read_quant_kernel<D, E4M3, BF16>
      <<<static_cast<unsigned>((warps + WARPS - 1) / WARPS), kReadThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows(const RowsParams& p, int mode, bool bf16, int d, cudaStream_t stream) {
  if (p.tokens == 0) return cudaSuccess;
  const bool rope = p.q != nullptr;  // the append alone has none, and neither norm nor rotation
#define FA_ROWS_CASE(DD, BF, M, R) \
  if (d == DD && bf16 == BF && mode == M && rope == R) return launch_rows_inst<DD, BF, M, R>(p, stream);
#define FA_ROWS_CASES(M, R)          \
  FA_ROWS_CASE(64, false, M, R)      \
  FA_ROWS_CASE(64, true, M, R)       \
  FA_ROWS_CASE(128, false, M, R)     \
  FA_ROWS_CASE(128, true, M, R)
  FA_ROWS_CASES(kRowsPlain, true)
  FA_ROWS_CASES(kRowsE4M3, true)
  FA_ROWS_CASES(kRowsInt8, true)
  FA_ROWS_CASES(kRowsE4M3, false)
  FA_ROWS_CASES(kRowsInt8, false)
#undef FA_ROWS_CASES
#undef FA_ROWS_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_rows_bwd(const RowsBwdParams& p, bool bf16, int d, cudaStream_t stream) {
  if (d == 64) return bf16 ? launch_rows_bwd_inst<64, true>(p, stream) : launch_rows_bwd_inst<64, false>(p, stream);
  return bf16 ? launch_rows_bwd_inst<128, true>(p, stream) : launch_rows_bwd_inst<128, false>(p, stream);
}

cudaError_t launch_read_quant(const ReadParams& p, bool e4m3, bool bf16, int d, cudaStream_t stream) {
  if (p.total == 0) return cudaSuccess;
#define FA_READ_CASE(DD, E4, BF) \
  if (d == DD && e4m3 == E4 && bf16 == BF) return launch_read_inst<DD, E4, BF>(p, stream);
  FA_READ_CASE(64, false, false)
  FA_READ_CASE(64, false, true)
  FA_READ_CASE(64, true, false)
  FA_READ_CASE(64, true, true)
  FA_READ_CASE(128, false, false)
  FA_READ_CASE(128, false, true)
  FA_READ_CASE(128, true, false)
  FA_READ_CASE(128, true, true)
#undef FA_READ_CASE
  return cudaErrorInvalidValue;
}

}  // namespace fa
