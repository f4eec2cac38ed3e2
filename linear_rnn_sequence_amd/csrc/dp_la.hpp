// dp_la.hpp -- linear attention with a decay per head on gfx950: the chunked
// form for prompts (one length or packed), its gradient, and the shared pieces.
//
// Per value head, with a state S [dk, dv] and a log decay l_t (natural log):
//
//   S_t = e^{l_t} S_{t-1} + k_t v_t^T,     o_t = S_t^T q_t
//
// Chunk form.  With G_i the inclusive cumulative log decay inside a chunk of C
// tokens and S the state at its start,
//
//   o_i = e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j
//   S'  = e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
//
// Gradient.  With D the gradient on the state at the chunk's end,
//
//   dq_i = e^{G_i} S do_i          + sum_{j <= i} e^{G_i - G_j} (do_i . v_j) k_j
//   dk_j = e^{G_C - G_j} D v_j     + sum_{i >= j} e^{G_i - G_j} (v_j . do_i) q_i
//   dv_j = e^{G_C - G_j} D^T k_j   + sum_{i >= j} e^{G_i - G_j} (k_j . q_i) do_i
//   D'   = e^{G_C} D + sum_i e^{G_i} q_i do_i^T      (gradient on the chunk's start state)
//
// so forward and gradient are one walk over chunks with other operands: rows a,
// columns b, values c, a state X, forwards (mask j <= i) or backwards (mask
// j >= i).  LaWalk below is that walk.
//
// The gradient of the log decay, dl_t = <D_t, e^{l_t} S_{t-1}>, needs no division by the
// decay.  Take apart q_i . dq_i = a_i + r_i + o_i and k_j . dk_j = b_j + c_j + o_j into the
// state's part, the scores' part of other tokens and that of the token itself (which is
// the same for both and cancels: left in, it leaves its rounding in the gradient of short
// or quickly forgetting sequences, where it is the largest term).  Pairs (i, j) of one
// chunk with i >= t > j give the sums of r - c from t to the chunk's end, or those of c - r
// before t, the same number: the shorter sum is taken (none at a chunk's first token, so
// that the first one of a sequence without an initial state gets exactly 0); everything
// that crosses the chunk's borders gives F - sum_{i < t} a_i + sum_{j < t} b_j, where F =
// <S, D> at the segment's start and the sums run from there.  (Summing q . dq - k . dk alone, from the segment's end, is the
// same number, but its rounding grows with the segment where the true value is as small
// as one token's terms; a and b shrink with the decay and take their rounding along.)
//
// Split over the sequence.  A sequence is cut into segments of whole chunks.
// With one segment a single launch walks it.  With several, dp_la_states_kernel
// sums each segment's own contribution to the state (it reads two of the
// tensors), dp_la_scan_kernel runs the decayed prefix sum over the segments in
// fp32, and the walks start from the result (where their states are few or small they
// add them up themselves: they come from L2, and a launch is saved).  The first segment starts from the
// initial state and the last ends with the final one, so a sequence of one segment
// takes no part in either.
//
// Precision.  States, scores and sums are fp32; cumulative log decays are fp64
// (a difference of two of them is an exponent, and a chunk with strong decays
// has large sums).  On the bf16 path the inputs are MFMA operands as they are.
// Computed operands (scores, the state where it is read, the weighted values that
// build it) are split into three bf16 terms, x = h + m + l with h = bf16(x), m = bf16(x - h),
// l = bf16(x - h - m), one MFMA per term: 24 bits, so that the only rounding to fewer is
// the result's, and a result's bits do not depend on which others are asked for.  Two
// terms (17 bits) are quicker (B = 4, H = 16, L = 4096, d = 128: forward 114 against 122
// us, gradient 355 against 383, without the decays' gradient 280 against 330) and leave a
// bf16 result's error against fp64 where it is, 1.66e-3 of its size; but 0.2% of the
// elements then round otherwise than the fp32 value (of a forward at that size; three terms:
// 0.02%, as many as another order of the sums), and the fp32 results (states, decays'
// gradient) are off by 1e-6 to 7e-6.  The fp32 path runs fp32 MFMA.
#pragma once

#include <atomic>

#include "dp_device.hpp"

namespace dp {

typedef float f32x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ operands
//
// A 32-deep product step over the index set a 16x16 accumulator pair holds:
// lane group g = lane >> 4 covers {4g + e} and {16 + 4g + e}, e = 0..3 (see the
// fp16 helpers in dp_device.hpp).  row(): 8 values of one row, tr(): 8 rows of
// one column, split(): the values of two accumulator tiles as operands.
//
// They read LDS tiles [rows][pitch] with per-lane offsets that are set up once:
// row_lane for row (lane & 15) of a 16-row tile, moved by row_step to the ks-th 32
// columns, and tr_lane, moved by tr_step to the m-th 16 columns.
//
// bf16 tiles are unpadded and swizzled: the 16-byte block c of row r sits at block
// c ^ swz(r).  A row read takes one block of 16 rows at a time, a transposed read two
// adjacent blocks of 8 rows; swz gives the 16 rows of a tile different blocks and 8
// neighbouring rows different pairs of blocks, so both touch every bank once.  (Padded
// rows served one of the two: 43% of the walk's LDS cycles were conflicts.)  Tiles that
// are only read by rows (a and the scores) are "packed": in every 32 columns the 8 of
// lane group g stand together, one 16-byte read.  (Two 8-byte reads are merged by the
// compiler across row tiles and then moved into place, one move a register.)  Such a read
// takes 16 lanes at a time, half of them of each of two lane groups (rows 0..3 and 12..15
// of one, 4..11 of the next): swzp gives these different blocks.
// fp32 tiles are padded by 16 bytes, which serves both of their reads.
template <typename T>
struct LaOp;

template <>
struct LaOp<bf16_t> {
  using frag_t = bf16x8_t;
  static constexpr int C = 64;  // tokens per chunk
  static constexpr int NS = 3;  // terms of a computed operand
  static constexpr int pitch(int d) { return d < 32 ? 32 : d; }
  // block 0 of row r, in elements, for rows of `ld` elements (16 / CH rows span the banks)
  __device__ __forceinline__ static int swz(int r, int ld) {
    const int ch = ld / 8, h = (r & 15) * ch / 16;
    return 8 * (2 * (h % (ch / 2)) + h / (ch / 2));
  }
  // the same of a packed tile
  __device__ __forceinline__ static int swzp(int r, int ld) {
    const int ch = ld / 8, h = (r & 15) * ch / 16;
    return 8 * (ch == 4 ? ((h & 1) << 1) ^ (h >> 1) * 3 : h);
  }
  __device__ __forceinline__ static int at(int r, int c8, int ld) { return r * ld + ((8 * c8) ^ swz(r, ld)); }
  // 16 bytes, block c8 of row r, into a plain or a packed tile
  __device__ __forceinline__ static void put16(bf16_t* s, int r, int c8, int ld, const u32x4_t& v) {
    st16(s + at(r, c8, ld), v);
  }
  __device__ __forceinline__ static void put16_packed(bf16_t* s, int r, int c8, int ld, const u32x4_t& v) {
    // columns 8 c8 .. + 3 are group 2 (c8 & 1)'s, the next four the next group's; half (c8 >> 1) & 1 of theirs
    const int o = r * ld + ((8 * ((c8 & ~3) + 2 * (c8 & 1))) ^ swzp(r, ld)) + 4 * ((c8 >> 1) & 1);
    *reinterpret_cast<u32x2_t*>(s + o) = u32x2_t{v[0], v[1]};
    *reinterpret_cast<u32x2_t*>(s + (o ^ 8)) = u32x2_t{v[2], v[3]};
  }
  __device__ __forceinline__ static int row_lane(int ld) {  // plain
    const int l = threadIdx.x & 63, n = l & 15, g = l >> 4;
    return n * ld + ((8 * (g >> 1)) ^ swz(n, ld)) + 4 * (g & 1);
  }
  __device__ __forceinline__ static int prow_lane(int ld) {  // packed
    const int l = threadIdx.x & 63, n = l & 15, g = l >> 4;
    return n * ld + ((8 * g) ^ swzp(n, ld));
  }
  __device__ __forceinline__ static int row_step(int off, int ks) { return off ^ (32 * ks); }
  // four columns of tile ct for lane group g in a packed tile: prow_lane moved
  __device__ __forceinline__ static int pcol_step(int off, int ct) { return (off ^ (32 * (ct >> 1))) + 4 * (ct & 1); }
  __device__ __forceinline__ static frag_t row(const bf16_t* p, int off) {
    const s16x4_t a = *reinterpret_cast<const s16x4_t*>(p + off), b = *reinterpret_cast<const s16x4_t*>(p + (off ^ 16));
    return __builtin_bit_cast(frag_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  __device__ __forceinline__ static frag_t prow(const bf16_t* p, int off) {
    return __builtin_bit_cast(frag_t, ld16(p + off));
  }
  __device__ __forceinline__ static int tr_lane(int ld) {
    const int l = threadIdx.x & 63, i = l & 15, g = l >> 4, r = 4 * g + (i >> 2);
    return r * ld + ((8 * ((i & 3) >> 1)) ^ swz(r, ld)) + 4 * (i & 1);
  }
  __device__ __forceinline__ static int tr_step(int off, int m) { return off ^ (16 * m); }
  __device__ __forceinline__ static frag_t tr(const bf16_t* p, int ld) {
    const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p);
    const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 16 * ld));
    return __builtin_bit_cast(frag_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  // four consecutive values as loaded, and as fp32
  __device__ __forceinline__ static u32x4_t load4(const bf16_t* p) {
    const u32x2_t u = *reinterpret_cast<const u32x2_t*>(p);
    return u32x4_t{u[0], u[1], 0, 0};
  }
  __device__ __forceinline__ static f32x4_t widen4(const u32x4_t& u) {
    return f32x4_t{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u), __uint_as_float(u[1] << 16),
                   __uint_as_float(u[1] & 0xffff0000u)};
  }
  __device__ __forceinline__ static f32x8_t widen(const frag_t& f) {
    const u32x4_t u = __builtin_bit_cast(u32x4_t, f);
    f32x8_t x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    return x;
  }
  // two values rounded to one register of bf16, and its halves as fp32 again: one
  // conversion a pair (a vector conversion there and back converts every value twice)
  __device__ __forceinline__ static uint32_t cvt2(float a, float b) {
    const f32x2_t x = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2_t));
  }
  template <int NS>
  __device__ __forceinline__ static void split(f32x8_t x, frag_t* out) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      u32x4_t u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] = cvt2(x[2 * i], x[2 * i + 1]);
        if (s + 1 < NS) {
          x[2 * i] -= __uint_as_float(u[i] << 16);
          x[2 * i + 1] -= __uint_as_float(u[i] & 0xffff0000u);
        }
      }
      out[s] = __builtin_bit_cast(frag_t, u);
    }
  }
  __device__ __forceinline__ static f32x4_t mma(const frag_t& a, const frag_t& b, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // four consecutive values as NS terms, `plane` elements apart
  template <int NS>
  __device__ __forceinline__ static void put(bf16_t* p, int plane, f32x4_t x) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      u32x2_t u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        u[i] = cvt2(x[2 * i], x[2 * i + 1]);
        if (s + 1 < NS) {
          x[2 * i] -= __uint_as_float(u[i] << 16);
          x[2 * i + 1] -= __uint_as_float(u[i] & 0xffff0000u);
        }
      }
      *reinterpret_cast<u32x2_t*>(p + s * plane) = u;
    }
  }
};

template <>
struct LaOp<float> {
  using frag_t = f32x8_t;
  static constexpr int C = 32;  // half the scores per token: fp32 MFMA is the bound
  static constexpr int NS = 1;
  static constexpr int pitch(int d) { return (d < 32 ? 32 : d) + 4; }
  __device__ __forceinline__ static int at(int r, int c4, int ld) { return r * ld + 4 * c4; }
  __device__ __forceinline__ static void put16(float* s, int r, int c4, int ld, const u32x4_t& v) { st16(s + at(r, c4, ld), v); }
  __device__ __forceinline__ static void put16_packed(float* s, int r, int c4, int ld, const u32x4_t& v) {
    st16(s + at(r, c4, ld), v);
  }
  __device__ __forceinline__ static int row_lane(int ld) {
    const int l = threadIdx.x & 63;
    return (l & 15) * ld + 4 * (l >> 4);
  }
  __device__ __forceinline__ static int prow_lane(int ld) { return row_lane(ld); }
  __device__ __forceinline__ static int row_step(int off, int ks) { return off + 32 * ks; }
  __device__ __forceinline__ static int pcol_step(int off, int ct) { return off + 16 * ct; }
  __device__ __forceinline__ static frag_t row(const float* p, int off) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p + off), b = *reinterpret_cast<const f32x4_t*>(p + off + 16);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __device__ __forceinline__ static frag_t prow(const float* p, int off) { return row(p, off); }
  __device__ __forceinline__ static int tr_lane(int ld) {
    const int l = threadIdx.x & 63;
    return 4 * (l >> 4) * ld + (l & 15);
  }
  __device__ __forceinline__ static int tr_step(int off, int m) { return off + 16 * m; }
  __device__ __forceinline__ static frag_t tr(const float* p, int ld) {
    frag_t f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = p[e * ld];
      f[4 + e] = p[(16 + e) * ld];
    }
    return f;
  }
  __device__ __forceinline__ static u32x4_t load4(const float* p) { return ld16(p); }
  __device__ __forceinline__ static f32x4_t widen4(const u32x4_t& u) { return __builtin_bit_cast(f32x4_t, u); }
  __device__ __forceinline__ static f32x8_t widen(const frag_t& f) { return f; }
  template <int NS>
  __device__ __forceinline__ static void split(const f32x8_t& x, frag_t* out) {
    out[0] = x;
  }
  __device__ __forceinline__ static f32x4_t mma(const frag_t& a, const frag_t& b, f32x4_t c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  template <int NS>
  __device__ __forceinline__ static void put(float* p, int, const f32x4_t& x) {
    *reinterpret_cast<f32x4_t*>(p) = x;
  }
};

__device__ __forceinline__ f32x8_t la_cat(const f32x4_t& a, const f32x4_t& b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Log decays below this (-inf, a reset, among them) are taken as this: e^-1000
// is zero in fp32, and sums of 64 of them stay finite.  NaN passes.
constexpr float kLaMinLog = -1000.f;
constexpr double kLog2E = 1.4426950408889634;

// Inclusive prefix sum over a wavefront, by DPP.
__device__ __forceinline__ double la_scan64(double x) {
  auto step = [](double v, auto ctrl, auto rows) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    return v + __builtin_bit_cast(double, ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
  };
  x = step(x, std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});  // row_shr:1
  x = step(x, std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});  // row_shr:2
  x = step(x, std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});  // row_shr:4
  x = step(x, std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});  // row_shr:8
  x = step(x, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // row_bcast:15
  x = step(x, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});  // row_bcast:31
  return x;
}

// ------------------------------------------------------------ geometry

// Sequences and their segments.  One length: sequence d is rows d L .. d L + L - 1,
// cut into `nps` segments.  Packed (cu given): rows cu[d] .. cu[d+1] - 1, its first
// segment tab[d] (dp_la_table_kernel; tab[nseq] segments in all, tab[nseq + 1] =
// the first row behind the last sequence).  Every sequence has one segment at
// least, so that an empty one still passes its state on.  Packed segments differ in
// length; `order` lists them with the whole ones first and the shorter halves last, and
// the workgroups take them in that order, so that the last to start are short.
struct LaGeo {
  const int* cu;
  const int* tab;
  const int* order;
  int nseq, L, seg, nps, nwork;  // nwork: segments (packed: an upper bound)
};

struct LaSeg {
  int d, index, count;  // sequence; which of its segments, and of how many
  int first, last;
  long long row;       // first row
  int len;             // tokens
};

__device__ __forceinline__ bool la_segment(const LaGeo& g, int s, LaSeg& o) {
  int i, n, d, count;
  long long base;
  if (g.cu == nullptr) {
    count = g.nps;
    d = s / g.nps;
    i = s - d * g.nps;
    n = g.L;
    base = (long long)d * g.L;
  } else {
    if (s >= g.tab[g.nseq]) return false;
    int lo = 0, hi = g.nseq;  // tab[lo] <= s < tab[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g.tab[mid] <= s) lo = mid;
      else hi = mid;
    }
    d = lo;
    i = s - g.tab[d];
    count = g.tab[d + 1] - g.tab[d];
    const bool ok = g.tab[g.nseq + 1] >= 0;  // offsets that break their order: every sequence is empty
    base = ok ? g.cu[d] : 0;
    n = ok ? g.cu[d + 1] - g.cu[d] : 0;
  }
  const int t0 = i * g.seg;
  o.d = d;
  o.index = i;
  o.count = count;
  o.first = i == 0;
  o.last = n - t0 <= g.seg;
  o.row = base + t0;
  o.len = n - t0 < g.seg ? n - t0 : g.seg;
  return true;
}

// Segment and head of workgroup b.  Workgroups go round the 8 XCDs in turn, each with an
// L2 of its own: the value heads of one query / key head follow each other on one XCD,
// so that their common rows come from HBM once (groups past the last whole eight stay in
// plain order).
__device__ __forceinline__ void la_block(int b, const LaGeo& g, int H, int Hk, int* s, int* h) {
  if (Hk == H) {
    *s = b / H;
    *h = b - *s * H;
    return;
  }
  const int r = H / Hk, whole = g.nwork * Hk / 8 * 8;
  int grp, u;  // (segment, key head), and which of its value heads
  if (b < whole * r) {
    const int j = b >> 3;
    grp = j / r * 8 + (b & 7);
    u = j - j / r * r;
  } else {
    grp = b / r;
    u = b - grp * r;
  }
  *s = grp / Hk;
  *h = (grp - *s * Hk) * r + u;
}

// The segment a workgroup's place in the order stands for; false behind the last.
__device__ __forceinline__ bool la_in_order(const LaGeo& g, int* s) {
  if (g.cu == nullptr) return true;
  if (*s >= g.tab[g.nseq]) return false;
  *s = g.order[*s];
  return true;
}

// ------------------------------------------------------------ shared steps

// One tensor of a walk: rows [row][nh][D], head h of H reads h * nh / H.
struct LaTen {
  const void* p;
  int nh;
};

// The decays of one chunk in LDS: G (fp64, log2 units), e^{G_i}, e^{G_C - G_i} and
// e^{G_C}; C * 16 + 16 bytes.
template <int C>
struct LaDecays {
  double* G;
  float *E, *W, *tot;
  __device__ __forceinline__ explicit LaDecays(char* p)
      : G(reinterpret_cast<double*>(p)),
        E(reinterpret_cast<float*>(p + C * 8)),
        W(reinterpret_cast<float*>(p + C * 12)),
        tot(reinterpret_cast<float*>(p + C * 16)) {}
};

// Written by one wavefront.  `v` is lane i's token's log decay (0 behind the end).
template <int C>
__device__ __forceinline__ void la_decays(float v, const LaDecays<C>& d) {
  const int l = threadIdx.x & 63;
  v = v < kLaMinLog ? kLaMinLog : v;
  const double G = la_scan64((double)v * kLog2E);
  const uint64_t u = __builtin_bit_cast(uint64_t, G);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, C - 1);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), C - 1);
  const double tot = __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
  if (l < C) {
    d.G[l] = G;
    d.E[l] = __builtin_amdgcn_exp2f((float)G);
    d.W[l] = __builtin_amdgcn_exp2f((float)(tot - G));
  }
  if (l == 0) *d.tot = __builtin_amdgcn_exp2f((float)tot);
}

// A walk's decays, four chunks at a time: wavefront w takes chunk w of a group, from
// log decays loaded while the group before was worked on.  (One chunk at a time kept the
// other three wavefronts waiting for the scan in every chunk.)
template <int C>
struct LaDecayRing {
  static constexpr int BYTES = C * 16 + 16;  // of one chunk; four in LDS
  char* lds;
  const float* ld;
  long long row0;
  int len, nc, rev, head, h, H;
  float v;
  // chunk of the walk's step `it`
  __device__ __forceinline__ int chunk(int it) const { return rev ? nc - 1 - it : it; }
  __device__ __forceinline__ LaDecays<C> at(int it) const { return LaDecays<C>(lds + (it & 3) * BYTES); }
  __device__ __forceinline__ void load(int it0, int wave) {
    v = 0.f;
    if (ld == nullptr || it0 + wave >= nc) return;
    const int t = chunk(it0 + wave) * C + (threadIdx.x & 63);
    if ((threadIdx.x & 63) < C && t < len) v = head ? ld[h] : ld[(row0 + t) * H + h];
  }
  // before step `it` (a multiple of four): everybody is past step it - 1's last read
  __device__ __forceinline__ void fill(int it, int wave) {
    la_decays<C>(v, at(wave));
    load(it + 4, wave);
  }
};

// 16-byte vectors of a chunk's rows of width D, per thread of a block of NT: vector i
// is row tok + i NT / VPR, block c.  Rows behind the chunk's n read the last row instead
// and are written to LDS as zeros: loads without a branch, since the compiler ends a
// predicated group of loads with a wait before the next one's addresses, which left the
// memory latency of each tensor exposed in turn.  (32-bit offsets: a chunk's rows span
// less than 2 GB, a row less than 2^24 elements.)
template <typename T, int D, int C, int NT>
struct LaRows {
  static constexpr int VE = 16 / (int)sizeof(T);
  static constexpr int VPR = D / VE;  // vectors per row
  static constexpr int N = (C * VPR + NT - 1) / NT;
  static constexpr int STEP = NT / VPR;  // rows between a thread's vectors
  static_assert(NT % VPR == 0, "rows");
  u32x4_t r[N];

  __device__ __forceinline__ void load(const LaTen& t, long long row, int n, int h, int H) {
    const int rs = t.nh * D, tok = (int)threadIdx.x / VPR, c = (int)threadIdx.x % VPR;
    const int hd = t.nh == H ? h : h * t.nh / H;
    const char* base = static_cast<const char*>(t.p) + (row * rs + (long long)hd * D) * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int rr = tok + i * STEP < n ? tok + i * STEP : n - 1;
      r[i] = ld16(base + (__umul24((unsigned)rr, (unsigned)rs) + (unsigned)(c * VE)) * (unsigned)sizeof(T));
    }
  }
  template <bool PACKED>
  __device__ __forceinline__ void put(T* s, int ld, int n) {
    const int tok = (int)threadIdx.x / VPR, c = (int)threadIdx.x % VPR;
    if (n < C) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (tok + i * STEP >= n) r[i] = u32x4_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (C % STEP == 0 || tok + i * STEP < C) {
        if constexpr (PACKED) LaOp<T>::put16_packed(s, tok + i * STEP, c, ld, r[i]);
        else LaOp<T>::put16(s, tok + i * STEP, c, ld, r[i]);
      }
  }
};

// The blocks of a tile's rows past a real width of 16 (padded to 32) as zeros.
template <typename T, int C, bool PACKED>
__device__ __forceinline__ void la_zero_pad(T* s, int ld) {
  constexpr int VE = 16 / (int)sizeof(T), B = 16 / VE;
  const u32x4_t z = {0, 0, 0, 0};
  for (int i = threadIdx.x; i < C * B; i += blockDim.x) {
    if constexpr (PACKED) LaOp<T>::put16_packed(s, i / B, B + i % B, ld, z);
    else LaOp<T>::put16(s, i / B, B + i % B, ld, z);
  }
}

// Keeps a lane offset's derived addresses inside the chunk loop: hoisted out of it they
// would hold a register each across everything.
__device__ __forceinline__ int la_here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Wavefronts of a workgroup, and those of them that hold columns of a state with dv of
// them: all share the loads and the scores, the columns of a narrow head belong to the
// first dv / 16.  A chunk is a chain of short steps, so its time on an idle CU is issue
// and latency of one wavefront: with eight, each holds half as much.  The forward takes
// eight where dv = 128 fills them (B = 16, H = 16, L = 1024, d = 128: 87 us with one
// workgroup a CU against 114 with two of four wavefronts and twice the segments; 512
// tokens of 8 heads 17.6 against 20.7).  The gradient keeps two workgroups of four, whose
// reads of the shared rows are fewer (B = 4, H = 16, d = 128: L = 2048 190 against 203
// us, L = 4096 395 against 386; d = 64, L = 4096 180 against 230; fp32 406 against 459).
constexpr int la_fwd_waves(int dv) { return dv == 128 ? 8 : 4; }
constexpr int kLaBwdWaves = 4;
constexpr int la_waves(int dv, int nw) { return dv / 16 < nw ? dv / 16 : nw; }

// X <- tot X + sum over the chunk's tokens of (w_j c_j) b_j, this wavefront's CT column
// tiles: A = b transposed, B = the weighted values split into terms.  The decay stays in
// a factor (the state is scale x) and the weights are divided by it, so that a chunk
// multiplies 64 values a lane only where the factor has left [2^-40, 2^40] (or is NaN).
template <typename T, int DKP, int CT, int LB, int LC>
__device__ __forceinline__ void la_update(f32x4_t (&x)[DKP / 16][CT], float& scale, const T* sB, const T* sC,
                                          const float* sW, float tot, int col0) {
  using Op = LaOp<T>;
  constexpr int C = Op::C, NS = Op::NS;
  const int g = (threadIdx.x >> 4) & 3;
  scale = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(scale * tot)));
  if (!(scale >= 0x1p-40f && scale <= 0x1p40f)) {
#pragma unroll
    for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
      for (int t = 0; t < CT; ++t) x[m][t] *= scale;
    scale = 1.f;
  }
  const float inv = __builtin_amdgcn_rcpf(scale);
  const int ob = la_here(Op::tr_lane(LB)), oc = la_here(Op::tr_lane(LC));
#pragma unroll
  for (int ks = 0; ks < C / 32; ++ks) {
    const f32x4_t w0 = *reinterpret_cast<const f32x4_t*>(sW + 32 * ks + 4 * g);
    const f32x4_t w1 = *reinterpret_cast<const f32x4_t*>(sW + 32 * ks + 16 + 4 * g);
    const f32x8_t w = la_cat(w0, w1) * inv;
    typename Op::frag_t vf[CT][NS];
#pragma unroll
    for (int t = 0; t < CT; ++t)
      Op::template split<NS>(Op::widen(Op::tr(sC + 32 * ks * LC + Op::tr_step(oc, col0 / 16 + t), LC)) * w, vf[t]);
    // a product's terms follow each other 2 CT products apart, not back to back
#pragma unroll
    for (int m = 0; m < DKP / 16; m += 2) {
      const typename Op::frag_t a[2] = {Op::tr(sB + 32 * ks * LB + Op::tr_step(ob, m), LB),
                                        Op::tr(sB + 32 * ks * LB + Op::tr_step(ob, m + 1), LB)};
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < CT; ++t) x[m + u][t] = Op::mma(a[u], vf[t][s], x[m + u][t]);
    }
  }
}

// A state tile set from / to memory: X[row][col] at p[row * DV + col], or with
// tr the transpose, p[col * DK + row].  Rows past DK (padding of dk = 16) are 0.
// One branch around all of the loads: with one per tile the compiler waits for each
// group of them in turn.
template <int DK, int DV, int DKP, int CT>
__device__ __forceinline__ void la_state_load(f32x4_t (&x)[DKP / 16][CT], const float* p, bool tr, int col0) {
  const int l = threadIdx.x & 63, g = l >> 4, n = l & 15;
#pragma unroll
  for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
    for (int t = 0; t < CT; ++t) x[m][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (p == nullptr) return;
  if (tr) {
    const float* q = p + (col0 + n) * DK + 4 * g;
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int t = 0; t < CT; ++t) x[m][t] = *reinterpret_cast<const f32x4_t*>(q + 16 * t * DK + 16 * m);
  } else {
    const float* q = p + 4 * g * DV + col0 + n;
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[m][t][e] = q[(16 * m + e) * DV + 16 * t];
  }
}
template <int DK, int DV, int DKP, int CT>
__device__ __forceinline__ void la_state_store(const f32x4_t (&x)[DKP / 16][CT], float scale, float* p, bool tr, int col0) {
  const int l = threadIdx.x & 63, g = l >> 4, n = l & 15;
  if (tr) {
    float* q = p + (col0 + n) * DK + 4 * g;
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int t = 0; t < CT; ++t) *reinterpret_cast<f32x4_t*>(q + 16 * t * DK + 16 * m) = x[m][t] * scale;
  } else {
    float* q = p + 4 * g * DV + col0 + n;
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) q[(16 * m + e) * DV + 16 * t] = x[m][t][e] * scale;
  }
}

// ------------------------------------------------------------ the walk

// One row's product with its result tiles, summed over the lane groups.
template <typename Op, int CT>
__device__ __forceinline__ float la_dot(const u32x4_t (&q)[CT], const f32x4_t (&a)[CT]) {
  float s = 0.f;
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const f32x4_t w = Op::widen4(q[t]);
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fmaf(w[e], a[t][e], s);
  }
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  return s;
}

struct LaWalkArgs {
  LaTen a, b, c;      // rows, columns [.., DK] and values [.., DV]
  LaTen dot;          // rows [.., DV] whose products with the result rows are wanted, or null
  float2* dots;       // [row][H]: with the state's part of the result row, with the scores' part (`apart`: i != j)
  int apart;          // each token's own score goes into its row after the products with `dot`
  void* r;            // result [row][H][DV], T or fp32
  const float* ld;    // log decays, or null
  int ld_head;        // one per head ([H]) instead of [row][H]
  const float* x0;    // the state the walk starts from, or null (zero)
  const float *loc, *dec;  // nloc earlier segments' own contributions and decays to add up from it,
  int nloc, loc_step;      // loc_step segments apart (backwards: -1)
  float* x1;          // where its last state goes, or null
  int rev, tr, r_f32, H;
};

template <typename T, int DK, int DV, int NW>
struct LaWalk {
  using Op = LaOp<T>;
  using frag_t = typename Op::frag_t;
  static constexpr int C = Op::C, R = C / 16, NS = Op::NS;
  static constexpr int DKP = DK < 32 ? 32 : DK;
  static constexpr int WV = la_waves(DV, NW);  // wavefronts that hold columns
  static constexpr int CT = DV / 16 / WV;      // column tiles of each
  static constexpr int NT = 64 * NW;
  static constexpr int LA = Op::pitch(DK), LC = Op::pitch(DV), LP = Op::pitch(C);
  static constexpr int oA = 0;
  static constexpr int oB = oA + C * LA * (int)sizeof(T);
  static constexpr int oC = oB + C * LA * (int)sizeof(T);
  static constexpr int oP = oC + C * LC * (int)sizeof(T);
  static constexpr int oG = oP + NS * C * LP * (int)sizeof(T);
  static constexpr int oOwn = oG + 4 * LaDecayRing<C>::BYTES;
  static constexpr int oDot = oOwn + C * 4;
  static constexpr int LDS = oOwn, LDS_DOTS = oDot + WV * C * 8;  // without and with `apart` and `dots`

  __device__ __forceinline__ static void run(const LaWalkArgs& p, char* lds, long long row0, int len, int h) {
    T* sA = reinterpret_cast<T*>(lds + oA);
    T* sB = reinterpret_cast<T*>(lds + oB);
    T* sC = reinterpret_cast<T*>(lds + oC);
    T* sP = reinterpret_cast<T*>(lds + oP);
    float* sOwn = reinterpret_cast<float*>(lds + oOwn);
    float2* sDot = reinterpret_cast<float2*>(lds + oDot);
    const int tid = threadIdx.x, l = tid & 63, g = l >> 4, n = l & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool active = wave < WV;
    const int col0 = active ? wave * 16 * CT : 0;
    const bool rev = p.rev != 0;

    if constexpr (DK < 32) {  // the padded columns of rows a and b stay zero
      la_zero_pad<T, C, true>(sA, LA);
      la_zero_pad<T, C, false>(sB, LA);
    }
    const int ra_lane = Op::prow_lane(LA), rb_lane = Op::row_lane(LA), rp_lane = Op::prow_lane(LP);
    f32x4_t x[DKP / 16][CT];
    if (active) la_state_load<DK, DV, DKP, CT>(x, p.x0, p.tr != 0, col0);
    if (active) {
      // two segments' values in flight at a time
      for (int j = 0; j < p.nloc; j += 2) {
        const bool two = j + 1 < p.nloc;
        f32x4_t y0[DKP / 16][CT], y1[DKP / 16][CT];
        const long long o0 = (long long)j * p.loc_step * p.H, o1 = (long long)(two ? j + 1 : j) * p.loc_step * p.H;
        la_state_load<DK, DV, DKP, CT>(y0, p.loc + o0 * (DK * DV), p.tr != 0, col0);
        la_state_load<DK, DV, DKP, CT>(y1, p.loc + o1 * (DK * DV), p.tr != 0, col0);
        const float d0 = p.dec[o0], d1 = p.dec[o1];
#pragma unroll
        for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
          for (int t = 0; t < CT; ++t) {
            x[m][t] = x[m][t] * d0 + y0[m][t];
            if (two) x[m][t] = x[m][t] * d1 + y1[m][t];
          }
      }
    }
    float scale = 1.f;  // the state is scale x
    const int nc = (len + C - 1) / C;

    LaRows<T, DK, C, NT> ra, rb;
    LaRows<T, DV, C, NT> rc;
    LaDecayRing<C> ring{lds + oG, p.ld, row0, len, nc, rev, p.ld_head, h, p.H, 0.f};
    auto fetch = [&](int ci) {
      const int t0 = ci * C, m = len - t0 < C ? len - t0 : C;
      ra.load(p.a, row0 + t0, m, h, p.H);
      rb.load(p.b, row0 + t0, m, h, p.H);
      rc.load(p.c, row0 + t0, m, h, p.H);
    };
    if (nc > 0) {
      ring.load(0, wave);
      fetch(ring.chunk(0));
    }

    for (int it = 0; it < nc; ++it) {
      const int ci = ring.chunk(it);
      const LaDecays<C> dec = ring.at(it);
      const double* sG = dec.G;
      const int t0 = ci * C, m = len - t0 < C ? len - t0 : C;
      const int ra0 = la_here(ra_lane), rb0 = la_here(rb_lane), rp0 = la_here(rp_lane);
      ra.template put<true>(sA, LA, m);
      rb.template put<false>(sB, LA, m);
      rc.template put<false>(sC, LC, m);
      if ((it & 3) == 0 && wave < 4) ring.fill(it, wave);
      block_sync_lds();
      if (it + 1 < nc) fetch(ring.chunk(it + 1));
      // the rows the result is multiplied with (behind the chunk's end: its last row)
      u32x4_t dq[R][CT];
      if (p.dots != nullptr) {
        const int hd = p.dot.nh == p.H ? h : h * p.dot.nh / p.H;
        const T* base = static_cast<const T*>(p.dot.p) + ((row0 + t0) * p.dot.nh + hd) * (long long)DV + col0 + 4 * g;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int rr = 16 * r + n < m ? 16 * r + n : m - 1;
          const T* q = base + __umul24((unsigned)rr, (unsigned)(p.dot.nh * DV));
#pragma unroll
          for (int t = 0; t < CT; ++t) dq[r][t] = Op::load4(q + 16 * t);
        }
      }
      float ds[R];  // products with the state's part

      // scores, transposed (rows: columns j of P, columns: rows i): lane (g, n) holds
      // P[i = n][j = 4g..4g+3], stored as four consecutive values per term.  The
      // tiles beyond the diagonal that a 32-deep step covers come out as zeros.
      // All of a wavefront's tiles go through each step together: one alone leaves the
      // wavefront waiting for its reads, products and exponentials in turn.
      static_assert((NW == 4 || NW == 8) && (R == 4 || R == 2), "tiles");
      constexpr int NTL = R == 2 ? 1 : NW == 4 ? 3 : 2;
      const int flip = rev ? R - 1 : 0;
      f32x4_t sc[NTL];
      int rt[NTL], ct[NTL];
#pragma unroll
      for (int u = 0; u < NTL; ++u) {
        // rows 0 and 1 (backwards 3 and 2) reach one 32-deep step, the others both: four
        // tiles each for three passes of four wavefronts.  Eight take the first two in one
        // pass and the last one twice
        const int w = wave & 3, pass = NW == 8 && R == 4 ? u + (u == 0 ? wave >> 2 : 1) : u;
        rt[u] = (pass == 0 ? w >> 1 : pass + 1) ^ flip;
        ct[u] = (pass == 0 ? w & 1 : w) ^ flip;
        sc[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int ks = 0; ks < DKP / 32; ++ks)
#pragma unroll
        for (int u = 0; u < NTL; ++u)
          sc[u] = Op::mma(Op::row(sB + 16 * ct[u] * LA, Op::row_step(rb0, ks)), Op::prow(sA + 16 * rt[u] * LA, Op::row_step(ra0, ks)),
                          sc[u]);
#pragma unroll
      for (int u = 0; u < NTL; ++u) {
        const double gi = sG[16 * rt[u] + n];
        const double* gj = sG + 16 * ct[u] + 4 * g;
        const int edge = 16 * (rt[u] - ct[u]) + n - 4 * g;  // j = i: e = edge; forwards j <= i: e <= edge
        const int last = rev ? edge + p.apart : edge - p.apart;
        if (p.apart && rt[u] == ct[u] && n >> 2 == g)
          sOwn[16 * rt[u] + n] = n & 2 ? (n & 1 ? sc[u][3] : sc[u][2]) : (n & 1 ? sc[u][1] : sc[u][0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float d = rev ? (float)(gj[e] - gi) : (float)(gi - gj[e]);
          const float v = sc[u][e] * __builtin_amdgcn_exp2f(d);
          sc[u][e] = (rev ? e >= last : e <= last) ? v : 0.f;
        }
        Op::template put<NS>(sP + 16 * rt[u] * LP + Op::pcol_step(rp0, ct[u]), C * LP, sc[u]);
      }

      // the state's part of the result, transposed (lane: token n, columns 4g..4g+3)
      f32x4_t acc[R][CT];
      if (active) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t = 0; t < CT; ++t) acc[r][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < DKP / 32; ++ks) {
          frag_t xf[CT][NS];
#pragma unroll
          for (int t = 0; t < CT; ++t) Op::template split<NS>(la_cat(x[2 * ks][t], x[2 * ks + 1][t]), xf[t]);
          frag_t a[R];
#pragma unroll
          for (int r = 0; r < R; ++r) a[r] = Op::prow(sA + 16 * r * LA, Op::row_step(ra0, ks));
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int t = 0; t < CT; ++t) acc[r][t] = Op::mma(xf[t][s], a[r], acc[r][t]);
        }
        const float* fac = rev ? dec.W : dec.E;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float f = fac[16 * r + n] * scale;
#pragma unroll
          for (int t = 0; t < CT; ++t) acc[r][t] *= f;
        }
        if (p.dots != nullptr) {
#pragma unroll
          for (int r = 0; r < R; ++r) ds[r] = la_dot<Op, CT>(dq[r], acc[r]);
        }
      }
      block_sync_lds();

      if (active) {
        // the scores' part
        const int oc = la_here(Op::tr_lane(LC));
#pragma unroll
        for (int ks = 0; ks < C / 32; ++ks) {
          frag_t vf[CT];
#pragma unroll
          for (int t = 0; t < CT; ++t) vf[t] = Op::tr(sC + 32 * ks * LC + Op::tr_step(oc, col0 / 16 + t), LC);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (rev ? ks < r / 2 : ks > r / 2) continue;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              const frag_t pf = Op::prow(sP + s * C * LP + 16 * r * LP, Op::row_step(rp0, ks));
#pragma unroll
              for (int t = 0; t < CT; ++t) acc[r][t] = Op::mma(vf[t], pf, acc[r][t]);
            }
          }
        }
        // the rows' products with those of `dot`, then each token's own score times its values
        if (p.dots != nullptr) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float all = la_dot<Op, CT>(dq[r], acc[r]);
            if (g == 0) sDot[wave * C + 16 * r + n] = float2{ds[r], all - ds[r]};
          }
        }
        if (p.apart) {
          const int ov = la_here(Op::row_lane(LC));
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float own = sOwn[16 * r + n];
#pragma unroll
            for (int t = 0; t < CT; ++t)
              acc[r][t] += Op::widen4(Op::load4(sC + 16 * r * LC + Op::tr_step(ov, col0 / 16 + t))) * own;
          }
        }
        // write the rows
        const int ro = n * p.H * DV + col0 + 4 * g;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const bool in = m == C || 16 * r + n < m;
          const long long row = row0 + t0 + 16 * r, o = (row * p.H + h) * DV;
          if (in) {
#pragma unroll
            for (int t = 0; t < CT; ++t) {
              if (p.r_f32)
                *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.r) + o + (ro + 16 * t)) = acc[r][t];
              else
                Op::template put<1>(static_cast<T*>(p.r) + o + (ro + 16 * t), 0, acc[r][t]);
            }
          }
        }
        if (it + 1 < nc || p.x1 != nullptr)
          la_update<T, DKP, CT, LA, LC>(x, scale, sB, sC, rev ? dec.E : dec.W, *dec.tot, col0);
      }
      block_sync_lds();
      if (p.dots != nullptr && tid < C && tid < m) {
        float2 sum = sDot[tid];
#pragma unroll
        for (int w = 1; w < WV; ++w) {
          sum.x += sDot[w * C + tid].x;
          sum.y += sDot[w * C + tid].y;
        }
        p.dots[(row0 + t0 + tid) * p.H + h] = sum;
      }
    }
    if (active && p.x1 != nullptr) la_state_store<DK, DV, DKP, CT>(x, scale, p.x1, p.tr != 0, col0);
  }
};

// ------------------------------------------------------------ kernels

struct LaArgs {
  const void *q, *k, *v, *dout;  // [row][Hk][dk], [row][Hk][dk], [row][H][dv], [row][H][dv]
  const float* ld;
  const float *h0, *dfinal;      // [nseq][H][dk][dv] or null
  void* out;                     // [row][H][dv]
  float* fstate;                 // [nseq][H][dk][dv] or null
  void *dq, *dk, *dv;            // gradients; dq and dk fp32 [row][H][dk] (partial) when Hk < H
  float *dld, *dh0;
  float *st, *rt;                // state at a segment's start, state gradient at its end: [nwork][H][dk dv]
  float *sdec, *rdec;            // decay over the segment before / behind [nwork][H]
  float2 *xq, *xk;               // q . dq and k . dk  [row][H]: the state's part, the scores' part
  float *ldpart;                 // per-segment sums of dld [nwork][H] (one decay per head)
  LaGeo geo;
  int H, Hk, ld_head, out_f32, qk_f32;
  int sum_in_walk;               // the walks add the other segments' contributions up themselves
  int h0_in_st;                  // h0 is overwritten by fstate: cut sequences have it in st, at their first segment
};

// Each segment's own contribution to the state (role 0: k, v; to the next segment's
// place) and to the state gradient (role 1: q, dout, walking backwards; to the previous
// segment's place), with the segment's decay.  A sequence's last segment (role 1: its
// first) contributes to no other: the walk over it ends with the final state.  It reads two
// of the tensors once and writes dk dv fp32 per segment: 39 to 47 us in a trace (minimum
// and median; its clocks are lower than an untraced call's) at B = 4, H = 16, L = 4096, d =
// 128, 3 TB/s, half way between HBM and the issue of its products.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(64 * la_fwd_waves(DV), la_fwd_waves(DV) / 2) void dp_la_states_kernel(LaArgs p) {
  using Op = LaOp<T>;
  constexpr int C = Op::C, NW = la_fwd_waves(DV), NT = 64 * NW, WV = la_waves(DV, NW), CT = DV / 16 / WV;
  constexpr int DKP = DK < 32 ? 32 : DK;
  constexpr int LB = Op::pitch(DK), LC = Op::pitch(DV);
  extern __shared__ __align__(16) char lds[];
  T* sB = reinterpret_cast<T*>(lds);
  T* sC = sB + C * LB;
  char* sD = reinterpret_cast<char*>(sC + C * LC);
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int s, h;
  la_block(blockIdx.x, p.geo, p.H, p.Hk, &s, &h);
  const bool rev = blockIdx.y != 0;
  LaSeg sg;
  if (!la_in_order(p.geo, &s) || !la_segment(p.geo, s, sg)) return;
  if (rev ? sg.first : sg.last) return;  // nothing of its sequence follows in this direction
  if (p.h0_in_st && sg.first) {  // no segment writes this place: keep h0 there for the walks
    const float* from = p.h0 + ((long long)sg.d * p.H + h) * DK * DV;
    float* to = p.st + ((long long)s * p.H + h) * DK * DV;
    for (int i = 4 * tid; i < DK * DV; i += 4 * NT)
      *reinterpret_cast<f32x4_t*>(to + i) = *reinterpret_cast<const f32x4_t*>(from + i);
  }
  const LaTen tb = rev ? LaTen{p.q, p.Hk} : LaTen{p.k, p.Hk};
  const LaTen tc = rev ? LaTen{p.dout, p.H} : LaTen{p.v, p.H};
  if constexpr (DK < 32) la_zero_pad<T, C, false>(sB, LB);
  const bool active = wave < WV;
  const int col0 = active ? wave * 16 * CT : 0;
  f32x4_t x[DKP / 16][CT];
#pragma unroll
  for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
    for (int t = 0; t < CT; ++t) x[m][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int nc = (sg.len + C - 1) / C;
  LaRows<T, DK, C, NT> rb;
  LaRows<T, DV, C, NT> rc;
  LaDecayRing<C> ring{sD, p.ld, sg.row, sg.len, nc, rev, p.ld_head, h, p.H, 0.f};
  auto fetch = [&](int ci) {
    const int t0 = ci * C, m = sg.len - t0 < C ? sg.len - t0 : C;
    rb.load(tb, sg.row + t0, m, h, p.H);
    rc.load(tc, sg.row + t0, m, h, p.H);
  };
  if (nc > 0) {
    ring.load(0, wave);
    fetch(ring.chunk(0));
  }
  float scale = 1.f;
  double total = 0.0;  // the segment's log decay
  for (int it = 0; it < nc; ++it) {
    const int ci = ring.chunk(it), m = sg.len - ci * C < C ? sg.len - ci * C : C;
    rb.template put<false>(sB, LB, m);
    rc.template put<false>(sC, LC, m);
    if ((it & 3) == 0 && wave < 4) ring.fill(it, wave);
    block_sync_lds();
    if (it + 1 < nc) fetch(ring.chunk(it + 1));
    const LaDecays<C> dec = ring.at(it);
    total += dec.G[C - 1];
    if (active) la_update<T, DKP, CT, LB, LC>(x, scale, sB, sC, rev ? dec.E : dec.W, *dec.tot, col0);
    block_sync_lds();
  }
  float* dst = (rev ? p.rt : p.st) + ((long long)(rev ? s - 1 : s + 1) * p.H + h) * DK * DV;
  if (active) la_state_store<DK, DV, DKP, CT>(x, scale, dst, false, col0);
  if (tid == 0) (rev ? p.rdec : p.sdec)[(long long)(rev ? s - 1 : s + 1) * p.H + h] = __builtin_amdgcn_exp2f((float)total);
}
template <typename T, int DK, int DV>
constexpr int la_states_lds() {
  return LaOp<T>::C * (LaOp<T>::pitch(DK) + LaOp<T>::pitch(DV)) * (int)sizeof(T) + 4 * LaDecayRing<LaOp<T>::C>::BYTES;
}

// Where a forward walk over segment s starts: the state at its start, or (sum_in_walk)
// the initial state and what the segments before contribute.
__device__ __forceinline__ void la_start(const LaArgs& p, const LaSeg& sg, int s, int h, long long per, LaWalkArgs& w) {
  if (!sg.first && !p.sum_in_walk) w.x0 = p.st + ((long long)s * p.H + h) * per;
  else if (p.h0_in_st && sg.count > 1) w.x0 = p.st + ((long long)(s - sg.index) * p.H + h) * per;
  else w.x0 = p.h0 == nullptr ? nullptr : p.h0 + ((long long)sg.d * p.H + h) * per;
  if (p.sum_in_walk && !sg.first) {
    const long long at = (long long)(s - sg.index + 1) * p.H + h;
    w.loc = p.st + at * per;
    w.dec = p.sdec + at;
    w.nloc = sg.index;
    w.loc_step = 1;
  }
}
// Where a backward walk over it starts: the gradient on the state at its end.
__device__ __forceinline__ void la_end(const LaArgs& p, const LaSeg& sg, int s, int h, long long per, LaWalkArgs& w) {
  if (sg.last || p.sum_in_walk) w.x0 = p.dfinal == nullptr ? nullptr : p.dfinal + ((long long)sg.d * p.H + h) * per;
  else w.x0 = p.rt + ((long long)s * p.H + h) * per;
  if (p.sum_in_walk && !sg.last) {
    const long long at = (long long)(s - sg.index + sg.count - 2) * p.H + h;
    w.loc = p.rt + at * per;
    w.dec = p.rdec + at;
    w.nloc = sg.count - 1 - sg.index;
    w.loc_step = -1;
  }
}

// The forward walk: one workgroup per segment and head.  B = 4, H = 16, L = 4096, d = 128:
// the call takes 122 to 128 us (traced, at lower clocks, this kernel 102 to 120 and the
// states 39 to 47), 16 chunks a workgroup; bound by the issue of its products (64 GFLOP
// with the terms, 51 us at the 1.27 PFLOP/s of a large library product) and of the
// exponentials, splits and LDS reads between them, which overlap in part.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(64 * la_fwd_waves(DV), 2) void dp_la_fwd_kernel(LaArgs p) {
  extern __shared__ __align__(16) char lds[];
  int s, h;
  la_block(blockIdx.x, p.geo, p.H, p.Hk, &s, &h);
  LaSeg sg;
  if (!la_in_order(p.geo, &s) || !la_segment(p.geo, s, sg)) return;
  const long long per = DK * DV, so = ((long long)sg.d * p.H + h) * per;
  LaWalkArgs w{};
  w.a = LaTen{p.q, p.Hk};
  w.b = LaTen{p.k, p.Hk};
  w.c = LaTen{p.v, p.H};
  w.r = p.out;
  w.r_f32 = p.out_f32;
  w.ld = p.ld;
  w.ld_head = p.ld_head;
  w.H = p.H;
  la_start(p, sg, s, h, per, w);
  w.x1 = sg.last && p.fstate != nullptr ? p.fstate + so : nullptr;
  LaWalk<T, DK, DV, la_fwd_waves(DV)>::run(w, lds, sg.row, sg.len, h);
}

// The gradient's walks, one workgroup per segment, head and role: dq (forwards
// over the transposed state), dk (backwards, transposed) and dv (backwards).  B = 4, H =
// 16, L = 4096, d = 128, with the decays' gradient: the call takes 388 to 404 us (traced,
// this kernel 339 to 355), bound as the forward: 245 GFLOP in all, 193 us at that rate.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(64 * kLaBwdWaves, 2) void dp_la_bwd_kernel(LaArgs p) {
  extern __shared__ __align__(16) char lds[];
  int s, h;
  la_block(blockIdx.x, p.geo, p.H, p.Hk, &s, &h);
  const int role = blockIdx.y;
  LaSeg sg;
  if (!la_in_order(p.geo, &s) || !la_segment(p.geo, s, sg)) return;
  const long long per = DK * DV, so = ((long long)sg.d * p.H + h) * per;
  const LaTen q{p.q, p.Hk}, k{p.k, p.Hk}, v{p.v, p.H}, dout{p.dout, p.H};
  LaWalkArgs w{};
  w.ld = p.ld;
  w.ld_head = p.ld_head;
  w.H = p.H;
  w.rev = role != 0;
  w.tr = role != 2;
  if (role == 0) {
    la_start(p, sg, s, h, per, w);
  } else {
    la_end(p, sg, s, h, per, w);
    w.x1 = sg.first && role == 2 && p.dh0 != nullptr ? p.dh0 + so : nullptr;
  }
  if (role == 2) {
    w.a = k;
    w.b = q;
    w.c = dout;
    w.r = p.dv;
  } else {
    w.a = role == 0 ? dout : v;
    w.b = role == 0 ? v : dout;
    w.c = role == 0 ? k : q;
    w.r = role == 0 ? p.dq : p.dk;
    w.r_f32 = p.qk_f32;
    w.apart = 1;  // whether the decays' gradient is asked for or not: the same bits
    w.dot = role == 0 ? q : k;
    w.dots = role == 0 ? p.xq : p.xk;
  }
  if (DK != DV && role == 2)
    LaWalk<T, DK, DV, kLaBwdWaves>::run(w, lds, sg.row, sg.len, h);
  else
    LaWalk<T, DV, DK, kLaBwdWaves>::run(w, lds, sg.row, sg.len, h);
}

// ------------------------------------------------------------ launches

// A kernel's LDS limit is a property of the device: raised at its first launch on each.
inline void la_allow_lds(const void* fn, std::atomic<uint64_t>& seen) {
  int d = 0;
  if (hipGetDevice(&d) != hipSuccess) return;  // the launch reports it
  const uint64_t bit = d < 64 ? 1ull << d : 0;
  if ((seen.load(std::memory_order_relaxed) & bit) != 0) return;
  (void)allow_big_lds(fn);
  seen.fetch_or(bit, std::memory_order_relaxed);
}

template <typename T, int DK, int DV>
hipError_t la_states_launch(const LaArgs& a, int roles, hipStream_t st) {
  constexpr int lds = la_states_lds<T, DK, DV>();
  static std::atomic<uint64_t> seen{0};
  la_allow_lds(reinterpret_cast<const void*>(&dp_la_states_kernel<T, DK, DV>), seen);
  hipLaunchKernelGGL((dp_la_states_kernel<T, DK, DV>), dim3((unsigned)(a.geo.nwork * a.H), roles),
                     dim3(64 * la_fwd_waves(DV)), lds, st, a);
  return hipGetLastError();
}

template <typename T, int DK, int DV>
hipError_t la_fwd_launch(const LaArgs& a, hipStream_t st) {
  using W = LaWalk<T, DK, DV, la_fwd_waves(DV)>;
  static std::atomic<uint64_t> seen{0};
  la_allow_lds(reinterpret_cast<const void*>(&dp_la_fwd_kernel<T, DK, DV>), seen);
  hipLaunchKernelGGL((dp_la_fwd_kernel<T, DK, DV>), dim3((unsigned)(a.geo.nwork * a.H)), dim3(W::NT), W::LDS, st, a);
  return hipGetLastError();
}

template <typename T, int DK, int DV>
hipError_t la_bwd_launch(const LaArgs& a, hipStream_t st) {
  constexpr int l0 = LaWalk<T, DV, DK, kLaBwdWaves>::LDS_DOTS, l1 = LaWalk<T, DK, DV, kLaBwdWaves>::LDS;
  static std::atomic<uint64_t> seen{0};
  la_allow_lds(reinterpret_cast<const void*>(&dp_la_bwd_kernel<T, DK, DV>), seen);
  hipLaunchKernelGGL((dp_la_bwd_kernel<T, DK, DV>), dim3((unsigned)(a.geo.nwork * a.H), 3), dim3(64 * kLaBwdWaves),
                     l0 > l1 ? l0 : l1, st, a);
  return hipGetLastError();
}

enum LaStage { kLaStates, kLaFwd, kLaBwd };

// One launch of a forward or gradient: `roles` for kLaStates (1: states, 2: and
// state gradients).
template <typename T, int DK, int DV>
hipError_t la_stage(LaStage stage, const LaArgs& a, int roles, hipStream_t st) {
  if (stage == kLaStates) return la_states_launch<T, DK, DV>(a, roles, st);
  return stage == kLaFwd ? la_fwd_launch<T, DK, DV>(a, st) : la_bwd_launch<T, DK, DV>(a, st);
}

}  // namespace dp

#define DP_LA_DECLARE(tn, DK) \
  hipError_t dp_la_stage_##tn##_##DK(dp::LaStage, const dp::LaArgs&, int dv, int roles, hipStream_t);
#define DP_LA_DEFINE(T, tn, DK)                                                                              \
  hipError_t dp_la_stage_##tn##_##DK(dp::LaStage s, const dp::LaArgs& a, int dv, int roles, hipStream_t st) { \
    switch (dv) {                                                                                            \
      case 16: return dp::la_stage<T, DK, 16>(s, a, roles, st);                                              \
      case 32: return dp::la_stage<T, DK, 32>(s, a, roles, st);                                              \
      case 64: return dp::la_stage<T, DK, 64>(s, a, roles, st);                                              \
      case 128: return dp::la_stage<T, DK, 128>(s, a, roles, st);                                            \
    }                                                                                                        \
    return hipErrorInvalidValue;                                                                             \
  }
