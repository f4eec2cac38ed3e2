// dp_norm.hpp -- group norm with an activation, channels last, and its gradient.
//
// x [rows, G, D]: the G groups of D channels of a row are normalised on their own,
//
//   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps)    (rms: m = 0)
//   n = (x - m) r,   a = n w + b
//   y = a,  a sigma(a)  (silu)   or   a z sigma(z)  (gate z)
//
// with w, b [G, D] fp32.  A group is held in registers by LPR lanes of one
// wavefront (NV 16-byte vectors each), so x is read once and the variance is the
// mean of squared differences, not a difference of sums.  Everything is fp32; a
// result is rounded once.  Bound by HBM: forward 2 tensors (3 with a gate), gradient 3
// (5).  bf16, 16384 x 16 x 128 with a gate: forward 43 us, 4.7 TB/s; gradient 75 us, 4.5
// TB/s.  Groups of 100 channels start anywhere: the gradient of 5001 x 12 x 100 takes 27.4
// us, 2.2 TB/s, bound by the shifts and selects of its last vectors, by the lanes that 12
// groups leave idle (a workgroup has 16 places for them) and by the sums' own launch (4 us).
//
// Gradient, with da = dy times the activation's slope or gate and dn = da w:
//   dx = r (dn - mean(dn) - n mean(dn n))     (rms: no mean(dn))
//   dw = sum over rows of da n, db = sum of da, dz = dy a (sigma(z) + z sigma(z) (1 - sigma(z)))
#pragma once

#include "dp_device.hpp"

namespace dp {

struct NormArgs {
  const void *x, *gate, *dy;
  const float *w, *b;
  void *y, *dx, *dgate;
  float *dw, *db;
  float* part;  // gradient: [2][parts][G D] partial sums of dw and db
  long long rows;
  int G, D, parts;
  float eps;
  int rms, silu;
};

// 1 / (1 + e^-a) by the hardware's exponential and reciprocal (one unit in the last
// place each); e^-a past the range gives 0.
__device__ __forceinline__ float norm_sigmoid(float a) { return __builtin_amdgcn_rcpf(1.f + __expf(-a)); }

// Sum over the LPR lanes of a group, the same value in each.
template <int LPR>
__device__ __forceinline__ float norm_sum(float x) {
  x = dpp_group_sum<(LPR < 16 ? LPR : 16)>(x);
  if constexpr (LPR >= 32) x += __shfl_xor(x, 16);
  if constexpr (LPR >= 64) x += __shfl_xor(x, 32);
  return x;
}

// 16, 8 or 4 bytes at the element type's alignment: a group of an odd width starts
// anywhere.
template <typename V, int A>
struct NormVec {
  typedef V __attribute__((aligned(A))) type;
};

// One lane's share of a group: element i of vector v is channel (lane + v LPR) VE + i.
// Where the width D is no multiple of VE, the group's last vector is read so that it
// ends with the group and is shifted into place when it is used, not when it is loaded
// (a shift would wait for the load, and the next row's loads are meant to stay in flight).
template <typename T, int LPR, int NV>
struct NormRow {
  static constexpr int VE = 16 / (int)sizeof(T), N = NV * VE;
  using vec_t = typename NormVec<u32x4_t, sizeof(T)>::type;
  // channel of element e, for this lane of the group
  __device__ __forceinline__ static int channel(int lane, int e) { return (lane + (e / VE) * LPR) * VE + e % VE; }
  // the raw vectors (zero past D); widen() makes them fp32
  struct Raw {
    u32x4_t v[NV];
  };
  __device__ __forceinline__ static void load(const T* p, int lane, int D, Raw& r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (lane + v * LPR) * VE;
      r.v[v] = u32x4_t{0, 0, 0, 0};
      if (D >= VE) {
        if (c < D) r.v[v] = *reinterpret_cast<const vec_t*>(p + (c + VE <= D ? c : D - VE));
      } else if (c < D) {  // fewer channels than a vector: lane 0, by elements
        T t[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) t[i] = i < D ? p[i] : T(0);
        __builtin_memcpy(&r.v[v], t, 16);
      }
    }
  }
  __device__ __forceinline__ static void widen(const Raw& r, int lane, int D, float* f) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      u32x4_t u = r.v[v];
      if (D % VE != 0 && D > VE) {
        const int c = (lane + v * LPR) * VE, over = c < D && c + VE > D ? c + VE - D : 0;
        const int b = over * 8 * (int)sizeof(T);  // 0 .. 127 bits to the right
        uint64_t lo = u[0] | ((uint64_t)u[1] << 32), hi = u[2] | ((uint64_t)u[3] << 32);
        if (b >= 64) {
          lo = hi;
          hi = 0;
        }
        const int m = b & 63;
        lo = (lo >> m) | ((hi << 1) << (63 - m));
        hi >>= m;
        u = u32x4_t{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
      }
      unpack16(u, f + v * VE, T(0));
    }
  }
  __device__ __forceinline__ static void load_f32(const float* p, int lane, int D, float* f) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int c = channel(lane, e);
      f[e] = c < D ? p[c] : 0.f;
    }
  }
  __device__ __forceinline__ static void store(T* p, int lane, int D, const float* f) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (lane + v * LPR) * VE;
      u32x4_t u;
      pack(f + v * VE, u);
      if (c + VE <= D) {
        *reinterpret_cast<vec_t*>(p + c) = u;
      } else if (c < D) {
        const int n = (D - c) * (int)sizeof(T);  // bytes left: 8, 4 and 2 of them at a time
        char* q = reinterpret_cast<char*>(p + c);
        if (n & 8) {
          *reinterpret_cast<typename NormVec<u32x2_t, sizeof(T)>::type*>(q) = u32x2_t{u[0], u[1]};
          u[0] = u[2];
          u[1] = u[3];
          q += 8;
        }
        if (n & 4) {
          *reinterpret_cast<typename NormVec<uint32_t, sizeof(T)>::type*>(q) = u[0];
          u[0] = u[1];
          q += 4;
        }
        if (n & 2) *reinterpret_cast<uint16_t*>(q) = (uint16_t)u[0];
      }
    }
  }
  __device__ __forceinline__ static void pack(const float* f, u32x4_t& u) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2_t x = {f[2 * i], f[2 * i + 1]};
        u[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2_t));
      }
    }
  }
  // x -> (x - m) r in place (elements past D: 0); returns r
  __device__ __forceinline__ static float normalise(float* f, int lane, int D, float inv, float eps, bool rms) {
    if (!rms) {
      // The mean, then the mean of what is left: the first is off by a few 2^-24 of an
      // offset far above the spread, which the second takes out.  The second divides: a
      // constant group then normalises to exact zeros.
      const bool full = D == LPR * N;
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) s += f[e];
        s = norm_sum<LPR>(s);
        float m = pass == 0 ? s * inv : s / (float)D;
        if (!__builtin_isfinite(s)) {  // values whose sum passes fp32's range: the sum of their D-ths
          s = 0.f;
#pragma unroll
          for (int e = 0; e < N; ++e) s = fmaf(f[e], inv, s);
          m = norm_sum<LPR>(s);
        }
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] -= m;
        if (!full) {
#pragma unroll
          for (int e = 0; e < N; ++e) f[e] = channel(lane, e) < D ? f[e] : 0.f;
        }
      }
    }
    auto squares = [&] {
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) q = fmaf(f[e], f[e], q);
      return norm_sum<LPR>(q);
    };
    float q = squares(), down = 1.f;
    if (__builtin_isinf(q)) {  // squares past fp32's range: of values 2^-80 as large
      down = 0x1p-80f;
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] *= down;
      q = squares();
    }
    // (the hardware's reciprocal root takes a denormal for zero: a spread below 1e-19 with
    // eps = 0 goes through it 2^64 times as large)
    const float m2 = fmaf(q, inv, eps * down * down);
    const bool tiny = m2 < 0x1p-120f;
    const float r = __builtin_amdgcn_rsqf(tiny ? m2 * 0x1p64f : m2) * (tiny ? 0x1p32f : 1.f);
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] *= r;
    return r * down;
  }
};

// Both kernels: a workgroup keeps to one block of GB groups (blockIdx.y), so that a
// lane sees the same channels in every row it takes: w and b are read once and, in the
// gradient, dw and db summed in registers.  TS = 256 / LPR / GB rows run side by side,
// and the next row's vectors are loaded before the current one is worked on.
template <typename T, int LPR, int NV, bool GATE>
__global__ __launch_bounds__(256) void dp_group_norm_kernel(NormArgs p, int GB, int TS) {
  using Row = NormRow<T, LPR, NV>;
  constexpr int N = Row::N;
  const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const int ts = slot / GB, g = blockIdx.y * GB + slot % GB;
  if (ts >= TS || g >= p.G) return;
  const long long go = (long long)g * p.D, C = (long long)p.G * p.D;
  float w[N], b[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    w[e] = 1.f;
    b[e] = 0.f;
  }
  if (p.w != nullptr) Row::load_f32(p.w + go, lane, p.D, w);
  if (p.b != nullptr) Row::load_f32(p.b + go, lane, p.D, b);
  const float inv = 1.f / (float)p.D;
  const T* x = static_cast<const T*>(p.x) + go;
  const T* z = static_cast<const T*>(p.gate) + go;
  T* y = static_cast<T*>(p.y) + go;
  long long row = (long long)blockIdx.x * TS + ts;
  const long long step = (long long)gridDim.x * TS;
  if (row >= p.rows) return;
  typename Row::Raw rx, rz;
  Row::load(x + row * C, lane, p.D, rx);
  if constexpr (GATE) Row::load(z + row * C, lane, p.D, rz);
  for (; row < p.rows; row += step) {
    float f[N], a[N];
    Row::widen(rx, lane, p.D, f);
    if constexpr (GATE) Row::widen(rz, lane, p.D, a);
    if (row + step < p.rows) {
      Row::load(x + (row + step) * C, lane, p.D, rx);
      if constexpr (GATE) Row::load(z + (row + step) * C, lane, p.D, rz);
    }
    Row::normalise(f, lane, p.D, inv, p.eps, p.rms != 0);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      f[e] = fmaf(f[e], w[e], b[e]);
      if constexpr (GATE) f[e] *= a[e] * norm_sigmoid(a[e]);
    }
    if constexpr (!GATE) {
      if (p.silu) {
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] *= norm_sigmoid(f[e]);
      }
    }
    Row::store(y + row * C, lane, p.D, f);
  }
}

// Gradient.  A workgroup adds the sums of dw and db of its side rows up through LDS and
// writes one line of `part`; dp_group_norm_sum_kernel adds the lines up, both in a fixed
// order.
template <typename T, int LPR, int NV, bool GATE>
__global__ __launch_bounds__(256) void dp_group_norm_bwd_kernel(NormArgs p, int GB, int TS) {
  using Row = NormRow<T, LPR, NV>;
  constexpr int N = Row::N;
  const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const int ts = slot / GB, g = blockIdx.y * GB + slot % GB;
  const bool live = ts < TS && g < p.G;  // the others only wait below
  const long long go = (long long)g * p.D, C = (long long)p.G * p.D;
  float w[N], b[N], dw[N], db[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    w[e] = 1.f;
    b[e] = dw[e] = db[e] = 0.f;
  }
  if (p.w != nullptr && live) Row::load_f32(p.w + go, lane, p.D, w);
  if (p.b != nullptr && live) Row::load_f32(p.b + go, lane, p.D, b);
  const float inv = 1.f / (float)p.D;
  const T* x = static_cast<const T*>(p.x) + go;
  const T* dy = static_cast<const T*>(p.dy) + go;
  const T* gate = static_cast<const T*>(p.gate) + go;
  long long row = live ? (long long)blockIdx.x * TS + ts : p.rows;
  const long long step = (long long)gridDim.x * TS;
  typename Row::Raw rx, rd, rz;
  auto fetch = [&](long long r) {
    if (r >= p.rows) return;
    Row::load(x + r * C, lane, p.D, rx);
    Row::load(dy + r * C, lane, p.D, rd);
    if constexpr (GATE) Row::load(gate + r * C, lane, p.D, rz);
  };
  fetch(row);
  for (; row < p.rows; row += step) {
    float n[N], da[N], z[N];
    Row::widen(rx, lane, p.D, n);
    Row::widen(rd, lane, p.D, da);
    if constexpr (GATE) Row::widen(rz, lane, p.D, z);
    fetch(row + step);
    const float r = Row::normalise(n, lane, p.D, inv, p.eps, p.rms != 0);
    if constexpr (GATE) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float s = norm_sigmoid(z[e]), a = fmaf(n[e], w[e], b[e]), t = da[e];
        da[e] = t * (z[e] * s);
        z[e] = t * a * fmaf(z[e] * s, 1.f - s, s);
      }
      Row::store(static_cast<T*>(p.dgate) + go + row * C, lane, p.D, z);
    } else if (p.silu) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float a = fmaf(n[e], w[e], b[e]), s = norm_sigmoid(a);
        da[e] *= fmaf(a * s, 1.f - s, s);
      }
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      dw[e] = fmaf(da[e], n[e], dw[e]);
      db[e] += da[e];
      da[e] *= w[e];
      s1 += da[e];
      s2 = fmaf(da[e], n[e], s2);
    }
    s1 = p.rms ? 0.f : norm_sum<LPR>(s1) * inv;
    s2 = norm_sum<LPR>(s2) * inv;
#pragma unroll
    for (int e = 0; e < N; ++e) n[e] = r * (da[e] - s1 - n[e] * s2);
    Row::store(static_cast<T*>(p.dx) + go + row * C, lane, p.D, n);
  }
  if (p.part == nullptr) return;
  extern __shared__ __align__(16) float norm_lds[];  // [256][N + 1], where TS > 1
  float* mine = norm_lds + threadIdx.x * (N + 1);
  float* out = p.part + (long long)blockIdx.x * C + go;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* sum = which == 0 ? dw : db;
    if (TS > 1) {
#pragma unroll
      for (int e = 0; e < N; ++e) mine[e] = sum[e];
      __syncthreads();
      if (live && ts == 0) {
        for (int i = 1; i < TS; ++i) {
#pragma unroll
          for (int e = 0; e < N; ++e) sum[e] += mine[i * GB * LPR * (N + 1) + e];
        }
      }
      __syncthreads();
    }
    if (live && ts == 0) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int c = Row::channel(lane, e);
        if (c < p.D) out[(long long)which * p.parts * C + c] = sum[e];
      }
    }
  }
}

// dw and db (blockIdx.y): the partial lines added up, 16 channels a workgroup, 64 groups
// of lanes on every 64th line each, then in a fixed order.  (64 channels and 16 groups
// left most of the chip idle: 2048 lines of 1000 channels took 25 us of a gradient's 37.)
static __global__ __launch_bounds__(1024) void dp_group_norm_sum_kernel(NormArgs p) {
  __shared__ float red[64][17];
  const long long C = (long long)p.G * p.D;
  const int l = threadIdx.x & 15, w = threadIdx.x >> 4;
  const long long c = (long long)blockIdx.x * 16 + l;
  const float* part = p.part + (long long)blockIdx.y * p.parts * C;
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int i = w; i < p.parts; i += 64) s += part[i * C + c];
  }
  red[w][l] = s;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) t += red[16 * w + i][l];
  t += __shfl_xor(t, 16);
  t += __shfl_xor(t, 32);
  float* out = blockIdx.y == 0 ? p.dw : p.db;
  if (w == 0 && c < C && out != nullptr) out[c] = t;
}

}  // namespace dp
