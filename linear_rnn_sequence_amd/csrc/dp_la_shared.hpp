// dp_la_shared.hpp -- the parts of linear attention that no head size or element
// type shapes: the segment table of a packed batch, the decayed sums over
// segments, the gradient of the log decays, and the sums and zeros that are left.  Included by the C ABI only.
#pragma once

#include "dp_la.hpp"

namespace dp {

// tab[d] = segments before sequence d (one at least each), tab[nseq] = all of them,
// tab[nseq + 1] = cu[nseq], or -1 if the offsets are not 0 = cu[0] <= cu[1] <= .. <=
// cu[nseq] <= L; order: the segments, whole ones first, then those of half the length
// and more, then the rest.  One workgroup; each thread sums a run of sequences.
static __global__ __launch_bounds__(256) void dp_la_table_kernel(const int* cu, int nseq, int L, int seg, int* tab,
                                                                 int* order) {
  __shared__ int wave_sum[3][4];
  __shared__ int bad;
  const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63;
  const int per = (nseq + 255) / 256;
  const int lo = tid * per < nseq ? tid * per : nseq;
  const int hi = lo + per < nseq ? lo + per : nseq;
  if (tid == 0) bad = (cu[0] != 0 || cu[nseq] > L || cu[nseq] < 0) ? 1 : 0;
  __syncthreads();
  int mybad = 0;
  for (int d = lo; d < hi; ++d) mybad |= (cu[d + 1] < cu[d] || cu[d] < 0 || cu[d + 1] > L) ? 1 : 0;
  if (mybad) atomicOr(&bad, 1);
  __syncthreads();
  const bool ok = bad == 0;
  auto length = [&](int d) { return ok ? cu[d + 1] - cu[d] : 0; };
  // whole segments, and whether a long or a short rest follows
  int mine[3] = {0, 0, 0};
  for (int d = lo; d < hi; ++d) {
    const int n = length(d), rest = n % seg;
    mine[0] += n / seg;
    mine[1] += rest >= (seg + 1) / 2;
    mine[2] += n == 0 || (rest > 0 && rest < (seg + 1) / 2);
  }
  int at[3], all[3];
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    int x = mine[c];
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(x, o);
      if (l >= o) x += y;
    }
    if (l == 63) wave_sum[c][wave] = x;
    at[c] = x - mine[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    all[c] = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) at[c] += wave_sum[c][w];
      all[c] += wave_sum[c][w];
    }
  }
  int id = at[0] + at[1] + at[2];  // segments before this thread's first sequence
  at[1] += all[0];
  at[2] += all[0] + all[1];
  for (int d = lo; d < hi; ++d) {
    tab[d] = id;
    const int n = length(d), whole = n / seg, rest = n % seg;
    for (int i = 0; i < whole; ++i) order[at[0]++] = id++;
    if (rest >= (seg + 1) / 2) order[at[1]++] = id++;
    else if (rest > 0 || n == 0) order[at[2]++] = id++;
  }
  if (tid == 0) {
    tab[nseq] = all[0] + all[1] + all[2];
    tab[nseq + 1] = ok ? cu[nseq] : -1;
  }
}

// Decayed sums over a sequence's segments, one thread per four state elements, in
// place.  Role 0: st[s] holds segment s - 1's own contribution and becomes the state at
// segment s's start.  Role 1: rt[s] holds segment s + 1's and becomes the gradient on
// the state at segment s's end.
static __global__ __launch_bounds__(256) void dp_la_scan_kernel(LaArgs p, int per) {
  const long long x = (long long)blockIdx.y * 256 + threadIdx.x;
  const int d = blockIdx.x / p.H, h = blockIdx.x - d * p.H;
  if (x >= per / 4) return;
  int s0, s1;
  if (p.geo.cu == nullptr) {
    s0 = d * p.geo.nps;
    s1 = s0 + p.geo.nps;
  } else {
    s0 = p.geo.tab[d];
    s1 = p.geo.tab[d + 1];
  }
  const int n = s1 - s0 - 1;  // segments that start from the sum
  if (n <= 0) return;
  const bool rev = blockIdx.z != 0;
  const float* init = rev ? p.dfinal : p.h0;
  f32x4_t cur = {0.f, 0.f, 0.f, 0.f};
  if (init != nullptr) cur = *reinterpret_cast<const f32x4_t*>(init + ((long long)d * p.H + h) * per + 4 * x);
  float* base = (rev ? p.rt : p.st) + (long long)h * per + 4 * x;
  const float* dec = rev ? p.rdec : p.sdec;
  const long long ss = (long long)p.H * per;
  // eight segments' values in flight at a time
  for (int i0 = 0; i0 < n; i0 += 8) {
    f32x4_t loc[8];
    float f[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u, s = rev ? s1 - 2 - i : s0 + 1 + i;
      if (i < n) {
        loc[u] = *reinterpret_cast<const f32x4_t*>(base + s * ss);
        f[u] = dec[(long long)s * p.H + h];
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u, s = rev ? s1 - 2 - i : s0 + 1 + i;
      if (i < n) {
        cur = cur * f[u] + loc[u];
        *reinterpret_cast<f32x4_t*>(base + s * ss) = cur;
      }
    }
  }
}

// dl of one segment and head (see the head of dp_la.hpp): <S, D> at the segment's start,
// plus the sums of b - a from there to before the token, plus what the token's chunk of C
// adds: the sums of c - r before it, in the chunk's second half those of r - c from it on,
// all in fp64.  A decay that erases the state has gradient
// zero (the difference of the sums would leave their rounding).  With one decay per head
// the segment's sum of dl goes to ldpart.
constexpr int kDldThreads = 512;
template <int C>
__global__ __launch_bounds__(kDldThreads) void dp_la_dld_kernel(LaArgs p, int per) {
  constexpr int NT = kDldThreads, NW = NT / 64, U = 2048 / NT;
  __shared__ double red[NW], run[NW];
  const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63;
  const int s = blockIdx.x / p.H, h = blockIdx.x - s * p.H;
  LaSeg sg;
  if (!la_segment(p.geo, s, sg)) {
    if (p.ld_head && tid == 0) p.ldpart[(long long)s * p.H + h] = 0.f;
    return;
  }
  // S and D at the segment's start: what a forward walk starts from, and the gradient the
  // segment before ends with; at the sequence's start h0 (none: zero) and its gradient
  LaWalkArgs wS{}, wD{};
  la_start(p, sg, s, h, per, wS);
  if (sg.first) {
    wD.x0 = wS.x0 == nullptr ? nullptr : p.dh0 + ((long long)sg.d * p.H + h) * per;
  } else {
    LaSeg before = sg;
    --before.index;
    before.last = 0;
    la_end(p, before, s - 1, h, per, wD);
  }
  auto state = [&](const LaWalkArgs& w, int i) {
    f32x4_t x = {0.f, 0.f, 0.f, 0.f};
    if (w.x0 != nullptr) x = *reinterpret_cast<const f32x4_t*>(w.x0 + i);
    for (int j = 0; j < w.nloc; ++j) {
      const long long o = (long long)j * w.loc_step * p.H;
      x = x * w.dec[o] + *reinterpret_cast<const f32x4_t*>(w.loc + o * per + i);
    }
    return x;
  };
  // the first tokens' terms on the way meanwhile
  float2 q, k;
  float ld;
  auto fetch = [&](int e) {
    const int i = e + tid;
    q = k = float2{0.f, 0.f};
    ld = 0.f;
    if (i < sg.len) {
      q = p.xq[(sg.row + i) * p.H + h];
      k = p.xk[(sg.row + i) * p.H + h];
      ld = p.ld_head ? p.ld[h] : p.ld[(sg.row + i) * p.H + h];
    }
  };
  fetch(0);
  double f = 0.0;
  auto dot = [&](const f32x4_t& a, const f32x4_t& b) {
    f += (double)(a[0] * b[0] + a[1] * b[1]) + (double)(a[2] * b[2] + a[3] * b[3]);
  };
  if (wS.nloc + wD.nloc > 0) {
    for (int i = 4 * tid; i < per; i += 4 * NT) dot(state(wS, i), state(wD, i));
  } else if (wS.x0 != nullptr && wD.x0 != nullptr) {
    // several vectors of each in flight
    for (int i0 = 4 * tid; i0 < per; i0 += 4 * NT * U) {
      f32x4_t a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + 4 * NT * u < per ? i0 + 4 * NT * u : i0;
        a[u] = *reinterpret_cast<const f32x4_t*>(wS.x0 + i);
        b[u] = *reinterpret_cast<const f32x4_t*>(wD.x0 + i);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + 4 * NT * u < per) dot(a[u], b[u]);
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) f += __shfl_xor(f, o);
  if (l == 0) red[wave] = f;
  __syncthreads();
  double carry = 0.0, sum = 0.0;
#pragma unroll
  for (int w = 0; w < NW; ++w) carry += red[w];
  for (int e = 0; e < sg.len; e += NT) {
    const double cross = (double)k.x - (double)q.x, in = (double)q.y - (double)k.y;
    const bool erases = ld <= kLaMinLog;
    if (e + NT < sg.len) fetch(e + NT);
    const double cc = la_scan64(cross), ci = la_scan64(in);
    if (l == 63) run[wave] = cc;
    // the sums of r - c up to the chunk's start and its end, which lanes 31 and 63 hold
    const double t0 = __shfl(ci, C - 1), t1 = __shfl(ci, 63);
    const bool lower = C == 64 || l < 32;
    const double inside = ((l & (C - 1)) < C / 2 ? (lower ? 0.0 : t0) : (lower ? t0 : t1)) - ci + in;
    __syncthreads();
    double before = carry + cc - cross;
    for (int w = 0; w < wave; ++w) before += run[w];
    const int i = e + tid;
    if (i < sg.len) {
      const double d = erases ? 0.0 : before + inside;
      sum += d;
      if (!p.ld_head) p.dld[(sg.row + i) * p.H + h] = (float)d;
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) carry += run[w];
    __syncthreads();
  }
  if (p.ld_head) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
    __syncthreads();  // red: everybody has read the first use
    if (l == 0) red[wave] = sum;
    __syncthreads();
    if (tid == 0) {
      double all = 0.0;
#pragma unroll
      for (int w = 0; w < NW; ++w) all += red[w];
      p.ldpart[(long long)s * p.H + h] = (float)all;
    }
  }
}

// What is left after the walks, by ranges of workgroups:
//  - shared query / key heads (nq workgroups, then as many): dq and dk of a group's value
//    heads summed in a fixed order, four elements a thread, rounded once;
//  - one decay per head (nl = H): dld[h] = the segments' sums of dl, in a fixed order;
//  - packed batches (the rest): zeros for the gradients of rows behind the last sequence.
template <typename T>
__global__ __launch_bounds__(256) void dp_la_finish_kernel(LaArgs p, void* dq, void* dk, int DK, int DV, long long rows,
                                                           int nq, int nl) {
  __shared__ double red[4];
  const int tid = threadIdx.x;
  int b = blockIdx.x;
  const bool packed = p.geo.cu != nullptr;
  const long long behind = packed ? (p.geo.tab[p.geo.nseq + 1] < 0 ? 0 : p.geo.tab[p.geo.nseq + 1]) : rows;
  if (b < 2 * nq) {
    const bool key = b >= nq;
    if (key) b -= nq;
    const long long n4 = behind * p.Hk * DK / 4;
    const int r = p.H / p.Hk;
    const float* part = static_cast<const float*>(key ? p.dk : p.dq);
    T* out = static_cast<T*>(key ? dk : dq);
    for (long long i = (long long)b * 256 + tid; i < n4; i += (long long)nq * 256) {
      const long long e = 4 * i, rk = e / DK;  // (row, key head)
      const int c = (int)(e - rk * DK);
      f32x4_t s = {0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < r; ++j) s += *reinterpret_cast<const f32x4_t*>(part + (rk * r + j) * DK + c);
      LaOp<T>::template put<1>(out + e, 0, s);
    }
    return;
  }
  b -= 2 * nq;
  if (b < nl) {
    double s = 0.0;
    for (int i = tid; i < p.geo.nwork; i += 256) s += (double)p.ldpart[(long long)i * p.H + b];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o);
    if ((tid & 63) == 0) red[tid >> 6] = s;
    __syncthreads();
    if (tid == 0) p.dld[b] = (float)(red[0] + red[1] + red[2] + red[3]);
    return;
  }
  b -= nl;
  const int nb = gridDim.x - 2 * nq - nl;
  const long long n = rows - behind, first = (long long)b * 256 + tid, step = (long long)nb * 256;
  if (n <= 0) return;
  auto zero = [&](void* q, long long row_bytes) {  // rows of a multiple of 16 bytes
    char* z = static_cast<char*>(q) + behind * row_bytes;
    for (long long i = first; i < n * row_bytes / 16; i += step) st16(z + 16 * i, u32x4_t{0, 0, 0, 0});
  };
  zero(dq, (long long)p.Hk * DK * (long long)sizeof(T));
  zero(dk, (long long)p.Hk * DK * (long long)sizeof(T));
  zero(p.dv, (long long)p.H * DV * (long long)sizeof(T));
  if (p.dld != nullptr && !p.ld_head)
    for (long long i = first; i < n * p.H; i += step) p.dld[behind * p.H + i] = 0.f;
}

}  // namespace dp
