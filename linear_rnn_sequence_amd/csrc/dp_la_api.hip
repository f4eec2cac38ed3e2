// dp_la_api.hip -- C ABI of linear attention with a decay per head: dp_la_fwd_*,
// dp_la_bwd_*, dp_la_decode_* (declared in include/dp.h).  Arguments are checked on
// the host before any HIP call; the library allocates nothing and keeps nothing.
#include <limits.h>
#include <stdint.h>

#include "dp.h"
#include "dp_la_decode.hpp"
#include "dp_la_shared.hpp"
#include "dp_overlap.hpp"

DP_LA_DECLARE(f32, 16)
DP_LA_DECLARE(f32, 32)
DP_LA_DECLARE(f32, 64)
DP_LA_DECLARE(f32, 128)
DP_LA_DECLARE(bf16, 16)
DP_LA_DECLARE(bf16, 32)
DP_LA_DECLARE(bf16, 64)
DP_LA_DECLARE(bf16, 128)

namespace {

constexpr size_t kWsAlign = 256;
constexpr int kChunk = 64;  // segments are whole chunks of either path

size_t up(size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

struct LaShape {
  int B, H, Hk, L, dk, dv, packed;
  long long rows() const { return packed ? L : (long long)B * L; }
};

// Bytes of the tensors of a call, elements of `elem` bytes.
struct LaBytes {
  size_t qk, v, out, ld, state, cu;
  LaBytes(const LaShape& s, int elem, int out_elem, bool head)
      : qk((size_t)s.rows() * s.Hk * s.dk * elem),
        v((size_t)s.rows() * s.H * s.dv * elem),
        out((size_t)s.rows() * s.H * s.dv * out_elem),
        ld((head ? (size_t)1 : (size_t)s.rows()) * s.H * 4),
        state((size_t)s.B * s.H * s.dk * s.dv * 4),
        cu((size_t)(s.B + 1) * 4) {}
};

int check(const LaShape& s) {
  if (s.B <= 0 || s.H <= 0 || s.Hk <= 0 || s.L < 0 || s.dk <= 0 || s.dv <= 0) return DP_EINVAL;
  if (s.Hk > s.H || s.H % s.Hk != 0) return DP_EINVAL;
  if (!dim_ok(s.dk) || !dim_ok(s.dv)) return DP_ENOTSUP;
  if (s.L > INT_MAX - 4 * kChunk || s.rows() > INT_MAX - 4 * kChunk) return DP_ENOTSUP;  // row indices are 32-bit
  // byte offsets inside a chunk are 32-bit: 64 rows x H max(dk, dv) x 4 bytes
  if ((long long)s.H * 128 * kChunk * 4 > INT_MAX) return DP_ENOTSUP;
  if ((long long)s.B + s.L / kChunk > INT_MAX) return DP_ENOTSUP;
  return DP_OK;
}
// A launch has less than 2^32 threads: a workgroup of 512 at most per segment and head.
int check_grid(const LaShape& s, const dp::LaGeo& g) {
  return (long long)g.nwork * s.H <= UINT_MAX / 512 ? DP_OK : DP_ENOTSUP;
}

// Segments: about `target` workgroups in all, of `least` chunks of 64 tokens at least.
// More segments give a short batch the whole chip (a workgroup walks its chunks one
// after another, 2 to 5 us each, fp32 3 to 13); each costs its state (dk dv fp32) being
// written, summed and read again, and the states' pass reads two tensors a second time.
// So a batch whose heads alone fill the chip is not cut, nor a sequence of `alone` chunks,
// for which one launch is quicker than two.
int segments(int L, int seg) { return (int)(((long long)L + seg - 1) / seg); }
void plan(const LaShape& s, int target, int least, int alone, dp::LaGeo* g, int* single) {
  const long long chunks = (s.rows() + kChunk - 1) / kChunk;
  long long segs = (target + s.H - 1) / s.H;  // wanted over all sequences
  if (segs < s.B) segs = s.B;
  long long per;  // chunks per segment
  if (s.packed) {
    per = (chunks + segs - 1) / segs;
  } else {
    const long long c = segments(s.L, kChunk), n = segs / s.B;
    per = (c + n - 1) / n;
  }
  if (segments(s.L, kChunk) <= alone) per = alone;
  if (per < least) per = least;
  g->nseq = s.B;
  g->L = s.L;
  g->seg = (int)(per * kChunk);
  *single = s.L <= g->seg;
  g->nps = s.L <= g->seg ? 1 : segments(s.L, g->seg);
  // packed: sum over sequences of max(1, ceil(len / seg)) <= nseq + L / seg
  g->nwork = s.packed ? s.B + s.L / g->seg : s.B * g->nps;  // no more than rows / 64 + B
}
// Forward: one workgroup of eight wavefronts a CU, or two of four.  A second launch and its
// workspace cost the host 4 us and the GPU 2: a sequence is walked alone for two chunks, and
// for three where a narrow state makes them short (8 heads, alone against cut, as the GPU
// runs them and as calls of one stream, which the host bounds: bf16 d = 128, 128 tokens
// 12.8 / 13.9 and 12.8 / 16.3 us, 256 tokens 22.1 / 15.1 and 22.2 / 16.3; d = 64, 192
// tokens 11.0 / 10.1 and 11.8 / 16.2, 256 tokens 13.6 / 10.6 and 13.9 / 16.3; fp32 d = 64,
// 192 tokens 17.7 / 13.2 and 17.8 / 16.2, 256 tokens 22.5 / 13.7 and 22.6 / 16.2, d = 128,
// 128 tokens 28.4 / 24.9, 256 tokens 53 / 26).  Types share the rule, as they share the
// workspace's size.
// Gradient: three roles of one workgroup a CU, two chunks a segment at least (8 heads of
// 128, 2048 tokens: 48 against 61 us with one), and four alone: 192 tokens are quicker so
// everywhere (8 heads of 128 28 / 34 us, 64 of them 30 / 40), 256 where heads are many
// and wide (64 of 128 38 / 42 us, 64 of 64 25.6 / 23.4, 8 of 128 36 / 34).
void plan_fwd(const LaShape& s, dp::LaGeo* g, int* single) {
  plan(s, dp::la_fwd_waves(s.dv) == 8 ? 256 : 512, 1, s.dk * s.dv <= 64 * 64 ? 3 : 2, g, single);
}
void plan_bwd(const LaShape& s, dp::LaGeo* g, int* single) { plan(s, 256, 2, 4, g, single); }
// Whether the walks add up the earlier segments' states themselves or start from the scan's
// sums, by what either costs a sequence of n segments, in microseconds (fp32 states either
// way, so the inputs' type does not matter):
//   scan: its launch, 4, and its chain over the segments, n / 8;
//   walk: the longest one reads n - 1 states first, at 128 KB a microsecond (the 64 bytes
//         a clock that a CU takes from L2); in the gradient three roles read them, two of
//         them side by side on a CU and the decays' gradient once more: 20 KB.
// Packed rows count half: only the bound of n is known, which one long sequence reaches,
// and others' products run beside its reads.  Timed both ways for 1 to 64 heads of 16 to
// 128 columns, 2 to 512 segments, one length and up to 48 packed sequences, both types and
// directions (796 cases): on average 0.4% slower than the quicker of the two.  d = 128, one
// length, walk against scan: 8 segments (32 heads) 66.6 / 67.4 us, 16 (16) 47.9 / 45.8, 32
// (8) 45.6 / 38.4; d = 64: 16 (32) 33.3 / 38.0, 64 (8) 29.2 / 31.9, 512 (1) 169 / 226.  24 packed
// sequences (d = 128, 16 heads) 139 / 144, 48 of them (43 segments, one long) 203 / 181.
// Gradient, d = 128: 2 segments (128 heads) 354 / 355, 4 (64) 362 / 357, 8 (16) 66 / 45; d =
// 32: 16 (16) 44.2 / 46.2, 128 (2) 97 / 89.
bool sum_in_walk(const LaShape& s, const dp::LaGeo& g, bool bwd) {
  const long long n = segments(s.L, g.seg), kb = (n - 1) * s.dk * s.dv * 4 / 1024;
  return 8 * kb <= (bwd ? 20 : 128) * (s.packed ? 2 : 1) * (32 + n);
}

struct LaWs {
  size_t tab, order, st, rt, sdec, rdec, xq, xk, dh0, ldpart, pq, pk, total;
};
LaWs layout(const LaShape& s, const dp::LaGeo& g, int single, bool bwd) {
  LaWs w{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up(bytes);
    return at;
  };
  const size_t state = (size_t)s.H * s.dk * s.dv * 4, tok = (size_t)s.rows() * s.H * 4;
  w.tab = take(s.packed ? (size_t)(s.B + 2) * 4 : 0);
  w.order = take(s.packed ? (size_t)g.nwork * 4 : 0);
  w.st = take(single ? 0 : (size_t)g.nwork * state);
  w.sdec = take(single ? 0 : (size_t)g.nwork * s.H * 4);
  if (bwd) {
    w.rt = take(single ? 0 : (size_t)g.nwork * state);
    w.rdec = take(single ? 0 : (size_t)g.nwork * s.H * 4);
    w.dh0 = take((size_t)s.B * state);
    w.xq = take(2 * tok);
    w.xk = take(2 * tok);
    w.ldpart = take((size_t)g.nwork * s.H * 4);
    w.pq = take(s.Hk < s.H ? tok * s.dk : 0);
    w.pk = take(s.Hk < s.H ? tok * s.dk : 0);
  }
  w.total = o;
  return w;
}

hipError_t stage(int elem, dp::LaStage st, const dp::LaArgs& a, int dk, int dv, int roles, hipStream_t str) {
  if (elem == 4) {
    switch (dk) {
      case 16: return dp_la_stage_f32_16(st, a, dv, roles, str);
      case 32: return dp_la_stage_f32_32(st, a, dv, roles, str);
      case 64: return dp_la_stage_f32_64(st, a, dv, roles, str);
      case 128: return dp_la_stage_f32_128(st, a, dv, roles, str);
    }
  } else {
    switch (dk) {
      case 16: return dp_la_stage_bf16_16(st, a, dv, roles, str);
      case 32: return dp_la_stage_bf16_32(st, a, dv, roles, str);
      case 64: return dp_la_stage_bf16_64(st, a, dv, roles, str);
      case 128: return dp_la_stage_bf16_128(st, a, dv, roles, str);
    }
  }
  return hipErrorInvalidValue;
}

int status(hipError_t e) { return e == hipSuccess ? DP_OK : DP_EHIP; }

// Segment table (packed), and with several segments the states and their sums.
hipError_t front(int elem, const LaShape& s, const dp::LaArgs& a, int single, int roles, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (s.packed) {
    hipLaunchKernelGGL(dp::dp_la_table_kernel, dim3(1), dim3(256), 0, st, a.geo.cu, a.geo.nseq, a.geo.L, a.geo.seg,
                       const_cast<int*>(a.geo.tab), const_cast<int*>(a.geo.order));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (single) return e;
  if ((e = stage(elem, dp::kLaStates, a, s.dk, s.dv, roles, st)) != hipSuccess || a.sum_in_walk) return e;
  const int per = s.dk * s.dv;
  hipLaunchKernelGGL(dp::dp_la_scan_kernel, dim3((unsigned)(s.B * s.H), (per / 4 + 255) / 256, roles), dim3(256), 0, st, a,
                     per);
  return hipGetLastError();
}

int la_fwd(int elem, const void* q, const void* k, const void* v, const float* ld, const int* cu, int B, int H, int Hk,
           int L, int dk, int dv, void* out, float* fstate, const float* h0, void* ws, size_t wsb, int flags,
           dp_stream stream) {
  const LaShape s{B, H, Hk, L, dk, dv, cu != nullptr};
  int rc = check(s);
  if (rc != DP_OK) return rc;
  if ((flags & ~(DP_OUT_F32 | DP_LA_HEAD_DECAY)) != 0) return DP_EINVAL;
  if ((flags & DP_LA_HEAD_DECAY) != 0 && ld == nullptr) return DP_EINVAL;
  if (L > 0 && (q == nullptr || k == nullptr || v == nullptr || out == nullptr)) return DP_EINVAL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(fstate, 16) ||
      !aligned(h0, 16) || !aligned(ld, 4) || !aligned(cu, 4))
    return DP_EINVAL;
  dp::LaArgs a{};
  int single = 0;
  plan_fwd(s, &a.geo, &single);
  if ((rc = check_grid(s, a.geo)) != DP_OK) return rc;
  const LaWs w = layout(s, a.geo, single, false);
  if (w.total > 0 && (ws == nullptr || wsb < w.total || !aligned(ws, kWsAlign))) return DP_EWORKSPACE;
  const bool f32_out = elem == 4 || (flags & DP_OUT_F32) != 0;
  const LaBytes n(s, elem, f32_out ? 4 : elem, (flags & DP_LA_HEAD_DECAY) != 0);
  if (!dp::outputs_apart({{fstate, n.state}, {out, n.out}, {ws, w.total}},
                         {{h0, n.state}, {q, n.qk}, {k, n.qk}, {v, n.v}, {ld, n.ld}, {cu, n.cu}}, {{0, 0}}))
    return DP_EINVAL;
  char* b = static_cast<char*>(ws);
  int* tab = s.packed ? reinterpret_cast<int*>(b + w.tab) : nullptr;
  a.q = q;
  a.k = k;
  a.v = v;
  a.ld = ld;
  a.h0 = h0;
  a.out = out;
  a.fstate = fstate;
  a.st = reinterpret_cast<float*>(b + w.st);
  a.sdec = reinterpret_cast<float*>(b + w.sdec);
  a.geo.cu = cu;
  a.geo.tab = tab;
  a.geo.order = s.packed ? reinterpret_cast<const int*>(b + w.order) : nullptr;
  a.H = H;
  a.Hk = Hk;
  a.ld_head = (flags & DP_LA_HEAD_DECAY) != 0;
  a.out_f32 = f32_out;
  a.sum_in_walk = !single && sum_in_walk(s, a.geo, false);
  // In one buffer, a sequence's last segment could write the state before another has
  // started from it (the XCDs take their workgroups each at its own pace).
  a.h0_in_st = !single && h0 != nullptr && h0 == fstate;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = front(elem, s, a, single, 1, st);
  if (e == hipSuccess) e = stage(elem, dp::kLaFwd, a, dk, dv, 0, st);
  return status(e);
}

int la_bwd(int elem, const void* q, const void* k, const void* v, const float* ld, const int* cu, const float* h0,
           const void* dout, const float* dfinal, int B, int H, int Hk, int L, int dk, int dv, void* dq, void* dk_out,
           void* dv_out, float* dld, float* dh0, void* ws, size_t wsb, int flags, dp_stream stream) {
  const LaShape s{B, H, Hk, L, dk, dv, cu != nullptr};
  int rc = check(s);
  if (rc != DP_OK) return rc;
  if ((flags & ~DP_LA_HEAD_DECAY) != 0) return DP_EINVAL;
  if ((flags & DP_LA_HEAD_DECAY) != 0 && ld == nullptr) return DP_EINVAL;
  if (L > 0 && (q == nullptr || k == nullptr || v == nullptr || dout == nullptr || dq == nullptr || dk_out == nullptr ||
                dv_out == nullptr))
    return DP_EINVAL;
  if (dld != nullptr && ld == nullptr) return DP_EINVAL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dout, 16) || !aligned(dq, 16) ||
      !aligned(dk_out, 16) || !aligned(dv_out, 16) || !aligned(h0, 16) || !aligned(dfinal, 16) || !aligned(dh0, 16) ||
      !aligned(ld, 4) || !aligned(dld, 4) || !aligned(cu, 4))
    return DP_EINVAL;
  dp::LaArgs a{};
  int single = 0;
  plan_bwd(s, &a.geo, &single);
  if ((rc = check_grid(s, a.geo)) != DP_OK) return rc;
  const LaWs w = layout(s, a.geo, single, true);
  if (w.total > 0 && (ws == nullptr || wsb < w.total || !aligned(ws, kWsAlign))) return DP_EWORKSPACE;
  const LaBytes n(s, elem, elem, (flags & DP_LA_HEAD_DECAY) != 0);
  if (!dp::outputs_apart(
          {{dq, n.qk}, {dk_out, n.qk}, {dv_out, n.v}, {dld, n.ld}, {dh0, n.state}, {ws, w.total}},
          {{q, n.qk}, {k, n.qk}, {v, n.v}, {dout, n.v}, {ld, n.ld}, {h0, n.state}, {dfinal, n.state}, {cu, n.cu}}))
    return DP_EINVAL;
  char* b = static_cast<char*>(ws);
  auto f = [&](size_t at) { return reinterpret_cast<float*>(b + at); };
  int* tab = s.packed ? reinterpret_cast<int*>(b + w.tab) : nullptr;
  const bool group = Hk < H;
  a.q = q;
  a.k = k;
  a.v = v;
  a.dout = dout;
  a.ld = ld;
  a.h0 = h0;
  a.dfinal = dfinal;
  a.dq = group ? f(w.pq) : dq;
  a.dk = group ? f(w.pk) : dk_out;
  a.dv = dv_out;
  a.dld = dld;
  // the decays' gradient starts from <h0, dh0>
  a.dh0 = dh0 == nullptr && dld != nullptr && h0 != nullptr ? f(w.dh0) : dh0;
  a.st = f(w.st);
  a.rt = f(w.rt);
  a.sdec = f(w.sdec);
  a.rdec = f(w.rdec);
  a.xq = dld != nullptr ? reinterpret_cast<float2*>(b + w.xq) : nullptr;
  a.xk = dld != nullptr ? reinterpret_cast<float2*>(b + w.xk) : nullptr;
  a.ldpart = f(w.ldpart);
  a.geo.cu = cu;
  a.geo.tab = tab;
  a.geo.order = s.packed ? reinterpret_cast<const int*>(b + w.order) : nullptr;
  a.H = H;
  a.Hk = Hk;
  a.ld_head = (flags & DP_LA_HEAD_DECAY) != 0;
  a.qk_f32 = group || elem == 4;
  a.sum_in_walk = !single && sum_in_walk(s, a.geo, true);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = front(elem, s, a, single, 2, st);
  if (e == hipSuccess) e = stage(elem, dp::kLaBwd, a, dk, dv, 0, st);
  if (e == hipSuccess && dld != nullptr) {
    const dim3 grid((unsigned)(a.geo.nwork * H));
    if (elem == 4)
      hipLaunchKernelGGL((dp::dp_la_dld_kernel<dp::LaOp<float>::C>), grid, dim3(dp::kDldThreads), 0, st, a, dk * dv);
    else
      hipLaunchKernelGGL((dp::dp_la_dld_kernel<dp::LaOp<dp::bf16_t>::C>), grid, dim3(dp::kDldThreads), 0, st, a, dk * dv);
    e = hipGetLastError();
  }
  const bool sums = dld != nullptr && a.ld_head;
  if (e == hipSuccess && ((group && s.rows() > 0) || sums || (s.packed && L > 0))) {
    const long long n4 = s.rows() * Hk * dk / 4, blocks = (n4 + 255) / 256;
    const int nq = group ? (int)(blocks < 2048 ? blocks : 2048) : 0, nl = sums ? H : 0, nz = s.packed && L > 0 ? 256 : 0;
    const dim3 grid((unsigned)(2 * nq + nl + nz));
    if (elem == 4)
      hipLaunchKernelGGL((dp::dp_la_finish_kernel<float>), grid, dim3(256), 0, st, a, dq, dk_out, dk, dv, s.rows(), nq, nl);
    else
      hipLaunchKernelGGL((dp::dp_la_finish_kernel<dp::bf16_t>), grid, dim3(256), 0, st, a, dq, dk_out, dk, dv, s.rows(), nq, nl);
    e = hipGetLastError();
  }
  return status(e);
}

int la_ws(int B, int H, int Hk, int L, int dk, int dv, int packed, bool bwd, size_t* bytes) {
  if (bytes == nullptr) return DP_EINVAL;
  const LaShape s{B, H, Hk, L, dk, dv, packed != 0};
  int rc = check(s);
  if (rc != DP_OK) return rc;
  dp::LaGeo g{};
  int single = 0;
  if (bwd) plan_bwd(s, &g, &single);
  else plan_fwd(s, &g, &single);
  if ((rc = check_grid(s, g)) != DP_OK) return rc;
  *bytes = layout(s, g, single, bwd).total;
  return DP_OK;
}

// Value columns per decode workgroup: the whole width where rows and heads alone
// give every CU a workgroup or two, else narrower ones (16 at least: 64-byte
// segments of a state row).
int decode_cw(long long bh, int dv) {
  int cw = dv;
  while (cw > 16 && bh * (dv / cw) < 512) cw /= 2;
  return cw;
}

template <typename T, int DK, int CW>
hipError_t decode_launch(const dp::LaDecodeArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((dp::dp_la_decode_kernel<T, DK, CW>), dim3((unsigned)((long long)a.B * a.H * (a.dv / CW))),
                     dim3(dp::la_decode_threads(DK, CW)), 0, st, a);
  return hipGetLastError();
}
template <typename T, int DK>
hipError_t decode_dk(const dp::LaDecodeArgs& a, hipStream_t st) {
  switch (decode_cw((long long)a.B * a.H, a.dv)) {
    case 16: return decode_launch<T, DK, 16>(a, st);
    case 32: return decode_launch<T, DK, 32>(a, st);
    case 64: return decode_launch<T, DK, 64>(a, st);
    default: return decode_launch<T, DK, 128>(a, st);
  }
}

template <typename T>
int la_decode(const void* q, const void* k, const void* v, const float* ld, const int* slots, int B, int H, int Hk,
              int nslots, int dk, int dv, void* out, float* state, int flags, dp_stream stream) {
  if (B <= 0 || H <= 0 || Hk <= 0 || Hk > H || H % Hk != 0 || nslots <= 0 || dk <= 0 || dv <= 0) return DP_EINVAL;
  if ((flags & ~(DP_OUT_F32 | DP_LA_HEAD_DECAY)) != 0) return DP_EINVAL;
  if ((flags & DP_LA_HEAD_DECAY) != 0 && ld == nullptr) return DP_EINVAL;
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr || state == nullptr) return DP_EINVAL;
  if (slots == nullptr && B > nslots) return DP_EINVAL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(state, 16) || !aligned(out, 4) ||
      !aligned(ld, 4) || !aligned(slots, 4))
    return DP_EINVAL;
  if (!dim_ok(dk) || !dim_ok(dv)) return DP_ENOTSUP;
  // a launch has less than 2^32 threads: 256 at most per row and head where those are many
  if (H > 65535 || (long long)B * H > UINT_MAX / 256) return DP_ENOTSUP;
  const LaShape s{B, H, Hk, B, dk, dv, 1};  // B tokens
  const LaBytes n(s, (int)sizeof(T), (flags & DP_OUT_F32) != 0 ? 4 : (int)sizeof(T), (flags & DP_LA_HEAD_DECAY) != 0);
  if (!dp::outputs_apart({{out, n.out}, {state, (size_t)nslots * H * dk * dv * 4}},
                         {{q, n.qk}, {k, n.qk}, {v, n.v}, {ld, n.ld}, {slots, (size_t)B * 4}}))
    return DP_EINVAL;
  const dp::LaDecodeArgs a{q, k, v, ld, slots, out, state, B, H, Hk, nslots, dv, (flags & DP_LA_HEAD_DECAY) != 0,
                           (flags & DP_OUT_F32) != 0};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  switch (dk) {
    case 16: return status(decode_dk<T, 16>(a, st));
    case 32: return status(decode_dk<T, 32>(a, st));
    case 64: return status(decode_dk<T, 64>(a, st));
    default: return status(decode_dk<T, 128>(a, st));
  }
}

}  // namespace

extern "C" {

int dp_la_fwd_workspace_size(int B, int H, int Hk, int L, int dk, int dv, int packed, size_t* bytes) {
  return la_ws(B, H, Hk, L, dk, dv, packed, false, bytes);
}
int dp_la_bwd_workspace_size(int B, int H, int Hk, int L, int dk, int dv, int packed, size_t* bytes) {
  return la_ws(B, H, Hk, L, dk, dv, packed, true, bytes);
}

int dp_la_fwd_f32(const float* q, const float* k, const float* v, const float* ld, const int* cu_seqlens, int B, int H,
                  int Hk, int L, int dk, int dv, float* out, float* final_state, const float* h0, void* workspace,
                  size_t workspace_bytes, int flags, dp_stream stream) {
  return la_fwd(4, q, k, v, ld, cu_seqlens, B, H, Hk, L, dk, dv, out, final_state, h0, workspace, workspace_bytes, flags,
                stream);
}
int dp_la_fwd_bf16(const void* q, const void* k, const void* v, const float* ld, const int* cu_seqlens, int B, int H,
                   int Hk, int L, int dk, int dv, void* out, float* final_state, const float* h0, void* workspace,
                   size_t workspace_bytes, int flags, dp_stream stream) {
  return la_fwd(2, q, k, v, ld, cu_seqlens, B, H, Hk, L, dk, dv, out, final_state, h0, workspace, workspace_bytes, flags,
                stream);
}

int dp_la_bwd_f32(const float* q, const float* k, const float* v, const float* ld, const int* cu_seqlens,
                  const float* h0, const float* dout, const float* dfinal, int B, int H, int Hk, int L, int dk, int dv,
                  float* dq, float* dk_out, float* dv_out, float* dld, float* dh0, void* workspace,
                  size_t workspace_bytes, int flags, dp_stream stream) {
  return la_bwd(4, q, k, v, ld, cu_seqlens, h0, dout, dfinal, B, H, Hk, L, dk, dv, dq, dk_out, dv_out, dld, dh0,
                workspace, workspace_bytes, flags, stream);
}
int dp_la_bwd_bf16(const void* q, const void* k, const void* v, const float* ld, const int* cu_seqlens,
                   const float* h0, const void* dout, const float* dfinal, int B, int H, int Hk, int L, int dk, int dv,
                   void* dq, void* dk_out, void* dv_out, float* dld, float* dh0, void* workspace,
                   size_t workspace_bytes, int flags, dp_stream stream) {
  return la_bwd(2, q, k, v, ld, cu_seqlens, h0, dout, dfinal, B, H, Hk, L, dk, dv, dq, dk_out, dv_out, dld, dh0,
                workspace, workspace_bytes, flags, stream);
}

int dp_la_decode_f32(const float* q, const float* k, const float* v, const float* ld, const int* slots, int B, int H,
                     int Hk, int nslots, int dk, int dv, float* out, float* state, int flags, dp_stream stream) {
  return la_decode<float>(q, k, v, ld, slots, B, H, Hk, nslots, dk, dv, out, state, flags, stream);
}
int dp_la_decode_bf16(const void* q, const void* k, const void* v, const float* ld, const int* slots, int B, int H,
                      int Hk, int nslots, int dk, int dv, void* out, float* state, int flags, dp_stream stream) {
  return la_decode<dp::bf16_t>(q, k, v, ld, slots, B, H, Hk, nslots, dk, dv, out, state, flags, stream);
}

}  // extern "C"
