// Norms before and after a block, fused with its gate and residual scale.
//
//   b_t = y_t / rms(y_t) (.) w_post      (y_t itself without w_post)
//   o_t = res_scale * x_t + g_t (.) b_t  (x_t itself without y)
//   n_t = o_t / rms(o_t) (.) w_next,     rms(v) = sqrt(mean v^2 + eps)
//
// The arithmetic is a few operations per value read, so HBM bounds it: the
// row is read once, kept in registers over both norms and written once.  All
// sums and statistics are FP32; o and n are each rounded once, n from the
// unrounded o.
//
// 16384 x 4096, BF16 rows: forward 96 us (537 MB at 5.6 TB/s; a copy of 4 GiB
// reaches 6.24), backward 149 + 5 us (806 MB at 5.2 TB/s).  One row of 2048:
// 2.9 us, the latency of a load, two reductions and a store.

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "internal.h"
#include "rows.h"

namespace moe {

namespace {

enum YKind { Y_NONE = 0, Y_BF16 = 1, Y_F32 = 2 };

struct NormArgs {
  int T, H, gate_kind;
  float a, eps, inv_h;
  float sq_in, sq_out;               // row sums of squares, see squares_of
  long long xs, ys;                  // elements between rows
  const void *x, *y, *wp, *wn, *gate;
  void *out, *n;                     // forward
  const void *go, *gn;               // backward
  void *dx, *dy, *dgate;
  float* part;                       // [3][parts][H] column sums
  int parts;
};

// Eight elements per vector; thread `tid` of the NT that share a row owns
// vectors tid, tid + NT, ... (VEC), or single elements tid, tid + NT, ...
// where a row's start or length is no multiple of 16 bytes.
template <int NT, bool VEC>
__device__ __forceinline__ int column(int v, int i, int tid) {
  return VEC ? (v * NT + tid) * 8 + i : (v * 8 + i) * NT + tid;
}

// Eight elements of a row as stored.  A thread past the row's end reads its
// first columns instead and has them cleared by `unpack`: loads without a
// branch of their own are all in flight before the first one is waited for.
template <bool F32, bool VEC> struct Row {
  Raw8<F32> raw;
};
template <bool F32> struct Row<F32, false> {
  uint32_t raw[8];
};

template <bool F32, int NT, bool VEC>
__device__ __forceinline__ Row<F32, VEC> fetch(const void* p, size_t base, int v, int tid, int H) {
  Row<F32, VEC> r;
  if constexpr (VEC) {
    const int c = column<NT, true>(v, 0, tid);
    const size_t at = base + (c < H ? c : 0);
    if constexpr (F32) {
      const float* q = reinterpret_cast<const float*>(p) + at;
      r.raw.a[0] = load16(q);
      r.raw.a[1] = load16(q + 4);
    } else {
      r.raw.a = load16(reinterpret_cast<const uint16_t*>(p) + at);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<NT, false>(v, i, tid);
      const size_t at = base + (c < H ? c : 0);
      if constexpr (F32) r.raw[i] = reinterpret_cast<const uint32_t*>(p)[at];
      else r.raw[i] = reinterpret_cast<const uint16_t*>(p)[at];
    }
  }
  return r;
}

template <bool F32, int NT, bool VEC>
__device__ __forceinline__ void unpack(float (&f)[8], const Row<F32, VEC>& r, int v, int tid,
                                       int H) {
  if constexpr (VEC) {
    const uint32_t keep = column<NT, true>(v, 0, tid) < H ? 0xffffffffu : 0u;
    Raw8<F32> w = r.raw;
    if constexpr (F32) w.a[0] &= keep, w.a[1] &= keep;
    else w.a &= keep;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = w.get(i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = column<NT, false>(v, i, tid) < H ? r.raw[i] : 0u;
      f[i] = __uint_as_float(F32 ? w : w << 16);
    }
  }
}

template <bool F32, int NT, bool VEC, int V>
__device__ __forceinline__ void fetch_all(Row<F32, VEC> (&r)[V], const void* p, size_t base, int tid,
                                          int H) {
#pragma unroll
  for (int v = 0; v < V; ++v) r[v] = fetch<F32, NT, VEC>(p, base, v, tid, H);
}

template <bool F32, int NT, bool VEC, int V>
__device__ __forceinline__ void unpack_all(float (&f)[V][8], const Row<F32, VEC> (&r)[V], int tid,
                                           int H) {
#pragma unroll
  for (int v = 0; v < V; ++v) unpack<F32, NT, VEC>(f[v], r[v], v, tid, H);
}

template <bool F32, int NT, bool VEC, bool PAST = false>
__device__ __forceinline__ void store_row(const float (&r)[8], void* p, size_t base, int v, int tid,
                                          int H) {
  if constexpr (VEC) {
    const int c = column<NT, true>(v, 0, tid);
    if (c < H) store8<F32, PAST>(p, base + c, r);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<NT, false>(v, i, tid);
      if (c < H) store1<F32>(p, base + c, r[i]);
    }
  }
}

// Sums of M values over the NT threads of a row.  One barrier: the next call
// writes the other half of `lds`, and a half is written again only after the
// barrier of the call between.
template <int NT, int M>
__device__ __forceinline__ void row_sums(float (&s)[M], float* lds, int& half) {
#pragma unroll
  for (int m = 0; m < M; ++m) s[m] = wave_sum(s[m]);
  if constexpr (NT > kWave) {
    constexpr int W = NT / kWave;
    float* p = lds + half * (W * 4);
    const int w = wave_in_block();
    if ((threadIdx.x & (kWave - 1)) == 0) {
#pragma unroll
      for (int m = 0; m < M; ++m) p[w * 4 + m] = s[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) {
      s[m] = 0.0f;
#pragma unroll
      for (int q = 0; q < W; ++q) s[m] += p[q * 4 + m];
    }
    half ^= 1;
  }
}

// This thread's part of a row's sum of squares, of the values times sq_in = 2^-k
// with 4^k >= H: it overflows no sooner than the mean square itself, which is
// the row's sum times sq_out = 4^k / H.  Powers of two change no bits: the sums
// differ from unscaled ones only where either leaves the normal range.
template <int V>
__device__ __forceinline__ float squares_of(const NormArgs& a, const float (&f)[V][8]) {
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = f[v][i] * a.sq_in;
      s = fmaf(q, q, s);
    }
  return s;
}

__device__ __forceinline__ float inv_rms(const NormArgs& a, float squares) {
  return rsqrtf(fmaf(squares, a.sq_out, a.eps));
}

template <bool XF, int Y, int NT, int V, bool VEC>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void block_norm_kernel(NormArgs a) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;   // rows per workgroup
  constexpr bool YF = Y == Y_F32;
  __shared__ float lds[NT > kWave ? 2 * (NT / kWave) * 4 : 1];
  const int tid = NT < 256 ? threadIdx.x % NT : threadIdx.x;
  const bool gate_row = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL;
  int half = 0;
  for (long long t = (long long)blockIdx.x * kRows + (NT < 256 ? wave_in_block() : 0); t < a.T;
       t += (long long)gridDim.x * kRows) {
    const size_t row = (size_t)t * a.H;
    Row<XF, VEC> xr[V], gr[V], pr[V], nr[V];
    Row<YF, VEC> yr[V];
    float gt = 1.0f;
    fetch_all<XF, NT, VEC>(xr, a.x, (size_t)t * a.xs, tid, a.H);
    if constexpr (Y != Y_NONE) {
      fetch_all<YF, NT, VEC>(yr, a.y, (size_t)t * a.ys, tid, a.H);
      if (gate_row)
        fetch_all<XF, NT, VEC>(gr, a.gate, a.gate_kind == MOE_GATE_FULL ? row : 0, tid, a.H);
      if (a.gate_kind == MOE_GATE_TOKEN) gt = reinterpret_cast<const float*>(a.gate)[t];
      if (a.wp) fetch_all<XF, NT, VEC>(pr, a.wp, 0, tid, a.H);
    }
    if (a.wn) fetch_all<XF, NT, VEC>(nr, a.wn, 0, tid, a.H);
    float o[V][8];
    unpack_all<XF, NT, VEC>(o, xr, tid, a.H);
    if constexpr (Y != Y_NONE) {
      float y[V][8], w[V][8];
      unpack_all<YF, NT, VEC>(y, yr, tid, a.H);
      if (a.wp) {
        float s[1] = {squares_of<V>(a, y)};
        row_sums<NT, 1>(s, lds, half);
        const float r = inv_rms(a, s[0]);
        unpack_all<XF, NT, VEC>(w, pr, tid, a.H);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) y[v][i] = y[v][i] * r * w[v][i];
      }
      if (gate_row) {
        unpack_all<XF, NT, VEC>(w, gr, tid, a.H);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) y[v][i] *= w[v][i];
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[v][i] = fmaf(a.a, o[v][i], y[v][i] * gt);
        store_row<XF, NT, VEC, true>(o[v], a.out, row, v, tid, a.H);
      }
    }
    if (a.wn) {
      float s[1] = {squares_of<V>(a, o)}, w[V][8];
      row_sums<NT, 1>(s, lds, half);
      const float r = inv_rms(a, s[0]);
      unpack_all<XF, NT, VEC>(w, nr, tid, a.H);
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[v][i] = o[v][i] * r * w[v][i];
        store_row<XF, NT, VEC, true>(w[v], a.n, row, v, tid, a.H);
      }
    }
  }
}

// Threads of a workgroup of the backward pass: one row, or as many rows as
// wavefronts, whose column sums then meet in 32 KB of LDS.
__host__ __device__ constexpr int back_threads(int nt, int v) { return nt == kWave ? 1024 / v : nt; }

// The backward pass, with x the stored o:
//   D  = do + r (w_next (.) dn - o c),  c = r^2/H <w_next (.) dn, o>   r = 1/rms(o)
//   dx = res_scale D,   q = g (.) D,   dg = D (.) b
//   dy = r (w_post (.) q - y c),        c = r^2/H <w_post (.) q, y>    r = 1/rms(y)
//   dw_next = sum_t dn o r,  dw_post = sum_t q y r
// c is about 1 / rms, as r is, and formed from the product with the row, which
// is about rms, one r after the other: r^3 alone would leave FP32's range for
// rows of 1e13 and of 1e-13.
// The three sums of squares and products that D needs come from one
// reduction over the row, the product that dy (and a token's gate) needs from
// a second one.  A workgroup walks rows with a fixed stride and keeps its
// columns' sums over them in registers; a second kernel adds the workgroups'
// sums in order, so equal inputs give equal bits.
template <bool XF, int Y, int NT, int V, bool VEC>
__global__ __launch_bounds__(back_threads(NT, V)) void block_norm_back_kernel(NormArgs a) {
  constexpr int kRows = back_threads(NT, V) / NT;
  constexpr bool YF = Y == Y_F32;
  __shared__ float lds[NT > kWave ? 2 * (NT / kWave) * 4 : 1];
  const int tid = NT == kWave ? threadIdx.x % NT : threadIdx.x;
  const int sub = NT == kWave ? wave_in_block() : 0;
  int half = 0;
  Row<XF, VEC> wn[V], wp[V], gc[V];
  float swn[V][8] = {}, swp[V][8] = {}, sg[V][8] = {};
  if (a.wn) fetch_all<XF, NT, VEC>(wn, a.wn, 0, tid, a.H);
  if constexpr (Y != Y_NONE) {
    if (a.wp) fetch_all<XF, NT, VEC>(wp, a.wp, 0, tid, a.H);
    if (a.gate_kind == MOE_GATE_CHANNEL) fetch_all<XF, NT, VEC>(gc, a.gate, 0, tid, a.H);
  }
  for (long long t = (long long)blockIdx.x * kRows + sub; t < a.T; t += (long long)gridDim.x * kRows) {
    const size_t row = (size_t)t * a.H;
    Row<XF, VEC> dr[V], orow[V], gr[V];
    Row<YF, VEC> yr[V];
    float gt = 1.0f;
    if (a.go) fetch_all<XF, NT, VEC>(dr, a.go, row, tid, a.H);
    if (a.wn) {
      fetch_all<XF, NT, VEC>(orow, a.x, (size_t)t * a.xs, tid, a.H);
      fetch_all<XF, NT, VEC>(gr, a.gn, row, tid, a.H);
    }
    if constexpr (Y != Y_NONE) {
      fetch_all<YF, NT, VEC>(yr, a.y, (size_t)t * a.ys, tid, a.H);
      if (a.gate_kind == MOE_GATE_FULL) fetch_all<XF, NT, VEC>(gc, a.gate, row, tid, a.H);
      if (a.gate_kind == MOE_GATE_TOKEN) gt = reinterpret_cast<const float*>(a.gate)[t];
    }
    float d[V][8] = {}, y[V][8];
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (a.go) unpack_all<XF, NT, VEC>(d, dr, tid, a.H);
    if constexpr (Y != Y_NONE) {
      unpack_all<YF, NT, VEC>(y, yr, tid, a.H);
      s[2] = squares_of<V>(a, y);
    }
    if (a.wn) {
      float o[V][8], g[V][8], w[V][8];
      unpack_all<XF, NT, VEC>(o, orow, tid, a.H);
      unpack_all<XF, NT, VEC>(g, gr, tid, a.H);
      unpack_all<XF, NT, VEC>(w, wn, tid, a.H);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[1] = fmaf(w[v][i] * g[v][i], o[v][i], s[1]);
      s[0] = squares_of<V>(a, o);
      row_sums<NT, 3>(s, lds, half);
      const float r = inv_rms(a, s[0]);
      const float c = r * (r * (s[1] * a.inv_h));
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[v][i] = fmaf(r, fmaf(w[v][i], g[v][i], -(o[v][i] * c)), d[v][i]);
          swn[v][i] = fmaf(g[v][i] * o[v][i], r, swn[v][i]);
        }
    } else if (Y != Y_NONE && a.wp) {
      row_sums<NT, 3>(s, lds, half);
    }
    const float scale = Y != Y_NONE ? a.a : 1.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = scale * d[v][i];
      store_row<XF, NT, VEC, true>(w, a.dx, row, v, tid, a.H);
    }
    if constexpr (Y != Y_NONE) {
      const float ry = a.wp ? inv_rms(a, s[2]) : 1.0f;
      const bool gate_row = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL;
      float w[V][8], g[V][8];
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[v][i] = 1.0f, g[v][i] = gt;
      if (a.wp) unpack_all<XF, NT, VEC>(w, wp, tid, a.H);
      if (gate_row) unpack_all<XF, NT, VEC>(g, gc, tid, a.H);
      // u = <q w_post, y>; a token's gate enters as a factor of it
      float u[1] = {0.0f};
      if (a.wp || a.gate_kind == MOE_GATE_TOKEN) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            u[0] = fmaf(d[v][i] * (gate_row ? g[v][i] : 1.0f) * w[v][i], y[v][i], u[0]);
        row_sums<NT, 1>(u, lds, half);
        if (a.gate_kind == MOE_GATE_TOKEN && tid == 0)
          reinterpret_cast<float*>(a.dgate)[t] = ry * u[0];
      }
      const float c = a.wp ? ry * (ry * (gt * u[0] * a.inv_h)) : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float dg[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float q = d[v][i] * g[v][i], yn = y[v][i] * ry;
          dg[i] = d[v][i] * (yn * w[v][i]);
          swp[v][i] = fmaf(q, yn, swp[v][i]);
          sg[v][i] += dg[i];
          // without w_post y itself has no part in dy: an infinity in it would
          y[v][i] = a.wp ? ry * fmaf(w[v][i], q, -(y[v][i] * c)) : q;
        }
        if (a.gate_kind == MOE_GATE_FULL) store_row<XF, NT, VEC>(dg, a.dgate, row, v, tid, a.H);
        store_row<YF, NT, VEC, true>(y[v], a.dy, row, v, tid, a.H);
      }
    }
  }
  // this workgroup's sums: one row of each plane
  const size_t at = (size_t)blockIdx.x * a.H, plane = (size_t)a.parts * a.H;
  auto join = [&](float (&sum)[V][8], float* dst) {
    if constexpr (kRows == 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) store_row<true, NT, VEC>(sum[v], dst, at, v, tid, a.H);
    } else {
      __shared__ float cols[kRows][NT * 8 * V];
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) cols[sub][column<NT, VEC>(v, i, tid)] = sum[v][i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.H; c += back_threads(NT, V)) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += cols[r][c];
        dst[at + c] = s;
      }
    }
  };
  if (a.wn) join(swn, a.part);
  if constexpr (Y != Y_NONE) {
    if (a.wp) join(swp, a.part + plane);
    if (a.gate_kind == MOE_GATE_CHANNEL) join(sg, a.part + 2 * plane);
  }
}

// Column sums of the workgroups' partial sums, in order: plane blockIdx.y of
// part [3][parts][H] -> its gradient.  64 columns per workgroup, the parts
// split over 16 wavefronts.
constexpr int kSumWaves = 16;

struct SumArgs {
  const float* part;
  int parts, H;
  void* dst[3];
};

__global__ __launch_bounds__(kWave* kSumWaves) void column_sums_kernel(SumArgs a) {
  __shared__ float lds[kSumWaves][kWave];
  void* dst = a.dst[blockIdx.y];
  if (!dst) return;
  const int c = blockIdx.x * kWave + (threadIdx.x & (kWave - 1)), w = wave_in_block();
  const float* p = a.part + (size_t)blockIdx.y * a.parts * a.H;
  float s = 0.0f;
  if (c < a.H) {
#pragma unroll 8
    for (int i = w; i < a.parts; i += kSumWaves) s += p[(size_t)i * a.H + c];
  }
  lds[w][threadIdx.x & (kWave - 1)] = s;
  __syncthreads();
  if (w == 0 && c < a.H) {
    s = 0.0f;
#pragma unroll
    for (int q = 0; q < kSumWaves; ++q) s += lds[q][threadIdx.x];
    reinterpret_cast<float*>(dst)[c] = s;
  }
}

// One workgroup for each row, or for four short ones (16384 x 4096, y and a
// channel gate: 94.9 us, with two workgroups per CU that walk the rows 92.8;
// 16384 x 2048: 59 us and 65).  A launch counts its threads in 32 bits, so those
// of a larger batch walk rows too.
constexpr int kMaxGroups = 1 << 20;

struct Shape {
  int nt, v;
};

// Threads per row and vectors per thread: few threads with much in flight
// each, several rows a CU.  BF16, in us:
//   20000 x 256     64 x 1:  9.7    256 x 1: 21.4    1024 x 1: 94.6
//   16384 x 2048   256 x 1: 57.5    256 x 2: 58.3    1024 x 1: 104.5
//   16384 x 4096   256 x 2: 94.6   1024 x 1: 129.3
//    4096 x 7168   256 x 4: 43.6    512 x 2: 46.1    1024 x 1: 47.8   1024 x 2: 69.4
// but 1024 x 1 for rows read by element (1000 x 8191: 19.2, 256 x 4: 26.1) and
// for fewer rows than CUs (64 x 7168: 4.1, 256 x 4: 4.3).  Only 1024 x 2 spills
// registers, read by element with y (85 to 117 of them).
Shape shape_of(int H, int T, bool vec) {
  if (H <= 512) return {64, 1};
  if (H <= 2048) return {256, 1};
  if (H <= 4096) return {256, 2};
  if (H <= 8192) return vec && T > device_num_cus() ? Shape{256, 4} : Shape{1024, 1};
  return {1024, 2};
}

// The backward pass keeps three column sums beside the row.  In us:
//   20000 x 256     64 x 1: 21     256 x 1: 68
//    4096 x 2048   256 x 1: 33     256 x 2: 36
//   16384 x 4096   256 x 2: 157    512 x 2: 235
//     515 x 7168   512 x 2: 26     512 x 4: 182 (registers spilled to scratch)
// 64 x 1 (128 registers a thread at 1024 threads) spills 5 to 30 of them with y,
// and by element 83 to 103; 512 x 2 spills 17 in FP32 with y, and by element 139
// to 172; 512 x 4 spills 226 to 331, and without y up to 59 or, by element, 279.
Shape back_shape_of(int H) {
  if (H <= 512) return {64, 1};
  if (H <= 2048) return {256, 1};
  if (H <= 4096) return {256, 2};
  if (H <= 8192) return {512, 2};
  return {512, 4};
}

bool vectors_ok(const moe_block& B, std::initializer_list<const void*> rows) {
  if (B.H % 8 || (B.T > 1 && (B.x_stride % 8 || B.y_stride % 8))) return false;
  for (const void* p : rows)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
  return true;
}

NormArgs args_of(const moe_block& B) {
  NormArgs a{};
  a.T = B.T;
  a.H = B.H;
  a.gate_kind = B.gate_kind;
  a.a = B.res_scale;
  a.eps = B.eps;
  a.inv_h = 1.0f / (float)B.H;
  int k = 0;
  while ((1 << 2 * k) < B.H) ++k;
  a.sq_in = std::ldexp(1.0f, -k);
  a.sq_out = std::ldexp(a.inv_h, 2 * k);
  a.xs = B.x_stride;
  a.ys = B.y_stride;
  a.x = B.x;
  a.y = B.y;
  a.wp = B.w_post;
  a.wn = B.w_next;
  a.gate = B.gate;
  return a;
}

template <bool XF, int Y, int NT, int V>
void launch_forward(const NormArgs& a, bool vec, unsigned grid, hipStream_t s) {
  const dim3 block(NT < 256 ? 256 : NT);
  if (vec) hipLaunchKernelGGL((block_norm_kernel<XF, Y, NT, V, true>), dim3(grid), block, 0, s, a);
  else hipLaunchKernelGGL((block_norm_kernel<XF, Y, NT, V, false>), dim3(grid), block, 0, s, a);
}

template <bool XF, int Y, int NT, int V>
void launch_back(const NormArgs& a, bool vec, unsigned grid, hipStream_t s) {
  const dim3 block(back_threads(NT, V));
  if (vec) hipLaunchKernelGGL((block_norm_back_kernel<XF, Y, NT, V, true>), dim3(grid), block, 0, s, a);
  else hipLaunchKernelGGL((block_norm_back_kernel<XF, Y, NT, V, false>), dim3(grid), block, 0, s, a);
}

template <bool BACK, bool XF, int Y>
void launch_typed(const NormArgs& a, Shape sh, bool vec, unsigned grid, hipStream_t s) {
  const int shape = sh.nt * 8 + sh.v;
  if constexpr (BACK) {
    switch (shape) {
      case 64 * 8 + 1: return launch_back<XF, Y, 64, 1>(a, vec, grid, s);
      case 256 * 8 + 1: return launch_back<XF, Y, 256, 1>(a, vec, grid, s);
      case 256 * 8 + 2: return launch_back<XF, Y, 256, 2>(a, vec, grid, s);
      case 512 * 8 + 2: return launch_back<XF, Y, 512, 2>(a, vec, grid, s);
      default: return launch_back<XF, Y, 512, 4>(a, vec, grid, s);
    }
  } else {
    switch (shape) {
      case 64 * 8 + 1: return launch_forward<XF, Y, 64, 1>(a, vec, grid, s);
      case 256 * 8 + 1: return launch_forward<XF, Y, 256, 1>(a, vec, grid, s);
      case 256 * 8 + 2: return launch_forward<XF, Y, 256, 2>(a, vec, grid, s);
      case 256 * 8 + 4: return launch_forward<XF, Y, 256, 4>(a, vec, grid, s);
      case 1024 * 8 + 1: return launch_forward<XF, Y, 1024, 1>(a, vec, grid, s);
      default: return launch_forward<XF, Y, 1024, 2>(a, vec, grid, s);
    }
  }
}

template <bool BACK>
void launch_any(const moe_block& B, const NormArgs& a, Shape sh, bool vec, unsigned grid,
                hipStream_t s) {
  if (B.x_dtype == MOE_DT_F32) {
    if (B.y) launch_typed<BACK, true, Y_F32>(a, sh, vec, grid, s);
    else launch_typed<BACK, true, Y_NONE>(a, sh, vec, grid, s);
  } else if (!B.y) {
    launch_typed<BACK, false, Y_NONE>(a, sh, vec, grid, s);
  } else if (B.y_dtype == MOE_DT_F32) {
    launch_typed<BACK, false, Y_F32>(a, sh, vec, grid, s);
  } else {
    launch_typed<BACK, false, Y_BF16>(a, sh, vec, grid, s);
  }
}

int rows_per_group(Shape sh) { return sh.nt < 256 ? 256 / sh.nt : 1; }

// Workgroups of the backward pass: enough to fill the CUs, few enough that
// their partial column sums stay small next to the rows (16384 x 4096 with one,
// two and four per CU: 206, 157 and 162 us; 515 x 7168: 26, 30 and 34; 20000 x
// 256: 21, 24 and 30).
int back_groups(int T, int H) {
  const Shape sh = back_shape_of(H);
  const int rows = back_threads(sh.nt, sh.v) / sh.nt;
  const int most = device_num_cus() * (sh.nt == 256 ? 2 : 1);
  return T > 0 ? std::min(most, (T - 1) / rows + 1) : 0;
}

}  // namespace

hipError_t launch_block_norm(const moe_block& B, void* out, void* n, hipStream_t s) {
  NormArgs a = args_of(B);
  a.out = out;
  a.n = n;
  const bool vec = vectors_ok(B, {B.x, B.y, B.w_post, B.w_next,
                                  B.gate_kind == MOE_GATE_TOKEN ? nullptr : B.gate, out, n});
  const Shape sh = shape_of(B.H, B.T, vec);
  const int rows = rows_per_group(sh);
  launch_any<false>(B, a, sh, vec, (unsigned)std::min(kMaxGroups, (B.T - 1) / rows + 1), s);
  return hipGetLastError();
}

size_t block_norm_backward_workspace(int T, int H) {
  return (size_t)3 * back_groups(T, H) * H * sizeof(float);
}

hipError_t launch_block_norm_backward(const moe_block& B, const void* go, const void* gn, void* dx,
                                      void* dy, void* dgate, float* dwp, float* dwn, float* part,
                                      hipStream_t s) {
  const Shape sh = back_shape_of(B.H);
  NormArgs a = args_of(B);
  a.go = go;
  a.gn = gn;
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.part = part;
  const int groups = back_groups(B.T, B.H);
  a.parts = groups;
  const bool token = B.gate_kind == MOE_GATE_TOKEN;
  if (groups > 0) {
    const bool vec = vectors_ok(B, {B.x, B.y, B.w_post, B.w_next, token ? nullptr : B.gate, go, gn,
                                    dx, dy, token ? nullptr : dgate, part});
    launch_any<true>(B, a, sh, vec, (unsigned)groups, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  SumArgs r{};
  r.part = part;
  r.parts = a.parts;
  r.H = B.H;
  r.dst[0] = dwn;
  r.dst[1] = dwp;
  r.dst[2] = B.gate_kind == MOE_GATE_CHANNEL ? dgate : nullptr;
  if (dwn || dwp || r.dst[2])
    hipLaunchKernelGGL(column_sums_kernel, dim3((B.H + kWave - 1) / kWave, 3),
                       dim3(kWave * kSumWaves), 0, s, r);
  return hipGetLastError();
}

}  // namespace moe
