// Router statistics and losses, and the router's gradient.
//
// For every sequence s with the n_s counting tokens t, p_t = softmax(scores_t):
//   c_se = routed slots of expert e,   f_se = E c_se / (k n_s)
//   P_se = mean_t p_te,   L_s = sum_e f_se P_se,   Z_s = mean_t lse(scores_t)^2
// and, c held constant (it is a count),
//   d scores_te = p_te / n_s (gL_s (f_se - <f_s, p_t>) + 2 gZ_s lse_t)
//                 + sum_{j: id_tj = e} w_tj (dw_tj - <w_t, dw_t>)
// the last term being the softmax over the selected scores (moe_topk_route).
//
// A row's arithmetic is a softmax over E <= 1024 values, so a group of 16, 32
// or 64 lanes takes a row with up to 16 values per lane: four rows per
// wavefront at the usual E, reductions of four DPP steps, each score read
// once.  65536 tokens x 256 experts, top-8, 24 sequences: 20 us for the rows
// (69 MB, 3.5 TB/s: one workgroup per CU, see block_rows_of) and 6 us for the
// partial sums; the gradient 36 us (141 MB, 3.9 TB/s).  32 tokens x 128 experts
// 4.1 us, the gradient of 333 tokens 4.6 us: a chain of loads and reductions.

#include <algorithm>

#include "internal.h"
#include "rows.h"

namespace moe {

namespace {

struct BalanceArgs {
  const float* scores;
  const int32_t* ids;
  const uint8_t* mask;      // nullable
  const int32_t* offsets;   // nullable: one sequence of all tokens
  int T, E, k, S;
  int block_rows;
  float* part_p;            // [slots][E]
  int32_t* part_c;          // [slots][E]
  float* part_z;            // [slots]
  int32_t* part_n;          // [slots]
  float* dots;              // [S][chunks]
  unsigned* arrived;        // [S]
  int32_t* counts;          // [S][E]
  int32_t* tokens;          // [S]
  float* loss;              // [S][2]
  const float* grad_loss;   // backward: [S][2] or null
  const float *wts, *grad_wts;   // [T][k] or null
  float* grad;              // [T][E]
};

// An id outside [0, E) is read as expert 0, as everywhere in the library.
__device__ __forceinline__ int expert_of(int id, int E) { return (unsigned)id < (unsigned)E ? id : 0; }

// Token bounds as the kernels read them: inside [0, T] whatever is stored.
__device__ __forceinline__ int bound(const BalanceArgs& a, int s) {
  if (!a.offsets) return s == 0 ? 0 : a.T;
  return max(0, min(a.T, a.offsets[s]));
}

// The last sequence that starts at or before token t (-1: none, S: t lies
// behind the last one).  Of sequences that start at the same token the last
// one is the one that is not empty.  By one lane:
__device__ __forceinline__ int sequence_of(const BalanceArgs& a, int t) {
  if (!a.offsets) return 0;
  int lo = 0, hi = a.S + 1;   // first index in [0, S + 1] whose start is past t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (bound(a, mid) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo - 1;
}

// and by a whole wavefront, 64 starts at a time.
__device__ __forceinline__ int sequence_of_wave(const BalanceArgs& a, int t) {
  if (!a.offsets) return 0;
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, n = a.S + 1;
  while (n > kWave) {
    const int stride = (n + kWave - 1) / kWave;
    const bool before = lane * stride < n && bound(a, min(lo + lane * stride, a.S)) <= t;
    const int c = __popcll(__ballot(before));
    if (c == 0) return lo - 1;
    lo += (c - 1) * stride;
    n = min(stride, n - (c - 1) * stride);
  }
  return lo - 1 + __popcll(__ballot(lane < n && bound(a, min(lo + lane, a.S)) <= t));
}

// Lane `li` of a group of LPR holds PER values of a row: vectors of four
// (VEC) or single values, strided over the group.
template <int LPR, int PER, bool VEC>
__device__ __forceinline__ int expert_at(int i, int li) {
  return VEC ? ((i >> 2) * LPR + li) * 4 + (i & 3) : i * LPR + li;
}

template <int LPR, int PER, bool VEC>
__device__ __forceinline__ void load_scores(float (&v)[PER], const BalanceArgs& a, int t, int li) {
  const float* row = a.scores + (size_t)t * a.E;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const int e = expert_at<LPR, PER, true>(i, li);
      const u32x4 w = load16(row + (e < a.E ? e : 0));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = __uint_as_float(w[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = expert_at<LPR, PER, false>(i, li);
      v[i] = row[e < a.E ? e : 0];
    }
  }
}

// v -> exp(v - max), 0 past E; returns the sum (0 if the row has no score, else
// at least 1 or NaN), the maximum by reference.  The difference is taken first:
// it is exact near the maximum and finite wherever the result is not 0, also
// for rows of the type's lowest value; 2^x is the hardware's, off by one unit
// in the last place.
template <int LPR, int PER, bool VEC>
__device__ __forceinline__ float exponentials(float (&v)[PER], float& m, int E, int li) {
  if (E < LPR * PER) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (expert_at<LPR, PER, VEC>(i, li) >= E) v[i] = -INFINITY;
  }
  m = v[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) m = fmaxf(m, v[i]);
  m = group_max<LPR>(m);
  const float base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = __builtin_amdgcn_exp2f((v[i] - base) * 1.44269504088896341f);
    s += v[i];
  }
  return group_sum<LPR>(s);
}

// log of a row's sum, which is at least 1.
__device__ __forceinline__ float log_of(float s) { return __builtin_amdgcn_logf(s) * 0.693147180559945309f; }

// 512 threads: 4.1 us for 32 tokens x 128 experts and 8.1 us for 2048, with 1024
// 4.5 and 9.2; 25.3 and 25.0 us for 65536 x 256.
constexpr int kBalanceBlock = 512;

// Loss of one sequence from its column sums (p and c of expert e in LDS) and
// its z sum and token count; every thread of the workgroup calls it.
__device__ __forceinline__ void finish_sequence(const BalanceArgs& a, int s, const float* p,
                                                const int32_t* c, float z, int n, float* red) {
  float sum = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    a.counts[(size_t)s * a.E + e] = c[e];
    sum = fmaf((float)c[e], p[e], sum);
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0f;
    for (int q = 0; q < (int)blockDim.x / kWave; ++q) sum += red[q];
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
    a.loss[2 * (size_t)s] = sum * inv * inv * ((float)a.E / (float)a.k);
    a.loss[2 * (size_t)s + 1] = z * inv;
    a.tokens[s] = n;
  }
  __syncthreads();
}

// One workgroup takes `block_rows` consecutive tokens, the part of each
// sequence among them on its own.  SINGLE: it takes all tokens and writes the
// results; else it writes the partial sums of block b and sequence s to slot
// b + s, which no other pair has, since both only grow along the tokens.
template <int LPR, int PER, bool VEC, bool SINGLE>
__global__ __launch_bounds__(kBalanceBlock) void balance_kernel(BalanceArgs a) {
  constexpr int kGroups = kBalanceBlock / LPR;
  constexpr int kWaves = kBalanceBlock / kWave;
  __shared__ float s_p[kWaves][LPR * PER];
  __shared__ int32_t s_c[LPR * PER];
  __shared__ float s_z[kWaves];
  __shared__ int32_t s_n[kWaves];
  __shared__ float s_red[kWaves];
  const int li = threadIdx.x % LPR, g = threadIdx.x / LPR;
  const int wave = wave_in_block(), lane = threadIdx.x & (kWave - 1);
  const int r0 = blockIdx.x * a.block_rows;
  const int r1 = min(a.T, r0 + a.block_rows);
  if constexpr (SINGLE) {
    // sequences without a token are met by no row
    for (int s = wave; s < a.S; s += kWaves) {
      if (bound(a, s + 1) > bound(a, s)) continue;
      for (int e = lane; e < a.E; e += kWave) a.counts[(size_t)s * a.E + e] = 0;
      if (lane == 0) a.tokens[s] = 0, a.loss[2 * s] = 0.0f, a.loss[2 * s + 1] = 0.0f;
    }
  }
  if constexpr (!SINGLE) {
    // for the workgroups of the next launch
    if (blockIdx.x == 0)
      for (int s = threadIdx.x; s < a.S; s += kBalanceBlock) a.arrived[s] = 0;
  }
  int r = r0;
  while (r < r1) {
    const int seq = sequence_of_wave(a, r);
    if (seq >= a.S) break;
    if (seq < 0) {
      r = max(r + 1, bound(a, 0));
      continue;
    }
    const int end = max(r + 1, min(r1, bound(a, seq + 1)));
    for (int e = threadIdx.x; e < LPR * PER; e += kBalanceBlock) s_c[e] = 0;
    __syncthreads();
    float acc[PER] = {}, z = 0.0f;
    int n = 0;
    for (int t = r + g; t < end; t += kGroups) {
      if (a.mask && !a.mask[t]) continue;
      float v[PER], m;
      load_scores<LPR, PER, VEC>(v, a, t, li);
      int id[64 / LPR];
#pragma unroll
      for (int q = 0; q < 64 / LPR; ++q) {
        if (LPR * q >= a.k) break;
        id[q] = a.ids[(size_t)t * a.k + min(li + LPR * q, a.k - 1)];
      }
      const float sum = exponentials<LPR, PER, VEC>(v, m, a.E, li);
      if (sum == 0.0f) continue;
      const float inv = __builtin_amdgcn_rcpf(sum);
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
      const float lse = m + log_of(sum);
      z = fmaf(lse, lse, z);
      ++n;
#pragma unroll
      for (int q = 0; q < 64 / LPR; ++q) {
        if (LPR * q >= a.k) break;
        if (li + LPR * q < a.k) atomicAdd(&s_c[expert_of(id[q], a.E)], 1);
      }
    }
    // the wavefront's groups, then the wavefronts
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if constexpr (LPR == 16) acc[i] += __shfl_xor(acc[i], 16, kWave);
      if constexpr (LPR <= 32) acc[i] += __shfl_xor(acc[i], 32, kWave);
      if (lane < LPR) s_p[wave][expert_at<LPR, PER, VEC>(i, li)] = acc[i];
    }
    z = li == 0 ? z : 0.0f;
    z = wave_sum(z);
    n = li == 0 ? n : 0;
    for (int off = kWave / 2; off > 0; off >>= 1) n += __shfl_xor(n, off, kWave);
    if (lane == 0) s_z[wave] = z, s_n[wave] = n;
    __syncthreads();
    z = 0.0f, n = 0;
    for (int w = 0; w < kWaves; ++w) z += s_z[w], n += s_n[w];
    const size_t slot = (size_t)blockIdx.x + seq;
    for (int e = threadIdx.x; e < a.E; e += kBalanceBlock) {
      float p = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) p += s_p[w][e];
      if constexpr (SINGLE) {
        s_p[0][e] = p;
      } else {
        a.part_p[slot * a.E + e] = p;
        a.part_c[slot * a.E + e] = s_c[e];
      }
    }
    if constexpr (SINGLE) {
      __syncthreads();
      finish_sequence(a, seq, s_p[0], s_c, z, n, s_red);
    } else {
      if (threadIdx.x == 0) a.part_z[slot] = z, a.part_n[slot] = n;
      __syncthreads();
    }
    r = end;
  }
}

// A workgroup adds the slots of one sequence for 64 experts, in order; the one
// that arrives last for its sequence adds the experts' terms of the loss, in
// order too, whichever it is.
__global__ __launch_bounds__(kBalanceBlock) void balance_finish_kernel(BalanceArgs a) {
  constexpr int kWaves = kBalanceBlock / kWave;
  __shared__ float s_p[kWaves][kWave];
  __shared__ int32_t s_c[kWaves][kWave];
  const int s = blockIdx.x, chunk = blockIdx.y, chunks = gridDim.y;
  const int lane = threadIdx.x & (kWave - 1), w = wave_in_block();
  const int first = bound(a, s), end = bound(a, s + 1);
  const int b0 = end > first ? first / a.block_rows : 0;
  const int b1 = end > first ? (end - 1) / a.block_rows + 1 : 0;
  const int e = chunk * kWave + lane;
  float p = 0.0f;
  int c = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int b = b0 + w; b < b1; b += kWaves) {
      p += a.part_p[((size_t)b + s) * a.E + e];
      c += a.part_c[((size_t)b + s) * a.E + e];
    }
  }
  s_p[w][lane] = p;
  s_c[w][lane] = c;
  __syncthreads();
  if (w != 0) return;
  p = 0.0f, c = 0;
#pragma unroll
  for (int q = 0; q < kWaves; ++q) p += s_p[q][lane], c += s_c[q][lane];
  if (e < a.E) a.counts[(size_t)s * a.E + e] = c;
  float dot = wave_sum((float)c * p);
  float z = 0.0f;
  int n = 0;
  for (int b = b0 + lane; b < b1; b += kWave) z += a.part_z[(size_t)b + s], n += a.part_n[(size_t)b + s];
  z = wave_sum(z);
  for (int off = kWave / 2; off > 0; off >>= 1) n += __shfl_xor(n, off, kWave);
  if (lane != 0) return;
  if (chunks > 1) {
    float* dots = a.dots + (size_t)s * chunks;
    __hip_atomic_store(dots + chunk, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__hip_atomic_fetch_add(a.arrived + s, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) != (unsigned)chunks - 1)
      return;
    dot = 0.0f;
    for (int q = 0; q < chunks; ++q)
      dot += __hip_atomic_load(dots + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
  a.loss[2 * (size_t)s] = dot * inv * inv * ((float)a.E / (float)a.k);
  a.loss[2 * (size_t)s + 1] = z * inv;
  a.tokens[s] = n;
}

// The gradient of the scores.  A group keeps f of the sequence it is in.  The
// k terms of the routing weights go to their experts through a row of LDS:
// ids that are distinct need one store each; if two slots of the token name
// one expert, one lane adds the terms in slot order.
constexpr int kBackBlock = 256;

template <int LPR, int PER, bool VEC>
__global__ __launch_bounds__(kBackBlock) void router_back_kernel(BalanceArgs a) {
  constexpr int kGroups = kBackBlock / LPR;
  __shared__ __align__(16) float s_row[kGroups][LPR * PER];
  const int li = threadIdx.x % LPR, g = threadIdx.x / LPR;
  float* srow = s_row[g];
  const int r0 = blockIdx.x * a.block_rows;
  const int r1 = min(a.T, r0 + a.block_rows);
  if (a.grad_wts) {
    for (int e = li; e < LPR * PER; e += LPR) srow[e] = 0.0f;
    wave_fence();
  }
  int seq = a.grad_loss ? sequence_of_wave(a, r0) : 0;
  int seq_end = -1;   // f is not loaded yet
  float f[PER], gl = 0.0f, gz = 0.0f;
  for (int t = r0 + g; t < r1; t += kGroups) {
    bool live = a.grad_loss != nullptr && !(a.mask && !a.mask[t]);
    float d[PER];
    if (live) load_scores<LPR, PER, VEC>(d, a, t, li);
    // the routed slots of the token, one a lane
    constexpr int kSlots = 64 / LPR;
    int id[kSlots];
    float w[kSlots], dw[kSlots];
    if (a.grad_wts) {
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        if (LPR * q >= a.k) break;
        const size_t at = (size_t)t * a.k + min(li + LPR * q, a.k - 1);
        id[q] = a.ids[at], w[q] = a.wts[at], dw[q] = a.grad_wts[at];
      }
    }
    if (live && t >= seq_end) {
      // usually the next sequence or the one after it
      if (seq < 0 || bound(a, min(seq + 1, a.S)) <= t) seq = sequence_of(a, t);
      seq_end = seq >= a.S ? a.T : bound(a, seq + 1);
      const int n = seq >= 0 && seq < a.S ? a.tokens[seq] : 0;
      const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
      gl = gz = 0.0f;
      if (n > 0) {
        gl = a.grad_loss[2 * (size_t)seq] * inv;
        gz = 2.0f * a.grad_loss[2 * (size_t)seq + 1] * inv;
      }
      const float scale = inv * ((float)a.E / (float)a.k);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = expert_at<LPR, PER, VEC>(i, li);
        f[i] = n > 0 && e < a.E ? (float)a.counts[(size_t)seq * a.E + e] * scale : 0.0f;
      }
    }
    live = live && seq >= 0 && seq < a.S;
    if (live) {
      float m;
      const float sum = exponentials<LPR, PER, VEC>(d, m, a.E, li);
      const float inv = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
      float fp = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        d[i] *= inv;
        fp = fmaf(f[i], d[i], fp);
      }
      fp = group_sum<LPR>(fp);
      const float lse = sum == 0.0f ? 0.0f : m + log_of(sum);
      const float base = fmaf(gz, lse, -(gl * fp));
#pragma unroll
      for (int i = 0; i < PER; ++i) d[i] *= fmaf(gl, f[i], base);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) d[i] = 0.0f;
    }
    if (a.grad_wts) {
      float dot = 0.0f;
      bool alone = true;
      const auto slots = [&](auto use) {
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
          if (LPR * q >= a.k) break;
          if (li + LPR * q < a.k) use(q);
        }
      };
      slots([&](int q) {
        id[q] = expert_of(id[q], a.E);
        dot = fmaf(w[q], dw[q], dot);
        // every slot writes its number to its expert's place; one that does
        // not find its own there shares the expert with another one
        srow[id[q]] = (float)(li + LPR * q);
      });
      dot = group_sum<LPR>(dot);
      wave_fence();
      slots([&](int q) { alone = alone && srow[id[q]] == (float)(li + LPR * q); });
      wave_fence();
      if (__ballot(!alone) == 0) {
        slots([&](int q) { srow[id[q]] = w[q] * (dw[q] - dot); });
      } else if (li == 0) {
        const size_t at = (size_t)t * a.k;
        for (int j = 0; j < a.k; ++j) srow[expert_of(a.ids[at + j], a.E)] = 0.0f;
        for (int j = 0; j < a.k; ++j)
          srow[expert_of(a.ids[at + j], a.E)] += a.wts[at + j] * (a.grad_wts[at + j] - dot);
      }
      wave_fence();
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
          const u32x4 r = *reinterpret_cast<const u32x4*>(srow + expert_at<LPR, PER, true>(i, li));
#pragma unroll
          for (int j = 0; j < 4; ++j) d[i + j] += __uint_as_float(r[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) d[i] += srow[expert_at<LPR, PER, false>(i, li)];
      }
      wave_fence();
      slots([&](int q) { srow[id[q]] = 0.0f; });
      wave_fence();
    }
    float* out = a.grad + (size_t)t * a.E;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const int e = expert_at<LPR, PER, true>(i, li);
        if (e < a.E)
          *reinterpret_cast<u32x4*>(out + e) =
              u32x4{__float_as_uint(d[i]), __float_as_uint(d[i + 1]), __float_as_uint(d[i + 2]),
                    __float_as_uint(d[i + 3])};
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = expert_at<LPR, PER, false>(i, li);
        if (e < a.E) out[e] = d[i];
      }
    }
  }
}

// Lanes per row by E (up to 16 values per lane).
int lanes_of(int E) { return E <= 256 ? 16 : E <= 512 ? 32 : 64; }

// Tokens per workgroup of the forward pass: whole rounds of its groups, and
// one workgroup per CU, whose partial sums then stay few (65536 x 256, 24
// sequences, 1024 threads: 25.0 us, with two and four per CU 29.5 and 38.0).
int block_rows_of(int T, int E) {
  const int round = kBalanceBlock / lanes_of(E);
  const int cus = device_num_cus();
  const int rounds = std::max(1, (int)(((long long)T + (long long)round * cus - 1) / ((long long)round * cus)));
  return rounds * round;
}

// All tokens in one workgroup and one launch: up to eight rounds of its
// groups (256 tokens x 128 experts: 7.2 us, in two launches 7.8; 512 tokens
// 10.8 and 8.2), and few sequences, which it takes one after the other.
bool single_block(int T, int E, int S) { return S <= 4 && T <= 8 * (kBalanceBlock / lanes_of(E)); }

int blocks_of(int T, int E) {
  const int rows = block_rows_of(T, E);
  return std::max(1, (int)(((long long)T + rows - 1) / rows));   // one clears the counters if there is no token
}

int chunks_of(int E) { return (E + kWave - 1) / kWave; }

size_t padded(size_t v) { return (v + 255) / 256 * 256; }

template <int LPR, int PER>
void launch_forward(const BalanceArgs& a, bool vec, bool single, unsigned grid, hipStream_t s) {
  const dim3 block(kBalanceBlock);
  if (single) {
    if (vec) hipLaunchKernelGGL((balance_kernel<LPR, PER, true, true>), dim3(1), block, 0, s, a);
    else hipLaunchKernelGGL((balance_kernel<LPR, PER, false, true>), dim3(1), block, 0, s, a);
  } else {
    if (vec) hipLaunchKernelGGL((balance_kernel<LPR, PER, true, false>), dim3(grid), block, 0, s, a);
    else hipLaunchKernelGGL((balance_kernel<LPR, PER, false, false>), dim3(grid), block, 0, s, a);
  }
}

template <int LPR, int PER>
void launch_backward(const BalanceArgs& a, bool vec, unsigned grid, hipStream_t s) {
  if (vec) hipLaunchKernelGGL((router_back_kernel<LPR, PER, true>), dim3(grid), dim3(kBackBlock), 0, s, a);
  else hipLaunchKernelGGL((router_back_kernel<LPR, PER, false>), dim3(grid), dim3(kBackBlock), 0, s, a);
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) {
  if (single_block(T, E, S)) return 0;
  const size_t slots = (size_t)blocks_of(T, E) + S;
  return 2 * padded(slots * E * 4) + 2 * padded(slots * 4) + padded((size_t)S * chunks_of(E) * 4) + padded((size_t)S * 4);
}

hipError_t launch_balance(const float* scores, const int32_t* ids, const uint8_t* mask,
                          const int32_t* offsets, int T, int E, int k, int S, int32_t* counts,
                          int32_t* tokens, float* loss, void* ws, hipStream_t s) {
  BalanceArgs a{};
  a.scores = scores;
  a.ids = ids;
  a.mask = mask;
  a.offsets = offsets;
  a.T = T;
  a.E = E;
  a.k = k;
  a.S = S;
  a.counts = counts;
  a.tokens = tokens;
  a.loss = loss;
  const bool vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(scores) & 15u) == 0;
  const bool single = single_block(T, E, S);
  a.block_rows = single ? std::max(T, 1) : block_rows_of(T, E);
  const int blocks = single ? 1 : blocks_of(T, E);
  if (!single) {
    const size_t slots = (size_t)blocks + S;
    char* p = reinterpret_cast<char*>(ws);
    a.part_p = reinterpret_cast<float*>(p);
    a.part_c = reinterpret_cast<int32_t*>(p += padded(slots * E * 4));
    a.part_z = reinterpret_cast<float*>(p += padded(slots * E * 4));
    a.part_n = reinterpret_cast<int32_t*>(p += padded(slots * 4));
    a.dots = reinterpret_cast<float*>(p += padded(slots * 4));
    a.arrived = reinterpret_cast<unsigned*>(p += padded((size_t)S * chunks_of(E) * 4));
  }
  if (E <= 64) launch_forward<16, 4>(a, vec, single, blocks, s);
  else if (E <= 128) launch_forward<16, 8>(a, vec, single, blocks, s);
  else if (E <= 256) launch_forward<16, 16>(a, vec, single, blocks, s);
  else if (E <= 512) launch_forward<32, 16>(a, vec, single, blocks, s);
  else launch_forward<64, 16>(a, vec, single, blocks, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || single) return e;
  hipLaunchKernelGGL(balance_finish_kernel, dim3(S, chunks_of(E)), dim3(kBalanceBlock), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_router_backward(const float* scores, const int32_t* ids, const float* wts,
                                  const float* grad_wts, const uint8_t* mask,
                                  const int32_t* offsets, const int32_t* counts,
                                  const int32_t* tokens, const float* grad_loss, int T, int E,
                                  int k, int S, float* grad, hipStream_t s) {
  BalanceArgs a{};
  a.scores = scores;
  a.ids = ids;
  a.wts = wts;
  a.grad_wts = grad_wts;
  a.mask = mask;
  a.offsets = offsets;
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.grad_loss = grad_loss;
  a.T = T;
  a.E = E;
  a.k = k;
  a.S = S;
  a.grad = grad;
  const bool vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(scores) & 15u) == 0 &&
                   (reinterpret_cast<uintptr_t>(grad) & 15u) == 0;
  const int round = kBackBlock / lanes_of(E);
  // four workgroups per CU (65536 x 256: 36.0 us, with two 44.1, with sixteen 42.7)
  const long long most = (long long)device_num_cus() * 4 * round;
  a.block_rows = (int)std::max(1LL, ((long long)T + most - 1) / most) * round;
  const unsigned grid = (unsigned)(((long long)T + a.block_rows - 1) / a.block_rows);
  if (E <= 64) launch_backward<16, 4>(a, vec, grid, s);
  else if (E <= 128) launch_backward<16, 8>(a, vec, grid, s);
  else if (E <= 256) launch_backward<16, 16>(a, vec, grid, s);
  else if (E <= 512) launch_backward<32, 16>(a, vec, grid, s);
  else launch_backward<64, 16>(a, vec, grid, s);
  return hipGetLastError();
}

}  // namespace moe
