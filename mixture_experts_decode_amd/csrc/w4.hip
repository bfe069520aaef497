// Products with 4-bit weights and group scales:
//   y[n] = sum_k s[n][k / G] (q[n][k] - z[n][k / G]) x[k]
// for a few rows x at once, with one matrix or the routed experts' matrices.
//
// Every weight is used for at most a few x rows, so its bytes (K/2 a row, plus
// scales) are what it cannot do without.  v_mfma_f32_16x16x32_bf16 takes x rows
// as its 16 A rows and 16 weight rows as its B columns: the products q x are
// exact (a 4-bit integer and a BF16 value), the matrix core adds them in FP32,
// and a lane ends with four x rows of one weight row, so a group is finished
// with one scale per lane:  y += s (sum q x - z sum x),  the sum of x by an MFMA
// against ones.
//
// A wavefront takes a part of K of a tile of 16 weight rows and requests all of
// it together, with the part's scales, which lie side by side in their rows
// and go through its own LDS (read one here and one there by the lanes that
// use them they cost a cache line each: 84.6 us against 46.6 without them, for
// the first product below).  Many short wavefronts keep the loads of a CU in
// flight and even out by themselves; persistent workgroups with x in LDS and a
// ring of steps in flight took 59 us.  40961 x 7168 for 5 rows: 51.0 us, 170.6 MB
// of weights and scales at 3.35 TB/s, which no unit explains by itself: HBM is at
// 54% of the copy rate and the vector unit busy for 46% of the time.  A wavefront
// issues about 209 vector instructions for 256 inputs of 16 rows, some 160 in the
// loop (56 convert the codes, 48 finish four groups), the rest before and after
// it; x goes through L2 once for every 16 weight rows (1.69 M L2 hits beside
// 1.35 M misses).  The time between is waits.
//
// A code becomes BF16 without a table: as an E4M3 byte the codes 0..15 stand
// for 0..15 times 2^-9 (eight subnormals and the first binade), which the
// FP8-to-BF16 conversion multiplies by 2^9.

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "rows.h"

namespace moe {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct W4Args {
  const uint8_t* q;
  const void* scale;
  const uint8_t* zero;
  const uint16_t* x;
  const int32_t* ids;     // [T][k], null: one matrix
  const float* wts;       // [T][k], null: 1
  void* y;
  int N, K, E, groups, group_shift;   // group_shift: log2(G / 32)
  int T, k, entries;
  int x_per_slot, swiglu, y_f32;
  int by_expert;          // a grid row is an expert, else a touched one
};

constexpr int kW4MaxEntries = kDecodeMaxEntries;

// Lane (row n, group g) has loaded elements 32 g .. 32 g + 31 of its row;
// afterwards its dword j holds elements 32 j + 8 g .. + 7, the ones that MFMA j
// (inputs 32 j .. 32 j + 31) takes from it: a 4 x 4 transposition over the
// four lane groups.
__device__ __forceinline__ u32x4 transpose4(u32x4 w) {
  auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

// The routed entries as every workgroup finds them: the experts that any entry
// names, and one expert's entries in order.
struct Lists {
  unsigned touched[kMaxExpertsTotal / 32];
  unsigned long long mask[kW4MaxEntries / kWave];
  int16_t list[kW4MaxEntries];
};

// Marks the experts that any entry names; returns their number.
__device__ __forceinline__ int touched_experts(Lists& s, const W4Args& a) {
  const int words = (a.E + 31) / 32;
  for (int i = threadIdx.x; i < words; i += blockDim.x) s.touched[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.entries; i += blockDim.x) {
    const int id = (unsigned)a.ids[i] < (unsigned)a.E ? a.ids[i] : 0;
    atomicOr(&s.touched[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
  int n = 0;
  for (int i = 0; i < words; ++i) n += __popc(s.touched[i]);
  return n;
}

// The want-th of them, or -1 if there are fewer.
__device__ __forceinline__ int touched_expert(const Lists& s, const W4Args& a, int want) {
  const int words = (a.E + 31) / 32;
  for (int i = 0; i < words; ++i) {
    unsigned w = s.touched[i];
    const int c = __popc(w);
    if (want < c) {
      for (; want > 0; --want) w &= w - 1;
      return 32 * i + __ffs(w) - 1;
    }
    want -= c;
  }
  return -1;
}

// Expert e's entries, in order, into s.list; returns their number.
__device__ __forceinline__ int entries_of(Lists& s, const W4Args& a, int e) {
  const int lane = threadIdx.x & (kWave - 1), wave = wave_in_block(), nw = blockDim.x / kWave;
  const int chunks = (a.entries + kWave - 1) / kWave;
  for (int c = wave; c < chunks; c += nw) {
    const int i = c * kWave + lane;
    int id = -1;
    if (i < a.entries) id = (unsigned)a.ids[i] < (unsigned)a.E ? a.ids[i] : 0;
    const unsigned long long m = __ballot(id == e);
    if (lane == 0) s.mask[c] = m;
  }
  __syncthreads();
  int count = 0;
  for (int c = 0; c < chunks; ++c) {
    const unsigned long long m = s.mask[c];
    if (c % nw == wave && ((m >> lane) & 1))
      s.list[count + __popcll(m & ((1ull << lane) - 1))] = (int16_t)(c * kWave + lane);
    count += __popcll(m);
  }
  __syncthreads();
  return count;
}

// Waits for the wavefront's own LDS accesses and for the other wavefronts;
// global loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Codes 0, 2, 4, 6 and 1, 3, 5, 7 of a dword -> BF16 integers in that order.
__device__ __forceinline__ bf16x8 codes_even_odd(uint32_t w) {
  const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
  union {
    bf16x2 p[4];
    bf16x8 v;
  } u;
  u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, false);
  u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, true);
  u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, false);
  u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, true);
  return u.v;
}

// Eight x values in the order of codes_even_odd.
__device__ __forceinline__ u32x4 even_odd(u32x4 v) {
  return u32x4{__builtin_amdgcn_perm(v[1], v[0], 0x05040100u), __builtin_amdgcn_perm(v[3], v[2], 0x05040100u),
               __builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
}

// Inputs of a wavefront's part, and wavefronts of a workgroup at most; they
// take the parts of K in turn.  Dense products have the same parts whatever the
// number of x rows, so that a row's sums do not depend on the batch.
// Dense products take parts of 256: 51.0 us for 40961 x 7168 (G = 64, float
// scales, zero points) and 5 x rows; with parts of 512 52.3, with 4 and 16
// wavefronts 52.8 and 63.4, with the next part's weights requested ahead 51.8.
// With routed experts every workgroup first lists its expert's entries, which
// longer parts spread over more work: 55.6 us for the gate and up products of
// 32 tokens and 128 experts (1536 x 2048 each, top-8), 67 and 103 with parts of
// 512 and 256.
__host__ __device__ constexpr int part_inputs(int sets, bool routed) { return sets == 1 && routed ? 1024 : 256; }
constexpr int kTileWaves = 8;

// Dwords of a row of `groups` scales (or zero points) in LDS: an odd number,
// so that 16 rows start in different banks.
__host__ __device__ constexpr int staged_dwords(int groups, int size) { return (groups * size + 3) / 4 | 1; }

// The scales (SIZE bytes each) of 16 rows over a part, `count` of them a row, a
// power of two -> the wavefront's LDS.  DW: as dwords, else one by one.
// kMost: pieces of a lane if there is a scale for every 32 inputs.
template <int PART, int SIZE, bool DW>
struct PartScales {
  static constexpr int kMost = (16 * (PART / 32) / (DW ? 4 / SIZE : 1) + kWave - 1) / kWave;
  uint32_t v[kMost];

  // p: the tile's first row; of_row: pieces of a row, first: the part's first
  // one; row_at(i): row i of the tile, from its first one
  template <class RowAt>
  __device__ __forceinline__ void load(const uint8_t* p, RowAt row_at, int of_row, int first, int log2n, int lane) {
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int at = lane + kWave * i, r = at >> log2n;
      if (i > 0 && (kWave * i >> log2n) >= 16) break;
      const size_t piece = row_at(r & 15) * of_row + min(first + (at & ((1 << log2n) - 1)), of_row - 1);
      if constexpr (DW || SIZE == 4) v[i] = reinterpret_cast<const uint32_t*>(p)[piece];
      else if constexpr (SIZE == 2) v[i] = reinterpret_cast<const uint16_t*>(p)[piece];
      else v[i] = p[piece];
    }
  }
  __device__ __forceinline__ void store(uint32_t* lds, int stride, int log2n, int lane) const {
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int at = lane + kWave * i, r = at >> log2n, c = at & ((1 << log2n) - 1);
      if (i > 0 && (kWave * i >> log2n) >= 16) break;
      if (r >= 16) continue;
      if constexpr (DW || SIZE == 4) lds[r * stride + c] = v[i];
      else if constexpr (SIZE == 2) reinterpret_cast<uint16_t*>(lds + r * stride)[c] = (uint16_t)v[i];
      else reinterpret_cast<uint8_t*>(lds + r * stride)[c] = (uint8_t)v[i];
    }
  }
};

__device__ __forceinline__ int log2_of(int v) { return 31 - __clz(v); }

// The x rows come in sets of eight.  Rows 0..7 of the A operand are their inputs
// of one MFMA (even j), rows 8..15 those of the next one (odd j), so a load
// serves two MFMAs.  Each of the two has its own accumulator, of which only its
// rows are meant; a lane picks its four rows from the one that they belong to,
// and the sums of x take one MFMA for both.  The order of a row's sums is the
// same whatever the number of sets.
template <int SETS, bool ROUTED, int GM, bool SF, bool ZP, bool DW>
__global__ __launch_bounds__(kTileWaves * kWave) void w4_tile_kernel(W4Args a) {
  extern __shared__ __align__(16) uint32_t lds[];
  __shared__ Lists s_entries;
  constexpr int kSize = SF ? 4 : 2, kPer = DW ? 4 / kSize : 1, kPerZ = DW ? 4 : 1;
  constexpr int kPart = part_inputs(SETS, ROUTED), kHalves = kPart / 128, kRows = 8 * SETS;
  constexpr int kAhead = SETS == 1 ? 2 : 1;   // halves of x in flight before the current one
  const int lane = threadIdx.x & (kWave - 1), wave = wave_in_block(), waves = blockDim.x / kWave;
  const int n16 = lane & 15, g = lane >> 4, odd = g >> 1;
  const int outs = a.swiglu ? a.N / 2 : a.N;
  const int tile_outs = a.swiglu ? 8 : 16;
  const int shift = 5 + a.group_shift;
  int e = 0, begin = 0, count = a.T;
  if constexpr (ROUTED) {
    if (a.by_expert) {
      e = blockIdx.y;
    } else {
      if ((int)blockIdx.y >= touched_experts(s_entries, a)) return;
      e = touched_expert(s_entries, a, blockIdx.y);
    }
    count = entries_of(s_entries, a, e);
    if (count == 0) return;
  } else {
    begin = blockIdx.y * kRows;
    count = min(a.T, begin + kRows);
  }
  // row i of the tile, from its first one: with SwiGLU eight gate rows and the
  // same outputs' eight up rows
  const int n0 = blockIdx.x * tile_outs, n_last = outs - 1 - n0;
  const size_t row0 = (size_t)e * a.N + n0;
  auto row_at = [&](int i) {
    return a.swiglu ? min(i & 7, n_last) + (i >= 8 ? outs : 0) : min(i, n_last);
  };
  const uint8_t* q = a.q + (row0 + row_at(n16)) * (size_t)(a.K / 2) + 16 * g;
  const uint8_t* scale0 = reinterpret_cast<const uint8_t*>(a.scale) + row0 * a.groups * kSize;
  const uint8_t* zero0 = a.zero + row0 * a.groups;
  // scales of a part in LDS, per wavefront
  const int part_groups = min(kPart / 32, max(1, kPart >> shift));
  const int s_row = staged_dwords(part_groups, kSize), z_row = staged_dwords(part_groups, 1);
  uint32_t* scales = lds + wave * 16 * (s_row + (ZP ? z_row : 0));
  uint32_t* zeros = scales + 16 * s_row;
  const int s_log = log2_of(max(1, part_groups / kPer)), z_log = log2_of(max(1, part_groups / kPerZ));
  float* sums = reinterpret_cast<float*>(lds + waves * 16 * (s_row + (ZP ? z_row : 0)));
  const uint8_t* sl = reinterpret_cast<const uint8_t*>(scales + n16 * s_row);
  const uint8_t* zl = reinterpret_cast<const uint8_t*>(zeros + n16 * z_row);
  const bf16x8 ones = {(__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f,
                       (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f};
  // inputs within a half that this lane holds: of load i, kLoadStep further
  const int lane_k = GM == 4 ? 32 * g + 8 * (n16 >> 3) : 8 * g + 32 * (n16 >> 3);
  constexpr int kLoadStep = GM == 4 ? 16 : 64;
  for (int first = begin; first < count; first += kRows) {
    const int rows = min(kRows, count - first);
    const uint16_t* xp[SETS];
#pragma unroll
    for (int m = 0; m < SETS; ++m) {
      int xi = first + min(8 * m + (n16 & 7), rows - 1);
      if constexpr (ROUTED) xi = a.x_per_slot ? s_entries.list[xi] : s_entries.list[xi] / a.k;
      xp[m] = a.x + (size_t)xi * a.K + lane_k;
    }
    f32x4 acc[SETS];
#pragma unroll
    for (int m = 0; m < SETS; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // WHOLE: the part lies within K
    auto part_of = [&](int k0, auto whole) {
      constexpr bool WHOLE = decltype(whole)::value;
      u32x4 w[kHalves], x[kAhead + 1][SETS][2];
      PartScales<kPart, kSize, DW> sv;
      PartScales<kPart, 1, DW> zv;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        w[h] = load16(WHOLE ? q + k0 / 2 + 64 * h : q + (min(k0 + 128 * h + 32 * g, a.K - 32) - 32 * g) / 2);
      const int g0 = k0 >> shift;
      sv.load(scale0, row_at, a.groups / kPer, g0 / kPer, s_log, lane);
      if constexpr (ZP) zv.load(zero0, row_at, a.groups / kPerZ, g0 / kPerZ, z_log, lane);
      auto load_x = [&](u32x4 (&v)[SETS][2], int h) {
#pragma unroll
        for (int m = 0; m < SETS; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int k = k0 + 128 * h + kLoadStep * i;
            v[m][i] = load16(xp[m] + (WHOLE ? k : min(k, a.K - 8 - lane_k)));
          }
      };
#pragma unroll
      for (int h = 0; h < kAhead; ++h) load_x(x[h], h);
      wave_fence();
      sv.store(scales, s_row, s_log, lane);
      if constexpr (ZP) zv.store(zeros, z_row, z_log, lane);
      wave_fence();
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        __builtin_amdgcn_sched_barrier(0);   // a half's temporaries at a time
        const int kh = k0 + 128 * h;
        // a long part's halves behind K (experts of 2048 x 768, 32 tokens: 47.3 -> 44.8 us)
        if (ROUTED && !WHOLE && kh >= a.K) break;
        if (h + kAhead < kHalves) load_x(x[(h + kAhead) % (kAhead + 1)], h + kAhead);
        // a group of 128 or more spans the half: each lane keeps its own 32
        // inputs of it, x is read to match
        const u32x4 wh = GM == 4 ? w[h] : transpose4(w[h]);
        f32x4 part[SETS][2], xs[SETS];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bf16x8 we = codes_even_odd(wh[2 * i]), wo = codes_even_odd(wh[2 * i + 1]);
          const uint32_t keep = WHOLE || kh + kLoadStep * i + lane_k < a.K ? 0xffffffffu : 0u;
#pragma unroll
          for (int m = 0; m < SETS; ++m) {
            u32x4 v = x[h % (kAhead + 1)][m][i];
            if constexpr (!WHOLE) v &= keep;
            const bf16x8 xb = __builtin_bit_cast(bf16x8, even_odd(v));
            if (i == 0 || GM < 4) part[m][0] = part[m][1] = xs[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            xs[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, ones, xs[m], 0, 0, 0);
            part[m][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, we, part[m][0], 0, 0, 0);
            part[m][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, wo, part[m][1], 0, 0, 0);
          }
          if (i == 1 || GM < 4) {
            // the group of this lane's rows: its own MFMA's if there is one
            // for every MFMA
            int gr = ((kh + (GM == 4 ? 0 : GM == 2 ? 64 * i : 64 * i + 32 * odd)) >> shift) - g0;
            if constexpr (!WHOLE) gr = min(gr, a.groups - 1 - g0);
            float f;
            if constexpr (SF) f = reinterpret_cast<const float*>(sl)[gr];
            else f = bf16_lo(reinterpret_cast<const uint16_t*>(sl)[gr]);
            float z = 8.0f;
            if constexpr (ZP) z = (float)zl[gr];
#pragma unroll
            for (int m = 0; m < SETS; ++m)
#pragma unroll
              for (int p = 0; p < 4; ++p)
                acc[m][p] = fmaf(f, fmaf(-z, xs[m][p], odd ? part[m][1][p] : part[m][0][p]), acc[m][p]);
          }
        }
      }
    };
    for (int k0 = kPart * wave; k0 < a.K; k0 += kPart * waves) {
      if (k0 + kPart <= a.K) part_of(k0, std::true_type{});
      else part_of(k0, std::false_type{});
    }
    // rows 8..15 of a set belong to the same x rows as rows 0..7
#pragma unroll
    for (int m = 0; m < SETS; ++m)
#pragma unroll
      for (int p = 0; p < 4; ++p) acc[m][p] += __shfl_xor(acc[m][p], 32, kWave);
    // the sums over the parts of K, added in order; wavefront w finishes the
    // sets w, w + waves, ...
    if (waves > 1) {
      if (first > begin) lds_barrier();   // the last ones have been read
      if (odd == 0) {
#pragma unroll
        for (int m = 0; m < SETS; ++m)
          *reinterpret_cast<f32x4*>(sums + (wave * SETS + m) * 128 + 4 * lane) = acc[m];
      }
      lds_barrier();
    }
#pragma unroll
    for (int m = 0; m < SETS; ++m) {
      if (m % waves != wave) continue;
      f32x4 v = acc[m];
      if (waves > 1) {
        v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int p = 0; p < waves; ++p)
          v += *reinterpret_cast<const f32x4*>(sums + (p * SETS + m) * 128 + 4 * (lane & 31));
      }
      // output column n16 of the tile for x rows 8 m + 4 g ..
      const int n = n0 + n16;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int i = 8 * m + 4 * g + p;
        float r = v[p];
        if (a.swiglu) r = swiglu(r, dpp_f32<0x128>(r));   // row_ror:8: the up row's sum
        if (odd == 0 && i < rows && n16 < tile_outs && n < outs) {
          const int entry = ROUTED ? s_entries.list[first + i] : first + i;
          if (a.wts) r *= a.wts[entry];
          const size_t to = (size_t)entry * outs + n;
          if (a.y_f32) reinterpret_cast<float*>(a.y)[to] = r;
          else reinterpret_cast<__bf16*>(a.y)[to] = (__bf16)r;
        }
      }
    }
  }
}

template <int SETS, bool ROUTED, int GM, bool DW>
void launch_scaled(const W4Args& a, bool sf, dim3 grid, int waves, size_t lds, hipStream_t s) {
  const dim3 block(waves * kWave);
  if (a.zero) {
    if (sf) hipLaunchKernelGGL((w4_tile_kernel<SETS, ROUTED, GM, true, true, DW>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((w4_tile_kernel<SETS, ROUTED, GM, false, true, DW>), grid, block, lds, s, a);
  } else {
    if (sf) hipLaunchKernelGGL((w4_tile_kernel<SETS, ROUTED, GM, true, false, DW>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((w4_tile_kernel<SETS, ROUTED, GM, false, false, DW>), grid, block, lds, s, a);
  }
}

template <int SETS, bool ROUTED, bool DW>
void launch_grouped(const W4Args& a, bool sf, dim3 grid, int waves, size_t lds, hipStream_t s) {
  if (a.group_shift == 0) launch_scaled<SETS, ROUTED, 1, DW>(a, sf, grid, waves, lds, s);
  else if (a.group_shift == 1) launch_scaled<SETS, ROUTED, 2, DW>(a, sf, grid, waves, lds, s);
  else launch_scaled<SETS, ROUTED, 4, DW>(a, sf, grid, waves, lds, s);
}

template <int SETS>
void launch_sets(const W4Args& a, bool sf, bool dwords, dim3 grid, int waves, size_t lds, hipStream_t s) {
  if (a.ids) {
    if (dwords) launch_grouped<SETS, true, true>(a, sf, grid, waves, lds, s);
    else launch_grouped<SETS, true, false>(a, sf, grid, waves, lds, s);
  } else {
    if (dwords) launch_grouped<SETS, false, true>(a, sf, grid, waves, lds, s);
    else launch_grouped<SETS, false, false>(a, sf, grid, waves, lds, s);
  }
}

}  // namespace

hipError_t launch_w4_linear(const moe_w4_weights& W, const uint16_t* x, const int32_t* ids,
                            const float* wts, int T, int k, int x_per_slot, int swiglu, void* y,
                            int y_dtype, hipStream_t s) {
  W4Args a{};
  a.q = reinterpret_cast<const uint8_t*>(W.q);
  a.scale = W.scale;
  a.zero = W.zero;
  a.x = x;
  a.ids = ids;
  a.wts = wts;
  a.y = y;
  a.N = W.rows;
  a.K = W.cols;
  a.E = W.num_mats;
  a.groups = W.cols / W.group;
  while ((32 << a.group_shift) < W.group) ++a.group_shift;
  a.T = T;
  a.k = k;
  a.entries = ids ? T * k : T;
  a.x_per_slot = x_per_slot;
  a.swiglu = swiglu;
  a.y_f32 = y_dtype == MOE_DT_F32;
  const bool sf = W.scale_dtype == MOE_DT_F32;
  const int outs = swiglu ? a.N / 2 : a.N;
  const int per = swiglu ? 8 : 16, tiles = (outs + per - 1) / per;
  a.by_expert = a.entries >= a.E;
  const int mats = ids ? std::min(a.E, a.entries) : 1;
  // x rows that one matrix meets at a time: all of them, or what an expert is
  // likely to get (one with more takes its rows in several passes)
  const int rows = ids ? (3 * a.entries + a.E - 1) / a.E : T;
  const int sets = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  const int inputs = part_inputs(sets, ids != nullptr);
  const int waves = std::min(kTileWaves, (a.K + inputs - 1) / inputs);
  const int part = std::min(inputs / 32, std::max(1, inputs >> (5 + a.group_shift)));
  // whole dwords of scales in a row and in a part of it
  const bool dwords = (sf || (a.groups % 2 == 0 && part % 2 == 0)) &&
                      (!a.zero || (a.groups % 4 == 0 && part % 4 == 0)) &&
                      (reinterpret_cast<uintptr_t>(a.scale) & 3) == 0 &&
                      (reinterpret_cast<uintptr_t>(a.zero) & 3) == 0;
  const size_t lds = (size_t)waves * 64 * (staged_dwords(part, sf ? 4 : 2) + (a.zero ? staged_dwords(part, 1) : 0)) +
                     (waves > 1 ? (size_t)waves * sets * 512 : 0);
  const dim3 grid(tiles, ids ? mats : (T + 8 * sets - 1) / (8 * sets));
  if (sets == 1) launch_sets<1>(a, sf, dwords, grid, waves, lds, s);
  else if (sets == 2) launch_sets<2>(a, sf, dwords, grid, waves, lds, s);
  else launch_sets<4>(a, sf, dwords, grid, waves, lds, s);
  return hipGetLastError();
}

}  // namespace moe
