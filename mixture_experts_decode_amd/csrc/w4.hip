// Products with 4-bit weights and group scales:
//   y[n] = sum_k s[n][k / G] (q[n][k] - z[n][k / G]) x[k]
// for a few rows x at once, with one matrix or the routed experts' matrices.
//
// Every weight is used for at most a few x rows, so its bytes (K/2 a row, plus
// scales) bound the product.  v_mfma_f32_16x16x32_bf16 takes the x rows as its
// 16 A rows and 16 weight rows as its B columns: the products q x are exact (a
// 4-bit integer and a BF16 value), the matrix core adds them in FP32, and a
// lane ends with four x rows of one weight row, so a group is finished with
// one scale per lane:  y += s (sum q x - z sum x),  the sum of x by an MFMA
// against ones.
//
// A code becomes BF16 without a table: as an E4M3 byte the codes 0..15 stand
// for 0..15 times 2^-9 (eight subnormals and the first binade), which the
// FP8-to-BF16 conversion multiplies by 2^9.

#include <algorithm>

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
};

constexpr int kW4MaxEntries = kDecodeMaxEntries;

// Eight codes of one dword (element 0 in the lowest nibble) -> BF16 integers.
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t w) {
  const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u);   // elements 0..3
  const uint32_t hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);   // elements 4..7
  union {
    bf16x2 p[4];
    bf16x8 v;
  } u;
  u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
  u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
  u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
  u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
  return u.v;
}

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

// Weights, scales and zero points, as stored, of one 128-input step of NR row
// tiles; they are converted where they are used, so that the loads of the
// next step stay in flight over the current one.
// GM: MFMAs (32 inputs each) to a scale group within the step.
template <int NR, int GM>
struct Step {
  u32x4 w[NR];
  uint32_t s[NR][4 / GM], z[NR][4 / GM];
};

template <int NR, int GM, bool SF, bool ZP>
__device__ __forceinline__ void load_step(Step<NR, GM>& st, const W4Args& a, const size_t (&row)[NR],
                                          int k0, int g) {
  const int k = min(k0 + 32 * g, a.K - 32);
#pragma unroll
  for (int r = 0; r < NR; ++r)
    st.w[r] = load_stream16(a.q + row[r] * (size_t)(a.K / 2) + k / 2);
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int j = 0; j < 4 / GM; ++j) {
      const int gr = min((k0 + 32 * GM * j) >> (5 + a.group_shift), a.groups - 1);
      const size_t at = row[r] * a.groups + gr;
      if constexpr (SF) st.s[r][j] = reinterpret_cast<const uint32_t*>(a.scale)[at];
      else st.s[r][j] = reinterpret_cast<const uint16_t*>(a.scale)[at];
      if constexpr (ZP) st.z[r][j] = a.zero[at];
    }
}

// MT tiles of 16 x rows, NR tiles of 16 weight rows per workgroup; its
// wavefronts take 128-input steps in turn and add their sums through LDS.
template <int MT, int NR, int GM, bool SF, bool ZP>
__global__ __launch_bounds__(MT == 1 ? 1024 : MT == 2 ? 512 : 256) void w4_kernel(W4Args a) {
  extern __shared__ float lds[];
  __shared__ unsigned long long s_mask[kW4MaxEntries / kWave];
  __shared__ int16_t s_list[kW4MaxEntries];
  const int lane = threadIdx.x & (kWave - 1), wave = wave_in_block();
  const int nw = blockDim.x / kWave;
  const int n16 = lane & 15, g = lane >> 4;
  const int outs = a.swiglu ? a.N / 2 : a.N;
  const int e = a.ids ? blockIdx.y : 0;
  int first = 0, count;
  if (a.ids) {
    // the entries of expert e, in order
    const int chunks = (a.entries + kWave - 1) / kWave;
    for (int c = wave; c < chunks; c += nw) {
      const int i = c * kWave + lane;
      int id = -1;
      if (i < a.entries) id = (unsigned)a.ids[i] < (unsigned)a.E ? a.ids[i] : 0;
      const unsigned long long m = __ballot(id == e);
      if (lane == 0) s_mask[c] = m;
    }
    __syncthreads();
    count = 0;
    for (int c = 0; c < chunks; ++c) {
      const unsigned long long m = s_mask[c];
      if (c % nw == wave && ((m >> lane) & 1))
        s_list[count + __popcll(m & ((1ull << lane) - 1))] = (int16_t)(c * kWave + lane);
      count += __popcll(m);
    }
    if (count == 0) return;
    __syncthreads();
  } else {
    first = blockIdx.y * (16 * MT);
    count = min(a.T - first, 16 * MT);
  }
  // weight rows of the tiles; with SwiGLU the first half of them are gate
  // rows, the second the same outputs' up rows
  constexpr int kHalf = NR == 1 ? 1 : NR / 2;
  const int tile_rows = a.swiglu ? 16 * kHalf : 16 * NR;
  const int r0 = blockIdx.x * tile_rows;
  size_t row[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const bool up = a.swiglu && r >= kHalf;
    const int n = min(r0 + 16 * (up ? r - kHalf : r) + n16, outs - 1);
    row[r] = (size_t)e * a.N + n + (up ? outs : 0);
  }
  const bf16x8 ones = {(__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f,
                       (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f};
  for (int tile = 0; tile < count; tile += 16 * MT) {
    const uint16_t* xr[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int i = min(tile + 16 * m + n16, count - 1);
      int xi = first + i;
      if (a.ids) xi = a.x_per_slot ? s_list[i] : s_list[i] / a.k;
      xr[m] = a.x + (size_t)xi * a.K;
    }
    f32x4 acc[MT][NR];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[m][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int stride = 128 * nw;
    Step<NR, GM> cur, nxt;
    int k0 = 128 * wave;
    if (k0 < a.K) load_step<NR, GM, SF, ZP>(cur, a, row, k0, g);
    for (; k0 < a.K; k0 += stride) {
      u32x4 xv[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = min(k0 + 32 * j, a.K - 32) + 8 * g;
          xv[m][j] = load16(xr[m] + k);
        }
      if (k0 + stride < a.K) load_step<NR, GM, SF, ZP>(nxt, a, row, k0 + stride, g);
#pragma unroll
      for (int r = 0; r < NR; ++r) cur.w[r] = transpose4(cur.w[r]);
      f32x4 part[MT][NR], xs[MT];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j % GM == 0) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            xs[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int r = 0; r < NR; ++r) part[m][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          }
        }
        if (k0 + 32 * j < a.K) {
          bf16x8 xb[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            xb[m] = __builtin_bit_cast(bf16x8, xv[m][j]);
            xs[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[m], ones, xs[m], 0, 0, 0);
          }
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const bf16x8 wb = codes_to_bf16(cur.w[r][j]);
#pragma unroll
            for (int m = 0; m < MT; ++m)
              part[m][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[m], wb, part[m][r], 0, 0, 0);
          }
        }
        if (j % GM == GM - 1) {
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float sc = __uint_as_float(SF ? cur.s[r][j / GM] : cur.s[r][j / GM] << 16);
            const float zp = ZP ? (float)cur.z[r][j / GM] : 8.0f;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[m][r][i] = fmaf(sc, fmaf(-zp, xs[m][i], part[m][r][i]), acc[m][r][i]);
          }
        }
      }
      cur = nxt;
    }
    // the wavefronts' sums, added in order
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          lds[((wave * MT + m) * NR + r) * 256 + (4 * g + i) * 16 + n16] = acc[m][r][i];
    __syncthreads();
    const int out_tiles = a.swiglu ? kHalf : NR;
    for (int o = threadIdx.x; o < MT * out_tiles * 256; o += blockDim.x) {
      const int c = o & 15, m16 = (o >> 4) & 15, r = (o >> 8) % out_tiles, m = (o >> 8) / out_tiles;
      const int i = tile + 16 * m + m16, n = r0 + 16 * r + c;
      if (i >= count || n >= outs) continue;
      float v = 0.0f, up = 0.0f;
      for (int w = 0; w < nw; ++w) {
        v += lds[((w * MT + m) * NR + r) * 256 + m16 * 16 + c];
        if (a.swiglu) up += lds[((w * MT + m) * NR + r + kHalf) * 256 + m16 * 16 + c];
      }
      if (a.swiglu) v = swiglu(v, up);
      const int entry = a.ids ? s_list[i] : first + i;
      if (a.wts) v *= a.wts[entry];
      const size_t at = (size_t)entry * outs + n;
      if (a.y_f32) reinterpret_cast<float*>(a.y)[at] = v;
      else reinterpret_cast<__bf16*>(a.y)[at] = (__bf16)v;
    }
    __syncthreads();
  }
}

template <int MT, int NR, int GM>
void launch_scaled(const W4Args& a, bool sf, dim3 grid, int waves, hipStream_t s) {
  const size_t lds = (size_t)waves * MT * NR * 256 * sizeof(float);
  const dim3 block(waves * kWave);
  if (a.zero) {
    if (sf) hipLaunchKernelGGL((w4_kernel<MT, NR, GM, true, true>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((w4_kernel<MT, NR, GM, false, true>), grid, block, lds, s, a);
  } else {
    if (sf) hipLaunchKernelGGL((w4_kernel<MT, NR, GM, true, false>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((w4_kernel<MT, NR, GM, false, false>), grid, block, lds, s, a);
  }
}

template <int MT, int NR>
void launch_grouped(const W4Args& a, bool sf, dim3 grid, int waves, hipStream_t s) {
  if (a.group_shift == 0) launch_scaled<MT, NR, 1>(a, sf, grid, waves, s);
  else if (a.group_shift == 1) launch_scaled<MT, NR, 2>(a, sf, grid, waves, s);
  else launch_scaled<MT, NR, 4>(a, sf, grid, waves, s);
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
  const int steps = (a.K + 127) / 128;
  // x rows that one matrix meets: all of them, or the mean over the experts
  const int rows = ids ? (a.entries + a.E - 1) / a.E : T;
  const int mt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  const int nr = swiglu || outs > 16 * 1024 ? 2 : 1;
  const int tiles = (outs + (swiglu ? 16 : 16 * nr) - 1) / (swiglu ? 16 : 16 * nr);
  const int most = mt == 1 ? 16 : mt == 2 ? 8 : 4;
  int waves = 4;
  while (waves < most && waves < steps && (long long)tiles * (ids ? a.E : 1) * waves < 4096) waves *= 2;
  const dim3 grid(tiles, ids ? a.E : (T + 16 * mt - 1) / (16 * mt));
  if (nr == 2) {
    if (mt == 1) launch_grouped<1, 2>(a, sf, grid, waves, s);
    else if (mt == 2) launch_grouped<2, 2>(a, sf, grid, waves, s);
    else launch_grouped<4, 2>(a, sf, grid, waves, s);
  } else {
    if (mt == 1) launch_grouped<1, 1>(a, sf, grid, waves, s);
    else if (mt == 2) launch_grouped<2, 1>(a, sf, grid, waves, s);
    else launch_grouped<4, 1>(a, sf, grid, waves, s);
  }
  return hipGetLastError();
}

}  // namespace moe
