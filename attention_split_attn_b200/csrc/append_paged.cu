// append_paged.cu -- new K/V rows written through a slot map into a paged
// cache: copied (rounded once where the types differ), or quantized to e4m3 /
// int8 codes with one F32 scale per (slot, KV head).
//
//   scale = rn(amax / 448)  or  rn(amax / 127),   code = rn(x / scale)
//
// The quotient is rounded once: x / scale is taken toward zero and its last
// bit set when a remainder is left (round to odd), and rounding that to the
// code's few bits gives the nearest code to the exact quotient.  A plain F32
// quotient would land on ties that the exact one misses, and ties are common
// (amax / 448 of 8-bit significands).
//
// 14001 rows of 4 x 256 f16 take 17.7 us (115 MB, 6.5 TB/s).
// Both kernels move bytes and little else (each row read once, each cell
// written once).  Copy: a CTA's 256 threads span one row's K and V in
// 16-byte pieces, so the loads and stores of a head are whole 128-byte lines
// whatever the cache's strides, and take 4 rows at a time to keep 4 loads in
// flight per thread.  Quantization: a warp per (row, KV head), K then V, one
// reduction each.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace attn {

namespace {

constexpr int kApThreads = 256;
constexpr int kApRows = 4;   // rows in flight per thread

__device__ __forceinline__ int64_t cell_offset(const attn_append_args& a, int32_t slot) {
  const int32_t page = slot / a.page_size;
  return (int64_t)page * a.kv_stride_page + (int64_t)(slot - page * a.page_size) * a.kv_stride_cell;
}

__device__ __forceinline__ bool slot_valid(const attn_append_args& a, int32_t slot) {
  return slot >= 0 && slot < a.n_pages * a.page_size;
}

// 8 values at `src` as 8 16-bit values of the cache type.
template <int NEW, int KV>
__device__ __forceinline__ uint4 load8(const void* src, int64_t i) {
  if constexpr (NEW == KV) {
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + i));
  } else {
    float f[8];
    if constexpr (NEW == ATTN_F32) {
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(src) + i);
      unpack_vec<float>(__ldg(s), f);
      unpack_vec<float>(__ldg(s + 1), f + 4);
    } else if constexpr (NEW == ATTN_F16) {
      unpack_vec<__half>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + i)), f);
    } else {
      unpack_vec<__nv_bfloat16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + i)), f);
    }
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (KV == ATTN_F16) {
        const __half2 h = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// CTA blockIdx.x takes rows [rpc * blockIdx.x, + rpc); pieces of 8 values:
// the K heads, then the V heads.
template <int NEW, int KV>
__global__ void __launch_bounds__(kApThreads) append_copy_kernel(const attn_append_args a, int rpc) {
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int r0 = blockIdx.x * rpc, r1 = min(r0 + rpc, a.n_rows);
  const int per_head = a.head_dim / 8, half = a.n_head_kv * per_head;
  for (int c = threadIdx.x; c < 2 * half; c += kApThreads) {
    const bool is_v = c >= half;
    const int cc = is_v ? c - half : c;
    const int g = cc / per_head, d = (cc - g * per_head) * 8;
    const void* src = is_v ? a.v_new : a.k_new;
    uint16_t* dst = static_cast<uint16_t*>(is_v ? a.v : a.k) + (int64_t)g * a.kv_stride_head + d;
    const int64_t s0 = (int64_t)g * a.new_stride_head + d;
    for (int r = r0; r < r1; r += kApRows) {
      int32_t slot[kApRows];
      uint4 w[kApRows];
#pragma unroll
      for (int k = 0; k < kApRows; ++k) slot[k] = r + k < r1 ? __ldg(a.slot + r + k) : -1;
#pragma unroll
      for (int k = 0; k < kApRows; ++k)
        if (slot_valid(a, slot[k])) w[k] = load8<NEW, KV>(src, s0 + (int64_t)(r + k) * a.new_stride_row);
#pragma unroll
      for (int k = 0; k < kApRows; ++k)
        if (slot_valid(a, slot[k])) *reinterpret_cast<uint4*>(dst + cell_offset(a, slot[k])) = w[k];
    }
  }
}

// x / s rounded to odd (toward zero, the last bit set when that is not exact:
// S. Boldo and G. Melquiond, "Emulation of a FMA and correctly rounded sums",
// 2008).  div_odd_fast, for s far from the ends of the range and inv = 1 / s:
// one Newton step on the quotient (P. Markstein's division with a fused
// multiply-add, 1990) puts q within an ulp of it, where the remainder x - q s
// is exact; a remainder of the other sign means that q lies beyond the
// quotient, and one step of its bits back truncates it.  (A division per value
// took 79% of the issue slots.)
__device__ __forceinline__ float div_odd_fast(float x, float s, float inv) {
  const float q0 = x * inv;
  const float q = fmaf(fmaf(-q0, s, x), inv, q0);
  const float rem = fmaf(-q, s, x);
  const uint32_t b = __float_as_uint(q);
  if (rem == 0.f) return q;
  return __uint_as_float((b - ((b ^ __float_as_uint(rem)) >> 31)) | 1u);
}
// At the ends: x and s of 1e-30 and below are scaled up, or the remainder would
// be a fraction of the smallest float and round to 0 (a tie that is none).
__device__ __forceinline__ float div_odd(float x, float s) {
  const float up = s < 1.f ? 0x1p96f : 1.f;
  x *= up;
  s *= up;
  const float q = __fdiv_rz(x, s);
  const float rem = fmaf(-q, s, x);
  return rem != 0.f ? __uint_as_float(__float_as_uint(q) | 1u) : q;
}

// Two floats to e4m3 codes (lo in the low byte): to nearest even, beyond 448
// to 448, NaN to the NaN code.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int NEW, bool E4M3, int D>
__global__ void __launch_bounds__(kApThreads) append_quant_kernel(const attn_append_args a) {
  constexpr int N = D / 32;   // values per lane: 2, 4 or 8
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int64_t w = ((int64_t)blockIdx.x * kApThreads + threadIdx.x) >> 5;
  const int64_t r = w / a.n_head_kv;
  const int g = (int)(w - r * a.n_head_kv);
  if (r >= a.n_rows) return;
  const int32_t slot = __ldg(a.slot + r);
  if (!slot_valid(a, slot)) return;
  const int64_t src = r * a.new_stride_row + (int64_t)g * a.new_stride_head + lane * N;
  const int64_t dst = cell_offset(a, slot) + (int64_t)g * a.kv_stride_head + lane * N;
  float x[2][N];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const void* base = t ? a.v_new : a.k_new;
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      if constexpr (NEW == ATTN_F32) {
        const float2 f = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(base) + src + k));
        x[t][k] = f.x;
        x[t][k + 1] = f.y;
      } else {
        const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + src + k));
        if constexpr (NEW == ATTN_F16) unpack_f16x2(v, x[t][k], x[t][k + 1]);
        else unpack_bf16x2(v, x[t][k], x[t][k + 1]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) m = fmax_nan(m, fabsf(x[t][k]));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float s = __fdiv_rn(m, E4M3 ? 448.f : 127.f);
    const bool mid = s > 1e-30f && s < 1e30f;   // (the same in every lane)
    const float inv = __frcp_rn(s);
    uint8_t* out = static_cast<uint8_t*>(t ? a.v : a.k) + dst;
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      float lo = 0.f, hi = 0.f;
      if (mid) {
        lo = div_odd_fast(x[t][k], s, inv);
        hi = div_odd_fast(x[t][k + 1], s, inv);
      } else if (s > 0.f) {
        lo = div_odd(x[t][k], s);
        hi = div_odd(x[t][k + 1], s);
      }
      uint32_t two;
      if constexpr (E4M3) {
        two = to_e4m3x2(lo, hi);
      } else {   // NaN (an infinite scale) converts to 0
        const int a0 = max(-127, min(127, __float2int_rn(lo))), a1 = max(-127, min(127, __float2int_rn(hi)));
        two = (uint32_t)(a0 & 0xff) | ((uint32_t)(a1 & 0xff) << 8);
      }
      *reinterpret_cast<uint16_t*>(out + k) = (uint16_t)two;
    }
    if (lane == 0) (t ? a.v_scale : a.k_scale)[(int64_t)slot * a.scale_stride_cell + g] = s;
  }
}

template <typename Kern, typename... Args>
cudaError_t launch_pdl(Kern kern, int64_t blocks, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kApThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int NEW>
cudaError_t launch_new(const attn_append_args& a, int sms, cudaStream_t stream) {
  if (a.kv_type == ATTN_F16 || a.kv_type == ATTN_BF16) {
    // rows per CTA: one while that leaves at most 8 CTAs per SM, else as many
    // as keep it there
    const int rpc = (int)std::max<int64_t>(1, ((int64_t)a.n_rows + 8LL * sms - 1) / (8LL * sms));
    const int64_t blocks = ((int64_t)a.n_rows + rpc - 1) / rpc;
    return a.kv_type == ATTN_F16 ? launch_pdl(append_copy_kernel<NEW, ATTN_F16>, blocks, stream, a, rpc)
                                 : launch_pdl(append_copy_kernel<NEW, ATTN_BF16>, blocks, stream, a, rpc);
  }
  const int64_t blocks = ((int64_t)a.n_rows * a.n_head_kv * 32 + kApThreads - 1) / kApThreads;
  const bool e4 = a.kv_type == ATTN_FP8_E4M3;
  switch (a.head_dim) {
    case 64: return e4 ? launch_pdl(append_quant_kernel<NEW, true, 64>, blocks, stream, a)
                       : launch_pdl(append_quant_kernel<NEW, false, 64>, blocks, stream, a);
    case 128: return e4 ? launch_pdl(append_quant_kernel<NEW, true, 128>, blocks, stream, a)
                        : launch_pdl(append_quant_kernel<NEW, false, 128>, blocks, stream, a);
    default: return e4 ? launch_pdl(append_quant_kernel<NEW, true, 256>, blocks, stream, a)
                       : launch_pdl(append_quant_kernel<NEW, false, 256>, blocks, stream, a);
  }
}

}  // namespace

cudaError_t launch_append_paged(const attn_append_args& a, int sms, cudaStream_t stream) {
  switch (a.new_type) {
    case ATTN_F32: return launch_new<ATTN_F32>(a, sms, stream);
    case ATTN_F16: return launch_new<ATTN_F16>(a, sms, stream);
    default: return launch_new<ATTN_BF16>(a, sms, stream);
  }
}

}  // namespace attn
