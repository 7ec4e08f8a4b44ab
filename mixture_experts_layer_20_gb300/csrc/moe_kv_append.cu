// Writes new keys and values into a paged 8-bit cache ('PagedAttention,
// speculative decoding, MoE and Blackwell', section 1: the cache in fixed
// pages behind a block table; 'Hosting Qwen on Blackwell': pages laid out
// head by head).
//
// A block is 16 consecutive tokens of one sequence and KV head, keys and
// values apart.  It holds E4M3 codes and one power of two 2^(X - 127) by the
// MXFP8 rule of the weights: X = floor(log2 amax) - 8 + 127 clamped to
// 0..254, values x 2^(127 - X) rounded to nearest even and saturated at
// +-448, -0 as +0.  A block that already held tokens keeps the larger of its
// stored X and the new tokens' X; where that grows, the codes held are scaled
// down by the (exact) power of two and rounded again.
//
// Bound by memory: 2 bytes read and 1 written per value.  One warp takes one
// (block, head): its 2 x 16 x D values are loaded at once (sixteen 16-byte
// loads a lane for D = 128), so the amax and the codes come from one read and
// the chain of dependent loads before it (sequence, length, page) is paid once
// for K and V.  Measured: 64 sequences with one new token, 4 heads of 128: 6.6 us
// (that chain and the launch); 6000 new tokens of 8 heads: 13.5 us, 2.7 TB/s.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "moe_internal.h"
#include "moe_kv.cuh"

namespace moe {
namespace {

constexpr int kAppendWarps = 4;

__device__ __forceinline__ uint32_t drop_minus_zero(uint32_t w) {
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (((w >> (8 * b)) & 0xffu) == 0x80u) w &= ~(0xffu << (8 * b));
  return w;
}

// Eight values times 2^k (k in -127 .. 127, exact but for underflow) as codes.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float mul) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * h] * mul, v[4 * h + 1] * mul), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * h + 2] * mul, v[4 * h + 3] * mul), __NV_SATFINITE, __NV_E4M3);
    w[h] = drop_minus_zero(static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16));
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float2 decode2(uint32_t two) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32) moe_kv_append_kernel(const KvAppend a) {
  constexpr int kLanes = D / 8;            // lanes of one token's row
  constexpr int kPerLoad = 32 / kLanes;    // tokens a warp load covers
  constexpr int kLoads = kKvBlock / kPerLoad;
  pdl_wait_and_release();
  const int lane = threadIdx.x & 31;
  const int head = blockIdx.y * kAppendWarps + (threadIdx.x >> 5);
  if (head >= a.cache.heads) return;

  // Sequence s owns the slots from offsets[s] / 16 + 2 s on: at least as many
  // as the blocks that its new tokens can touch.
  const int slot = blockIdx.x;
  // Offsets that go down may hide their sequence from the search below: the first
  // n_seqs slots look at one sequence's each.
  if (slot < a.n_seqs && head == 0 && lane == 0) {
    const int from = __ldg(a.offsets + slot), to = __ldg(a.offsets + slot + 1);
    if (from < 0 || to < from || to > a.T) atomicOr(a.status, kStatusDeviceCheck);
  }
  const int s = warp_find(a.n_seqs, [&](int i) { return __ldg(a.offsets + i) / kKvBlock + 2 * i <= slot; });
  const int t0 = __ldg(a.offsets + s), t1 = __ldg(a.offsets + s + 1);
  const int len = __ldg(a.kv_lens + s);
  const int fresh = t1 - t0;
  if (t0 < 0 || fresh < 0 || t1 > a.T || len < fresh ||
      len > a.max_pages * static_cast<long long>(a.cache.page)) {
    if (lane == 0) atomicOr(a.status, kStatusDeviceCheck);
    return;
  }
  const int first = len - fresh;  // position of the first new token
  const int block = first / kKvBlock + (slot - (t0 / kKvBlock + 2 * s));
  // (positions go up to 2^31 - 1: none past the last block is computed)
  if (slot < t0 / kKvBlock + 2 * s || fresh == 0 || block > (len - 1) / kKvBlock) return;
  const int begin = max(first, block * kKvBlock);
  const int end = block * kKvBlock + min(len - block * kKvBlock, kKvBlock);
  const int page = __ldg(a.block_table + static_cast<size_t>(s) * a.max_pages +
                         block * kKvBlock / a.cache.page);

  // The new values, whatever page they go to.
  uint4 raw[2][kLoads];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(kv ? a.v : a.k) +
                               static_cast<size_t>(head) * D + (lane % kLanes) * 8;
    const long long stride = kv ? a.v_stride : a.k_stride;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int pos = block * kKvBlock + i * kPerLoad + lane / kLanes;
      raw[kv][i] = make_uint4(0, 0, 0, 0);
      if (pos >= begin && pos < end)
        raw[kv][i] = __ldg(reinterpret_cast<const uint4*>(src + (t0 + pos - first) * stride));
    }
  }
  if (page < 0 || page >= a.cache.pages) {
    if (lane == 0) atomicOr(a.status, kStatusDeviceCheck);
    return;
  }
  const int in_page = block * kKvBlock % a.cache.page;
  const int held = begin - block * kKvBlock;
  auto row_of = [&](int kv) {
    return (static_cast<size_t>(page) * 2 + kv) * a.cache.heads + head;
  };
  auto scale_of = [&](int kv) {
    return a.cache.scales + row_of(kv) * (a.cache.page / kKvBlock) + in_page / kKvBlock;
  };
  int stored[2] = {0, 0};
  if (held) {
    stored[0] = min(static_cast<int>(*scale_of(0)), 254);
    stored[1] = min(static_cast<int>(*scale_of(1)), 254);
  }

#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t* codes = a.cache.codes + (row_of(kv) * a.cache.page + in_page) * D + (lane % kLanes) * 8;
    // the largest magnitude: bf16 patterns without their signs order as numbers
    // do, and those above infinity (NaN) count as nothing
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t w[4] = {raw[kv][i].x, raw[kv][i].y, raw[kv][i].z, raw[kv][i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
        top = max(top, lo > 0x7f80u ? 0u : lo);
        top = max(top, hi > 0x7f80u ? 0u : hi);
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    // floor(log2 amax) - 8 + 127 is the exponent field less 8 (0 for smaller values)
    const int need = max(0, static_cast<int>(top >> 7) - 8);
    const int byte = held ? max(stored[kv], need) : need;

    if (held && byte > stored[kv]) {
      const int down = byte - stored[kv];  // 2^-down; past 2^-126 every code becomes 0
      const float mul = down > 126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 - down) << 23);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = i * kPerLoad + lane / kLanes;
        if (at >= held) continue;
        uint2* c = reinterpret_cast<uint2*>(codes + static_cast<size_t>(at) * D);
        const uint2 old = *c;
        const float2 x0 = decode2(old.x), x1 = decode2(old.x >> 16), x2 = decode2(old.y),
                     x3 = decode2(old.y >> 16);
        const float v[8] = {x0.x, x0.y, x1.x, x1.y, x2.x, x2.y, x3.x, x3.y};
        *c = encode8(v, mul);
      }
    }
    // 2^(127 - byte); 2^-127, for byte 254, is subnormal
    const float mul =
        __uint_as_float(byte == 254 ? 0x00400000u : static_cast<uint32_t>(254 - byte) << 23);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = i * kPerLoad + lane / kLanes;
      const int pos = block * kKvBlock + at;
      if (pos < begin || pos >= end) continue;
      const uint32_t w[4] = {raw[kv][i].x, raw[kv][i].y, raw[kv][i].z, raw[kv][i].w};
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
      *reinterpret_cast<uint2*>(codes + static_cast<size_t>(at) * D) = encode8(v, mul);
    }
    if (lane == 0) *scale_of(kv) = static_cast<uint8_t>(byte);
  }
}

}  // namespace

cudaError_t launch_kv_append(cudaStream_t s, const KvAppend& a) {
  const long long slots = a.T / kKvBlock + 2LL * a.n_seqs + 1;
  const dim3 grid(static_cast<unsigned>(slots),
                  static_cast<unsigned>((a.cache.heads + kAppendWarps - 1) / kAppendWarps));
  KernelScope scope(s, "moe_kv_append");
  return a.cache.dim == 64
             ? launch_kernel(moe_kv_append_kernel<64>, grid, dim3(kAppendWarps * 32), 0, s, a)
             : launch_kernel(moe_kv_append_kernel<128>, grid, dim3(kAppendWarps * 32), 0, s, a);
}

}  // namespace moe
