// What the kernels of attention over the paged 8-bit cache share: how the work
// is dealt out, and the kernel that joins the parts.  A unit is (sequence, KV
// head, group of query rows); its keys come in steps.  The steps of all units,
// one after another, are dealt out evenly over the workers of the grid: worker
// w takes steps [w per, (w + 1) per).
#pragma once

#include <cuda_fp16.h>

#include <algorithm>

#include "moe_attention.cuh"
#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_kv.cuh"

namespace moe {
namespace {

constexpr float kGrow = 8.0f;    // log2 growth over a row's reference that moves it
constexpr int kPBits = 6;        // p <= 2^8 enters the MMA times 2^6: below 2^16
constexpr int kSeqCache = 256;   // sequences whose lengths are kept in shared memory

// Rows of a unit, tokens of a step, fewest steps that a worker takes.
template <int ROWS, int STEP, int MIN>
struct DealOf {
  static constexpr int kRows = ROWS, kStep = STEP, kMinSteps = MIN;
};

// The two E4M3 codes in the low half of w as f16x2.
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
  uint32_t r;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}\n"
      : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t codes_f16_hi(uint32_t w) {
  uint32_t r;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, hi;\n}\n"
      : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

// 2^(byte - 127) for a scale byte.
__device__ __forceinline__ float byte_scale(int byte) {
  return __uint_as_float(byte ? static_cast<uint32_t>(byte) << 23 : 0x00400000u);
}
// A score's factor from its parts.  Finite: beside an infinite key the other keys of
// its block are zeros, whose scores are 0 and not 0 x inf.
__device__ __forceinline__ float score_factor(float key_scale, float row_scale) {
  return fminf(key_scale * row_scale, 3.402823466e38f);
}
// 2^k, 0 below the normal range.
__device__ __forceinline__ float pow2i(int k) {
  return k < -126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(min(k, 127) + 127) << 23);
}

// What O is in units of while a unit's blocks of values, each with a scale of its
// own, go by.  A weight enters the second product as f16 p 2^6 2^(X - ref), X the
// scale byte of its value block, O in units of 2^(ref - 127 - 6).  f16 has its 11
// bits down to 2^-14 and nothing below 2^-25, so X may lie at most kNear under
// ref: a weight of 2^-16 of its row's largest then still has all of them, and
// what is lost at the low end is 2^-27 of the largest.  ref follows the blocks up
// and down, from kLeast to kMost (block maxima of 2^-55 to 2^25; O is moved with it,
// exactly in fp32).  A step of blocks further apart, or beyond these, makes the unit
// `far` for the rest of its steps here: each block is then added to O by itself, in
// fp32, and O is in units of 2^(kFarRef - 127 - 6).  That holds values of 2^-100 to
// 2^110 beside each other, whatever their blocks' scales and weights.
// Blocks with byte 0 (no value above 2^-118; zeros, as a rule) are left out of
// account.
constexpr int kNear = 4, kLeast = 64, kMost = 144, kFarRef = 151;
// Whether ref serves for a step whose blocks' bytes lie in lo .. hi (255 .. 0: none).
__device__ __forceinline__ bool units_hold(int ref, int lo, int hi) {
  return hi <= ref && lo >= ref - kNear;
}
// The ref that does (ref: the last one, 0 before any values), -1: none, it is far.
__device__ __forceinline__ int next_units(int ref, int lo, int hi) {
  const int top = max(ref, hi);
  const int next = lo < top - kNear ? hi : top;
  const bool near = lo >= next - kNear &&
                    (next == 0 || static_cast<unsigned>(next - kLeast) <= kMost - kLeast);
  return near ? next : -1;
}

// One sequence, with indexes that do not fit turned into nothing to do: offsets
// into no rows, a length into no keys.
struct Seq {
  int row0, fresh, len;  // rows of q and their number, keys
};
// Its units: row groups, steps of each (1 without keys: the zeros still have
// to be written), steps over all heads and row groups.
struct SeqWork {
  int groups, steps;
  long long weight;
};

__device__ __forceinline__ Seq read_seq(const KvAttention& a, int s) {
  Seq q;
  q.row0 = __ldg(a.offsets + s);
  q.fresh = __ldg(a.offsets + s + 1) - q.row0;
  q.len = __ldg(a.kv_lens + s);
  const long long most = static_cast<long long>(a.max_pages) * a.cache.page;
  const bool bad_rows =
      q.row0 < 0 || q.fresh < 0 || q.row0 + static_cast<long long>(q.fresh) > a.T;
  if (bad_rows || q.len < 0 || q.len > most) {
    atomicOr(a.status, kStatusDeviceCheck);
    if (bad_rows) q.fresh = 0;
    if (q.len < 0 || q.len > most) q.len = 0;
  }
  return q;
}

template <class Deal>
__device__ __forceinline__ SeqWork work_of(const KvAttention& a, const Seq& q) {
  SeqWork w;
  w.groups = static_cast<int>((static_cast<long long>(q.fresh) * a.group + Deal::kRows - 1) / Deal::kRows);
  w.steps = max(1, (q.len + Deal::kStep - 1) / Deal::kStep);
  w.weight = static_cast<long long>(w.steps) * w.groups * a.cache.heads;
  return w;
}

// Steps that each of the grid's workers takes.
template <class Deal>
__device__ __forceinline__ long long share_of(long long total, int workers) {
  return max(static_cast<long long>(Deal::kMinSteps), (total + workers - 1) / workers);
}

// A worker's share of the steps, walked unit by unit.
template <class Deal>
struct Walk {
  Seq q;
  int groups, steps;         // of the sequence
  int s, head, group, step;  // current unit, its first step of this share
  long long left;            // steps of the share still to come, this unit's among them
  __device__ __forceinline__ int end() const {
    return static_cast<int>(min(static_cast<long long>(steps), step + left));
  }
  __device__ __forceinline__ bool next(const KvAttention& a, const Seq* cache) {
    left -= end() - step;
    if (left <= 0) return false;
    step = 0;
    if (++group < groups) return true;
    group = 0;
    if (++head < a.cache.heads) return true;
    head = 0;
    for (;;) {
      ++s;
      q = s < kSeqCache ? cache[s] : read_seq(a, s);
      const SeqWork w = work_of<Deal>(a, q);
      groups = w.groups;
      steps = w.steps;
      if (w.weight > 0) return true;
    }
  }
};

// The share of `left` steps that starts at step `first` of all, by a whole warp
// (there is such a step).  w: a walk, of this deal or of another.
template <class Deal, class W>
__device__ __forceinline__ void find_share(const KvAttention& a, const Seq* cache, long long first,
                                           long long left, W& w) {
  const int lane = threadIdx.x & 31;
  long long before = 0;
  for (int s0 = 0;; s0 += 32) {
    Seq q{};
    SeqWork k{};
    if (s0 + lane < a.n_seqs) {
      q = s0 + lane < kSeqCache ? cache[s0 + lane] : read_seq(a, s0 + lane);
      k = work_of<Deal>(a, q);
    }
    long long c = k.weight;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += u;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + c > first);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        const long long at = first - (before + c - k.weight);
        const int unit = static_cast<int>(at / k.steps);
        w.q = q;
        w.groups = k.groups;
        w.steps = k.steps;
        w.s = s0 + lane;
        w.head = unit / k.groups;
        w.group = unit - w.head * k.groups;
        w.step = static_cast<int>(at - static_cast<long long>(unit) * k.steps);
        w.left = left;
      }
      break;
    }
    before += __shfl_sync(0xffffffffu, c, 31);
  }
}

__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

// Adds a part with maximum m, sum l and u = O / l (O itself if `weighted`) to a
// running maximum, sum and O.
__device__ __forceinline__ void add_part(float& top, float& sum, float4& v, float m, float l,
                                         float4 u, bool weighted = false) {
  const float nt = fmaxf(top, m);
  const float at = nt == -INFINITY ? 0.0f : nt;
  const float old = ex2(top - at), f = ex2(m - at);
  const float wu = weighted ? f : l * f;
  top = nt;
  sum = sum * old + l * f;
  v.x = v.x * old + wu * u.x;
  v.y = v.y * old + wu * u.y;
  v.z = v.z * old + wu * u.z;
  v.w = v.w * old + wu * u.w;
}

// Four columns of a result row, and the logarithm of its sum.
template <int D>
__device__ __forceinline__ void write_row(const KvAttention& a, int row0, int head, int row,
                                          int col, float m, float l, float4 u) {
  const int i = row / a.group;
  const size_t to =
      static_cast<size_t>(row0 + i) * a.heads + head * a.group + (row - i * a.group);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to * D + col) =
      make_uint2(pack_bf16x2(u.x, u.y), pack_bf16x2(u.z, u.w));
  if (col == 0 && a.lse) a.lse[to] = log_sum(m, l);
}

// Adds the parts of the units of one sequence and head, in an order that the
// lengths alone decide.  A warp takes a row (its lanes four columns each) and,
// where there are more warps than rows, a share of the parts.  Few units of
// many parts have their rows split over several CTAs, up to two an SM (6
// sequences of up to 131000 keys, 8 heads, L2 flushed before each call: 199 us in all
// instead of 209; four an SM cost 64 shorter sequences 3 us).
constexpr int kJoinWarps = 16;
constexpr int kJoinAt = 4;  // parts that a warp has under way
template <int D, class Deal>
__global__ void __launch_bounds__(kJoinWarps * 32)
    moe_kv_attention_join_kernel(const KvAttention a, int workers) {
  constexpr int ROWS = Deal::kRows;
  const int here = ROWS / gridDim.z;          // rows of this CTA
  const int turn = min(here, kJoinWarps);     // at a time
  const int shares = kJoinWarps / turn;       // of the parts
  __shared__ long long s_before[kJoinWarps], s_total[kJoinWarps];
  __shared__ float4 s_v[kJoinWarps][32];
  __shared__ float2 s_ml[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.x, head = blockIdx.y;
  // What the lengths say is there before the parts are: the first kernel's CTAs
  // let this one start only after their own wait.
  long long before = 0, total = 0;
  for (int i = threadIdx.x; i < a.n_seqs; i += kJoinWarps * 32) {
    const long long k = work_of<Deal>(a, read_seq(a, i)).weight;
    total += k;
    if (i < s) before += k;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    s_before[warp] = before;
    s_total[warp] = total;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    before += s_before[i];
    total += s_total[i];
  }
  const Seq q = read_seq(a, s);
  const SeqWork k = work_of<Deal>(a, q);
  const long long per = share_of<Deal>(total, workers);
  pdl_wait_and_release();
  for (int group = 0; group < k.groups; ++group) {
    const long long begin = before + (static_cast<long long>(head) * k.groups + group) * k.steps;
    const long long first = begin / per;
    const int parts = static_cast<int>((begin + k.steps - 1) / per - first) + 1;
    if (parts == 1) continue;
    const int rows = min(ROWS, q.fresh * a.group - group * ROWS);
    const float* p0 = a.partial + (static_cast<size_t>(first) * 2 + 1) * ROWS * (D + 2);
    for (int rr = 0; rr < here; rr += turn) {
      const int r = blockIdx.z * here + rr + warp % turn, share = warp / turn;
      float top = -INFINITY, sum = 0.0f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      const bool mine = r < rows && lane < D / 4;
      if (mine) {
        for (int i0 = share; i0 < parts; i0 += kJoinAt * shares) {
          float2 ml[kJoinAt], u0[kJoinAt], u1[kJoinAt];
#pragma unroll
          for (int i = 0; i < kJoinAt; ++i) {
            const int part = i0 + i * shares;
            if (part >= parts) continue;
            // part 0 is the second slot of its warp, the others the first of theirs
            const float2* src = reinterpret_cast<const float2*>(
                p0 + (part == 0 ? 0 : (static_cast<size_t>(part) * 2 - 1) * ROWS * (D + 2)) +
                r * (D + 2));
            ml[i] = __ldcg(src + D / 2);
            u0[i] = __ldcg(src + 2 * lane);
            u1[i] = __ldcg(src + 2 * lane + 1);
          }
#pragma unroll
          for (int i = 0; i < kJoinAt; ++i) {
            if (i0 + i * shares >= parts) continue;
            add_part(top, sum, v, ml[i].x, ml[i].y,
                     make_float4(u0[i].x, u0[i].y, u1[i].x, u1[i].y));
          }
        }
      }
      if (shares > 1) {
        __syncthreads();
        s_v[warp][lane] = v;
        if (lane == 0) s_ml[warp] = make_float2(top, sum);
        __syncthreads();
        if (share == 0)
          for (int i = 1; i < shares; ++i)
            add_part(top, sum, v, s_ml[warp + i * turn].x, s_ml[warp + i * turn].y,
                     s_v[warp + i * turn][lane], true);
      }
      if (mine && share == 0) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        write_row<D>(a, q.row0, head, group * ROWS + r, 4 * lane, top, sum,
                     make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
      }
    }
  }
}

// steps: the most a unit has.
template <int D, class Deal>
cudaError_t launch_join(cudaStream_t s, const KvAttention& a, long long steps, int workers) {
  if (steps <= 1) return cudaSuccess;  // units of one step are not split
  const long long joins = static_cast<long long>(a.n_seqs) * a.cache.heads;
  const long long parts = std::min(workers / joins, steps / Deal::kMinSteps + 1);  // of a unit
  unsigned split = 1;
  while (split < Deal::kRows && joins * split * 2 <= 2LL * device_sm_count() &&
         parts * Deal::kRows > static_cast<long long>(kJoinWarps) * kJoinAt * split)
    split *= 2;
  KernelScope scope(s, "moe_kv_attention_join");
  return launch_kernel(moe_kv_attention_join_kernel<D, Deal>,
                       dim3(static_cast<unsigned>(a.n_seqs), static_cast<unsigned>(a.cache.heads), split),
                       dim3(kJoinWarps * 32), 0, s, a, workers);
}

}  // namespace
}  // namespace moe
