// Attention of new tokens over the paged 8-bit cache where a unit has many
// query rows (drafted tokens, large groups; head dimension 128): the same work
// and results as moe_kv_attention.cu, with both products on tcgen05.
//
// Warp MMAs of 32 query rows cost about 900 instructions per 32 tokens, and
// with 7 warps an SM they, not the memory, set the pace (4.9 of 6.8 TB/s; 32
// sequences of up to 6000 with 4 new tokens, 64 heads over 8: 82 us, here 77 us
// or 3.6 TB/s).  With 16 rows both do as well (45 and 48 us for 64 sequences of
// 4096): those stay with the warp MMAs.
// Here a group of four warps takes 128 tokens at a time, one token a thread:
//   S^T [token, row] = K Q^T: each thread turns its token's codes into f16
//     (exact) and stores them to tensor memory, the MMA's A operand; Q is B;
//   P^T: each thread has its token's scores of all rows, so the running sums
//     stay in the threads until the unit's end, and a row's reference m moves
//     only when some score passes it by 2^8 (one vote a step);
//   O^T [column, row] += V^T P^T: V as f16 in shared memory, read M-major, so
//     that the transposition costs nothing; P as f16 2^6 2^(X - ref), X the
//     block's value scale and ref the unit's (next_units).
// Where value scales lie far apart, O's part of a step is added up in fp32
// instead (far_steps): no block's scale takes bits from another's weights.
// Two groups an SM, each with its own share of the steps, its own loading warp
// and a ring of 64-token halves of K and V; the loading warp looks pages up
// two steps and scales one step ahead.
//
// What bounds it now: a group's step takes 3300 cycles, a chain of its own
// latencies (the two conversions, a vote, exponentials, the P stores), against
// 2800 that the memory would allow; a change of unit costs 7000, the start 5 us
// and the join 5 us.

#include <climits>

#include "moe_kv_attention.cuh"

namespace moe {
namespace {

constexpr int D = 128;
constexpr int ROWS = 32;          // query rows of a unit
constexpr int kGroups = 2;        // of four warps, an SM
constexpr int kTokens = 128;      // of a step
constexpr int kHalfBytes = 64 * D;
constexpr int kSlots = 7;         // of 64 tokens' codes, K or V, in a group's ring
constexpr int kScaleSlots = 4;    // steps whose scales are kept
constexpr int kThreads = (kGroups + 1) * 128;  // the last warpgroup: a loading and an MMA warp a group
constexpr int kBars = 2 * kSlots + 4;
constexpr uint32_t kGroupCols = 256;           // tensor memory: K, S, O; a far unit's O, sums
constexpr uint32_t kColS = 64, kColO = 96, kColFar = 128, kColFarSum = 160;

using Deal = DealOf<ROWS, kTokens, 1>;
constexpr int kVBytes = kTokens * D * 2;     // V as f16
constexpr int kPBytes = ROWS * kTokens * 2;  // P as f16
constexpr int kQBytes = ROWS * D * 2;        // Q as f16
constexpr int kGroupBytes = kSlots * kHalfBytes + kVBytes + kPBytes + kQBytes;
constexpr int kSmem = 1024 + kGroups * kGroupBytes;

// f16 in, fp32 out; A from tensor memory, or M-major from shared memory.
__device__ constexpr uint32_t idesc_f16(int n, bool a_m_major) {
  return (1u << 4) | (a_m_major ? 1u << 15 : 0u) | (static_cast<uint32_t>(n / 8) << 17) |
         (static_cast<uint32_t>(128 / 16) << 24);
}

// The four warps of a group.
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(group + 1) : "memory");
}
__device__ __forceinline__ bool group_any(int group, bool v) {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "setp.ne.u32 p, %2, 0;\n"
      "barrier.cta.red.or.pred q, %1, 128, p;\n"
      "selp.u32 %0, 1, 0, q;\n"
      "}\n"
      : "=r"(r)
      : "r"(group + 1), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x) {
  asm volatile("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\nst.shared.b16 [%0], lo;\n}\n" ::"r"(a),
               "r"(x)
               : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Floats in the order of signed integers (NaN counts as -infinity).
__device__ __forceinline__ int ordered(float v) {
  const int i = __float_as_int(fmaxf(v, -INFINITY));
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) {
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// A group's ring: slot of its n-th half (K first, K second, V first, V second
// of each step), and the phase its barriers are in.
struct Half {
  uint32_t slot, phase;
  __device__ __forceinline__ explicit Half(uint32_t n) : slot(n % kSlots), phase(n / kSlots & 1) {}
};

__device__ __forceinline__ void load_group(const KvAttention& a, const CUtensorMap* map, Walk<Deal> w,
                                           const Seq* cache, uint8_t (*scales)[16], uint32_t* range,
                                           uint32_t ring, uint32_t full, uint32_t empty,
                                           const WaitCtx& wc) {
  const int lane = threadIdx.x & 31;
  const int P = a.cache.page, ps = __ffs(P) - 1, box = min(P, 32);  // P is a power of two
  const int block = lane & 7;  // of the step, that this lane is for
  // A step, as far as it is known.
  struct Step {
    bool there;
    int at, len, head;  // of this lane's block: position; keys of the sequence
    int page;           // lanes 0 .. 7; -1: past the end, or
    bool none;          // outside the pool
    int scale;          // lanes 0 .. 7 K's, 8 .. 15 V's
  };
  bool more = true;
  int t = 0, t1 = 0;
  auto unit = [&]() {
    while (more && w.q.len == 0) more = w.next(a, cache);
    if (more) {
      t = w.step;
      t1 = w.end();
    }
  };
  unit();
  auto look_up = [&]() {
    Step s{};
    s.there = more;
    if (!more) return s;
    s.at = t * kTokens + block * kKvBlock;
    s.len = w.q.len;
    s.head = w.head;
    s.page = -1;
    if (lane < 8 && s.at < s.len)
      s.page = __ldg(a.block_table + static_cast<size_t>(w.s) * a.max_pages + (s.at >> ps));
    if (++t >= t1) {
      more = w.next(a, cache);
      unit();
    }
    return s;
  };
  auto ask_scales = [&](Step& s) {
    if (!s.there) return;
    const bool in = s.at < s.len;
    s.page = __shfl_sync(0xffffffffu, s.page, block);
    const bool ok = s.page >= 0 && s.page < a.cache.pages;
    if (in && !ok && lane < 8) atomicOr(a.status, kStatusDeviceCheck);
    if (!in || !ok) s.page = -1;
    s.none = in && !ok;
    s.scale = 0;
    if (lane < 16 && s.page >= 0)
      s.scale = __ldg(a.cache.scales +
                      ((static_cast<size_t>(s.page * 2 + (lane >> 3)) * a.cache.heads + s.head)
                       << (ps - 4)) +
                      (s.at & (P - 1)) / kKvBlock);
  };
  Step s0 = look_up(), s1 = look_up();
  ask_scales(s0);
  uint32_t n = 0;  // halves issued
  bool ok = true;
  for (int step = 0; s0.there; ++step) {
    Step s2 = look_up();
    ask_scales(s1);
    for (int part = 0; part < 4 && ok; ++part) {
      const Half h(n);
      ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * h.slot, h.phase ^ 1u, wc));
      if (!ok) break;
      const bool mine = lane < 8 && (block >> 2) == (part & 1) && s0.page >= 0 &&
                        (s0.at & (box - 1)) == 0;
      const unsigned boxes = __popc(__ballot_sync(0xffffffffu, mine));
      if (mine)
        tma_load_2d(ring + h.slot * kHalfBytes + (block & 3) * (kKvBlock * D), map,
                    full + 8 * h.slot, 0,
                    (((s0.page * 2 + (part >> 1)) * a.cache.heads + s0.head) << ps) +
                        (s0.at & (P - 1)));
      // the scales may still be on their way: they go with the first arrival
      if (part == 0) {
        const unsigned v = lane >= 8 && lane < 16 ? s0.scale : 0;  // the values'
        const unsigned hi = __reduce_max_sync(0xffffffffu, v);
        const unsigned lo = __reduce_min_sync(0xffffffffu, v ? v : 255u);
        if (lane < 16) scales[step % kScaleSlots][lane] = static_cast<uint8_t>(s0.scale);
        const unsigned none = __ballot_sync(0xffffffffu, lane < 8 && s0.none);
        if (lane == 0) range[step % kScaleSlots] = lo | hi << 8 | none << 16;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(full + 8 * h.slot, boxes * box * D);
      ++n;
    }
    if (!ok) break;
    s0 = s1;
    s1 = s2;
  }
  if (!ok && lane == 0)  // the last loads may still be landing
    for (uint32_t i = n > kSlots ? n - kSlots : 0; i < n; ++i) {
      const Half h(i);
      mbar_wait_drain(full + 8 * h.slot, h.phase, a.status);
    }
}

// What a step that holds the sequence's end, a block without a page, or new tokens
// that some rows do not see, needs before a token's values (a row at `src`, its
// 16-byte units turned by x; `at`: see step_token) meet the MMAs.  Codes past the end
// are whatever was in the page, those without one whatever the ring held: they
// become zeros.  A NaN among the new tokens concerns only the rows that see its
// token, but would meet the others' p = 0: it becomes zero too, and
// nan_from[column] keeps the first position of one, for the end of the unit.
__device__ __noinline__ void clean_row(uint32_t src, int x, int at, int len, int fresh,
                                       int* nan_from, int* nans) {
  if (at > len - fresh) {
#pragma unroll 1
    for (int u = 0; u < 8; ++u) {
      const uint32_t addr = src + ((u ^ x) << 4);
      if (at >= len) {
        sts128(addr, 0, 0, 0, 0);
        continue;
      }
      const uint4 v = lds128(addr);
      uint32_t c[4] = {v.x, v.y, v.z, v.w}, any = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) any |= (c[i] & 0x7f7f7f7fu) + 0x01010101u;
      if (!(any & 0x80808080u)) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int shift = 8 * (i & 3);
        if ((c[i >> 2] >> shift & 0x7f) == 0x7f) {
          c[i >> 2] &= ~(0xffu << shift);
          atomicMin(&nan_from[u * 16 + i], at);
          *nans = 1;
        }
      }
      sts128(addr, c[0], c[1], c[2], c[3]);
    }
    // TMA writes here next
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncwarp();
}

// A group's MMAs, by one warp: at each unit's start S of its first step, then
// for each step O += V P and S of the next.
__device__ __forceinline__ void issue_group(const KvAttention& a, Walk<Deal> w, const Seq* cache,
                                            uint32_t tm, uint32_t q_smem,
                                            uint32_t p_smem, uint32_t v_smem, uint32_t s_done,
                                            uint32_t o_done, uint32_t ready, const WaitCtx& wc) {
  const bool leader = elect_one();
  const uint32_t q_desc = desc_k(q_smem), p_desc = desc_k(p_smem),
                 v_desc = desc_n(v_smem, kTokens * 128);
  uint32_t n = 0;
  auto wait = [&]() {
    mbar_wait(ready, n & 1, wc);
    __syncwarp();
    ++n;
    tc_fence_after_sync();
  };
  auto scores = [&]() {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      mma_ts(leader, tm + kColS, tm + 8 * i, q_desc + ((i / 4) * (ROWS * 128) + (i % 4) * 32) / 16,
             idesc_f16(ROWS, false), i != 0);
    commit(leader, s_done);
  };
  for (bool more = true; more; more = w.next(a, cache)) {
    const int t0 = w.step, t1 = w.end();
    if (w.q.len == 0) continue;
    wait();
    scores();
    for (int t = t0; t < t1; ++t) {
      wait();
#pragma unroll
      for (int i = 0; i < kTokens / 16; ++i)
        mma_ss(leader, tm + kColO, v_desc + i * (2048 / 16),
               p_desc + ((i / 4) * (ROWS * 128) + (i % 4) * 32) / 16, idesc_f16(ROWS, true),
               t != t0 || i != 0);
      commit(leader, o_done);
      if (t + 1 < t1) scores();
    }
  }
}

// One thread of a group: its group's places, and its own.
struct GroupAt {
  uint32_t ring, full, empty, s_done, o_done, ready;
  uint32_t v_smem, q_smem, p_smem;
  uint32_t mine;  // tensor memory, at this warp's lanes
  int group, tid, half;  // tid: token of a step, column of O; half: of the step's tokens
};

// The K half of step i (of this group's, in turn) into tensor memory.  Here and
// below: whether no wait has given up, in the warp, so far.  After one that has no
// slot of the ring is given back: its load may still be under way, and another
// arrival in that phase of its barrier would be one too many.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t phase, const WaitCtx& wc, bool ok) {
  return __all_sync(0xffffffffu, mbar_wait(bar, phase, wc)) && ok;
}
__device__ __forceinline__ bool take_k(const GroupAt& g, uint32_t i, const WaitCtx& wc, bool ok) {
  const Half h(4 * i + g.half);
  ok = wait_all(g.full + 8 * h.slot, h.phase, wc, ok);
  const uint32_t src = g.ring + h.slot * kHalfBytes + static_cast<uint32_t>(g.tid & 63) * D;
  const int x = g.tid & 7;  // swizzle of this token's rows
  uint4 k[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) k[u] = lds128(src + ((u ^ x) << 4));
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    uint32_t f[32];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t v[4] = {k[4 * hh + u].x, k[4 * hh + u].y, k[4 * hh + u].z, k[4 * hh + u].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[8 * u + 2 * j] = codes_f16(v[j]);
        f[8 * u + 2 * j + 1] = codes_f16_hi(v[j]);
      }
    }
    tmem_st_x32(g.mine + 32 * hh, f);
  }
  __syncwarp();
  if ((g.tid & 31) == 0 && ok) mbar_arrive(g.empty + 8 * h.slot);
  return ok;
}
// V of step n as f16, over the last one (whose product is complete).
__device__ __forceinline__ bool take_v(const GroupAt& g, uint32_t n, bool zone, int at, int len,
                                       int fresh, int* nan_from, int* nans, const WaitCtx& wc,
                                       bool ok) {
  const Half h(4 * n + 2 + g.half);
  ok = wait_all(g.full + 8 * h.slot, h.phase, wc, ok);
  const uint32_t src = g.ring + h.slot * kHalfBytes + static_cast<uint32_t>(g.tid & 63) * D;
  const int x = g.tid & 7;
  if (zone) clean_row(src, x, at, len, fresh, nan_from, nans);
  uint4 v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u] = lds128(src + ((u ^ x) << 4));
  if (n > 0) ok = wait_all(g.o_done, (n - 1) & 1, wc, ok);
#pragma unroll
  for (int u = 0; u < 16; ++u) {  // 8 columns each
    const uint32_t lo = u & 1 ? v[u >> 1].z : v[u >> 1].x;
    const uint32_t hi = u & 1 ? v[u >> 1].w : v[u >> 1].y;
    sts128(g.v_smem + (u >> 3) * (kTokens * 128) + g.tid * 128 + (((u & 7) ^ x) << 4),
           codes_f16(lo), codes_f16_hi(lo), codes_f16(hi), codes_f16_hi(hi));
  }
  // Only now is the slot given back: the loads are known to be done where their values
  // have been used.  (Given back right after them, with the wait in between, some of
  // the loads were done after it, when the slot was being filled again.)
  __syncwarp();
  if ((g.tid & 31) == 0 && ok) mbar_arrive(g.empty + 8 * h.slot);
  return ok;
}
// This warp's operands are written: to the MMA warp.
__device__ __forceinline__ void hand_over(const GroupAt& g) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tmem_st_wait();
  tc_fence_before_sync();
  __syncwarp();
  if ((g.tid & 31) == 0) mbar_arrive(g.ready);
}

// What a CTA's threads share.
struct Shared {
  alignas(8) uint64_t bar[kGroups * kBars];
  Walk<Deal> walk[kGroups];
  alignas(16) float scale[kGroups][ROWS];   // of a row's scores, from its f16
  alignas(16) int limit[kGroups][ROWS];     // last position that a row sees
  alignas(16) float m[kGroups][ROWS];       // its reference
  alignas(16) float f[kGroups][ROWS];       // factors for all threads
  float red[kGroups][4][ROWS];
  alignas(16) uint8_t bytes[kGroups][kScaleSlots][16];
  // the values' bytes: smallest (but 0), largest; from bit 16 on, blocks on no page of
  // the pool
  uint32_t range[kGroups][kScaleSlots];
  int nan[kGroups][D];  // first position of a NaN among the new tokens' values
  int nans[kGroups];
  uint32_t tmem_base;
  int abort;
};

// Position of a thread's token in step t; past all where its block lies on no page.
__device__ __forceinline__ int step_token(uint32_t range, int t, int tid) {
  return range >> (16 + tid / kKvBlock) & 1 ? INT_MAX : t * kTokens + tid;
}

__device__ __forceinline__ GroupAt group_at(Shared& sh, uint32_t base, int group) {
  const uint32_t ring = base + group * kGroupBytes, full = smem_u32(&sh.bar[group * kBars]);
  const int tid = threadIdx.x & 127;
  GroupAt g;
  g.ring = ring;
  g.v_smem = ring + kSlots * kHalfBytes;
  g.q_smem = g.v_smem + kVBytes;
  g.p_smem = g.q_smem + kQBytes;
  g.full = full;
  g.empty = full + 8 * kSlots;
  g.s_done = full + 16 * kSlots;
  g.o_done = g.s_done + 8;
  g.ready = g.s_done + 16;
  g.mine = sh.tmem_base + group * kGroupCols + (static_cast<uint32_t>(tid & 96) << 16);
  g.group = group;
  g.tid = tid;
  g.half = tid >> 6;
  return g;
}

// The steps from t on of a group's unit whose value scales lie far apart (n: steps of
// this group so far), the first with its V in place and its scores at kColS: O += V P
// in fp32, 8 rows a warp, 4 columns a lane, so that no block's scale takes bits from
// another's weights.  O comes from kColO in units of 2^(was - 127 - kPBits) and goes to
// kColFar in units of 2^(kFarRef - 127 - kPBits), the sums are at kColFarSum; the MMA
// warp goes on as ever, what it adds up is not used.  32 sequences of up to 6000 with 4
// new tokens, 64 heads over 8, half of the value blocks 2^12 above the others: 381 us for
// 85 (L2 flushed).  Out of line: in line it cost a change of unit 2 us where the code
// is cold.
// Returns n after it, with the top bit where a wait gave up.
__device__ __noinline__ uint32_t far_steps(const KvAttention& a, Shared& sh, uint32_t base, int t,
                                           uint32_t n, int was) {
  const int group = threadIdx.x >> 7;
  const GroupAt g = group_at(sh, base, group);
  const WaitCtx wc{a.timeout_ns, a.status, &sh.abort};
  const Walk<Deal>& w = sh.walk[group];
  const int len = w.q.len, fresh = w.q.fresh, t1 = w.end();
  const int lane = g.tid & 31, quarter = g.tid >> 5, x = g.tid & 7;
  bool ok = true;
  uint64_t o[4][4];  // column 4 lane + c of rows 8 quarter + 2 j, + 1
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[c][j] = 0;
  if (t != w.step) {  // in the new units, in two factors (each a normal number)
    const int down = was - kFarRef;
    const float f0 = pow2i(down / 2), f1 = pow2i(down - down / 2);
    uint32_t r[ROWS];
    tmem_ld_x32(g.mine + kColO, r);
    tmem_ld_wait();
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // from a column a thread, 16 rows at a time
#pragma unroll
      for (int j = 0; j < 16; ++j)
        sts32(g.p_smem + (j * D + g.tid) * 4,
              __float_as_uint(__uint_as_float(r[16 * h + j]) * f0 * f1));
      group_sync(group);
      if ((quarter >> 1) == h) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t at = g.p_smem + ((8 * (quarter & 1) + 2 * j) * D + 4 * lane) * 4;
          const uint4 x0 = lds128(at), x1 = lds128(at + D * 4);
          o[0][j] = pair(__uint_as_float(x0.x), __uint_as_float(x1.x));
          o[1][j] = pair(__uint_as_float(x0.y), __uint_as_float(x1.y));
          o[2][j] = pair(__uint_as_float(x0.z), __uint_as_float(x1.z));
          o[3][j] = pair(__uint_as_float(x0.w), __uint_as_float(x1.w));
        }
      }
      group_sync(group);
    }
  }
  for (bool entry = true; t < t1; ++t, ++n, entry = false) {
    const uint32_t range = sh.range[group][n % kScaleSlots];
    const int at = step_token(range, t, g.tid);
    const bool zone = range >> 16 || t * kTokens + kTokens - 1 > len - fresh;
    if (!entry) {
      ok = take_v(g, n, zone, at, len, fresh, sh.nan[group], &sh.nans[group], wc, ok);
      ok = wait_all(g.s_done, n & 1, wc, ok);
      tc_fence_after_sync();
    }
    uint32_t s[ROWS];
    tmem_ld_x32(g.mine + kColS, s);
    const uint8_t* const bytes = sh.bytes[group][n % kScaleSlots];
    const float ks = byte_scale(bytes[g.tid / kKvBlock]);
    tmem_ld_wait();
    if (!entry && t + 1 < t1) ok = take_k(g, n + 1, wc, ok);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const float y = __uint_as_float(s[j]) * score_factor(ks, sh.scale[group][j]);
      s[j] = at > sh.limit[group][j] ? 0xff800000u : __float_as_uint(y);
      const int top = __reduce_max_sync(0xffffffffu, ordered(__uint_as_float(s[j])));
      if (lane == j) sh.red[group][quarter][j] = unordered(top);
    }
    group_sync(group);
    if (g.tid < ROWS) {
      const float old = sh.m[group][g.tid];
      const float u = fmaxf(fmaxf(sh.red[group][0][g.tid], sh.red[group][1][g.tid]),
                            fmaxf(sh.red[group][2][g.tid], sh.red[group][3][g.tid]));
      sh.f[group][g.tid] = u > old ? ex2(old - u) : 1.0f;
      sh.m[group][g.tid] = fmaxf(old, u);
    }
    group_sync(group);
    {
      uint32_t l[ROWS];
      tmem_ld_x32(g.mine + kColFarSum, l);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const float m = sh.m[group][j];
        const float p = ex2(__uint_as_float(s[j]) - (m == -INFINITY ? 0.0f : m));
        s[j] = __float_as_uint(p);
        l[j] = __float_as_uint(fmaf(__uint_as_float(l[j]), sh.f[group][j], p));
      }
      tmem_st_x32(g.mine + kColFarSum, l);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = *reinterpret_cast<const float2*>(&sh.f[group][8 * quarter + 2 * j]);
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c][j] = mul2(o[c][j], pair(f.x, f.y));
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {  // 64 tokens' weights at a time, where P has its place
      // a token's weights: 128 bytes, their 16-byte units turned by the token
      if ((g.tid >> 6) == i) {
#pragma unroll
        for (int u = 0; u < ROWS / 4; ++u)
          sts128(g.p_smem + (g.tid & 63) * (ROWS * 4) + ((u ^ x) << 4), s[4 * u], s[4 * u + 1],
                 s[4 * u + 2], s[4 * u + 3]);
      }
      group_sync(group);
      const uint32_t v = g.v_smem + (lane >> 4) * (kTokens * 128) + i * (64 * 128) + (lane & 1) * 8;
      const int unit = lane >> 1 & 7;  // of the columns, in a token's 128 bytes
#pragma unroll 1
      for (int b = 0; b < 64 / kKvBlock; ++b) {
        const float scale = byte_scale(bytes[8 + 4 * i + b]) * pow2i(127 - kFarRef + kPBits);
#pragma unroll 4
        for (int k = 0; k < kKvBlock; ++k) {
          const int token = b * kKvBlock + k;
          uint32_t h[2];
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                       : "=r"(h[0]), "=r"(h[1])
                       : "r"(v + token * 128 + ((unit ^ (k & 7)) << 4))
                       : "memory");
          const uint32_t row = g.p_smem + token * (ROWS * 4);
          const uint4 p0 = lds128(row + (((2 * quarter) ^ (k & 7)) << 4));
          const uint4 p1 = lds128(row + (((2 * quarter + 1) ^ (k & 7)) << 4));
          const uint64_t p[4] = {pair(__uint_as_float(p0.x), __uint_as_float(p0.y)),
                                 pair(__uint_as_float(p0.z), __uint_as_float(p0.w)),
                                 pair(__uint_as_float(p1.x), __uint_as_float(p1.y)),
                                 pair(__uint_as_float(p1.z), __uint_as_float(p1.w))};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[c >> 1]));
            const float value = (c & 1 ? f.y : f.x) * scale;
            const uint64_t v2 = pair(value, value);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[c][j] = fma2(p[j], v2, o[c][j]);
          }
        }
      }
      group_sync(group);
    }
    if (t + 1 == t1) {  // to a column a thread, through V's memory
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y[4] = {unpair(o[0][j]), unpair(o[1][j]), unpair(o[2][j]), unpair(o[3][j])};
        const uint32_t at = g.v_smem + ((8 * quarter + 2 * j) * D + 4 * lane) * 4;
        sts128(at, __float_as_uint(y[0].x), __float_as_uint(y[1].x), __float_as_uint(y[2].x),
               __float_as_uint(y[3].x));
        sts128(at + D * 4, __float_as_uint(y[0].y), __float_as_uint(y[1].y),
               __float_as_uint(y[2].y), __float_as_uint(y[3].y));
      }
      group_sync(group);
      uint32_t r[ROWS];
#pragma unroll
      for (int j = 0; j < ROWS; ++j) r[j] = lds32(g.v_smem + (j * D + g.tid) * 4);
      tmem_st_x32(g.mine + kColFar, r);
    }
    hand_over(g);
  }
  return n | (ok ? 0u : 0x80000000u);
}

// After a wait that gave up, every wait returns at once: the groups' warps then
// run their loops to the end with what there is, so that all of a group meet at
// its barriers; the loading warps stop.
__global__ void __launch_bounds__(kThreads, 1)
    moe_kv_attention_wide_kernel(const __grid_constant__ CUtensorMap map,
                                 const __grid_constant__ KvAttention a) {
  constexpr int kPerRow = kTokens / ROWS;  // threads that share a query row's load
  constexpr int kCols = D / kPerRow;       // its values that each takes
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  __shared__ Seq s_seqs[kSeqCache];
  __shared__ int s_to[kGroups][ROWS];                    // a row's place among the results, or -1
  __shared__ long long s_sum[kThreads / 32];
  __shared__ bool s_any[kGroups], s_more[kGroups];
  auto& s_bar = sh.bar;
  auto& s_walk = sh.walk;
  auto& s_scale = sh.scale;
  auto& s_limit = sh.limit;
  auto& s_m = sh.m;
  auto& s_f = sh.f;
  auto& s_red = sh.red;
  auto& s_bytes = sh.bytes;
  auto& s_range = sh.range;
  auto& s_nan = sh.nan;
  auto& s_nans = sh.nans;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const bool loads = warp >= 4 * kGroups;
  const int group = loads ? (warp - 4 * kGroups) % kGroups : warp >> 2;
  const bool issues = warp >= 5 * kGroups;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring = base + group * kGroupBytes;
  const uint32_t v_smem = ring + kSlots * kHalfBytes, q_smem = v_smem + kVBytes,
                 p_smem = q_smem + kQBytes;
  const uint32_t full = smem_u32(&s_bar[group * kBars]), empty = full + 8 * kSlots;
  // S and O complete; operands written (by the group's four warps); all MMAs complete
  const uint32_t s_done = empty + 8 * kSlots, o_done = s_done + 8, ready = s_done + 16,
                 drained = s_done + 24;
  if (threadIdx.x == 0) {
    for (int g = 0; g < kGroups; ++g) {
      const uint32_t b = smem_u32(&s_bar[g * kBars]);
      for (int i = 0; i < kSlots; ++i) {
        mbar_init(b + 8 * i, 1);
        mbar_init(b + 8 * (kSlots + i), 2);  // the two warps that read it
      }
      mbar_init(b + 16 * kSlots, 1);
      mbar_init(b + 16 * kSlots + 8, 1);
      mbar_init(b + 16 * kSlots + 16, 4);
      mbar_init(b + 16 * kSlots + 24, 1);
    }
    sh.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map);
  }
  pdl_wait_and_release();
  const WaitCtx wc{a.timeout_ns, a.status, &sh.abort};

  // All steps, then this group's share of them.
  long long total = 0;
  for (int s = threadIdx.x; s < a.n_seqs; s += kThreads) {
    const Seq q = read_seq(a, s);
    if (s < kSeqCache) s_seqs[s] = q;
    total += work_of<Deal>(a, q).weight;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) s_sum[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) total += s_sum[i];
  const long long per = share_of<Deal>(total, gridDim.x * kGroups);
  if (per * (static_cast<long long>(blockIdx.x) * kGroups) >= total) return;  // the whole CTA
  const int worker = blockIdx.x * kGroups + group;
  if (warp == 0) {
    tmem_alloc(smem_u32(&sh.tmem_base), kGroups * kGroupCols);
    tmem_relinquish();
  }
  if (loads && !issues) {
    const long long first = per * worker;
    if (first < total)
      find_share<Deal>(a, s_seqs, first, std::min(per, total - first), s_walk[group]);
    if (lane == 0) s_any[group] = first < total;
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const bool any = s_any[group];
  // Registers go where the scores are: 256 x 224 + 128 x 56 of 384 x 168.
  if (loads) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    Walk<Deal> share{};
    if (any) share = s_walk[group];
    __syncthreads();  // the loading warps have their copies of the walks
    if (any && !issues)
      load_group(a, &map, share, s_seqs, s_bytes[group], s_range[group], ring, full, empty, wc);
    if (any && issues) {
      const uint32_t tm = __shfl_sync(0xffffffffu, sh.tmem_base, 0) + group * kGroupCols;
      issue_group(a, share, s_seqs, tm, q_smem, p_smem, v_smem, s_done, o_done, ready, wc);
      // Every MMA issued completes before tensor memory is freed.
      const bool leader = elect_one();
      commit(leader, drained);
      if (leader) mbar_wait_drain(drained, 0, a.status);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    __syncthreads();
    const int tid = threadIdx.x & 127;  // token of a step, column of O
    const int quarter = warp & 3, half = quarter >> 1;
    const uint32_t tm = __shfl_sync(0xffffffffu, sh.tmem_base, 0) + group * kGroupCols;
    const uint32_t mine = tm + (static_cast<uint32_t>(quarter * 32) << 16);
    const GroupAt g{ring, full, empty, s_done, o_done, ready, v_smem, q_smem, p_smem, mine, group, tid,
                    half};
    uint32_t n = 0;         // steps so far
    const Walk<Deal>& w = s_walk[group];
    s_nan[group][tid] = INT_MAX;
    if (tid == 0) s_nans[group] = 0;

    bool ok = true;  // see take_k
    auto wait = [&](uint32_t bar, uint32_t phase) { ok = wait_all(bar, phase, wc, ok); };

    // A unit, and this thread's part of its query rows.
    struct Unit {
      int len, fresh, row0, head, r0, t0, t1, steps;
    };
    const int q_row = tid / kPerRow, q_at = tid % kPerRow;
    uint4 raw[kCols / 8];
    auto read_unit = [&]() {
      const Unit u{w.q.len, w.q.fresh, w.q.row0, w.head, w.group * ROWS, w.step, w.end(), w.steps};
      const int r = u.r0 + q_row;
      const bool valid = r < u.fresh * a.group;
      const int i = valid ? r / a.group : 0;
      const int gh = valid ? r - i * a.group : 0;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                 (u.row0 + i) * a.q_stride +
                                 static_cast<size_t>(u.head * a.group + gh) * D + q_at * kCols;
#pragma unroll
      for (int c = 0; c < kCols / 8; ++c)
        raw[c] = valid ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
      return u;
    };
    Unit unit{};
    if (any) unit = read_unit();

    for (bool go = any; go;) {
      const int len = unit.len, fresh = unit.fresh, row0 = unit.row0, head = unit.head;
      const int rows = fresh * a.group;  // of the sequence and head
      const int r0 = unit.r0, t0 = unit.t0, t1 = unit.t1;

      // Query rows as f16, each over 2^e of its largest value.
      {
        const int rr = q_row, r = r0 + rr, at = q_at;
        const bool valid = r < rows;
        const int i = valid ? r / a.group : 0;
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < kCols / 8; ++c) {
          const uint32_t v[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[j] << 16)),
                                   fabsf(__uint_as_float(v[j] & 0xffff0000u))));
        }
#pragma unroll
        for (int o = 1; o < kPerRow; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // exponent field e: values over 2^(e - 127) lie in [-2, 2]
        const int e = min(253, max(1, static_cast<int>(__float_as_uint(top) >> 23)));
        const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
        for (int c = 0; c < kCols / 8; ++c) {
          const uint32_t v[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
          uint32_t f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            f[j] = pack_f16x2(__uint_as_float(v[j] << 16) * down,
                              __uint_as_float(v[j] & 0xffff0000u) * down);
          const int unit = at * (kCols / 8) + c;
          sts128(q_smem + (unit >> 3) * (ROWS * 128) + rr * 128 + (((unit & 7) ^ (rr & 7)) << 4),
                 f[0], f[1], f[2], f[3]);
        }
        if (at == 0) {
          s_scale[group][rr] =
              a.scale_log2 * __uint_as_float(static_cast<uint32_t>(e) << 23);
          s_limit[group][rr] = valid ? len - fresh + i : -1;
          s_m[group][rr] = -INFINITY;
        }
      }
      if (len > 0) {
        ok = take_k(g, n, wc, ok);
        hand_over(g);
      }
      group_sync(group);  // the rows' factors and limits

      uint64_t nm[ROWS / 2], l[ROWS / 2];  // references (0 for -infinity), negative; sums
#pragma unroll
      for (int j = 0; j < ROWS / 2; ++j) nm[j] = l[j] = 0;
      int ref = 0;  // O's units, see next_units
      bool far = false;

      int t = t0;
      for (; t < t1 && len > 0; ++t, ++n) {
        const uint32_t range = s_range[group][n % kScaleSlots];  // came with the step's K
        const int at = step_token(range, t, tid);  // this thread's token
        // some row may not see all
        const bool zone = range >> 16 || t * kTokens + kTokens - 1 > len - fresh;
        ok = take_v(g, n, zone, at, len, fresh, s_nan[group], &s_nans[group], wc, ok);
        wait(s_done, n & 1);
        tc_fence_after_sync();
        uint32_t s[ROWS];
        tmem_ld_x32(mine + kColS, s);
        const uint8_t* const bytes = s_bytes[group][n % kScaleSlots];
        const int kb = bytes[tid / kKvBlock];
        const int vb = bytes[8 + tid / kKvBlock];
        const int lo = range & 0xff, hi = range >> 8 & 0xff;
        tmem_ld_wait();
        if (t + 1 < t1) ok = take_k(g, n + 1, wc, ok);
        // Scores over the references: s c - m, c the factor of a block and row.  What of the
        // block's scale is above 2^60 meets the score first: beside an infinite key the
        // block's other keys are zeros, whose scores are 0 and not 0 x inf.
        const float low = byte_scale(min(kb, 187)), high = byte_scale(max(kb, 187) - 60);
        const uint64_t ks2 = pair(low, low), high2 = pair(high, high);
        float top = -INFINITY;
        auto over = [&]() {
          top = -INFINITY;
          uint64_t y[ROWS / 2];
#pragma unroll
          for (int j = 0; j < ROWS; j += 4) {
            const float4 c = *reinterpret_cast<const float4*>(&s_scale[group][j]);
            y[j / 2] = fma2(mul2(pair(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), high2),
                            mul2(pair(c.x, c.y), ks2), nm[j / 2]);
            y[j / 2 + 1] =
                fma2(mul2(pair(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3])), high2),
                     mul2(pair(c.z, c.w), ks2), nm[j / 2 + 1]);
          }
#pragma unroll
          for (int j = 0; j < ROWS; j += 2) {
            const float2 z = unpair(y[j / 2]);
            s[j] = __float_as_uint(z.x);
            s[j + 1] = __float_as_uint(z.y);
          }
          if (zone) {
#pragma unroll
            for (int j = 0; j < ROWS; j += 4) {
              const int4 last = *reinterpret_cast<const int4*>(&s_limit[group][j]);
              if (at > last.x) s[j] = 0xff800000u;
              if (at > last.y) s[j + 1] = 0xff800000u;
              if (at > last.z) s[j + 2] = 0xff800000u;
              if (at > last.w) s[j + 3] = 0xff800000u;
            }
          }
#pragma unroll
          for (int j = 0; j < ROWS; j += 2)
            top = max3(top, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
        };
        over();
        const bool first = t == t0;
        if (group_any(group, first || top > kGrow || !units_hold(ref, lo, hi))) {
          // Each row's largest score, over its reference, in all of the step.
#pragma unroll
          for (int j = 0; j < ROWS; ++j) {
            const int k = __reduce_max_sync(0xffffffffu, ordered(__uint_as_float(s[j])));
            if (lane == j) s_red[group][quarter][j] = unordered(k);
          }
          const int next = next_units(ref, lo, hi);
          // One word for all: all go through the same barriers, and after a wait that gave
          // up the threads may differ in what they read.
          if (group_any(group, next < 0)) {
            far = true;
            break;
          }
          if (tid < ROWS) {
            const float was = s_m[group][tid], zero = was == -INFINITY ? 0.0f : was;
            const float u = zero + fmaxf(fmaxf(s_red[group][0][tid], s_red[group][1][tid]),
                                         fmaxf(s_red[group][2][tid], s_red[group][3][tid]));
            s_f[group][tid] = u > was ? ex2(was - u) : 1.0f;
            s_m[group][tid] = fmaxf(was, u);
          }
          group_sync(group);
          const float fr = pow2i(ref - next);
          ref = next;
          uint64_t f[ROWS / 2];
#pragma unroll
          for (int j = 0; j < ROWS; j += 2) {
            const float2 ff = *reinterpret_cast<const float2*>(&s_f[group][j]);
            const float2 now = *reinterpret_cast<const float2*>(&s_m[group][j]);
            const uint64_t to = pair(now.x == -INFINITY ? 0.0f : -now.x,
                                     now.y == -INFINITY ? 0.0f : -now.y);
            // the scores' distance from the reference moves with it
            const float2 was = unpair(nm[j / 2]), is = unpair(to);
            s[j] = __float_as_uint(__uint_as_float(s[j]) + (is.x - was.x));
            s[j + 1] = __float_as_uint(__uint_as_float(s[j + 1]) + (is.y - was.y));
            nm[j / 2] = to;
            f[j / 2] = pair(ff.x, ff.y);
            l[j / 2] = mul2(l[j / 2], f[j / 2]);
          }
          if (!first) {  // the last product is complete
            uint32_t o[ROWS];
            tmem_ld_x32(mine + kColO, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < ROWS; j += 2) {
              const float2 v = unpair(f[j / 2]);
              o[j] = __float_as_uint(__uint_as_float(o[j]) * (v.x * fr));
              o[j + 1] = __float_as_uint(__uint_as_float(o[j + 1]) * (v.y * fr));
            }
            tmem_st_x32(mine + kColO, o);
          }
        }
        {
          const float vf = pow2i(vb - ref + kPBits);
          const uint64_t vf2 = pair(vf, vf);
          // row j of P: 128 bytes for each 64 tokens, units of 8 tokens turned by j
          const uint32_t p_dst = p_smem + half * (ROWS * 128) + (tid & 7) * 2;
          const int unit = (tid & 63) >> 3;
#pragma unroll
          for (int j = 0; j < ROWS; j += 2) {
            const uint64_t p2 = pair(ex2(__uint_as_float(s[j])), ex2(__uint_as_float(s[j + 1])));
            l[j / 2] = add2(l[j / 2], p2);
            const float2 v = unpair(mul2(p2, vf2));
            const uint32_t w16 = pack_f16x2(v.x, v.y);
            sts16(p_dst + j * 128 + ((unit ^ (j & 7)) << 4), w16);
            sts16(p_dst + (j + 1) * 128 + ((unit ^ ((j + 1) & 7)) << 4), w16 >> 16);
          }
        }
        hand_over(g);
      }
      if (far) {
        uint32_t sum[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; j += 2) {
          const float2 v = unpair(l[j / 2]);
          sum[j] = __float_as_uint(v.x);
          sum[j + 1] = __float_as_uint(v.y);
        }
        tmem_st_x32(mine + kColFarSum, sum);
        tmem_st_wait();
        n = far_steps(a, sh, base, t, n, ref);
        ok = ok && !(n >> 31);
        n &= 0x7fffffffu;
        ref = kFarRef;
        tmem_ld_x32(mine + kColFarSum, sum);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < ROWS; j += 2)
          l[j / 2] = pair(__uint_as_float(sum[j]), __uint_as_float(sum[j + 1]));
      }

      // ---- O / l in the values' own scale: the result, or a part of it
      // O through V's memory, so that a warp stores whole rows.
      if (len > 0) {
        wait(o_done, (n - 1) & 1);
        tc_fence_after_sync();
        uint32_t o[ROWS];
        tmem_ld_x32(mine + (far ? kColFar : kColO), o);
        tmem_ld_wait();
        tc_fence_before_sync();
#pragma unroll
        for (int j = 0; j < ROWS; ++j) sts32(v_smem + (j * D + tid) * 4, o[j]);
      } else {
#pragma unroll 1
        for (int j = 0; j < ROWS; ++j) sts32(v_smem + (j * D + tid) * 4, 0);
      }
      {  // a row's sum over the tokens: each warp's in its part of Q's and P's memory
        static_assert(kQBytes + kPBytes == 4 * ROWS * 32 * 4);
        const uint32_t mem = q_smem + quarter * (ROWS * 32 * 4);
#pragma unroll
        for (int j = 0; j < ROWS; j += 2) {
          const float2 v = unpair(l[j / 2]);
          sts32(mem + (j * 32 + (lane ^ j)) * 4, __float_as_uint(v.x));
          sts32(mem + ((j + 1) * 32 + (lane ^ (j + 1))) * 4, __float_as_uint(v.y));
        }
        __syncwarp();
        if (lane < ROWS) {
          float sum = 0.0f;
#pragma unroll 8
          for (int i = 0; i < 32; ++i)
            sum += __uint_as_float(lds32(mem + (lane * 32 + (i ^ lane)) * 4));
          s_red[group][quarter][lane] = sum;
        }
      }
      group_sync(group);
      const bool whole = t0 == 0 && t1 == unit.steps;
      // The unit's first part lies in the second slot of its worker, the others
      // in the first of theirs.
      float* const part = a.partial + (static_cast<size_t>(worker) * 2 + (t0 == 0 ? 1 : 0)) *
                                          ROWS * (D + 2);
      if (tid == 0) s_more[group] = s_walk[group].next(a, s_seqs);
      if (tid < ROWS) {
        const float sum = (s_red[group][0][tid] + s_red[group][1][tid]) +
                          (s_red[group][2][tid] + s_red[group][3][tid]);
        const float up = byte_scale(ref) * (1.0f / (1 << kPBits));
        s_f[group][tid] = sum == 0.0f ? 0.0f : up / sum;
        const int row = r0 + tid;
        int to = -1;
        if (row < rows) {
          if (whole) {
            const int i = row / a.group;
            to = (row0 + i) * a.heads + head * a.group + (row - i * a.group);
            if (a.lse) a.lse[to] = log_sum(s_m[group][tid], sum);
          } else {
            to = tid;
            *reinterpret_cast<float2*>(part + tid * (D + 2) + D) =
                make_float2(s_m[group][tid], sum);
          }
        }
        s_to[group][tid] = to;  // (2^31 rows of results would not fit the memory)
      }
      const bool nans = s_nans[group];
      group_sync(group);
      go = s_more[group];
      if (go) unit = read_unit();  // its queries come while this one's results go
#pragma unroll 2
      for (int j = quarter; j < ROWS; j += 4) {
        const int to = s_to[group][j];
        if (to < 0) break;  // rows past the unit's
        const uint4 u = lds128(v_smem + (j * D + lane * 4) * 4);
        const float f = s_f[group][j];
        float v[4] = {__uint_as_float(u.x) * f, __uint_as_float(u.y) * f, __uint_as_float(u.z) * f,
                      __uint_as_float(u.w) * f};
        if (nans) {
          for (int i = 0; i < 4; ++i)
            if (s_nan[group][lane * 4 + i] <= s_limit[group][j]) v[i] = NAN;
        }
        if (whole) {
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(to) * D +
                                    lane * 4) =
              make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
          float2* const dst = reinterpret_cast<float2*>(part + j * (D + 2)) + 2 * lane;
          dst[0] = make_float2(v[0], v[1]);
          dst[1] = make_float2(v[2], v[3]);
        }
      }
      group_sync(group);  // what the next unit overwrites is read
      if (nans) {
        s_nan[group][tid] = INT_MAX;
        if (tid == 0) s_nans[group] = 0;
        group_sync(group);
      }
    }
    tc_fence_before_sync();
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(sh.tmem_base, kGroups * kGroupCols);
  }
}

}  // namespace

cudaError_t launch_kv_attention_wide(cudaStream_t s, const KvAttention& a) {
  CUtensorMap map;
  const uint64_t rows = 2ull * a.cache.pages * a.cache.heads * a.cache.page;
  const uint64_t dims[2] = {static_cast<uint64_t>(D), rows};
  const uint64_t strides[1] = {static_cast<uint64_t>(D)};
  const uint32_t box[2] = {static_cast<uint32_t>(D),
                           static_cast<uint32_t>(std::min(a.cache.page, 32))};
  cudaError_t e = make_u8_map_nd(&map, a.cache.codes, 2, dims, strides, box, D);
  if (e != cudaSuccess) return e;
  e = allow_dynamic_smem(reinterpret_cast<const void*>(moe_kv_attention_wide_kernel),
                         kSmem);
  if (e != cudaSuccess) return e;
  // No more groups than shares there can be.
  const long long steps =
      (static_cast<long long>(a.max_pages) * a.cache.page + kTokens - 1) / kTokens;
  const long long units =
      ((static_cast<long long>(a.T) * a.group + ROWS - 1) / ROWS + a.n_seqs) * a.cache.heads;
  const long long ctas = (std::min(steps * units, 1LL << 40) + kGroups - 1) / kGroups;
  const int grid = static_cast<int>(std::min<long long>(
      {std::max(1LL, ctas), static_cast<long long>(device_sm_count()),
       static_cast<long long>(kKvAttentionWarps / kGroups)}));
  {
    KernelScope scope(s, "moe_kv_attention");
    e = launch_kernel(moe_kv_attention_wide_kernel, dim3(grid), dim3(kThreads), kSmem, s,
                      map, a);
  }
  return e == cudaSuccess ? launch_join<D, Deal>(s, a, steps, grid * kGroups) : e;
}

}  // namespace moe
