// Attention of one or a few new tokens per sequence over the paged 8-bit
// cache: per query row, a pass over its sequence's keys and values with a
// running maximum and sum.
//
// Bound by reading the cache, one byte a value.  A unit is (sequence, KV head,
// group of at most 8 NT query rows: all heads of the group, all new tokens;
// units of more than 16 rows with head dimension 128 go to
// moe_kv_attention_wide.cu);
// its keys come in steps of 32 tokens, two blocks of the cache.  The steps of
// all units, one after another, are dealt out evenly over the warps: warp w of
// the grid takes steps [w per, (w + 1) per), so ragged lengths and few
// sequences load every SM alike, and no warp waits for another.  A unit that
// ends up in several warps leaves partial results (O / l, m, l) in the
// workspace; a second kernel adds them in warp order, so the sum does not
// depend on timing.  (Sharing each tile among a CTA's warps, with an exchange
// at every unit's end, cost about 30 us in barriers and round trips on a batch
// of 64 sequences.)
//
// Measured: 6 sequences of up to 131000 keys, 64 heads over 8: 164 us, 6.1 TB/s
// (90 % of a copy); 64 sequences of up to 4096, 64 heads over 4: 45 us, 4.0 TB/s
// (59 %): about 5 us pass before the first scores (lengths, share, page numbers,
// first tiles: four round trips to memory), 5 us in joining the parts, the rest
// at 5.9 TB/s.
//
// Each consumer warp has a ring of steps in shared memory; one or two warps of
// the CTA load for all, a lane for each ring: TMA boxes of up to 32 rows of a
// page (128- or 64-byte swizzle), K refilled as soon as the scores are done, V
// at the end of the step.  The block table's words come by cp.async four steps
// ahead and the scale bytes by cp.async onto the barrier of their K, so the
// loading warps themselves wait for no memory.
// The tokens are the M side of the m16n8k16 MMAs and the query rows the N
// side, 8 at a time: S^T = K Q^T and O^T = V^T P^T, in fp32.  E4M3 codes
// become f16 exactly (cvt) on their way into the A fragments; a query row is
// scaled by a power of two into f16, exact but for values 2^-24 below its
// largest.  The order of the contraction is free: the lane that holds a K
// row's bytes 32 t .. 32 t + 31 feeds them to the MMAs as they lie.  V comes
// transposed by ldmatrix in pairs of bytes, which a byte permute splits into
// even and odd columns (rows g and g + 8 of A), P by movmatrix.  The weights
// p = 2^(s - m) enter as f16 p 2^6 2^(X - ref), X the block's value scale and ref
// the unit's (next_units): 11 significant bits, three more than bf16.  A row's
// reference m is moved (a reduction over the warp, and O rescaled) only when
// some score passes it by 2^8.

#include <climits>

#include "moe_kv_attention.cuh"

namespace moe {
namespace {

constexpr int kStep = 32;        // tokens of a warp's step: two blocks

// Steps of a warp, at most, where a CTA has a unit of its own.  Against the even
// dealing with its second kernel, us with the L2 flushed, one sequence / eight:
//   8 rows, dim 128   100 keys 12.4 for 17.0 / 11.9 for 18.8, 1920 keys 19.9 for 20.8 / 20.4 for 22.7
//   16 rows, dim 128  100 keys 12.9 for 16.8 / 12.3 for 20.0, 1600 keys 20.4 for 20.7 / 21.2 for 21.6
//   8 rows, dim 64    100 keys  9.9 for 16.6 / 11.0 for 16.7, 1920 keys 17.5 for 18.8 / 19.2 for 20.7
//   16 rows, dim 64   100 keys 10.3 for 15.3 / 11.1 for 17.3, 1600 keys 18.0 for 18.7 / 17.7 for 20.2
//   32 rows, dim 64   100 keys 12.1 for 17.2 / 12.8 for 19.4, 1120 keys 19.5 for 21.7 / 20.1 for 22.9
// (the last of each: 5 steps a warp); past it 2500 keys took 22.5 for 19.9 (8 rows,
// dim 128, one sequence).  The block table's width stands for the lengths, which the
// host does not know: a table wider than this goes the other way whatever is in it.
constexpr int kOwnSteps = 5;
constexpr int kAheadPages = 4;   // steps ahead of the loads that pages are looked up

// NT tiles of 8 query rows, WARPS consumer warps with STAGES ring stages each,
// LOADERS loading warps.  One CTA per SM.
template <int D_, int NT_, int WARPS_, int STAGES_, int LOADERS_>
struct Shape {
  static constexpr int D = D_, NT = NT_, kWarps = WARPS_, kStages = STAGES_, kLoaders = LOADERS_;
  static constexpr int kRows = 8 * NT;
  using Deal = DealOf<kRows, moe::kStep, 4>;
  static constexpr int kThreads = 32 * (kWarps + kLoaders);
  static constexpr int kHalf = kStep * D;  // K or V of a warp's step
  static constexpr int kStage = 2 * kHalf;
  // Four row tiles leave no registers for the query fragments.
  static constexpr bool kQueryInSmem = NT > 2;
  static constexpr int kQuery = kQueryInSmem ? NT * (D / 16) * 32 * 8 : 0;  // a warp's
  static constexpr int kSmem = 1024 + kWarps * (kStages * kStage + kQuery);
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  // volatile: it stays before the return of the slot that its operands came from
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
               "{%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}

// Transposes an 8 x 8 matrix of 16-bit values: lane 4 g + t holds (g, 2 t) and
// (g, 2 t + 1).
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A step's block b that lies on a page outside the pool, from its word of Rings.
constexpr uint32_t kNoBlock = 0x80, kNoBlocks = kNoBlock | kNoBlock << 8;
__device__ __forceinline__ bool no_page(uint32_t word, int b) {
  return word >> (8 * b) & kNoBlock;
}

// What a step that holds the sequence's end, a block without a page (none), or new
// tokens that some rows do not see, needs before its values (32 tokens from position
// pos on, at v, swizzled) meet the MMAs.  Codes past the end are whatever was in the
// page, those without one whatever the ring held: they become zeros.  A NaN among the new tokens concerns only the rows that see its token,
// but would meet the others' p = 0: it becomes zero too, and nan_from[column]
// keeps the first position of one, for the end of the unit.  Returns whether
// there was one.  Called by a warp, a token a lane.
template <int D>
__device__ __noinline__ bool clean_values(uint32_t v, int pos, int len, int fresh, uint32_t none,
                                          int* nan_from) {
  const int lane = threadIdx.x & 31;
  const bool no_block = no_page(none, lane >> 4);
  const int at = pos + lane;
  bool found = false;
#pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    // the swizzle turns the chunk, and each lane has a row of its own: any order
    const uint32_t addr = v + lane * D + c * 16;
    uint4 w = lds128(addr);
    if (at >= len || no_block) {
      w = make_uint4(0, 0, 0, 0);
    } else if (at > len - fresh) {
      uint32_t words[4] = {w.x, w.y, w.z, w.w};
      const int chunk = c ^ (D == 128 ? lane & 7 : (lane >> 1) & 3);
      for (int i = 0; i < 4; ++i)
        for (int b = 0; b < 4; ++b)
          if ((words[i] >> (8 * b) & 0x7f) == 0x7f) {
            words[i] &= ~(0xffu << (8 * b));
            atomicMin(&nan_from[chunk * 16 + i * 4 + b], at);
            found = true;
          }
      w = make_uint4(words[0], words[1], words[2], words[3]);
    } else {
      continue;
    }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w.x), "r"(w.y),
                 "r"(w.z), "r"(w.w)
                 : "memory");
  }
  __syncwarp();
  return __any_sync(0xffffffffu, found);
}

// Arrives on `bar` once this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A loading warp: lane i fills ring first + i, its K halves and V halves in
// turn as they are given back.
template <class S>
struct Rings {
  static constexpr int kSlots = 2 * kAheadPages;
  uint4 scales[S::kWarps][S::kStages];          // words with the scale bytes: K, K, V, V
  // where in them (bits, a byte each); the top bit of the first two bytes: the block
  // lies on a page outside the pool
  uint32_t shifts[S::kWarps][S::kStages];
  int pages[S::kWarps][kSlots][2];              // of a step's two blocks
  int4 meta[S::kWarps][kSlots];                 // position, head, blocks inside
};

template <class S>
__device__ __forceinline__ void load_rings(const KvAttention& a, const CUtensorMap* map,
                                           const Walk<typename S::Deal>& share, bool any, int mine, bool ring,
                                           const Seq* cache, Rings<S>* r, uint32_t rings,
                                           uint32_t bars, const WaitCtx& wc) {
  constexpr int kN = S::kWarps * S::kStages;
  constexpr int kSlots = Rings<S>::kSlots;
  const int P = a.cache.page, ps = __ffs(P) - 1, box = min(P, kStep);  // P is a power of two
  const int v_rows = a.cache.heads * P;  // from K's rows of a page to V's
  const size_t v_scales = static_cast<size_t>(a.cache.heads) << (ps - 4);
  const uint8_t* const scales_end =
      a.cache.scales + (static_cast<size_t>(2 * a.cache.heads) * a.cache.pages << (ps - 4));
  auto valid = [&](int page) { return page >= 0 && page < a.cache.pages; };

  bool more = any;     // the walk has steps to look up
  Walk<typename S::Deal> w = share;
  int t = 0, t1 = 0;   // of its unit
  auto unit = [&]() {
    while (more && w.q.len == 0) more = w.next(a, cache);
    if (more) {
      t = w.step;
      t1 = w.end();
    }
  };
  unit();
  int looked = 0;  // steps looked up
  auto look_up = [&]() {
    if (!more) return;
    const int slot = looked % kSlots;
    const int pos = t * kStep;
    const bool in1 = pos + kKvBlock < w.q.len;
    r->meta[mine][slot] = make_int4(pos, w.head, in1, 0);
    const int32_t* row = a.block_table + static_cast<size_t>(w.s) * a.max_pages;
    const uint32_t dst = smem_u32(&r->pages[mine][slot][0]);
    cp_async4(dst, row + (pos >> ps), 4);
    if (in1) cp_async4(dst + 4, row + ((pos + kKvBlock) >> ps), 4);
    ++looked;
    if (++t >= t1) {
      more = w.next(a, cache);
      unit();
    }
  };
  for (int i = 0; i < kAheadPages; ++i) look_up();
  cp_async_commit();
  cp_async_wait<0>();

  int next = 0, stage = 0, half = 0;  // this lane's step and half
  int row0 = -1, row1 = -1;           // the step's boxes in the map (K's; -1: none)
  uint32_t phase = 0;
  unsigned long long idle_since = 0;
  for (;;) {
    // A step's page words were asked for at least 2 kAheadPages turns ago.
    cp_async_wait<2 * kAheadPages - 2>();
    const int slot = mine * S::kStages + stage;
    // barriers: K full, V full, K empty, V empty, each [warp][stage]
    const uint32_t full = bars + 8 * (half * kN + slot), empty = full + 16 * kN;
    const bool go = ring && next < looked && mbar_test_wait(empty, phase ^ 1u);
    if (go) {
      if (half == 0) {
        const int4 d = r->meta[mine][next % kSlots];
        const int p0 = r->pages[mine][next % kSlots][0];
        const int p1 = d.z ? r->pages[mine][next % kSlots][1] : p0;
        const int in0 = d.x & (P - 1), in1 = (d.x + kKvBlock) & (P - 1);
        const bool ok0 = valid(p0), ok1 = d.z && valid(p1);
        if (!ok0 || !valid(p1)) atomicOr(a.status, kStatusDeviceCheck);
        const int at0 = p0 * 2 * a.cache.heads + d.y, at1 = p1 * 2 * a.cache.heads + d.y;
        row0 = ok0 ? (at0 << ps) + in0 : -1;
        row1 = ok1 && box < kStep ? (at1 << ps) + in1 : -1;
        uint32_t shifts = (ok0 ? 0u : kNoBlock) | (d.z && !ok1 ? kNoBlock << 8 : 0u);
        const uint32_t dst = smem_u32(&r->scales[mine][stage]);
        auto word = [&](int i, bool ok, const uint8_t* src) {
          src = ok ? src : a.cache.scales;
          const uint32_t o = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 3);
          src -= o;
          cp_async4(dst + 4 * i, src,
                    ok ? static_cast<int>(min(static_cast<long long>(scales_end - src), 4LL)) : 0);
          shifts |= o << (8 * i + 3);
        };
        const uint8_t* s0 = a.cache.scales + (static_cast<size_t>(at0) << (ps - 4)) + in0 / kKvBlock;
        const uint8_t* s1 = a.cache.scales + (static_cast<size_t>(at1) << (ps - 4)) + in1 / kKvBlock;
        word(0, ok0, s0);
        word(1, ok1, s1);
        word(2, ok0, s0 + v_scales);
        word(3, ok1, s1 + v_scales);
        r->shifts[mine][stage] = shifts;
        cp_async_arrive(full);
      }
      mbar_arrive_expect_tx(full, static_cast<uint32_t>((row0 >= 0) + (row1 >= 0)) * box * S::D);
      const uint32_t dst = rings + slot * S::kStage + half * S::kHalf;
      if (row0 >= 0) tma_load_2d(dst, map, full, 0, row0 + half * v_rows);
      if (row1 >= 0) tma_load_2d(dst + box * S::D, map, full, 0, row1 + half * v_rows);
      half ^= 1;
      if (half == 0) {
        ++next;
        if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
        look_up();
      }
    }
    __syncwarp();
    cp_async_commit();
    if (__any_sync(0xffffffffu, go)) {
      idle_since = 0;
      continue;
    }
    if (__all_sync(0xffffffffu, !ring || next == looked)) break;
    if (*wc.abort_flag) break;
    const unsigned long long now = globaltimer_ns();
    if (idle_since == 0) idle_since = now;
    if (__any_sync(0xffffffffu, now - idle_since > wc.timeout_ns)) {
      if ((threadIdx.x & 31) == 0) give_up(wc);
      break;
    }
  }
  cp_async_wait<0>();
  // After a wait that gave up: the last loads may still be landing.
  if (*wc.abort_flag && ring) {
    const int issued = 2 * next + half;
    for (int i = max(0, issued - 2 * S::kStages); i < issued; ++i) {
      const int at = (i >> 1) % S::kStages;
      mbar_wait_drain(bars + 8 * ((i & 1) * kN + mine * S::kStages + at),
                      ((i >> 1) / S::kStages) & 1, a.status);
    }
  }
}

// A unit's query rows as f16 fragments, each row over 2^e of its largest value, in
// registers or at q_smem.  This lane loads row g of each tile; it keeps the scores'
// factors of rows 2 t4 and 2 t4 + 1, its columns of S^T.  limit: the last position
// that each row sees.
template <class S>
__device__ __forceinline__ void load_queries(const KvAttention& a, const Seq& q, int head, int r0,
                                             int* limit, uint32_t q_smem,
                                             uint32_t (&qf)[S::kQueryInSmem ? 1 : S::NT][S::D / 16][2],
                                             float (&row_scale)[S::NT][2]) {
  constexpr int D = S::D, NT = S::NT, kSteps = D / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int rows = q.fresh * a.group;  // of the sequence and head
  uint4 raw[NT][D / 32];  // all loads under way before the first is used
  int last[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + nt * 8 + g;
    const bool valid = r < rows;
    const int i = valid ? r / a.group : 0;
    const int gh = valid ? r - i * a.group : 0;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (q.row0 + i) * a.q_stride +
                               static_cast<size_t>(head * a.group + gh) * D + t4 * (D / 4);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      raw[nt][c] = valid ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
    last[nt] = valid ? q.len - q.fresh + i : -1;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const uint32_t v[4] = {raw[nt][c].x, raw[nt][c].y, raw[nt][c].z, raw[nt][c].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[j] << 16)),
                               fabsf(__uint_as_float(v[j] & 0xffff0000u))));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // exponent field e: values over 2^(e - 127) lie in [-2, 2]
    const int e = min(253, max(1, static_cast<int>(__float_as_uint(top) >> 23)));
    const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    const float rs = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      row_scale[nt][j] = __shfl_sync(0xffffffffu, rs, (2 * t4 + j) * 4);
    if (t4 == 0) limit[nt * 8 + g] = last[nt];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const uint32_t v0 = k & 1 ? raw[nt][k / 2].z : raw[nt][k / 2].x;
      const uint32_t v1 = k & 1 ? raw[nt][k / 2].w : raw[nt][k / 2].y;
      const uint32_t f0 =
          pack_f16x2(__uint_as_float(v0 << 16) * down, __uint_as_float(v0 & 0xffff0000u) * down);
      const uint32_t f1 =
          pack_f16x2(__uint_as_float(v1 << 16) * down, __uint_as_float(v1 & 0xffff0000u) * down);
      if constexpr (S::kQueryInSmem) {
        sts64(q_smem + (nt * kSteps + k) * 256, f0, f1);
      } else {
        qf[nt][k][0] = f0;
        qf[nt][k][1] = f1;
      }
    }
  }
  __syncwarp();
}

// O / l in the values' own scale, from units of 2^(ref - 127 - kPBits): the result,
// or a part of it.  nan_from: see clean_values; null where it noted nothing.
template <class S>
__device__ __forceinline__ void finish_unit(const KvAttention& a, const Seq& q, int head, int r0,
                                            bool whole, float* part, const int* limit, int* nan_from,
                                            int ref, float (&o)[S::D / 16][S::NT][4],
                                            const float (&m)[S::NT][2], const float (&l)[S::NT][2]) {
  constexpr int D = S::D, NT = S::NT, kChunks = D / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int rows = q.fresh * a.group;
  if (nan_from) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (nan_from[16 * c + 2 * g + (j >> 1)] <= limit[nt * 8 + 2 * t4 + (j & 1)])
            o[c][nt][j] = NAN;
    __syncwarp();
    for (int i = lane; i < D; i += 32) nan_from[i] = INT_MAX;
  }
  const float up = byte_scale(ref) * (1.0f / (1 << kPBits));
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float sum = l[nt][j];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int r = nt * 8 + 2 * t4 + j, row = r0 + r;
      if (row >= rows) continue;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      if (whole) {
        const int i = row / a.group;
        const size_t orow =
            static_cast<size_t>(q.row0 + i) * a.heads + head * a.group + (row - i * a.group);
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + orow * D);
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          out[8 * c + g] = pack_bf16x2(o[c][nt][j] * inv * up, o[c][nt][2 + j] * inv * up);
        if (g == 0 && a.lse) a.lse[orow] = log_sum(m[nt][j], sum);
      } else {
        float2* dst = reinterpret_cast<float2*>(part + r * (D + 2));
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          dst[8 * c + g] = make_float2(o[c][nt][j] * inv * up, o[c][nt][2 + j] * inv * up);
        if (g == 0) dst[D / 2] = make_float2(m[nt][j], sum);
      }
    }
}

// What a CTA's warps share.
template <class S>
struct Shared {
  alignas(8) uint64_t bar[4 * S::kWarps * S::kStages];  // K full, V full, K empty, V empty
  Rings<S> rings;
  Walk<typename S::Deal> walk[S::kWarps];
  int limit[S::kWarps][S::kRows];  // last position that a row sees
  int nan[S::kWarps][S::D];        // see clean_values
  int abort;
};

// Where a unit's part lies: the first in the second slot of its warp, the others in
// the first of theirs.
template <class S>
__device__ __forceinline__ float* part_slot(const KvAttention& a, int warp, int t0) {
  return a.partial + (static_cast<size_t>(blockIdx.x * S::kWarps + warp) * 2 + (t0 == 0 ? 1 : 0)) *
                         S::kRows * (S::D + 2);
}

// The steps from t on of a warp's unit whose value scales lie far apart (K of the first
// has landed), its steps before left as a part in its slot; the result, or a part of
// it.  Block by block: a block's weights over its own largest as f16 p 2^6, and its
// product (one MMA deep) added to O in fp32 with the block's factor, so that no
// block's scale or weight takes bits from another's.  Out of line, and the state
// handed over in memory: in line, or with O live across the call, the ordinary steps
// of 16 rows took 2 to 30 % longer (registers).  64 sequences of up to 4096, 64 heads over
// 4, half of the value blocks 2^12 above the others: 77 us for 55 (L2 flushed).
// Stage and phase (in the high half) are the ring's, and returned; ~0: a wait gave up.
template <class S, bool OWN>
__device__ __noinline__ uint32_t far_steps(const KvAttention& a, Shared<S>& sh, uint32_t base, int t,
                                           uint32_t at) {
  constexpr int D = S::D, NT = S::NT, kSteps = D / 16, kChunks = D / 16;
  constexpr int kN = S::kWarps * S::kStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const WaitCtx wc{a.timeout_ns, a.status, &sh.abort};
  const uint32_t ring = base + warp * S::kStages * S::kStage;
  const uint32_t q_smem = base + kN * S::kStage + warp * S::kQuery + lane * 8;
  const uint32_t k_full = smem_u32(&sh.bar[warp * S::kStages]);
  const uint32_t v_full = k_full + 8 * kN, k_empty = k_full + 16 * kN, v_empty = k_full + 24 * kN;
  const Walk<typename S::Deal>& w = sh.walk[warp];
  const Seq q = w.q;
  const int t1 = w.end(), r0 = w.group * S::kRows, rows = q.fresh * a.group;
  const bool whole = w.step == 0 && t1 == w.steps;
  int* const limit = sh.limit[warp];
  int* const nan_from = sh.nan[warp];
  // places of K's rows and V's matrices, as for the ordinary steps
  const int x = D == 128 ? g : (g >> 1) & 3;
  const int mi = lane >> 3, vr = lane & 7;
  const int vx = (mi >> 1) ^ (D == 128 ? vr : (vr >> 1) & 3);
  const uint32_t v_off = S::kHalf + static_cast<uint32_t>(((mi & 1) * 8 + vr) * D);
  int stage = at & 0xffff;
  uint32_t phase = at >> 16;
  uint32_t qf[S::kQueryInSmem ? 1 : NT][kSteps][2];
  float row_scale[NT][2];
  load_queries<S>(a, q, w.head, r0, limit, q_smem, qf, row_scale);

  // what the unit's earlier steps left
  const float* const slot = part_slot<S>(a, warp, w.step);
  constexpr float kDown = 1.0f / (1 << (kFarRef - 127 - kPBits));
  float o[kChunks][NT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = nt * 8 + 2 * t4 + j;
      const float2* src = reinterpret_cast<const float2*>(slot + r * (D + 2));
      const bool there = r0 + r < rows;
      const float2 ml = there ? src[D / 2] : make_float2(-INFINITY, 0.0f);
      m[nt][j] = ml.x;
      l[nt][j] = g == 0 ? ml.y : 0.0f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const float2 v = there ? src[8 * c + g] : make_float2(0.0f, 0.0f);
        o[c][nt][j] = v.x * kDown * ml.y;
        o[c][nt][2 + j] = v.y * kDown * ml.y;
      }
    }
  bool ok = true, nans = false;
#pragma unroll 1
  for (; t < t1; ++t) {
    const int pos = t * kStep;
    const uint32_t sb = ring + stage * S::kStage;
    ok = __all_sync(0xffffffffu, mbar_wait(k_full + 8 * stage, phase, wc));
    if (!ok) break;
    const uint4 words = sh.rings.scales[warp][stage];
    const uint32_t shifts = sh.rings.shifts[warp][stage];
    const bool zone = pos + kStep - 1 > q.len - q.fresh || (shifts & kNoBlocks);
    ok = __all_sync(0xffffffffu, mbar_wait(v_full + 8 * stage, phase, wc));
    if (!ok) break;
    if (zone && clean_values<D>(sb + S::kHalf, pos, q.len, q.fresh, shifts, nan_from)) nans = true;
#pragma unroll 1
    for (int b = 0; b < 2; ++b) {
      const float ks =
          byte_scale((b ? words.y >> (shifts >> 8 & 31) : words.x >> (shifts & 31)) & 0xff);
      const float vs =
          byte_scale((b ? words.w >> (shifts >> 24) : words.z >> (shifts >> 16 & 31)) & 0xff);
      const int at_g = no_page(shifts, b) ? INT_MAX - 8 : pos + 16 * b + g;
      uint32_t kw[2][D / 16];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const int chunk = D == 128 ? (2 * t4 + c) ^ x : t4 ^ x;
          const uint4 v = lds128(sb + (b * 16 + h * 8 + g) * D + chunk * 16);
          kw[h][4 * c] = v.x; kw[h][4 * c + 1] = v.y;
          kw[h][4 * c + 2] = v.z; kw[h][4 * c + 3] = v.w;
        }
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[nt][j] = 0.0f;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const uint32_t ka[4] = {codes_f16(kw[0][k]), codes_f16(kw[1][k]), codes_f16_hi(kw[0][k]),
                                codes_f16_hi(kw[1][k])};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (S::kQueryInSmem) {
            const uint2 qw = lds64(q_smem + (nt * kSteps + k) * 256);
            mma_f16(sc[nt], ka, qw.x, qw.y);
          } else {
            mma_f16(sc[nt], ka, qf[nt][k][0], qf[nt][k][1]);
          }
        }
      }
      uint32_t pb[NT][2];
      float gain[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f = score_factor(ks, row_scale[nt][j]);
          float s[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s[h] = sc[nt][2 * h + j] * f;
            if (at_g + 8 * h > limit[nt * 8 + 2 * t4 + j]) s[h] = -INFINITY;
          }
          float u = fmaxf(s[0], s[1]);
          u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 4));
          u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 8));
          u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 16));
          const float fm = u > m[nt][j] ? ex2(m[nt][j] - u) : 1.0f;
          m[nt][j] = fmaxf(m[nt][j], u);
          l[nt][j] *= fm;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            o[c][nt][j] *= fm;
            o[c][nt][2 + j] *= fm;
          }
          // a row that sees nothing of the block: weights and factor 0
          const float top = u == -INFINITY ? 0.0f : u;
          const float over = u == -INFINITY ? 0.0f : ex2(u - m[nt][j]);
#pragma unroll
          for (int h = 0; h < 2; ++h) p[h][j] = ex2(s[h] - top);
          l[nt][j] += (p[0][j] + p[1][j]) * over;
          gain[nt][j] = over * vs * pow2i(127 - kFarRef);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          pb[nt][h] = movmatrix(pack_f16x2(p[h][0] * (1 << kPBits), p[h][1] * (1 << kPBits)));
      }
#pragma unroll
      for (int c = 0; c < kChunks; c += 2) {
        uint32_t v[4];
        ldmatrix_x4_trans(sb + v_off + b * 16 * D + ((vx ^ c) * 16), v);
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const uint32_t a0 = __byte_perm(v[2 * cc], 0, 0x3120);
          const uint32_t a1 = __byte_perm(v[2 * cc + 1], 0, 0x3120);
          const uint32_t va[4] = {codes_f16(a0), codes_f16_hi(a0), codes_f16(a1), codes_f16_hi(a1)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_f16(d, va, pb[nt][0], pb[nt][1]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              o[c + cc][nt][j] = fmaf(d[j], gain[nt][j & 1], o[c + cc][nt][j]);
          }
        }
      }
    }
    // clean_values wrote through the generic proxy what TMA writes next
    if (zone) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();  // K, V and the scales are read
    if (lane == 0) {
      mbar_arrive(k_empty + 8 * stage);
      mbar_arrive(v_empty + 8 * stage);
    }
    if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
  }
  float* part = part_slot<S>(a, warp, w.step);
  if constexpr (OWN) {
    extern __shared__ uint8_t smem_raw[];
    part = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)));
  }
  finish_unit<S>(a, q, w.head, r0, whole, part, limit, nans ? nan_from : nullptr, kFarRef, o, m, l);
  return ok ? static_cast<uint32_t>(stage) | phase << 16 : ~0u;
}

// OWN: each CTA has a unit of its own and shares its steps out among its warps,
// which leave their parts in shared memory, where the CTA joins them: for few
// units of few steps, where the second kernel would cost more than the even
// dealing gains.
template <class S, bool OWN>
__global__ void __launch_bounds__(S::kThreads, 1)
    moe_kv_attention_kernel(const __grid_constant__ CUtensorMap map,
                            const __grid_constant__ KvAttention a) {
  constexpr int D = S::D, NT = S::NT;
  using Deal = typename S::Deal;
  constexpr int kSteps = D / 16;   // MMA steps of a score
  constexpr int kChunks = D / 16;  // 16-byte chunks of a row
  constexpr int kN = S::kWarps * S::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<S> sh;
  __shared__ Seq s_seqs[kSeqCache];
  __shared__ long long s_sum[S::kThreads / 32];
  __shared__ bool s_any[S::kWarps];
  uint64_t* const s_bar = sh.bar;
  auto& s_rings = sh.rings;
  auto& s_walk = sh.walk;
  auto& s_limit = sh.limit;
  auto& s_nan = sh.nan;
  int& s_abort = sh.abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4 * kN; ++i)  // K: the boxes, and the scale words
      mbar_init(smem_u32(&s_bar[i]), i < kN ? 2 : 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map);
  }
  pdl_wait_and_release();
  const WaitCtx wc{a.timeout_ns, a.status, &s_abort};

  // All steps (OWN: units), then this warp's share of them.
  using Units = DealOf<S::kRows, 1 << 30, 1>;  // a unit counts as one step
  long long total = 0;
  for (int s = threadIdx.x; s < a.n_seqs; s += S::kThreads) {
    const Seq q = read_seq(a, s);
    if (s < kSeqCache) s_seqs[s] = q;
    total += OWN ? work_of<Units>(a, q).weight : work_of<Deal>(a, q).weight;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) s_sum[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < S::kThreads / 32; ++i) total += s_sum[i];
  const long long per = OWN ? 0 : share_of<Deal>(total, gridDim.x * S::kWarps);
  if (OWN && blockIdx.x >= total) return;
  if (per * (static_cast<long long>(blockIdx.x) * S::kWarps) >= total) return;  // the whole CTA
  const int gw = blockIdx.x * S::kWarps + warp;  // of the grid's consumers
  Walk<Deal>& w = s_walk[warp < S::kWarps ? warp : 0];
  if (warp < S::kWarps) {
    if constexpr (OWN) {
      find_share<Units>(a, s_seqs, blockIdx.x, 1, w);
      __syncwarp();
      if (lane == 0) {
        const int steps = work_of<Deal>(a, w.q).steps;
        const int each = (steps + S::kWarps - 1) / S::kWarps;
        w.steps = steps;
        w.step = warp * each;
        w.left = min(each, steps - w.step);
        s_any[warp] = w.step < steps;
      }
    } else {
      const long long first = per * gw;
      if (first < total) find_share<Deal>(a, s_seqs, first, std::min(per, total - first), w);
      if (lane == 0) s_any[warp] = first < total;
    }
  }
  __syncthreads();
  if (warp >= S::kWarps) {
    constexpr int kEach = (S::kWarps + S::kLoaders - 1) / S::kLoaders;  // rings of a loading warp
    const int mine = (warp - S::kWarps) * kEach + lane;
    const bool ring = lane < kEach && mine < S::kWarps;
    const bool any = ring && s_any[mine];
    Walk<Deal> share{};
    if (any) share = s_walk[mine];
    __syncthreads();
    load_rings<S>(a, &map, share, any, ring ? mine : 0, ring, s_seqs, &s_rings, base,
                  smem_u32(&s_bar[0]), wc);
    return;
  }
  __syncthreads();  // the loading warps have their copies of the walks
  if (!OWN && !s_any[warp]) return;
  for (int i = lane; i < D; i += 32) s_nan[warp][i] = INT_MAX;

  const uint32_t ring = base + warp * S::kStages * S::kStage;
  const uint32_t k_full = smem_u32(&s_bar[warp * S::kStages]);  // stage i at + 8 i
  const uint32_t v_full = k_full + 8 * kN, k_empty = k_full + 16 * kN, v_empty = k_full + 24 * kN;
  int stage = 0;
  uint32_t phase = 0;
  const int g = lane >> 2, t4 = lane & 3;
  const int x = D == 128 ? g : (g >> 1) & 3;  // swizzle of this lane's K rows
  const uint32_t k_off = static_cast<uint32_t>(g * D);
  const int mi = lane >> 3, vr = lane & 7;
  const int vx = (mi >> 1) ^ (D == 128 ? vr : (vr >> 1) & 3);
  const uint32_t v_off = S::kHalf + static_cast<uint32_t>(((mi & 1) * 8 + vr) * D);
  const uint32_t q_smem = base + kN * S::kStage + warp * S::kQuery + lane * 8;
  static_assert(S::kRows * (D + 2) * 4 <= S::kStages * S::kStage);
  auto own_part = [&](int i) {
    return reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)) +
                                    i * S::kStages * S::kStage);
  };
  bool ok = true;

  for (bool go = !OWN || s_any[warp]; go;) {
    const int len = w.q.len, fresh = w.q.fresh;
    const int r0 = w.group * S::kRows;
    const int t0 = w.step, t1 = w.end();

    uint32_t qf[S::kQueryInSmem ? 1 : NT][kSteps][2];
    float row_scale[NT][2];
    load_queries<S>(a, w.q, w.head, r0, s_limit[warp], q_smem, qf, row_scale);

    float o[kChunks][NT][4];  // columns 16 c + 2 g, + 1 (rows g, g + 8 of A) of rows 2 t4, + 1
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[c][nt][j] = 0.0f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
    }
    int ref = 0;  // O's units, see next_units
    bool nans = false;

    int t = t0;
    for (; t < t1 && ok && len > 0; ++t) {
      const int pos = t * kStep;  // first token of the step
      const uint32_t sb = ring + stage * S::kStage;
      ok = __all_sync(0xffffffffu, mbar_wait(k_full + 8 * stage, phase, wc));
      if (!ok) break;
      uint32_t pb[2][NT][2];
      uint32_t none;  // see no_page
      int kbyte[2], vbyte[2];
      {
        const uint4 words = s_rings.scales[warp][stage];
        const uint32_t shifts = s_rings.shifts[warp][stage];
        kbyte[0] = words.x >> (shifts & 31) & 0xff;
        kbyte[1] = words.y >> (shifts >> 8 & 31) & 0xff;
        vbyte[0] = words.z >> (shifts >> 16 & 31) & 0xff;
        vbyte[1] = words.w >> (shifts >> 24) & 0xff;
        none = shifts & kNoBlocks;
      }
      const bool zone = none || pos + kStep - 1 > len - fresh;  // some row may not see all of it
      // byte 0, as where there is no block, is left out of account
      const int next = next_units(ref, min(vbyte[0] ? vbyte[0] : 255, vbyte[1] ? vbyte[1] : 255),
                                  max(vbyte[0], vbyte[1]));
      if (next < 0) break;  // far_steps does the rest
      {
        float sc[2][NT][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t kw[2][D / 16];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              const int chunk = D == 128 ? (2 * t4 + c) ^ x : t4 ^ x;
              const uint4 v = lds128(sb + k_off + (b * 16 + h * 8) * D + chunk * 16);
              kw[h][4 * c] = v.x; kw[h][4 * c + 1] = v.y;
              kw[h][4 * c + 2] = v.z; kw[h][4 * c + 3] = v.w;
            }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[b][nt][j] = 0.0f;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const uint32_t ka[4] = {codes_f16(kw[0][k]), codes_f16(kw[1][k]),
                                    codes_f16_hi(kw[0][k]), codes_f16_hi(kw[1][k])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (S::kQueryInSmem) {
                const uint2 q = lds64(q_smem + (nt * kSteps + k) * 256);
                mma_f16(sc[b][nt], ka, q.x, q.y);
              } else {
                mma_f16(sc[b][nt], ka, qf[nt][k][0], qf[nt][k][1]);
              }
            }
          }
        }
        __syncwarp();  // K and the scales are read
        if (lane == 0) mbar_arrive(k_empty + 8 * stage);

        // Scores are sc x f; the factor of a block and row.
        float f[2][NT][2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float ks = byte_scale(kbyte[b]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) f[b][nt][j] = score_factor(ks, row_scale[nt][j]);
        }
        if (zone) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int at = no_page(none, b) ? INT_MAX - 8 : pos + 16 * b + g;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                // -inf stays -inf with a factor that is not 0
                f[b][nt][j & 1] = fmaxf(f[b][nt][j & 1], 1.17549435e-38f);
                if (at + 8 * (j >> 1) > s_limit[warp][nt * 8 + 2 * t4 + (j & 1)])
                  sc[b][nt][j] = -INFINITY;
              }
          }
        }
        bool grow = next != ref;
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            top[nt][j] = fmaxf(fmaxf(sc[0][nt][j], sc[0][nt][2 + j]) * f[0][nt][j],
                               fmaxf(sc[1][nt][j], sc[1][nt][2 + j]) * f[1][nt][j]);
            grow = grow || top[nt][j] > m[nt][j] + kGrow;
          }
        if (__any_sync(0xffffffffu, grow)) {
          const float fr = pow2i(ref - next);
          ref = next;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float u = top[nt][j];
              u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 4));
              u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 8));
              u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 16));
              const float fm = u > m[nt][j] ? ex2(m[nt][j] - u) : 1.0f;
              m[nt][j] = fmaxf(m[nt][j], u);
              l[nt][j] *= fm;
#pragma unroll
              for (int c = 0; c < kChunks; ++c) {
                o[c][nt][j] *= fm * fr;
                o[c][nt][2 + j] *= fm * fr;
              }
            }
        }
        const float vf[2] = {pow2i(vbyte[0] - ref + kPBits), pow2i(vbyte[1] - ref + kPBits)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float r0m = m[nt][0] == -INFINITY ? 0.0f : m[nt][0];
          const float r1m = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float p0 = ex2(fmaf(sc[b][nt][2 * h], f[b][nt][0], -r0m));
              const float p1 = ex2(fmaf(sc[b][nt][2 * h + 1], f[b][nt][1], -r1m));
              l[nt][0] += p0;
              l[nt][1] += p1;
              pb[b][nt][h] = movmatrix(pack_f16x2(p0 * vf[b], p1 * vf[b]));
            }
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait(v_full + 8 * stage, phase, wc));
      if (!ok) break;
      if (zone && clean_values<D>(sb + S::kHalf, pos, len, fresh, none, s_nan[warp])) nans = true;
      {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
          for (int c = 0; c < kChunks; c += 2) {
            uint32_t v[4];
            ldmatrix_x4_trans(sb + v_off + b * 16 * D + ((vx ^ c) * 16), v);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              const uint32_t a0 = __byte_perm(v[2 * cc], 0, 0x3120);
              const uint32_t a1 = __byte_perm(v[2 * cc + 1], 0, 0x3120);
              const uint32_t va[4] = {codes_f16(a0), codes_f16_hi(a0), codes_f16(a1),
                                      codes_f16_hi(a1)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[c + cc][nt], va, pb[b][nt][0], pb[b][nt][1]);
            }
          }
        }
      }
      // clean_values wrote through the generic proxy what TMA writes next
      if (zone) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();  // V is read
      if (lane == 0) mbar_arrive(v_empty + 8 * stage);
      if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
    }

    // (OWN: a part lies in the warp's ring, whose loads are all read.)
    const bool far = ok && t < t1 && len > 0;
    const bool whole = t0 == 0 && t1 == w.steps;
    finish_unit<S>(a, w.q, w.head, r0, whole && !far,
                   OWN && !far ? own_part(warp) : part_slot<S>(a, warp, t0), s_limit[warp],
                   nans ? s_nan[warp] : nullptr, ref, o, m, l);
    if (far) {
      const uint32_t at = far_steps<S, OWN>(a, sh, base, t, stage | phase << 16);
      ok = at != ~0u;
      stage = at & 0xffff;
      phase = at >> 16;
    }
    // After a wait that gave up the other units are walked too: what is not
    // computed is written as it stands.
    __syncwarp();
    int more = 0;
    if (lane == 0) more = w.next(a, s_seqs);
    if (!__shfl_sync(0xffffffffu, more, 0)) break;
    __syncwarp();
  }
  if constexpr (OWN) {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * S::kWarps) : "memory");
    const int each = (w.steps + S::kWarps - 1) / S::kWarps;
    const int parts = (w.steps + each - 1) / each, r0 = w.group * S::kRows;
    const int rows = min(S::kRows, w.q.fresh * a.group - r0);
    if (parts == 1) return;
    constexpr int kLanes = D / 4;  // of a row, four columns each
    const int col = 4 * (lane % kLanes);
    for (int r = (warp * 32 + lane) / kLanes; r < rows; r += 32 * S::kWarps / kLanes) {
      float top = -INFINITY, sum = 0.0f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < parts; ++i) {  // in the order of the steps
        const float2* src = reinterpret_cast<const float2*>(own_part(i) + r * (D + 2));
        const float2 ml = src[D / 2], u0 = src[col / 2], u1 = src[col / 2 + 1];
        add_part(top, sum, v, ml.x, ml.y, make_float4(u0.x, u0.y, u1.x, u1.y));
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      write_row<D>(a, w.q.row0, w.head, r0 + r, col, top, sum,
                   make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    }
  }
}

template <class S>
cudaError_t launch(cudaStream_t s, const KvAttention& a) {
  using Deal = typename S::Deal;
  CUtensorMap map;
  const uint64_t rows = 2ull * a.cache.pages * a.cache.heads * a.cache.page;
  const uint64_t dims[2] = {static_cast<uint64_t>(S::D), rows};
  const uint64_t strides[1] = {static_cast<uint64_t>(S::D)};
  const uint32_t box[2] = {static_cast<uint32_t>(S::D),
                           static_cast<uint32_t>(std::min(a.cache.page, kStep))};
  cudaError_t e = make_u8_map_nd(&map, a.cache.codes, 2, dims, strides, box, S::D);
  if (e != cudaSuccess) return e;
  // No more warps than shares there can be.
  const long long steps = (static_cast<long long>(a.max_pages) * a.cache.page + kStep - 1) / kStep;
  const long long units = ((static_cast<long long>(a.T) * a.group + S::kRows - 1) / S::kRows +
                           a.n_seqs) * a.cache.heads;
  const long long ctas = (std::min(steps * units, 1LL << 40) + Deal::kMinSteps * S::kWarps - 1) /
                         (Deal::kMinSteps * S::kWarps);
  const int sms = device_sm_count();
  if (units <= sms && steps <= kOwnSteps * S::kWarps) {
    e = allow_dynamic_smem(reinterpret_cast<const void*>(moe_kv_attention_kernel<S, true>),
                           S::kSmem);
    if (e != cudaSuccess) return e;
    KernelScope scope(s, "moe_kv_attention");
    return launch_kernel(moe_kv_attention_kernel<S, true>, dim3(static_cast<unsigned>(units)),
                         dim3(S::kThreads), S::kSmem, s, map, a);
  }
  e = allow_dynamic_smem(reinterpret_cast<const void*>(moe_kv_attention_kernel<S, false>),
                         S::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = static_cast<int>(
      std::min<long long>({std::max(1LL, ctas), static_cast<long long>(sms),
                           static_cast<long long>(kKvAttentionWarps / S::kWarps)}));
  {
    KernelScope scope(s, "moe_kv_attention");
    e = launch_kernel(moe_kv_attention_kernel<S, false>, dim3(grid), dim3(S::kThreads), S::kSmem, s,
                      map, a);
  }
  return e == cudaSuccess ? launch_join<S::D, Deal>(s, a, steps, grid * S::kWarps) : e;
}

template <int D>
cudaError_t launch_dim(cudaStream_t s, const KvAttention& a) {
  constexpr int k = 128 / D;  // stages are in proportion
  switch (kv_attention_rows(a.T, a.n_seqs, a.group)) {
    case 8: return launch<Shape<D, 1, 12, 2 * k, 2>>(s, a);
    case 16: return launch<Shape<D, 2, 10, 2 * k, 2>>(s, a);
    default:
      if constexpr (D == 128) return launch_kv_attention_wide(s, a);
      else return launch<Shape<D, 4, 7, 2 * k, 1>>(s, a);
  }
}

}  // namespace

// Rows of a unit: 8, 16 or 32, what a sequence has on average.
int kv_attention_rows(int T, int n_seqs, int group) {
  const long long rows = (static_cast<long long>(T) * group + n_seqs - 1) / n_seqs;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

size_t kv_attention_workspace(int T, int n_seqs, int group, int dim) {
  return 256 + static_cast<size_t>(kKvAttentionWarps) * 2 * kv_attention_rows(T, n_seqs, group) *
                   (dim + 2) * sizeof(float);
}

cudaError_t launch_kv_attention(cudaStream_t s, const KvAttention& a) {
  return a.cache.dim == 64 ? launch_dim<64>(s, a) : launch_dim<128>(s, a);
}

}  // namespace moe
