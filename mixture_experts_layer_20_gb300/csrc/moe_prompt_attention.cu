// Causal attention over whole prompts, packed one after another (bf16 in and
// out, grouped heads):
//   o_i = sum_{j <= i} p_ij v_j,  p_ij = softmax_j(scale q_i . k_j),
//   lse_i = ln sum_{j <= i} exp(scale q_i . k_j).
//
// A CTA takes up to 256 rows of one KV head: two tiles of 128 rows, a row
// being (token, query head of the group), so the heads that share a KV head
// share its tiles, and a short prompt fills a tile with its heads.  It passes
// once over the keys in tiles of 128 with a running maximum and sum:
//   S = Q K^T (tcgen05, fp32 in tensor memory), P = 2^(c S - m) as bf16 over
//   S's own columns, O += P V (tcgen05, P read from tensor memory, V as it
//   lies in memory: N-major).
// Roles: warp 10 takes the next item (256 rows), warp 9 loads (TMA ring of K
// and V tiles), warp 8 issues every MMA, warps 0-3 and 4-7 do the softmax of
// one row tile each, one row a thread.  The two row tiles take turns: while one
// is in its softmax, the tensor cores work on the other.  One CTA per SM stays
// for all its items, so that the next one's loads and first scores run during
// the last one's epilogue; items are handed out by a counter, those with most
// keys first.
// O is rescaled in tensor memory only when a row's maximum grew by more than
// 2^8 since the last time: P then stays below 2^8, within bf16, and the sums
// are in fp32.  P's rounding to bf16 (its sum is taken before it) is what the
// tensor cores take; it adds about as much error as rounding the output.
//
// Measured (one prompt of 8192 tokens, 64 query heads over 8, head dimension
// 128): 605 us, 1.82 PFLOP/s, 96 % of a library GEMM's; the tensor pipe is
// active 81 % of the cycles, limited by its reads of shared memory (a pair of
// row tiles takes 2500 cycles a key tile, 2048 of them in the MMAs).  Eleven
// prompts of 6000 tokens in all, 64 heads over 4: 90 us, 1.0 PFLOP/s.  There an
// item has 4 key tiles on average and each change of item costs about two more:
// the last product, the epilogue and the next item's first softmax follow one
// another.  Not faster: an epilogue by warps of its own (registers: 116 us),
// masked columns skipped 32 at a time (98), the next item taken ahead (95).
//
// Masked keys take no part whatever they hold: their scores are set by index.
// Their values do meet P = 0 in the MMA, where an infinity or NaN in a value
// row that a query may not see would make 0 x inf = NaN.  Where a row's result is
// not finite, its warp looks for the first such value of each column
// (not_finite): a column where the row sees one gets what that gives, and only a
// row with a column where it does not is computed again without the masked keys
// (at most the rows between a column's first such value and its key tile's start).
// 8192 tokens, 64 heads over 8, head dimension 128, a NaN among the values of the
// first token: 656 us; all values NaN: 3.4 ms (615 us without).  The other roles'
// waits run meanwhile: a row takes 20 instructions a key, 32 rows of 10^6 keys about
// a third of the default bound.

#include <algorithm>
#include <climits>

#include "moe_attention.cuh"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kTile = 128;        // rows of a row tile, and keys of a key tile
constexpr int kMmaWarp = 8, kLoadWarp = 9, kItemWarp = 10;
constexpr int kItems = 2;         // items taken ahead of the roles
constexpr int kThreads = 384;     // three warpgroups: two of softmax, one of the others
constexpr float kGrow = 8.0f;     // log2 growth of the maximum that rescales O
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // S (and P) of tile q at 128 q, O at 256 + 128 q

template <int D>
struct Cfg {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kBoxBytes = kTile * 128;  // 64 of the D columns
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kOut = 8 * 32 * 128;      // 64 columns of each softmax warp's rows, as bf16
  static constexpr int kSmem = (2 + kStages) * kTileBytes + kOut + 1024;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

struct PromptParams {
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const int32_t* offsets;
  int T, n_seqs, heads, kv_heads, group;
  int tok;    // tokens of a row tile: 128 / group
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  unsigned* status;
  unsigned long long timeout_ns;
  unsigned *item_ctr, *exit_ctr;  // at zero; the last CTA to leave resets both
};

// 256 rows of work: tokens first .. of the sequence from row `start` on.
struct Item {
  int start, first, kvh;
  int rows_tok[2];  // tokens of the two row tiles
  int tiles[2];     // and their key tiles (0: nothing to do)
  __device__ int n_tiles() const { return max(tiles[0], tiles[1]); }
};

// Items in order of their key tiles, most first, without a list of them: a
// sequence's blocks that see exactly L tiles are counted from its length.  A
// warp, which asks for growing indices.  It looks at 32 sequences at a time, goes on
// where the last search of the level ended, and passes over spans of sequences that
// are all too short for the level (each lane knows the longest of one span): with
// every search from the first sequence on, 4096 prompts of up to 20 tokens (32 heads over
// 4) took 2941 us instead of 482, with one of 8192 tokens among them 4457 instead of 760.
struct Order {
  int level, base, count;  // key tiles, index of the level's first item, its items
  int start, len;          // of sequence `lane`
  int most, span;          // the longest of `span` groups of 32 sequences, from lane x span on
  int at, before;          // the level's search: group it goes on from, blocks before that

  __device__ static void sequence(const PromptParams& p, int s, int& start, int& len) {
    start = len = 0;
    if (s >= p.n_seqs) return;
    start = __ldg(p.offsets + s);
    const int end = __ldg(p.offsets + s + 1);
    len = end - start;
    if (start < 0 || len < 0 || end > p.T) {
      atomicOr(p.status, kStatusDeviceCheck);
      len = 0;
    }
  }
  __device__ static int sum(int v) { return __reduce_add_sync(0xffffffffu, v); }
  __device__ static int tiles(int len) { return (len + kTile - 1) / kTile; }
  // Blocks of a sequence that see at most `tiles` key tiles.
  __device__ static int blocks(const PromptParams& p, int len, int tiles) {
    const int block = 2 * p.tok;
    return len <= tiles * kTile ? (len + block - 1) / block : tiles * kTile / block;
  }
  __device__ void group(const PromptParams& p, int g, int& st, int& l) const {
    st = start;
    l = len;
    if (g > 0) sequence(p, 32 * g + (threadIdx.x & 31), st, l);
  }
  // The first group from g on that may have blocks of this level; past all: none.
  __device__ int next_group(int g) const {
    const int lane = g / span;
    if (lane > 31) return INT_MAX;
    const unsigned mask =
        __ballot_sync(0xffffffffu, tiles(most) >= level) & (0xffffffffu << lane);
    if (mask == 0) return INT_MAX;
    return max(g, (__ffs(mask) - 1) * span);
  }
  __device__ void begin_level(const PromptParams& p) {
    before = at = 0;
    int n = 0;
    if (p.n_seqs <= 32) {
      n = blocks(p, len, level) - blocks(p, len, level - 1);
    } else {
      at = next_group(0);
      for (int g = at; g <= (p.n_seqs - 1) / 32; g = next_group(g + 1)) {
        int st, l;
        group(p, g, st, l);
        n += blocks(p, l, level) - blocks(p, l, level - 1);
      }
    }
    count = sum(n) * p.kv_heads;
  }
  __device__ void init(const PromptParams& p) {
    const int lane = threadIdx.x & 31, groups = (p.n_seqs + 31) / 32;
    sequence(p, lane, start, len);
    int top = len;
    span = 1;
    most = 0;
    if (groups > 1) {
      span = (groups + 31) / 32;
#pragma unroll 4
      for (int g = 0; g < groups; ++g) {
        int st, l;
        group(p, g, st, l);
        const int longest = __reduce_max_sync(0xffffffffu, l);
        if (g / span == lane) most = max(most, longest);
      }
      top = most;
    }
    level = tiles(__reduce_max_sync(0xffffffffu, top));
    base = count = 0;
    if (level > 0) begin_level(p);
  }
  // Item i (not below the last one asked for); false: there are not as many.
  __device__ bool get(const PromptParams& p, int i, Item& it) {
    while (level > 0 && i >= base + count) {
      base += count;
      if (--level > 0) begin_level(p);
    }
    if (level <= 0) return false;
    const int m = (i - base) / p.kv_heads;
    it.kvh = (i - base) - m * p.kv_heads;
    for (; at <= (p.n_seqs - 1) / 32; at = next_group(at + 1)) {
      int st, l;
      group(p, at, st, l);
      const int below = blocks(p, l, level - 1), n = blocks(p, l, level) - below;
      int c = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, c, o);
        if (static_cast<int>(threadIdx.x & 31) >= o) c += u;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + c > m);
      if (hit) {
        const int lane = __ffs(hit) - 1;
        const int block = __shfl_sync(0xffffffffu, below + m - before - (c - n), lane);
        it.start = __shfl_sync(0xffffffffu, st, lane);
        it.first = block * 2 * p.tok;
        const int length = __shfl_sync(0xffffffffu, l, lane);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int first = it.first + q * p.tok;
          it.rows_tok[q] = max(0, min(p.tok, length - first));
          it.tiles[q] = it.rows_tok[q] > 0 ? (first + it.rows_tok[q] - 1) / kTile + 1 : 0;
        }
        return true;
      }
      before += __shfl_sync(0xffffffffu, c, 31);
    }
    return false;
  }
};

// Row (token, head) again without the keys past `token`, one warp, from its running
// maximum m and sum l.
template <int D>
__device__ __forceinline__ void row_again(const PromptParams& p, int start, int token, int head,
                                          float m, float l, int lane) {
  constexpr int kCols = D / 32;  // of a lane
  const int j = head / p.group;
  const __nv_bfloat16* q = p.q + static_cast<long long>(token) * p.q_stride + head * D;
  const __nv_bfloat16* k = p.k + j * D;
  const __nv_bfloat16* v = p.v + j * D + lane * kCols;
  auto two = [](uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  };
  const float ref = m == -INFINITY ? 0.0f : m;
  float acc[kCols] = {};
  for (int t0 = start; t0 <= token; t0 += 32) {
    float s = 0.0f;
    const uint4* kr =
        reinterpret_cast<const uint4*>(k + static_cast<long long>(min(t0 + lane, token)) * p.k_stride);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(q) + i), b = __ldg(kr + i);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 x = two(aw[c]), y = two(bw[c]);
        s = fmaf(x.x, y.x, s);
        s = fmaf(x.y, y.y, s);
      }
    }
    const float w = t0 + lane <= token ? ex2(fmaf(s, p.scale_log2, -ref)) : 0.0f;
    const int n = min(32, token - t0 + 1);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const uint32_t* vr =
          reinterpret_cast<const uint32_t*>(v + static_cast<long long>(t0 + i) * p.v_stride);
#pragma unroll
      for (int c = 0; c < kCols; c += 2) {
        const float2 x = two(__ldg(vr + c / 2));
        acc[c] = fmaf(wi, x.x, acc[c]);
        acc[c + 1] = fmaf(wi, x.y, acc[c + 1]);
      }
    }
  }
  __nv_bfloat16* out = p.out + (static_cast<size_t>(token) * p.heads + head) * D + lane * kCols;
#pragma unroll
  for (int c = 0; c < kCols; ++c) out[c] = __float2bfloat16_rn(l == 0.0f ? 0.0f : acc[c] / l);
}

// The rows `rows` of a warp (one a lane, (token, head) of the sequence from `start` on),
// whose results are not finite though their sums are.  Keys 0 .. end - 1 met them,
// those up to first_tok all of them.
template <int D>
__device__ __noinline__ void not_finite(const PromptParams& p, int start, int first_tok, int end,
                                        unsigned rows, int token, int head, float m, float l) {
  constexpr int kLanes = D / 8;          // of a value row, 8 columns each
  constexpr int kPer = 32 / kLanes;      // rows at a time
  constexpr int kAt = 8;                 // loads under way
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* v = p.v + static_cast<long long>(start) * p.v_stride + head / p.group * D +
                           lane % kLanes * 8;
  // Whether a word's halves have all exponent bits set: in its top bits and theirs.
  auto odd = [](const uint4& x) {
    auto one = [](uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; };
    return ((one(x.x) | one(x.y) | one(x.z) | one(x.w)) & 0x80008000u) != 0;
  };
  // fn(key, its 8 values) for keys from .. end - 1, where not all are finite
  auto scan = [&](int from, auto fn) {
    for (int t0 = from + lane / kLanes; t0 < end; t0 += kAt * kPer) {
      uint4 x[kAt];
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        const int t = t0 + i * kPer;
        x[i] = t < end ? __ldg(reinterpret_cast<const uint4*>(v + static_cast<long long>(t) * p.v_stride))
                       : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kAt; ++i)
        if (odd(x[i])) fn(t0 + i * kPer, x[i]);
    }
  };
  // Values that every row sees give what they give.
  bool hidden = false;
  scan(first_tok + 1, [&](int, const uint4&) { hidden = true; });
  if (!__any_sync(0xffffffffu, hidden)) return;
  // The first NaN and infinity of either sign of each column.
  int nan[8], inf[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) nan[i] = inf[0][i] = inf[1][i] = INT_MAX;
  unsigned open = 0xff;  // columns without a NaN so far
  scan(0, [&](int t, const uint4& x) {
    if (open == 0) return;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t h = w[i / 2] >> (16 * (i & 1)) & 0xffffu;
      if ((h & 0x7f80u) != 0x7f80u) continue;
      if (h & 0x7fu) {
        nan[i] = min(nan[i], t);
        open &= ~(1u << i);
      } else if (h & 0x8000u) {
        inf[1][i] = min(inf[1][i], t);
      } else {
        inf[0][i] = min(inf[0][i], t);
      }
    }
  });
#pragma unroll
  for (int o = kLanes; o < 32; o *= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      nan[i] = min(nan[i], __shfl_xor_sync(0xffffffffu, nan[i], o));
      inf[0][i] = min(inf[0][i], __shfl_xor_sync(0xffffffffu, inf[0][i], o));
      inf[1][i] = min(inf[1][i], __shfl_xor_sync(0xffffffffu, inf[1][i], o));
    }
  while (rows) {
    const int r = __ffs(rows) - 1;
    rows &= rows - 1;
    const int tok = __shfl_sync(0xffffffffu, token, r), h = __shfl_sync(0xffffffffu, head, r);
    const float mr = __shfl_sync(0xffffffffu, m, r), lr = __shfl_sync(0xffffffffu, l, r);
    const int pos = tok - start;
    bool again = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int first = min(nan[i], min(inf[0][i], inf[1][i]));
      again = again || (first > pos && first < end);
    }
    if (__any_sync(0xffffffffu, again)) row_again<D>(p, start, tok, h, mr, lr, lane);
    __syncwarp();
    if (lane < kLanes) {
      __nv_bfloat16* out = p.out + (static_cast<size_t>(tok) * p.heads + h) * D + lane * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool up = inf[0][i] <= pos, down = inf[1][i] <= pos;
        if (nan[i] <= pos || (up && down)) out[i] = __ushort_as_bfloat16(0x7fff);
        else if (up || down) out[i] = __ushort_as_bfloat16(up ? 0x7f80 : 0xff80);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    moe_prompt_attention_kernel(const __grid_constant__ CUtensorMap map_q,
                                const __grid_constant__ CUtensorMap map_k,
                                const __grid_constant__ CUtensorMap map_v,
                                const __grid_constant__ PromptParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t s_bar[2 * C::kStages + 13 + 2 * kItems];
  __shared__ Item s_item[kItems];
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_base = base;
  const uint32_t ring = base + 2 * C::kTileBytes;
  const uint32_t out_smem = ring + C::kStages * C::kTileBytes;
  const uint32_t full_bar = smem_u32(&s_bar[0]);
  const uint32_t empty_bar = smem_u32(&s_bar[C::kStages]);
  const uint32_t qfull_bar = smem_u32(&s_bar[2 * C::kStages]);
  const uint32_t sfull_bar = qfull_bar + 16;  // S of tile q ready (and O of the tile before)
  const uint32_t pfull_bar = qfull_bar + 32;  // half h of P of tile q (at 2 h + q) ready, O rescaled
  const uint32_t ofull_bar = qfull_bar + 64;  // O of tile q complete
  const uint32_t qempty_bar = qfull_bar + 80;  // Q of tile q read
  const uint32_t drain_bar = qfull_bar + 96;
  const uint32_t ifull_bar = qfull_bar + 104;  // item ready
  const uint32_t iempty_bar = ifull_bar + 8 * kItems;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full_bar + 8 * s, 1);
      mbar_init(empty_bar + 8 * s, 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(qfull_bar + 8 * q, 1);
      mbar_init(sfull_bar + 8 * q, 1);
      mbar_init(pfull_bar + 8 * q, 4);
      mbar_init(pfull_bar + 16 + 8 * q, 4);
      mbar_init(ofull_bar + 8 * q, 1);
      mbar_init(qempty_bar + 8 * q, 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(ifull_bar + 8 * i, 1);
      mbar_init(iempty_bar + 8 * i, 10);  // the loading, MMA and softmax warps
    }
    mbar_init(drain_bar, 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&s_tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_wait_and_release();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem_base, 0);
  const WaitCtx wc{p.timeout_ns, p.status, &s_abort};

  // The next item, for a role's warp (no tiles: the end, or a wait gave up).
  int item_at = 0;
  auto next_item = [&]() {
    const int slot = item_at % kItems;
    const bool got =
        __all_sync(0xffffffffu, mbar_wait(ifull_bar + 8 * slot, (item_at / kItems) & 1, wc));
    ++item_at;
    Item it = s_item[slot];
    // A load in flight is not waited for by a later arrive: without the fence the slot
    // might be written again under it.
    asm volatile("fence.acq_rel.cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(iempty_bar + 8 * slot);
    // the broadcasts tell the compiler that the counts are uniform
#pragma unroll
    for (int q = 0; q < 2; ++q) it.tiles[q] = __shfl_sync(0xffffffffu, got ? it.tiles[q] : 0, 0);
    return it;
  };

  // Registers go where the rows of scores are: 256 x 208 + 128 x 88 of the
  // launch's 384 x 168, 208 the fewest that do not
  // spill (8192 tokens: 615 us; with 216 + 72, 622).
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kItemWarp) {
      Order order;
      order.init(p);
      int i = blockIdx.x;
      for (int n = 0;; ++n) {
        Item it{};
        const bool got = order.get(p, i, it);
        const int slot = n % kItems;
        if (!__all_sync(0xffffffffu,
                        mbar_wait(iempty_bar + 8 * slot, ((n / kItems) & 1) ^ 1u, wc)))
          break;
        if (lane == 0) {
          s_item[slot] = it;
          mbar_arrive(ifull_bar + 8 * slot);
          if (got) i = gridDim.x + atomicAdd(p.item_ctr, 1u);
        }
        if (!got) break;
        i = __shfl_sync(0xffffffffu, i, 0);
      }
      // The last CTA to come here resets the counters for the next call.
      if (lane == 0 && atomicAdd(p.exit_ctr, 1u) == gridDim.x - 1) {
        atomicExch(p.item_ctr, 0u);
        atomicExch(p.exit_ctr, 0u);
      }
    } else if (warp == kLoadWarp) {
      int stage = 0, issued = 0, q_loads[2] = {0, 0};
      uint32_t phase = 0;
      bool ok = true;
      for (;;) {
        const Item it = next_item();
        const int n_tiles = it.n_tiles();
        if (n_tiles == 0) break;
        if (lane == 0) {
          auto load_q = [&](int q) {
            if (it.tiles[q] == 0 || !ok) return;
            ok = mbar_wait(qempty_bar + 8 * q, (q_loads[q] & 1) ^ 1u, wc);
            if (!ok) return;
            mbar_arrive_expect_tx(qfull_bar + 8 * q,
                                  static_cast<uint32_t>(p.tok * p.group * 128 * (D / 64)));
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(q_base + q * C::kTileBytes + c * C::kBoxBytes, &map_q,
                          qfull_bar + 8 * q, 64 * c, it.kvh * p.group,
                          it.start + it.first + q * p.tok);
            ++q_loads[q];
          };
          auto load = [&](const CUtensorMap* map, int j) {
            ok = ok && mbar_wait(empty_bar + 8 * stage, phase ^ 1u, wc);
            if (!ok) return;
            const uint32_t fb = full_bar + 8 * stage;
            mbar_arrive_expect_tx(fb, C::kTileBytes);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(ring + stage * C::kTileBytes + c * C::kBoxBytes, map, fb, 64 * c, it.kvh,
                          it.start + j * kTile);
            ++issued;
            if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
          };
          load(&map_k, 0);
          load_q(0);
          load_q(1);
          for (int j = 0; j < n_tiles && ok; ++j) {
            load(&map_v, j);
            if (ok && j + 1 < n_tiles) load(&map_k, j + 1);
          }
        }
        __syncwarp();
      }
      // Drain: the last loads may still be landing.
      if (lane == 0) {
        for (int i = max(0, issued - C::kStages); i < issued; ++i)
          mbar_wait_drain(full_bar + 8 * (i % C::kStages), (i / C::kStages) & 1, p.status);
        for (int q = 0; q < 2; ++q)
          if (q_loads[q]) mbar_wait_drain(qfull_bar + 8 * q, (q_loads[q] - 1) & 1, p.status);
      }
    } else if (warp == kMmaWarp) {
      // The whole warp runs the loop, so that addresses and descriptors stay in
      // uniform registers; one elected lane's instructions take effect.  (From a
      // branch of one lane each MMA took about 80 cycles to issue, more than
      // the 64 it runs.)
      constexpr uint32_t idesc_s = idesc_bf16_f32(kTile, kTile);
      constexpr uint32_t idesc_o = idesc_bf16_f32(kTile, D) | (1u << 16);  // B (V) is N-major
      const bool leader = elect_one();
      int stage = 0;
      uint32_t phase = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
      bool ok = true;
      // The next tile of the ring, waited for: its stage.
      auto take = [&]() {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(full_bar + 8 * stage, phase, wc));
        tc_fence_after_sync();
        const int at = stage;
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        return at;
      };
      auto issue_s = [&](int q, int at) {
        const uint32_t qa = desc_k(q_base + q * C::kTileBytes);
        const uint32_t kb = desc_k(ring + at * C::kTileBytes);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t off = ((i / 4) * C::kBoxBytes + (i % 4) * 32) / 16;
          mma_ss(leader, tmem + kColS + 128 * q, qa + off, kb + off, idesc_s, i != 0);
        }
        commit(leader, sfull_bar + 8 * q);
      };

      while (ok) {
        const Item it = next_item();
        const int n_tiles = it.n_tiles();
        if (n_tiles == 0) break;
        int k_at = take();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (it.tiles[q] == 0 || !ok) continue;
          ok = __all_sync(0xffffffffu, mbar_wait(qfull_bar + 8 * q, q_phase[q], wc));
          q_phase[q] ^= 1u;
          if (!ok) continue;
          tc_fence_after_sync();
          issue_s(q, k_at);
          if (it.tiles[q] == 1) commit(leader, qempty_bar + 8 * q);
        }
        commit(leader, empty_bar + 8 * k_at);
        for (int j = 0; j < n_tiles && ok; ++j) {
          const int v_at = take();
          const bool more = j + 1 < n_tiles;
          if (more) k_at = take();
          const uint32_t vb = desc_n(ring + v_at * C::kTileBytes, C::kBoxBytes);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (j >= it.tiles[q] || !ok) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ok = ok &&
                   __all_sync(0xffffffffu, mbar_wait(pfull_bar + 16 * h + 8 * q, p_phase[q], wc));
              if (!ok) break;
              tc_fence_after_sync();
#pragma unroll
              for (int i = kTile / 32 * h; i < kTile / 32 * (h + 1); ++i)
                mma_ts(leader, tmem + kColO + 128 * q, tmem + kColS + 128 * q + 8 * i,
                       vb + i * (2048 / 16), idesc_o, j != 0 || i != 0);
            }
            p_phase[q] ^= 1u;
            if (!ok) continue;
            if (j + 1 < it.tiles[q]) {
              issue_s(q, k_at);
              if (j + 2 == it.tiles[q]) commit(leader, qempty_bar + 8 * q);
            } else {
              commit(leader, ofull_bar + 8 * q);
            }
          }
          commit(leader, empty_bar + 8 * v_at);
          if (more) commit(leader, empty_bar + 8 * k_at);
        }
      }
      // Drain: every MMA issued completes before tensor memory is freed.
      commit(leader, drain_bar);
      if (leader) mbar_wait_drain(drain_bar, 0, p.status);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int q = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int my_tok = row / p.group;  // of the tile
    const int row_at = my_tok * p.heads + row % p.group;  // of this thread's row in out, from the tile's
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + kColS + 128 * q;
    const uint32_t t_o = tmem + lanes + kColO + 128 * q;
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true;
    while (ok) {
      const Item it = next_item();
      if (it.n_tiles() == 0) break;
      const int n = q == 0 ? it.tiles[0] : it.tiles[1];
      if (n == 0) continue;
      const int head = it.kvh * p.group + row % p.group;
      const int first_tok = it.first + q * p.tok;
      const int pos = first_tok + my_tok;  // position in the sequence = last key seen
      // Rows past the sequence's end or the group's (their queries are the next sequence's,
      // or whatever was there) have no say below.
      const bool valid = my_tok < (q == 0 ? it.rows_tok[0] : it.rows_tok[1]);
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < n; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(sfull_bar + 8 * q, s_phase, wc));
        s_phase ^= 1u;
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t s[kTile];
        const int last = pos - j * kTile;  // last column seen
        const bool diagonal = j * kTile + kTile - 1 > first_tok;
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto half_max = [&](int h) {
          if (diagonal) {
#pragma unroll
            for (int c0 = kTile / 2 * h; c0 < kTile / 2 * (h + 1); c0 += 32) {
              if (j * kTile + c0 + 31 <= first_tok) continue;  // seen by all rows
#pragma unroll
              for (int c = c0; c < c0 + 32; ++c)
                if (c > last) s[c] = 0xff800000u;
            }
          }
#pragma unroll
          for (int c = kTile / 2 * h; c < kTile / 2 * (h + 1); c += 2)
            mx[(c >> 1) & 3] =
                max3(mx[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        };
        tmem_ld_x32(t_s, s);
        tmem_ld_x32(t_s + 32, s + 32);
        tmem_ld_wait();
        tmem_ld_x32(t_s + 64, s + 64);
        tmem_ld_x32(t_s + 96, s + 96);
        half_max(0);
        tmem_ld_wait();
        half_max(1);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, valid && top > m + kGrow)) {
          // The MMAs before this S, among them the last into O, are complete.
          const float f = top > m ? ex2(m - top) : 1.0f;  // 0 from -inf
          m = fmaxf(m, top);
          l *= f;
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld_x32(t_o + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st_x32(t_o + c, o);
          }
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), ref2 = pair(-ref, -ref);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int c = kTile / 2 * h; c < kTile / 2 * (h + 1); c += 2) {
            const float2 x = unpair(
                fma2(pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, ref2));
            const float a = ex2(x.x), b = ex2(x.y);
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pair(a, b));
            s[c >> 1] = pack_bf16x2(a, b);
          }
          tmem_st_x32(t_s + 32 * h, s + 32 * h);
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull_bar + 16 * h + 8 * q);
        }
        const float2 both = unpair(add2(sum[0], sum[1]));
        l += both.x + both.y;
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, mbar_wait(ofull_bar + 8 * q, o_phase, wc));
      o_phase ^= 1u;
      if (ok) {
        tc_fence_after_sync();
        const int token = it.start + pos;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        // Each thread has a row; through shared memory (16-byte units turned by
        // the row, so that neither side conflicts) eight lanes store 128 bytes
        // of one.  Stores straight from the rows' threads touch a line a lane:
        // 100 us instead of 92 for 11 prompts of 6000 tokens in all, 64 heads.
        __nv_bfloat16* const tile_out =
            p.out + (static_cast<long long>(it.start + first_tok) * p.heads + it.kvh * p.group) * D;
        const unsigned valid_rows = __ballot_sync(0xffffffffu, valid);
        const uint32_t mine = out_smem + warp * (32 * 128);
        const int sub = lane >> 3, unit = lane & 7;
        const uint64_t inv2 = pair(inv, inv);
        uint64_t odd[2] = {0, 0};  // stays 0 where all values are finite
#pragma unroll
        for (int c = 0; c < D; c += 64) {
          uint32_t o[64];
          tmem_ld_x32(t_o + c, o);
          tmem_ld_x32(t_o + c + 32, o + 32);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t x = fma2(pair(__uint_as_float(o[8 * i + 2 * k]),
                                           __uint_as_float(o[8 * i + 2 * k + 1])),
                                      inv2, 0);
              odd[k & 1] = fma2(x, 0, odd[k & 1]);
              const float2 y = unpair(x);
              v[k] = pack_bf16x2(y.x, y.y);
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             mine + lane * 128 + ((i ^ (lane & 7)) * 16)),
                         "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                         : "memory");
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + sub;
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(mine + r * 128 + ((unit ^ (r & 7)) * 16)));
            const int at = __shfl_sync(0xffffffffu, row_at, r);
            if (valid_rows >> r & 1)
              *reinterpret_cast<uint4*>(tile_out + static_cast<long long>(at) * D + c + unit * 8) = v;
          }
          __syncwarp();
        }
        const float2 rest = unpair(add2(odd[0], odd[1]));
        const bool finite = rest.x + rest.y == 0.0f;
        if (valid && p.lse)
          p.lse[static_cast<size_t>(token) * p.heads + head] =
              l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
        __syncwarp();  // the rows' first results are written before they are replaced
        // (a sum that is not finite is one of what the row sees)
        const unsigned odd_rows = __ballot_sync(0xffffffffu, valid && !finite && l < INFINITY);
        if (odd_rows)
          not_finite<D>(p, it.start, first_tok, min(n * kTile, p.T - it.start), odd_rows, token, head,
                        m, l);
      }
      tc_fence_before_sync();
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch(cudaStream_t s, const PromptAttention& a) {
  PromptParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.offsets = a.offsets;
  p.T = a.T;
  p.n_seqs = a.n_seqs;
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.group = a.heads / a.kv_heads;
  p.tok = kTile / p.group;
  p.scale_log2 = a.scale * 1.44269504088896341f;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  p.item_ctr = a.status + kTileCounterWord;
  p.exit_ctr = a.status + kTileExitWord;

  CUtensorMap mq, mk, mv;
  auto map = [&](CUtensorMap* m, const void* base, int heads, long long stride, uint32_t box_h,
                 uint32_t box_t) {
    const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(heads),
                              static_cast<uint64_t>(a.T)};
    const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(stride) * 2};
    const uint32_t box[3] = {64, box_h, box_t};
    return make_bf16_map_nd(m, base, 3, dims, strides, box);
  };
  cudaError_t e = map(&mq, a.q, a.heads, a.q_stride, p.group, p.tok);
  if (e == cudaSuccess) e = map(&mk, a.k, a.kv_heads, a.k_stride, 1, kTile);
  if (e == cudaSuccess) e = map(&mv, a.v, a.kv_heads, a.v_stride, 1, kTile);
  if (e != cudaSuccess) return e;
  e = allow_dynamic_smem(reinterpret_cast<const void*>(moe_prompt_attention_kernel<D>),
                         Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  KernelScope scope(s, "moe_prompt_attention");
  // no more CTAs than items there can be
  const long long items = (a.T / (2 * p.tok) + static_cast<long long>(a.n_seqs)) * p.kv_heads;
  const int grid = static_cast<int>(std::min<long long>(items, device_sm_count()));
  return launch_kernel(moe_prompt_attention_kernel<D>, dim3(grid), dim3(kThreads), Cfg<D>::kSmem, s,
                       mq, mk, mv, p);
}

}  // namespace

cudaError_t launch_prompt_attention(cudaStream_t s, const PromptAttention& a) {
  return a.dim == 64 ? launch<64>(s, a) : launch<128>(s, a);
}

}  // namespace moe
