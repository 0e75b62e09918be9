// Attention over packed prompts: TMA tile loads, tcgen05.mma with TMEM
// accumulators, warp-specialised, persistent.
//
// For row i of a sequence and the keys j it sees (j <= i when causal, all of
// the sequence otherwise): o_i = sum_j 2^(c s_ij - m) v_j / sum_j 2^(c s_ij - m),
// s = <q_i, k_j>, c = scale log2 e, m a per-row reference.
//
// A unit is two tiles of 128 query rows (A and B; one TMEM lane per row) that read
// the same keys: 256 rows of one query head, or 128 rows of two heads of one
// key/value head (prompt_shape).  Keys stream in blocks of 128 that both tiles
// use, so each K/V byte read from L2 serves 256 rows.  Where the units of a call
// would leave SMs idle, both tiles are the same 128 rows of a head instead and take
// every other block of keys each; their sums are joined through shared memory.
// Per SM one CTA, its warps:
//   warps 0-3 / 4-7  softmax of tile A / B, thread r owning row r: the block's
//            scores from TMEM into registers, their maximum, the weights in
//            base 2, written over the scores as 16-bit pairs;
//   warp 8   TMA loads: Q tiles, then K and V blocks through one ring;
//   warp 10  zeroes the V rows behind a sequence's end in its last block;
//   warp 9   products, one thread: S = Q K^T (128 x 128 x d) and
//            O += P V (128 x d x 128, P read from TMEM).  While one tile's
//            softmax runs, the tensor core works for the other tile.
//
// The reference of a row is its first block's maximum; it moves (rescaling O in
// TMEM) only when a later maximum exceeds it by more than 8, so a weight is at
// most 2^8, and O is touched by the softmax warps in few blocks.  Weights are
// rounded to the input type for the second product (relative 2^-8 in bf16, 2^-11 in
// fp16; the size of the output's own rounding and averaging out over the keys);
// their sum is taken from the unrounded ones.  In fp16 all weights carry a
// factor 2^7, which cancels, so that only weights below 2^-21 of the largest
// are subnormal.
//
// P overwrites S, and the documented order of two products covers only one
// accumulator, so the next S of a tile waits until the P V before it has completed.
//
// Keys past the end are masked, and the V rows that the last product reads past
// it are zeroed in shared memory: what the buffer holds there (NaN) reaches no
// output.  Units are walked longest first: query tiles in descending order,
// (sequence, head) within; each CTA finds its units by ballots over
// cu_seqlens, counting only those with rows, in alternating direction from
// round to round.  Every wait is bounded; a CTA that gives up records
// RRA_DEVERR_WAIT_TIMEOUT, lets copies and products in flight land, frees its
// TMEM and returns.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "block.cuh"
#include "tile_softmax.cuh"
#include "tc_ptx.cuh"
#include "softmax_tc.cuh"

namespace rra {
namespace {

constexpr int P_SOFTMAX_WARPS = 8;
constexpr int P_LOAD_WARP = 8, P_MMA_WARP = 9, P_TAIL_WARP = 10;
constexpr int P_THREADS = 384;               // three warpgroups; warp 11 only lends its registers
// Registers: 384 threads start with 168 each; the softmax warpgroups take 200
// (a row's 128 scores stay in registers), the third gives down to 104:
// 8 x 200 + 4 x 104 = 12 x 168.  At 216 and 72 the thread that issues the products
// spilled, between the products: 16 x 1024 tokens, 32 / 8 heads, d = 128, 153 against 127 us; one of 16384 1467 / 1401.
constexpr int P_REGS_SOFTMAX = 200, P_REGS_OTHER = 104;
static_assert(8 * P_REGS_SOFTMAX + 4 * P_REGS_OTHER <= 12 * 168, "register split exceeds the launch's registers");
constexpr uint32_t P_TMEM_COLS = 512;
constexpr uint32_t P_SUB = PT * 128;         // one 64-element column group of a tile: 128 rows x 128 B
// Bound on a wait that lasts a whole unit, of up to 2^23 blocks (the loading and the product warp, whose waits
// are of single steps, keep the usual one, and the flag they set ends this one too).
constexpr long long P_UNIT_WAIT_CYCLES = 1LL << 36;

template <int D>
struct PromptCfg {
  static constexpr uint32_t TILE = (D / 64) * P_SUB;              // a Q tile, a K block or a V block
  static constexpr int SLOTS = D == 128 ? 4 : 8;                  // K/V ring: 128 KB
  static constexpr uint32_t OFF_KV = 2 * TILE;
  static constexpr uint32_t OFF_OUT = OFF_KV + SLOTS * TILE;      // output staging, 4 KB a softmax warp
  static constexpr uint32_t OFF_BAR = OFF_OUT + P_SOFTMAX_WARPS * 4096;
  static constexpr uint32_t OFF_JOIN = OFF_BAR + 512;             // [2][128] reference and sum of a row (split units)
  static constexpr uint32_t SMEM = OFF_JOIN + 2 * PT * 8;
  // TMEM columns: S of A and B, O of A and B; P over S, or, where there is
  // room (d = 64), beside it: then the next S need not wait for this P V, and
  // goes as soon as the scores are in registers (32 heads, 8192 rows, not causal: 594 -> 547 us).
  static constexpr bool OWN_P = D == 64;
  static constexpr uint32_t T_S = 0, T_O = 2 * PT, T_P = OWN_P ? T_O + 2 * D : T_S, P_STEP = OWN_P ? PT / 2 : PT;
};

// Barrier and word offsets from OFF_BAR.
constexpr uint32_t PB_KV_FULL = 0;      // [8]
constexpr uint32_t PB_KV_EMPTY = 64;    // [8]
constexpr uint32_t PB_Q_FULL = 128;     // [2]
constexpr uint32_t PB_Q_EMPTY = 144;    // [2]
constexpr uint32_t PB_S_FULL = 160;     // [2] S product done
constexpr uint32_t PB_P_READY = 176;    // [2] P written (one arrival per softmax warp of the tile)
constexpr uint32_t PB_PV_DONE = 192;    // [2] P V product done
constexpr uint32_t PB_U_FULL = 208;     // [2] unit descriptor written
constexpr uint32_t PB_U_EMPTY = 224;    // [2] unit finished (softmax, product and tail warps)
constexpr uint32_t PB_DRAIN = 240;
constexpr uint32_t PW_TMEM = 248, PW_ABORT = 252;
constexpr uint32_t P_DESC = 256;        // [2] x 32 bytes: s0, n, q0, h (q0 < 0: no more units)
constexpr uint32_t PB_S_READ = 320;     // [2] the scores are in registers (one arrival per softmax warp of the tile)
constexpr uint32_t PB_TAIL = 336;       // [2] a V block's tail to zero; zeroed
constexpr uint32_t PB_JOIN = 352;       // [2] tile w's share for the other tile is in shared memory (one arrival per warp)

// How units are made up: `heads` query heads and `rows` rows (2 and 128, or 1 and 256), or
// `split`: 1 and 128, tile w taking the key blocks w, w + 2, ...
struct UnitShape {
  int heads, rows, split;
};

struct PromptUnit {
  int s0, n, q0, h;
  // First row and head of tile w.
  __device__ int row0(int w, const UnitShape& us) const { return us.heads == 2 || us.split ? q0 : q0 + w * PT; }
  __device__ int head(int w, const UnitShape& us) const { return us.heads == 2 ? h + w : h; }
  // Key blocks that the rows of tile w see; split: those of both tiles.
  __device__ int seen(int w, const UnitShape& us, int causal) const {
    if (w == 1 && us.heads == 1 && !us.split && n - q0 <= PT) return 0;
    const int all = (n + PT - 1) / PT;
    return causal ? min(all, row0(w, us) / PT + 1) : all;
  }
  // Key blocks of tile w, and of the unit.
  __device__ int blocks(int w, const UnitShape& us, int causal) const {
    return us.split ? (seen(0, us, causal) + 1 - w) / 2 : seen(w, us, causal);
  }
  __device__ int blocks(const UnitShape& us, int causal) const { return max(seen(0, us, causal), seen(1, us, causal)); }
};

// About how long a call takes with units of this shape, in key blocks of a unit (1.7 us at d = 128, 1.2 at
// d = 64): its longest unit alone, with 2 for its start and end, or all of them spread over the SMs, for sequences as
// long as the mean (causal: units of every length; not causal: rounds of equal ones), with 2 for a change of unit, 1
// where the next unit's first products go out under this one's last.  (0.52: at d = 128 a split unit's ring holds one
// block ahead for each tile; 32 heads of 16384, not causal: 3210 us split, 2820 whole.)
inline double prompt_time(const PromptArgs& a, const UnitShape& us, int d, int num_sms) {
  const int longest = std::min(a.max_seqlen, a.cap), mean_len = std::min(longest, std::max(1, a.cap / a.B));
  auto blocks = [&](int n) { return (n - 1) / PT + 1; };
  const long long tiles = std::min(a.B * ((a.max_seqlen - 1LL) / us.rows + 1), a.cap / us.rows + static_cast<long long>(a.B));
  const double rounds = static_cast<double>(tiles * (a.Hq / us.heads)) / num_sms, per = us.split ? (d == 128 ? 0.52 : 0.5) : 1.0;
  const double mean = (us.split ? 2 : 1) + per * (a.causal ? (blocks(mean_len) + us.rows / PT) / 2.0 : blocks(mean_len));
  const double alone = 2 + (us.split ? (blocks(longest) + 1) / 2 * 2 * per : blocks(longest));
  return std::max(alone, mean * (a.causal ? rounds + 1 / 3.0 : std::ceil(rounds)));
}

// Whole: two heads of a group at the same rows where the group is even, d = 128 and
// the prompts are not very long; else 256 rows of a head.  Two heads see the same blocks, so
// neither tile ever works alone, which the last rows of many sequences would; two
// successive tiles end one after the other, so that one's output leaves under the other's last
// block.  32 / 8 heads, d = 128, causal, heads paired against rows: 16 x 1024 tokens 127 / 140 us,
// 8 x 2048 207 / 222, eight of 1 to 4096 212 / 228; 8192 369 / 370, 16384 1406 / 1399 (within what two runs differ by); d = 64: 8192 281 / 263.
__host__ __device__ inline UnitShape whole_shape(int group, int d, int max_seqlen) {
  return group % 2 == 0 && d == 128 && max_seqlen <= 8192 ? UnitShape{2, PT, 0} : UnitShape{1, 2 * PT, 0};
}

// Split: where that takes less by prompt_time.  d = 128, causal, whole against split: 32 / 8 heads, 200 tokens 9.1 /
// 7.7 us, 1024 18.8 / 17.4, 4096 104 / 117, 16 x 512 47 / 80; 8 / 1 heads, 4096 58 / 34, 8192 111 / 109; d = 64, 12
// heads, not causal: 1024 15.0 / 11.3, 4096 85 / 68, 8192 237 / 243, 16 x 512 23.2 / 33.5.
inline UnitShape prompt_shape(const PromptArgs& a, int d, int num_sms) {
  const UnitShape whole = whole_shape(a.Hq / a.Hkv, d, a.max_seqlen), split{1, PT, 1};
  return prompt_time(a, split, d, num_sms) < prompt_time(a, whole, d, num_sms) ? split : whole;
}

// Walks the non-empty units in order (query tile descending, sequence, head);
// a warp's lanes look at 32 sequences at a time.  The walk only moves forward.
struct UnitWalk {
  UnitShape us;
  int qt;              // current query tile (us.rows rows), from the highest
  int b0;              // current group of 32 sequences
  long long before;    // non-empty units before the group (qt, b0)
  int lane;

  // Rows of sequence b, 0 for one that is not there or not valid (`record`: its code is recorded).
  __device__ int rows_of(const PromptArgs& a, int b, int& s0, int& n, bool record) const {
    if (b >= a.B) return 0;
    s0 = a.cu[b];
    n = a.cu[b + 1] - s0;
    if (n < 0 || n > a.max_seqlen || s0 < 0 || s0 > a.cap - n) {
      if (record)
        record_error(a.err, n < 0 ? RRA_DEVERR_SEQ_NEGATIVE
                                  : (n > a.max_seqlen ? RRA_DEVERR_SEQ_TOO_LONG : RRA_DEVERR_INDEX_RANGE));
      return 0;
    }
    return n;
  }

  // To the first tile of the longest sequence (max_seqlen may be far above it).
  __device__ void start(const PromptArgs& a, bool record) {
    int most = 0;
    for (int b = lane; b < a.B; b += 32) {
      int s0, n;
      most = max(most, rows_of(a, b, s0, n, record));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    qt = (most + us.rows - 1) / us.rows - 1;
    b0 = 0;
    before = 0;
  }

  // The unit with index `target` (not below any earlier target), or q0 < 0.
  __device__ PromptUnit find(const PromptArgs& a, long long target) {
    PromptUnit u;
    while (qt >= 0) {
      int s0 = 0, n = 0;
      const int rows = rows_of(a, b0 + lane, s0, n, false);
      const unsigned live = __ballot_sync(0xffffffffu, rows > qt * us.rows);
      const int per = a.Hq / us.heads;
      const long long here = static_cast<long long>(__popc(live)) * per;
      if (target < before + here) {
        const int k = static_cast<int>((target - before) / per);       // k-th live sequence of the group
        const bool mine = ((live >> lane) & 1u) && __popc(live & ((1u << lane) - 1u)) == k;
        const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        u.s0 = __shfl_sync(0xffffffffu, s0, src);
        u.n = __shfl_sync(0xffffffffu, n, src);
        u.q0 = qt * us.rows;
        u.h = static_cast<int>((target - before) % per) * us.heads;
        return u;
      }
      before += here;
      b0 += 32;
      if (b0 >= a.B) {
        b0 = 0;
        --qt;
      }
    }
    u.q0 = -1;
    return u;
  }
};

// LIMIT: the instantiation of launches made with a wait limit set (rra_set_wait_limit).
template <typename T, int D, bool SPLIT, bool LIMIT>
__global__ void __launch_bounds__(P_THREADS, 1)
    attend_prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const PromptArgs a) {
  using C = PromptCfg<D>;
  const UnitShape us = SPLIT ? UnitShape{1, PT, 1} : whole_shape(a.Hq / a.Hkv, D, a.max_seqlen);
  constexpr bool BF = IsBf16<T>::value == 1;
  extern __shared__ __align__(1024) uint8_t smem_prompt[];   // the swizzled tiles start 1024-byte aligned
  const uint32_t base = smem_u32(smem_prompt);
  const uint32_t bars = base + C::OFF_BAR;
  auto bar = [&](uint32_t kind, int i) { return bars + kind + 8 * static_cast<uint32_t>(i); };
  auto s_q = [&](int w) { return base + static_cast<uint32_t>(w) * C::TILE; };
  auto s_kv = [&](int i) { return base + C::OFF_KV + static_cast<uint32_t>(i) * C::TILE; };
  const uint32_t abort_flag = bars + PW_ABORT;
  const volatile uint32_t* tmem_ptr = reinterpret_cast<const volatile uint32_t*>(smem_prompt + C::OFF_BAR + PW_TMEM);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == P_MMA_WARP) {
    tmem_alloc(bars + PW_TMEM, P_TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(bar(PB_KV_FULL, i), 1);
      mbar_init(bar(PB_KV_EMPTY, i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(PB_Q_FULL, i), 1);
      mbar_init(bar(PB_Q_EMPTY, i), SPLIT ? P_SOFTMAX_WARPS / 2 : 1);
      mbar_init(bar(PB_JOIN, i), P_SOFTMAX_WARPS / 2);
      mbar_init(bar(PB_S_FULL, i), 1);
      mbar_init(bar(PB_P_READY, i), P_SOFTMAX_WARPS / 2);
      mbar_init(bar(PB_PV_DONE, i), 1);
      mbar_init(bar(PB_U_FULL, i), 1);
      mbar_init(bar(PB_U_EMPTY, i), P_SOFTMAX_WARPS + 2);
      mbar_init(bar(PB_TAIL, i), 1);
      mbar_init(bar(PB_S_READ, i), P_SOFTMAX_WARPS / 2);
    }
    mbar_init(bar(PB_DRAIN, 0), 1);
    st_shared_u32(abort_flag, 0u);
    fence_barrier_init();
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;
  dependent_launch();
  bool bad = false;
  // A bounded wait; every lane of the warp leaves with the same `bad`.
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (!mbar_wait_limited<LIMIT>(b, parity, abort_flag, a.wait_limit)) bad = true;
    bad = __any_sync(0xffffffffu, bad);
    return !bad;
  };
  // A wait that may last a whole unit: of the warp for the tails, and of the softmax warps of a tile
  // without rows for the next unit.
  auto wait_unit = [&](uint32_t b, uint32_t parity) {
    if (!mbar_wait_limited<LIMIT, P_UNIT_WAIT_CYCLES>(b, parity, abort_flag, a.unit_wait_limit)) bad = true;
    bad = __any_sync(0xffffffffu, bad);
    return !bad;
  };
  auto read_unit = [&](int i) {
    const uint32_t d = bars + P_DESC + 32u * static_cast<uint32_t>(i & 1);
    PromptUnit u;
    u.s0 = static_cast<int>(ld_shared_u32(d));
    u.n = static_cast<int>(ld_shared_u32(d + 4));
    u.q0 = static_cast<int>(ld_shared_u32(d + 8));
    u.h = static_cast<int>(ld_shared_u32(d + 12));
    return u;
  };

  if (warp >= P_SOFTMAX_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P_REGS_OTHER));
    if (warp == P_LOAD_WARP) {
      // ------------------------------------------------------------ loads
      UnitWalk walk{us, 0, 0, 0, lane};
      walk.start(a, blockIdx.x == 0);
      const long long G = gridDim.x, c = blockIdx.x;
      uint32_t it = 0, nq[2] = {0, 0};
      for (int i = 0; !bad; ++i) {
        // Round i of G units, walked forwards and backwards in turn.
        const PromptUnit u = walk.find(a, i * G + ((i & 1) ? G - 1 - c : c));
        if (i >= 2 && !wait(bar(PB_U_EMPTY, i & 1), ((i >> 1) - 1) & 1)) break;
        if (lane == 0) {
          const uint32_t d = bars + P_DESC + 32u * static_cast<uint32_t>(i & 1);
          st_shared_u32(d, static_cast<uint32_t>(u.s0));
          st_shared_u32(d + 4, static_cast<uint32_t>(u.n));
          st_shared_u32(d + 8, static_cast<uint32_t>(u.q0));
          st_shared_u32(d + 12, static_cast<uint32_t>(u.h));
          mbar_arrive(bar(PB_U_FULL, i & 1));
        }
        __syncwarp();
        if (u.q0 < 0) break;
        const int hk = u.h / (a.Hq / a.Hkv);
        const int nb = u.blocks(us, a.causal);
        auto load_q = [&](int w) {
          if (nq[w] > 0 && !wait(bar(PB_Q_EMPTY, w), (nq[w] - 1) & 1)) return;
          ++nq[w];
          if (lane == 0) {
            mbar_expect_tx(bar(PB_Q_FULL, w), C::TILE);
            for (int g = 0; g < D / 64; ++g)
              tma_load_3d(s_q(w) + g * P_SUB, &map_q, 64 * g, u.head(w, us), u.s0 + u.row0(w, us), bar(PB_Q_FULL, w));
          }
          __syncwarp();
        };
        auto load_kv = [&](const CUtensorMap* map, int j) {
          const int s = static_cast<int>(it % C::SLOTS);
          if (it >= C::SLOTS && !wait(bar(PB_KV_EMPTY, s), (it / C::SLOTS - 1) & 1)) return;
          ++it;
          if (lane == 0) {
            mbar_expect_tx(bar(PB_KV_FULL, s), C::TILE);
            for (int g = 0; g < D / 64; ++g)
              tma_load_3d(s_kv(s) + g * P_SUB, map, 64 * g, hk, u.s0 + j * PT, bar(PB_KV_FULL, s));
          }
          __syncwarp();
        };
        load_q(0);
        if (!bad) load_kv(&map_k, 0);
        if (!bad && u.blocks(1, us, a.causal) > 0) load_q(1);
        if (!bad) load_kv(&map_v, 0);
        for (int j = 1; j < nb && !bad; ++j) {
          load_kv(&map_k, j);
          if (!bad) load_kv(&map_v, j);
        }
      }
    } else if (warp == P_TAIL_WARP) {
      // ------------------------------------------------------------ tails
      // V rows [keys, 16 ceil(keys / 16)) of a unit's last block: zeros,
      // whatever lies behind the sequence.  The product thread hands the
      // block over once it has landed and gets it back before its P V.
      uint32_t kv0 = 0, done = 0;
      for (int i = 0;; ++i) {
        if (!wait_unit(bar(PB_U_FULL, i & 1), (i >> 1) & 1)) break;
        const PromptUnit u = read_unit(i);
        if (u.q0 < 0) break;
        const int nb = u.blocks(us, a.causal);
        const int keys = min(PT, u.n - (nb - 1) * PT), pad = -keys & 15;
        kv0 += 2 * static_cast<uint32_t>(nb);
        if (pad > 0) {
          if (!wait_unit(bar(PB_TAIL, 0), done & 1)) break;
          ++done;
          const uint32_t sv = s_kv(static_cast<int>((kv0 - 1) % C::SLOTS)) + keys * 128;
          for (int z = lane; z < pad * 8 * (D / 64); z += 32) {
            const int g = z / (pad * 8), r = z % (pad * 8);
            st_shared_v4(sv + g * P_SUB + r * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) {
          if (pad > 0) mbar_arrive(bar(PB_TAIL, 1));
          mbar_arrive(bar(PB_U_EMPTY, i & 1));
        }
      }
    } else if (warp == P_MMA_WARP) {
      // ------------------------------------------------------------ products
      // One thread does all of it: issuing from a branch inside each step cost
      // 95 to 150 cycles a product (against 64 of the tensor core).
      if (elect_one()) {
        auto wait1 = [&](uint32_t b, uint32_t parity) {
          if (!mbar_wait_limited<LIMIT>(b, parity, abort_flag, a.wait_limit)) bad = true;
          return !bad;
        };
        const uint32_t idesc_s = idesc_f16(BF ? 1u : 0u, 0, PT, PT);
        const uint32_t idesc_pv = idesc_f16(BF ? 1u : 0u, 1, PT, D);
        const uint64_t dq0 = sdesc(s_q(0), 16, 1024), dk0 = sdesc(s_kv(0), 16, 1024), dv0 = sdesc(s_kv(0), P_SUB, 1024);
        uint32_t kv0 = 0;                       // ring index of the unit's K block 0; K j at kv0 + 2j, V j one after
        // Q tiles, S products, P V products of each tile and tails so far.
        uint32_t nq_a = 0, nq_b = 0, ns_a = 0, ns_b = 0, npv_a = 0, npv_b = 0, ntail = 0;
        auto kv_slot = [&](uint32_t idx) { return static_cast<int>(idx % C::SLOTS); };
        auto kv_wait = [&](uint32_t idx) { return wait1(bar(PB_KV_FULL, kv_slot(idx)), (idx / C::SLOTS) & 1); };
        // S of tile w with the K block at ring index idx.
        auto issue_s = [&](int w, uint32_t idx, bool last) {
          tc_fence_after();
          const uint64_t dq = dq0 + static_cast<uint32_t>(w) * (C::TILE >> 4);
          const uint64_t dk = dk0 + static_cast<uint32_t>(kv_slot(idx)) * (C::TILE >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * P_SUB + (kk % 4) * 32) >> 4;
            umma_f16(tmem + C::T_S + w * PT, dq + off, dk + off, idesc_s, kk > 0 ? 1u : 0u);
          }
          umma_commit(bar(PB_S_FULL, w));
          if (last) umma_commit(bar(PB_Q_EMPTY, w));
        };
        auto release = [&](uint32_t idx) { umma_commit(bar(PB_KV_EMPTY, kv_slot(idx))); };
        // The S columns of tile w are free: P V done with the P over them, or (own P) the scores read.
        auto s_free = [&](int w) {
          const uint32_t n = C::OWN_P ? (w ? ns_b : ns_a) : (w ? npv_b : npv_a);
          return n == 0 || wait1(bar(C::OWN_P ? PB_S_READ : PB_PV_DONE, w), (n - 1) & 1);
        };
        // S of tile w of block j of a unit (block 0: its Q tile has landed).
        auto next_s = [&](int w, int j, uint32_t idx, bool last) {
          if (j == 0) {
            if (!wait1(bar(PB_Q_FULL, w), (w ? nq_b : nq_a) & 1)) return false;
            ++(w ? nq_b : nq_a);
          }
          if (!kv_wait(idx) || !s_free(w)) return false;
          ++(w ? ns_b : ns_a);
          issue_s(w, idx, last);
          return true;
        };
        // O (+)= P V of tile w for block j.
        auto next_pv = [&](int w, int j, int ksteps, uint32_t vi) {
          if (!wait1(bar(PB_P_READY, w), (w ? npv_b : npv_a) & 1)) return false;
          ++(w ? npv_b : npv_a);
          tc_fence_after();
          const uint64_t dv = dv0 + static_cast<uint32_t>(kv_slot(vi)) * (C::TILE >> 4);
          const uint32_t to = tmem + C::T_O + w * D, tp = tmem + C::T_P + w * C::P_STEP;
#pragma unroll
          for (int kk = 0; kk < PT / 16; ++kk) {
            if (kk < ksteps) umma_f16_tmem_a(to, tp + kk * 8, dv + kk * (2048 >> 4), idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(bar(PB_PV_DONE, w));
          return true;
        };
        PromptUnit u{0, 0, -1, 0};
        int started = 0;                        // tiles (bits) whose first S was issued during the previous unit
        if (wait1(bar(PB_U_FULL, 0), 0)) u = read_unit(0);
        for (int i = 0; !bad && u.q0 >= 0; ++i) {
          const int nba = u.blocks(0, us, a.causal), nbb = u.blocks(1, us, a.causal), nb = SPLIT ? u.seen(0, us, a.causal) : max(nba, nbb);
          PromptUnit next{0, 0, -2, 0};         // not read yet
          if constexpr (SPLIT) {
            // Block j for tile j & 1; S of its next block ahead of (own P) or behind its P V.  The Q tiles are
            // handed back by the join, so nothing of the next unit is issued ahead.
            auto s_of = [&](int j) {
              if (!next_s(j & 1, j >> 1, kv0 + 2 * j, false)) return false;
              release(kv0 + 2 * j);
              return true;
            };
            if (!s_of(0) || (nb > 1 && !s_of(1))) break;
            for (int j = 0; j < nb && !bad; ++j) {
              const uint32_t vi = kv0 + 2 * j + 1;
              if (!kv_wait(vi)) break;
              const int keys = min(PT, u.n - j * PT);
              if (keys & 15) {
                mbar_arrive(bar(PB_TAIL, 0));
                if (!wait1(bar(PB_TAIL, 1), ntail & 1)) break;
                ++ntail;
              }
              if (C::OWN_P && j + 2 < nb && !s_of(j + 2)) break;
              if (!next_pv(j & 1, j >> 1, (keys + 15) / 16, vi)) break;
              release(vi);
              if (!C::OWN_P && j + 2 < nb && !s_of(j + 2)) break;
            }
            if (bad || !wait1(bar(PB_U_FULL, (i + 1) & 1), ((i + 1) >> 1) & 1)) break;
            next = read_unit(i + 1);
            kv0 += 2 * static_cast<uint32_t>(nb);
            mbar_arrive(bar(PB_U_EMPTY, i & 1));
            u = next;
            continue;
          }
          if (!(started & 1) && !next_s(0, 0, kv0, nba == 1)) break;
          if (nbb > 0 && !(started & 2) && !next_s(1, 0, kv0, nbb == 1)) break;
          started = 0;
          release(kv0);
          for (int j = 0; j < nb && !bad; ++j) {
            const uint32_t vi = kv0 + 2 * j + 1, ki = vi + 1;
            if (!kv_wait(vi)) break;
            const int keys = min(PT, u.n - j * PT), ksteps = (keys + 15) / 16;
            if (keys & 15) {
              mbar_arrive(bar(PB_TAIL, 0));
              if (!wait1(bar(PB_TAIL, 1), ntail & 1)) break;
              ++ntail;
            }
            // With the next block's S ahead of this block's P V (own P), or right behind it.
            if constexpr (C::OWN_P) {
              if (j + 1 < nba && !next_s(0, j + 1, ki, j + 2 == nba)) break;
              if (j + 1 < nbb && !next_s(1, j + 1, ki, j + 2 == nbb)) break;
              if (j + 1 < nb) release(ki);
            } else {
              if (j < nba) {
                if (!next_pv(0, j, ksteps, vi)) break;
                if (j + 1 < nba && !next_s(0, j + 1, ki, j + 2 == nba)) break;
              }
            }
            if (j == nb - 1) {
              // Tile A's products are all issued (P over S) or it has ended (own P): its
              // first S of the next unit goes ahead of tile B's last P V.
              if (!wait1(bar(PB_U_FULL, (i + 1) & 1), ((i + 1) >> 1) & 1)) break;
              next = read_unit(i + 1);
              if (next.q0 >= 0 && (C::OWN_P ? nba < nbb : nbb > 0)) {
                if (!next_s(0, 0, kv0 + 2 * nb, next.blocks(0, us, a.causal) == 1)) break;
                started |= 1;
              }
            }
            if constexpr (C::OWN_P) {
              if (j < nba && !next_pv(0, j, ksteps, vi)) break;
              if (j < nbb && !next_pv(1, j, ksteps, vi)) break;
            } else {
              if (j < nbb) {
                if (!next_pv(1, j, ksteps, vi)) break;
                if (j + 1 < nbb && !next_s(1, j + 1, ki, j + 2 == nbb)) break;
              }
              if (j + 1 < nb) release(ki);
            }
            release(vi);
          }
          if (bad) break;
          kv0 += 2 * static_cast<uint32_t>(nb);
          mbar_arrive(bar(PB_U_EMPTY, i & 1));
          u = next;
        }
        if (!bad) {
          umma_commit(bar(PB_DRAIN, 0));
          wait1(bar(PB_DRAIN, 0), 0);
        }
      }
      bad = __any_sync(0xffffffffu, bad);
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P_REGS_SOFTMAX));
    const int w = warp >> 2, row = tid & (PT - 1);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::T_S + w * PT, tO = tmem + lane_off + C::T_O + w * D;
    const uint32_t tP = tmem + lane_off + C::T_P + w * C::P_STEP;
    uint32_t count = 0;                     // blocks of this tile so far
    uint32_t joins = 0;                     // units joined so far
    for (int i = 0;; ++i) {
      if (!wait_unit(bar(PB_U_FULL, i & 1), (i >> 1) & 1)) break;
      const PromptUnit u = read_unit(i);
      if (u.q0 < 0) break;
      const int nbw = u.blocks(w, us, a.causal), last = (SPLIT ? u.seen(w, us, a.causal) : nbw) - 1;
      float m_ref = -INFINITY, l_run = 0.f;
      for (int j = 0; j < nbw; ++j) {
        if (!wait(bar(PB_S_FULL, w), count & 1)) break;
        tc_fence_after();
        float s[PT], mx;
        const int jk = SPLIT ? 2 * j + w : j;           // the block of keys
        if (jk < last) {
          mx = prompt_scores<false>(tS, PT, s);
        } else {
          // The last block: the sequence's end, and the diagonal when causal.
          int lim = u.n - jk * PT;
          if (a.causal) lim = min(lim, u.row0(w, us) + row - jk * PT + 1);
          mx = prompt_scores<true>(tS, lim, s);
        }
        if constexpr (C::OWN_P) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(PB_S_READ, w));
          // P and O are free once the P V product before this one is done.
          if (count > 0 && !wait(bar(PB_PV_DONE, w), (count - 1) & 1)) break;
          tc_fence_after();
        }
        ++count;
        const float x = mx * a.scale_log2;
        const bool move = x > m_ref + P_MOVE;
        if (__any_sync(0xffffffffu, move)) {
          const float alpha = move ? fast_exp2(m_ref - x) : 1.f;
          if (move) m_ref = x;
          l_run *= alpha;
          if (j > 0) prompt_rescale<D>(tO, alpha);
        }
        l_run += prompt_weights<BF>(tP, s, a.scale_log2, m_ref);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PB_P_READY, w));
      }
      if (bad) break;
      if (SPLIT && last > 0) {
        // Both tiles hold the row: each hands the other the half of O's columns that it writes out (fp32, over the Q
        // tile that its own products have read), and reference and sum.
        if (!wait(bar(PB_PV_DONE, w), (count - 1) & 1)) break;
        tc_fence_after();
        constexpr int H = D / 2, CH = H / 8;               // columns of a tile; 16-byte chunks of a row's outputs
        auto at = [&](int tile, int c) { return s_q(tile) + row * (H * 4) + ((c ^ (row & 7)) << 4); };
        const uint32_t ml = bars + 512u + static_cast<uint32_t>(row) * 8u;
#pragma unroll
        for (int g = 0; g < H / 32; ++g) {
          float o[32];
          tmem_ld32(tO + (w ^ 1) * H + 32 * g, o);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_shared_v4(at(w, 8 * g + k), __float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]),
                         __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
        }
        st_shared_u32(ml + w * (PT * 8), __float_as_uint(m_ref));
        st_shared_u32(ml + w * (PT * 8) + 4, __float_as_uint(l_run));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PB_JOIN, w));
        if (!wait(bar(PB_JOIN, w ^ 1), joins & 1)) break;
        ++joins;
        const float m_o = __uint_as_float(ld_shared_u32(ml + (w ^ 1) * (PT * 8)));
        const float l_o = __uint_as_float(ld_shared_u32(ml + (w ^ 1) * (PT * 8) + 4));
        const float m = fmaxf(m_ref, m_o), mu = m == -INFINITY ? 0.f : m;
        const float f = fast_exp2(m_ref - mu), f_o = fast_exp2(m_o - mu), l = l_run * f + l_o * f_o;
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l), x = f * inv, x_o = f_o * inv;
        const uint32_t stg = base + C::OFF_OUT + static_cast<uint32_t>(warp) * 4096u;
        auto out_at = [&](int r, int c) { return stg + r * (H * 2) + ((c ^ ((CH == 8 ? r : r >> 1) & (CH - 1))) << 4); };
#pragma unroll
        for (int g = 0; g < H / 32; ++g) {
          float o[32];
          tmem_ld32(tO + w * H + 32 * g, o);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint4 v = ld_shared_v4(at(w ^ 1, 8 * g + k));
            o[4 * k] = o[4 * k] * x + __uint_as_float(v.x) * x_o;
            o[4 * k + 1] = o[4 * k + 1] * x + __uint_as_float(v.y) * x_o;
            o[4 * k + 2] = o[4 * k + 2] * x + __uint_as_float(v.z) * x_o;
            o[4 * k + 3] = o[4 * k + 3] * x + __uint_as_float(v.w) * x_o;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = pack2<Tout2<T>>(o[8 * k + 2 * e], o[8 * k + 2 * e + 1]);
            st_shared_v4(out_at(lane, 4 * g + k), p[0], p[1], p[2], p[3]);
          }
        }
        fence_proxy_async();                               // the next Q tile comes by TMA
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PB_Q_EMPTY, w ^ 1));
        const int r0 = u.q0 + (warp & 3) * 32;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int rr = (32 / CH) * k + lane / CH, cc = lane % CH;
          const uint4 v = ld_shared_v4(out_at(rr, cc));
          if (r0 + rr < u.n)
            *reinterpret_cast<uint4*>(static_cast<T*>(a.o) +
                                      (static_cast<long long>(u.s0 + r0 + rr) * a.Hq + u.h) * D + w * H + 8 * cc) = v;
        }
        __syncwarp();
        tc_fence_before();
      } else if (nbw > 0) {
        if (!wait(bar(PB_PV_DONE, w), (count - 1) & 1)) break;
        tc_fence_after();
        if (SPLIT && lane == 0) mbar_arrive(bar(PB_Q_EMPTY, 0));   // a unit of one block: tile A's alone
        const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);
        // 64 columns at a time through the warp's 4 KB of staging (rows of
        // 128 bytes, 16-byte chunks swizzled): whole row pieces leave, four to an
        // instruction.  Stored straight from the registers, a row a lane, the
        // epilogue held the tile for 4000 cycles.
        const uint32_t stg = base + C::OFF_OUT + static_cast<uint32_t>(warp) * 4096u;
        const int r0 = u.row0(w, us) + (warp & 3) * 32;
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
          float o[64];
          tmem_ld32_nowait(tO + 64 * g, o);
          tmem_ld32_nowait(tO + 64 * g + 32, o + 32);
          tmem_wait_ld32(o);
          tmem_wait_ld32(o + 32);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = pack2<Tout2<T>>(o[8 * k + 2 * e] * inv, o[8 * k + 2 * e + 1] * inv);
            st_shared_v4(stg + lane * 128 + ((k ^ (lane & 7)) << 4), p[0], p[1], p[2], p[3]);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rr = 4 * k + (lane >> 3), cc = lane & 7;
            const uint4 v = ld_shared_v4(stg + rr * 128 + ((cc ^ (rr & 7)) << 4));
            if (r0 + rr < u.n)
              *reinterpret_cast<uint4*>(static_cast<T*>(a.o) +
                                        (static_cast<long long>(u.s0 + r0 + rr) * a.Hq + u.head(w, us)) * D + 64 * g + 8 * cc) = v;
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(PB_U_EMPTY, i & 1));
    }
  }
  if (bad && lane == 0) {
    st_shared_u32(abort_flag, 1u);
    record_error(a.err, RRA_DEVERR_WAIT_TIMEOUT);
  }

  // Teardown: after an abort, copies and products still in flight get a
  // bounded grace period (~1 ms) to land before the TMEM is released.
  tc_fence_before();
  __syncthreads();
  if (warp == P_MMA_WARP) {
    if (lane == 0 && ld_shared_volatile_u32(abort_flag) != 0u) {
      const long long t0 = clock64();
      while (clock64() - t0 < 2000000LL) {
      }
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, P_TMEM_COLS);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 prompt_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 3-D map over a [rows, H, d] tensor with rows `stride` elements apart: box =
// 128 rows of 64 elements of one head, 128-byte swizzle.
cudaError_t make_map_rows(CUtensorMap* map, const void* ptr, int rows, int H, int d, long long stride, bool bf16) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {64, 1, PT};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = prompt_encode_fn()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                                  const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int D, bool SPLIT, bool LIMIT>
cudaError_t launch_shape(const PromptArgs& a, const UnitShape& us, int num_sms, cudaStream_t stream) {
  using C = PromptCfg<D>;
  auto kernel = attend_prompt_kernel<T, D, SPLIT, LIMIT>;
  constexpr int kMaxDevices = 64;
  static bool attr_set[kMaxDevices] = {};
  static std::mutex m;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(m);
    if (!attr_set[dev]) {
      if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess)
        return e;
      attr_set[dev] = true;
    }
  }
  const bool bf16 = IsBf16<T>::value == 1;
  CUtensorMap mq, mk, mv;
  if ((e = make_map_rows(&mq, a.q, a.cap, a.Hq, D, a.q_stride, bf16)) != cudaSuccess) return e;
  if ((e = make_map_rows(&mk, a.k, a.cap, a.Hkv, D, a.k_stride, bf16)) != cudaSuccess) return e;
  if ((e = make_map_rows(&mv, a.v, a.cap, a.Hkv, D, a.v_stride, bf16)) != cudaSuccess) return e;
  const long long units = static_cast<long long>(a.B) * (a.Hq / us.heads) * ((a.max_seqlen - 1) / us.rows + 1);
  const int grid = static_cast<int>(units < num_sms ? units : num_sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(P_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, a);
}

template <typename T, int D, bool LIMIT>
cudaError_t launch_lim(const PromptArgs& a, int num_sms, cudaStream_t stream) {
  const UnitShape us = prompt_shape(a, D, num_sms);
  return us.split ? launch_shape<T, D, true, LIMIT>(a, us, num_sms, stream)
                  : launch_shape<T, D, false, LIMIT>(a, us, num_sms, stream);
}

template <typename T, int D>
cudaError_t launch_d(PromptArgs a, int num_sms, cudaStream_t stream) {
  const long long each = std::min(a.wait_limit > 0 ? a.wait_limit : WAIT_LIMIT_CYCLES, 1LL << 38);
  a.unit_wait_limit = each * (1 + std::min(a.max_seqlen, a.cap) / PT);          // at most 2^38 x 2^23
  return a.wait_limit > 0 ? launch_lim<T, D, true>(a, num_sms, stream) : launch_lim<T, D, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_attend_prompt(const PromptArgs& a, int d, rra_dtype dt, int num_sms, cudaStream_t stream) {
  if (prompt_encode_fn() == nullptr) return cudaErrorNotSupported;
  if (dt == RRA_BF16)
    return d == 64 ? launch_d<__nv_bfloat16, 64>(a, num_sms, stream) : launch_d<__nv_bfloat16, 128>(a, num_sms, stream);
  return d == 64 ? launch_d<__half, 64>(a, num_sms, stream) : launch_d<__half, 128>(a, num_sms, stream);
}

}  // namespace rra
