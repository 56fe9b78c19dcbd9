// chunk_attn.cu -- attention of several query tokens per row over the cache, on
// the 5th-generation tensor cores.
//
// Mathematics.  The G query heads of a kv-head see the same keys, so the rows
// of a product are (token, head) pairs, TQ = 128 / G tokens by G heads: a query
// tile of 128 rows.  Over key tiles of 128 tokens, with running row maximum m,
// sum l and output O (online softmax):
//   S = Q K^T;  m' = max(m, max S);  P = 2^(c (S - m'));   c = scale log2 e
//   l = l 2^(c (m - m')) + sum P;  O = O 2^(c (m - m')) + P V.
// m only moves when a row's maximum rose by more than a factor 2^8 in weight
// (P then stays below 2^8 and l and O far inside fp32), so O is rescaled a few
// times per row and not once per tile; the quotient O / l does not depend on m.
// l sums the weights in fp32; the product with V takes them rounded to bf16, each
// off by 2^-8 of itself at most, up or down, so that outputs are off by 0.0020 to
// 0.0024 (2-norm) where the rounding of outputs alone gives 0.0016.  Two bf16
// pieces a weight, as the decode attention has them, would make three products of
// two: half as much again where products bound the call.
//
// Layout.  One CTA per SM holds two streams, each with its S and O in tensor
// memory (2 x (128 + D) of 512 columns; P overwrites the first half of S, or has
// columns of its own as kOne at D = 64) and four softmax warps of one row per
// thread: no shuffles.  While one stream's softmax runs, the tensor cores work
// for the other.
//   kPair  the streams are two query tiles over the same key tiles.
//   kOne   one query tile over the even and the odd key tiles, joined at the end.
//   kFew   as kOne with 32 query rows, four times in the tile: warp w of a stream
//          weighs only the keys [32 w, 32 w + 32) of a key tile (the other
//          weights of its copy are 0), so the four copies' outputs add up to the
//          rows' and the softmax of a tile takes a fourth of the time.  With few
//          rows the call is bound by reading K and V, and only then.  A weight of
//          0 times an infinity is NaN, in the three copies that should not weigh
//          it: where an output is NaN, V is looked through (settle).
// Two warps load keys and values (TMA; a page's rows of one kv-head are one
// box), one issues the products, one hands out the work.
//
// Work.  Items are (row, kv-head, tokens of a CTA), longest first within a row;
// the CTAs stay and take the next item when they are done, so that an item's
// loads and first product run under the epilogue of the one before.  Where the
// items do not fill the SMs evenly, their keys are split into parts of `part`
// tiles; the last CTA to finish a split item joins the parts in their order, so
// results do not depend on timing.
//
// Long axes.  The tensor cores add to O by cutting bits off: a tile takes up to
// 5.1e-7 of O away, always towards zero (values of mean 1 over 2^20 keys came out
// 0.4% low, over 2^24 6%).  So a CTA takes the tiles of an item or part in
// segments of kSegment (2.6e-4), O begins anew in each, and the segments are
// added up in fp32 with rounding, in a place of the CTA's in the workspace (2368
// queries over 131072 keys, 32 heads on 8 of 128: 4.28 -> 4.30 ms).  No wait for
// an item is then longer than a segment, about a millisecond.
#include "ksa_device.cuh"
#include "ksa_internal.h"
#include "tcgen05_device.cuh"

namespace ksa {

namespace {

constexpr int kQ = 128;        // query rows of a tile
constexpr int kKeys = 128;     // key tokens of a tile
// Keys of a tile whose weights are handed over before the others', so that their products run
// under the last exponentials (16384 keys, 2368 queries, 32 heads of 128: 96 took 531 us, 64 took
// 536).
constexpr int kEarly = 96;
constexpr int kSoftWarps = 8;  // four per stream
constexpr int kMmaWarp = 8, kKeyWarp = 9, kWorkWarp = 10, kValueWarp = 11;
// A thread is launched with 65536 / 384 registers, 168.  The softmax keeps a row of 128 scores
// in registers, so the third warpgroup passes its share on: 2 x 224 + 56 = 3 x 168.
constexpr int kThreads = 384;
constexpr int kSoftRegs = 224, kOtherRegs = 56;
constexpr int kBadRing = 32;   // key tiles whose page marks are kept (above any stage count)
constexpr int kWork = 2;       // items a CTA holds: the one it computes, and the next one
constexpr int kSegment = 512;  // key tiles that O is summed over in tensor memory, at most
constexpr int kPartsPerSm = 3;  // parts of split items, at most, per SM: the workspace's size
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kLead = 4, kLag = 10;  // stagger of the weights' loop, in pairs of keys
constexpr float kRescale = 8.f;      // log2 of the largest weight before m moves
constexpr int kCtlBytes = 3 * 1024;

enum Mode { kPair, kOne, kFew };

template <int D, Mode MODE>
struct Cfg {
  static constexpr bool kPairs = MODE == kPair, kFews = MODE == kFew;
  // At D = 64 tensor memory has room for weights beside the scores, so that a stream's next scores
  // are made while it weighs these.  6000 keys, 32 heads on 8, 2368 queries: 171 -> 163 us, 4800:
  // 346 -> 336; pairs (39 -> 40 over 1024 keys) and few rows (31.2 -> 31.6 us, 32 sequences of one
  // token) lose by it.
  static constexpr bool kApart = D == 64 && MODE == kOne;
  static constexpr int kWeights = kApart ? 2 * kKeys + 2 * D : 0;  // column of the weights,
  static constexpr int kPitch = kApart ? kKeys / 2 : kKeys;        // and of stream 1's behind it
  static constexpr int kQBytes = kQ * D * 2, kTileBytes = kKeys * D * 2;  // of Q, of K or V
  static constexpr int kQTiles = kPairs ? 2 : 1;
  static constexpr int kSumBytes = kFews ? 2 * D * 32 * 4 : 0;  // of the copies' sum, [2][D][32]
  // places of the rings: as many tiles as fit, the odd one for values (a tile's keys are done
  // with one product, its values wait for the softmax)
  static constexpr int kFit = (224 * 1024 - kQTiles * kQBytes - kSumBytes) / kTileBytes;
  static constexpr int kKeyPlaces = kFit / 2, kValuePlaces = kFit - kKeyPlaces;
  static constexpr int kRows = kFews ? 32 : kQ * kQTiles;  // query rows of a CTA
  static constexpr int kSmem = kQTiles * kQBytes + kFit * kTileBytes + kSumBytes + kCtlBytes;
};

struct Work {
  int b, g, token;   // row; kv-head; first token on the axis (-1: no more work)
  int tokens;        // query tokens of the item
  int seen;          // keys its first token sees (each further token one more when causal)
  int len;           // L of the row
  int t0, nt;        // key tiles of this part
  int parts, slot, z;  // parts of the item, the first part's place in the workspace, this part
                       // (and as multiples of kSegments the segments of it before this one, with
                       // kMore if others are behind it)
};

constexpr int kSegments = 1 << 12, kMore = 1 << 29;  // see Work::z

struct Ctl {  // in shared memory
  uint64_t q_full, q_empty, k_full[8], k_empty[8], v_full[8], v_empty[8];
  // per stream: scores ready, scores read, first kEarly weights and all of them ready, product with
  // V done
  uint64_t s_full[2], s_free[2], p_early[2], p_full[2], o_done[2];
  uint64_t work_full[kWork], work_empty[kWork], soft, drain;
  Work work[kWork];
  uint32_t tmem;
  int abort, alive;  // a wait gave up; when a warp that may work for longer than a wait last did
  int last;
  uint32_t bad[kBadRing];
  float2 ml[2][kQ];  // m and l of the streams' rows, for their join
};

struct Params {
  ChunkArgs a;
  uint32_t *next, *done;  // items handed out beyond the first of each CTA; CTAs that draw no more
  uint32_t *sem;          // [max_parts] parts finished, at the item's first part
  float *part;            // [max_parts] (m, l) of the rows, then O as [D / 4][rows][4]
  float *carry;           // [CTAs] (m, l) of the softmax threads, then O, of the segments so far
  int tq, max_parts;      // tq: query tokens of a tile
  int group;              // query heads of a kv-head
  bool wide_out;          // out is 32-byte aligned
};

// Time in units of 2^20 ns, as the word behind the abort mark holds it (Ctl::alive).
__device__ __forceinline__ uint32_t milliseconds() {
  return static_cast<uint32_t>(global_timer_ns() >> 20);
}

// Waits with a limit, which a warp at work puts off by Ctl::alive; false (and the CTA's abort mark)
// when it runs out.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, int *abort) {
  if (mbar_try_wait(bar, parity)) return true;
  volatile int *const word = abort;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (word[0] != 0) return false;
    if (global_timer_ns() - t0 > kWaitTimeoutNs &&
        milliseconds() - static_cast<uint32_t>(word[1]) > (kWaitTimeoutNs >> 20)) {
      word[0] = 1;
      return false;
    }
  }
  return true;
}

// The same for a whole warp: its lanes leave together, for a lane that goes on alone would wait for
// the others at the next vote.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *abort) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort));
}

// Largest of three, NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void exp2_in_place(uint32_t &x) {  // kept in program order
  asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+r"(x));
}

// 32 bytes to a 32-byte aligned address.
__device__ __forceinline__ void store_32(void *dst, const uint32_t *x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }  // a <= 2^30

// ---------------------------------------------------------------------------
// the work warp: rows -> items -> parts

struct Rows {  // 32 rows, one per lane
  int b, s0, n, L;   // row; first token, tokens, cached tokens
  int tiles, deep;   // CTAs' token groups; key tiles of the deepest one
};

__device__ __forceinline__ Rows load_rows(const ChunkArgs &a, int base, int TT, uint32_t *status) {
  Rows r{};
  const int b = base + static_cast<int>(threadIdx.x & 31);
  if (b < a.B) {
    const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], L = a.seq_lens[b];
    r.s0 = min(max(c0, 0), a.N);
    r.n = max(0, min(c1, a.N) - r.s0);
    r.L = min(max(L, 0), a.T);
    if (c0 != r.s0 || c1 < c0 || c1 > a.N || (r.n > 0 && L != r.L))
      flag_status(status, KSA_FLAG_SEQ_LEN_CLAMPED);
    r.tiles = ceil_div(r.n, TT);
    r.deep = r.n > 0 ? ceil_div(r.L, kKeys) : 0;
  }
  r.b = b;
  return r;
}

// The lanes' rows in order of depth, deepest first, so that what is handed out last is short.
__device__ __forceinline__ Rows sort_rows(const Rows &r) {
  const int lane = threadIdx.x & 31;
  const int after = __shfl_down_sync(0xffffffffu, r.deep, 1);
  if (__all_sync(0xffffffffu, lane == 31 || r.deep >= after)) return r;
  // bitonic; depths (below 2^24) with the lane behind them, so that the order is one
  int key = r.deep * 32 + 31 - lane;
#pragma unroll
  for (int k = 2; k <= 32; k *= 2)
#pragma unroll
    for (int d = k / 2; d > 0; d /= 2) {
      const int other = __shfl_xor_sync(0xffffffffu, key, d);
      key = ((lane & d) == 0) == ((lane & k) == 0) ? max(key, other) : min(key, other);
    }
  const int src = 31 - (key & 31);
  return {__shfl_sync(0xffffffffu, r.b, src),     __shfl_sync(0xffffffffu, r.s0, src),
          __shfl_sync(0xffffffffu, r.n, src),     __shfl_sync(0xffffffffu, r.L, src),
          __shfl_sync(0xffffffffu, r.tiles, src), __shfl_sync(0xffffffffu, r.deep, src)};
}

// In key tiles: what a part costs besides its tiles (its start and end), what it costs more if it
// is joined, and the last join: its start, and each of an item's parts (of full tiles).  A tile
// takes 1.8 us in pairs, half of that otherwise.
struct Costs {
  float start, part, join, each;
};
template <Mode MODE>
__device__ __forceinline__ constexpr Costs costs() {
  return MODE == kPair ? Costs{2.5f, 1.5f, 8.f, 0.8f}
         : MODE == kOne ? Costs{5.f, 3.f, 7.5f, 0.8f}
                        : Costs{2.5f, 1.5f, 4.5f, 0.15f};
}

// What is cut: items before `whole` are not, the others into parts of `part` key tiles.
struct Cut {
  int whole, part;
};

// Lane i < 16 tries all items with the deepest cut into i + 1 parts (lane 15: as many as fill the
// SMs), lane i >= 16 whole items but for the last round that does not fill the SMs, cut into
// i - 14 parts; every CTA gets the same answer.  Estimated ends, in key tiles of the form (see
// Costs).  Parts of mostly one size go round by round (6 rows of 29 to 60 thousand keys, 42 items:
// 146, 172, 272 and 330 parts took 120, 191, 137 and 170 us), others fill the SMs evenly but for a
// third of a part.
__device__ __forceinline__ Cut choose_cut(const ChunkArgs &a, const Rows &first, int TT, int ctas,
                                          int max_parts, Costs k) {
  const int lane = threadIdx.x & 31;
  float tiles = 0.f, items = 0.f, tokens = 0.f;
  int deepest = 0;
  Rows r = first;
  for (int base = 0; base < a.B; base += 32) {
    if (base > 0) r = load_rows(a, base, TT, nullptr);
    const float n = static_cast<float>(r.tiles) * a.Hkv;
    // mean depth of the row's groups: from the first group's last token to the last one's
    const int top = a.causal ? ceil_div(max(0, r.L - r.n + min(r.n, TT)), kKeys) : r.deep;
    items += n;
    tokens += n * min(r.n, TT);
    tiles += n * 0.5f * (top + r.deep);
    deepest = max(deepest, r.deep);
  }
  deepest = __reduce_max_sync(0xffffffffu, deepest);
  if (deepest < 4) return {0, max(deepest, 1)};
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    tiles += __shfl_xor_sync(0xffffffffu, tiles, off);
    items += __shfl_xor_sync(0xffffffffu, items, off);
    tokens += __shfl_xor_sync(0xffffffffu, tokens, off);
  }
  if (items > 1e6f) return {0, deepest};
  const int n = static_cast<int>(items), rem = n % ctas;
  const float mean = __fdividef(tiles, items), per_cta = 1.f / ctas;
  const bool equal = mean >= 0.85f * deepest;
  auto ends = [&](float parts, float extra, float even, float size) {
    const float one = __fdividef(tiles, parts), rounds = ceilf(parts * per_cta);
    return equal                ? rounds * (one + extra)
           : one >= 0.7f * size ? (rounds - 1.f) * (one + extra) + size + extra
                                : fmaxf(even + 0.35f * size, size + extra);
  };
  const float each = k.each * __fdividef(tokens, items * static_cast<float>(TT));
  {  // no cut can win (a look at 32 rows takes 1.3 us): c parts of the deepest item end at
     // deepest / c + each c behind their least cost, and that is 2 sqrt(deepest each) or more
    const float even = (tiles + k.start * items) * per_cta, x = deepest * each;
    const float least = k.join + fmaxf(even + 2.f * each, k.start + k.part + 2.f * x * rsqrtf(x));
    if (0.95f * ends(items, k.start, even, deepest) <= least) return {0, deepest};
  }
  const int cuts = lane < 15 ? lane + 1 : lane == 15 ? max(1, ctas / n) : lane - 14;
  const int s = max(2, ceil_div(deepest, cuts));
  float parts = 0.f, joined = 0.f;  // of cutting all items
  if (a.B <= 32) {
    const float own = static_cast<float>(first.tiles) * a.Hkv, per = __fdividef(1.f, s);
    const int deep = first.deep;
#pragma unroll 8
    for (int b = 0; b < a.B; ++b) {
      const float m = __shfl_sync(0xffffffffu, own, b);
      const float c = ceilf(__shfl_sync(0xffffffffu, deep, b) * per);
      parts += m * fmaxf(c, 1.f);
      if (c > 1.f) joined += m * c;
    }
  } else {  // all rows as deep as the mean
    const float c = fmaxf(1.f, ceilf(__fdividef(mean, s)));
    parts = items * c;
    joined = s < deepest ? parts : 0.f;
  }
  const float last = k.join + each * ceil_div(deepest, s);
  float cost;
  if (lane < 16) {
    const float even = (tiles + k.start * parts + k.part * joined) * per_cta;
    cost = ends(parts, k.start + (joined > 0.f ? k.part : 0.f), even, min(s, deepest));
    if (joined > 0.f) cost += last;
  } else {
    joined = static_cast<float>(rem) * cuts;
    cost = equal && rem > 0 && n > ctas
               ? (n / ctas) * (mean + k.start) +
                     ceilf(joined * per_cta) * (__fdividef(mean, cuts) + k.start + k.part) + last
               : INFINITY;
  }
  if (joined > max_parts) cost = INFINITY;
  if (lane == 0) cost *= 0.95f;
  float best = cost;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    best = fminf(best, __shfl_xor_sync(0xffffffffu, best, off));
  const int who = __ffs(__ballot_sync(0xffffffffu, cost == best)) - 1;
  return {who < 16 ? 0 : n - rem, __shfl_sync(0xffffffffu, s, who)};
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ int warp_scan(int x) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (static_cast<int>(threadIdx.x & 31) >= off) x += y;
  }
  return x;
}

__device__ __forceinline__ void hand_out_work(const Params &p, Ctl &ctl, int TT, Rows r,
                                              Costs k) {
  const ChunkArgs &a = p.a;
  const int lane = threadIdx.x & 31;
  const int ctas = static_cast<int>(gridDim.x);
  uint32_t *status = blockIdx.x == 0 ? a.status : nullptr;
  for (int base = 32; status != nullptr && base < a.B; base += 32) load_rows(a, base, TT, status);
  Cut cut = choose_cut(a, r, TT, ctas, p.max_parts, k);
  if (cut.whole == 0) {  // the choice was an estimate: the workspace must hold the real parts
    float joined = 0.f;
    Rows q = r;
    for (int b = 0; b < a.B; b += 32) {
      if (b > 0) q = load_rows(a, b, TT, nullptr);
      if (q.deep > cut.part)
        joined += static_cast<float>(q.tiles) * a.Hkv * ceil_div(q.deep, cut.part);
    }
    if (__any_sync(0xffffffffu, joined > 0.f)) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) joined += __shfl_xor_sync(0xffffffffu, joined, off);
      // (of whole items before a cut tail only the tail counts: at most `rem` items, see above)
      if (joined > p.max_parts) cut = {0, a.T};
    }
  }
  // the current 32 rows: parts [first, first + sum of units), whole items, places of parts to join
  int base = 0, first = 0, first_item = 0, first_slot = 0;
  int cuts, whole, units, slots, units_end, slots_end;
  auto measure = [&]() {
    r = sort_rows(r);
    const int items = r.tiles * a.Hkv, end = warp_scan(items);
    cuts = 1;
    whole = units = items;
    units_end = end;
    slots = slots_end = 0;
    if (__any_sync(0xffffffffu, r.deep > cut.part)) {
      cuts = max(1, ceil_div(r.deep, cut.part));
      whole = cuts == 1 ? items : min(max(cut.whole - (first_item + end - items), 0), items);
      units = whole + (items - whole) * cuts;
      slots = units - whole;
      units_end = warp_scan(units);
      slots_end = warp_scan(slots);
    }
    first_item += __shfl_sync(0xffffffffu, end, 31);
  };
  measure();
  int id = static_cast<int>(blockIdx.x), at = 0;
  uint32_t turn = 1;
  while (true) {
    int sum = __shfl_sync(0xffffffffu, units_end, 31);
    // (rows that overlap by a bad cu_q could count past 2^31: no more work from 2^30 on)
    while (id >= first + sum && base + 32 < a.B && first < (1 << 30)) {
      first += sum;
      first_slot += __shfl_sync(0xffffffffu, slots_end, 31);
      base += 32;
      r = load_rows(a, base, TT, nullptr);
      measure();
      sum = __shfl_sync(0xffffffffu, units_end, 31);
    }
    const bool end = id >= first + sum;
    Work w{};
    w.token = -1;
    bool use = true;
    if (!end) {
      const int local = id - first;
      const int who = __ffs(__ballot_sync(0xffffffffu, local < units_end)) - 1;
      const int c = __shfl_sync(0xffffffffu, cuts, who),
                tiles = __shfl_sync(0xffffffffu, r.tiles, who),
                n = __shfl_sync(0xffffffffu, r.n, who), L = __shfl_sync(0xffffffffu, r.L, who);
      const int in_row = local - __shfl_sync(0xffffffffu, units_end - units, who);
      const int slot0 = first_slot + __shfl_sync(0xffffffffu, slots_end - slots, who);
      const int uncut = __shfl_sync(0xffffffffu, whole, who);
      const bool is_cut = in_row >= uncut;
      const int item = is_cut ? uncut + (in_row - uncut) / c : in_row;
      const int group = item < a.Hkv ? 0 : item / a.Hkv;
      const int tile = tiles - 1 - group;  // when causal, the deepest first
      w.z = is_cut ? (in_row - uncut) % c : 0;
      w.g = item - group * a.Hkv;
      w.b = __shfl_sync(0xffffffffu, r.b, who);
      w.token = __shfl_sync(0xffffffffu, r.s0, who) + tile * TT;
      w.tokens = min(TT, n - tile * TT);
      w.seen = a.causal ? L - n + tile * TT + 1 : L;
      w.len = L;
      const int kend = a.causal ? max(0, w.seen + w.tokens - 1) : L;
      const int all = ceil_div(kend, kKeys), s = is_cut ? cut.part : max(all, 1);
      w.t0 = w.z * s;
      w.nt = min(s, all - w.t0);
      w.parts = is_cut ? max(1, ceil_div(all, s)) : 1;
      w.slot = is_cut ? slot0 + (item - uncut) * c : 0;
      use = w.z < w.parts;
    }
    const int all = w.nt, z = w.z;
    for (int done = 0; use; done += kSegment) {
      w.nt = min(all - done, kSegment);
      w.z = z + done / kSegment * kSegments + (all - done > kSegment ? kMore : 0);
      if (!warp_wait(&ctl.work_empty[at], turn, &ctl.abort)) return;
      if (lane == 0) {
        ctl.work[at] = w;
        mbar_arrive(&ctl.work_full[at]);
      }
      __syncwarp();
      if (++at == kWork) {
        at = 0;
        turn ^= 1u;
      }
      w.t0 += kSegment;
      use = all - done > kSegment;
    }
    if (end) break;
    // the next item, drawn behind this one's handing out: the first one does not wait for it
    uint32_t drawn = 0u;
    if (lane == 0) drawn = atomicAdd(p.next, 1u);
    id = ctas + static_cast<int>(__shfl_sync(0xffffffffu, drawn, 0));
  }
  // no CTA draws any more: the counters go back for the next call
  if (lane == 0 && atomicAdd(p.done, 1u) == gridDim.x - 1u) {
    *p.next = 0u;
    *p.done = 0u;
  }
}

// The next item, for a warp: waits until it is there; false after an aborted wait.
struct Take {
  int at = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ bool get(Ctl &ctl, Work &w) {
    if (!warp_wait(&ctl.work_full[at], turn, &ctl.abort)) return false;
    w = ctl.work[at];
    return true;
  }
  __device__ __forceinline__ void release(Ctl &ctl) {  // the warp reads the item no more
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl.work_empty[at]);
    if (++at == kWork) {
      at = 0;
      turn ^= 1u;
    }
  }
};

// Floats of a CTA's sums over segments: (m, l) of each softmax thread, then the O that it has.
__host__ __device__ constexpr size_t carry_floats(int rows, int D) {
  return 2 * kSoftWarps * 32 + static_cast<size_t>(rows) * D;
}

// Outputs of few rows that are not finite.  V is looked through: where a row's keys [first, end)
// hold infinities of one sign in a dim, and no NaN, that is the sum (finite keys add nothing to
// it); a row that sees nothing gets 0; all else stays as it is.  By a whole warp, whose rows share
// b and g and end within a tile's tokens of each other; `mine`: the lane has a row, with no NaN
// score.  Its outputs, `dims` from `dim` on: bf16 at `out` or, of a part, quads of fp32 `pitch`
// apart.
template <int D>
__device__ __noinline__ void settle(const ChunkArgs &a, Ctl &ctl, const Work &w, int first, int end,
                                    int dim, int dims, bool mine, uint16_t *out, float4 *part,
                                    int pitch) {
  uint32_t nan = 0u, pos = 0u, neg = 0u;  // a bit for each dim
  const int lane = threadIdx.x & 31;
  const auto look = [&](int t) {
    const long long at = kv_row(a.kv, w.b, w.g, a.Hkv, a.T, t);
    if (at < 0) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(a.V + at * D + dim);
    for (int i = 0; i < dims / 8; ++i) {
      const uint4 x = src[i];
      const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t h = y[e / 2] >> (16 * (e % 2)) & 0xffffu, bit = 1u << (8 * i + e);
        if ((h & 0x7f80u) != 0x7f80u) continue;
        if ((h & 0x7fu) != 0u)
          nan |= bit;
        else if (h >> 15)
          neg |= bit;
        else
          pos |= bit;
      }
    }
  };
  // the keys that all rows see (but those that see none) by all lanes, the others by the lanes
  // whose rows see them
  const int all = __reduce_min_sync(0xffffffffu, end > first ? end : INT32_MAX);
  if (all != INT32_MAX) {
    for (int t = first + lane, n = 1; t < all; t += 32, ++n) {
      look(t);
      if ((n & 4095) == 0)
        *const_cast<volatile int *>(&ctl.alive) = static_cast<int>(milliseconds());
    }
    nan = __reduce_or_sync(0xffffffffu, nan);
    pos = __reduce_or_sync(0xffffffffu, pos);
    neg = __reduce_or_sync(0xffffffffu, neg);
    for (int t = all; t < end; ++t) look(t);
  }
  if (!mine) return;
  const bool nothing = end <= first;
  for (int e = 0; e < dims; ++e) {
    const bool p = pos >> e & 1u, n = neg >> e & 1u;
    if (!nothing && (p == n || (nan >> e & 1u))) continue;
    const float x = nothing ? 0.f : p ? INFINITY : -INFINITY;
    if (out != nullptr)
      out[e] = static_cast<uint16_t>(__float_as_uint(x) >> 16);
    else
      reinterpret_cast<float *>(part + e / 4 * pitch)[e % 4] = x;
  }
}

// A segment that is not a part's only one, by a softmax warp: the segments before and O of the
// streams (the warp's own and, but for pairs, the other one; weights f0 and f1, below 0: none)
// go together.  If more segments follow, the sum goes to the workspace, else over the warp's own
// O.  Returns its (m, l).
template <int D, Mode MODE>
__device__ __forceinline__ float2 add_segment(const Params &p, const Ctl &ctl, const Work &w,
                                              float f0, float f1, float2 ml) {
  constexpr int DIMS = MODE == kPair ? D : D / 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s = warp >> 2;
  const float c = p.a.scale * kLog2e;
  const uint32_t at = ctl.tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 2 * kKeys +
                      (MODE == kPair ? 0 : s * DIMS);
  const uint32_t own = at + s * D, other = at + (s ^ 1) * D;
  float *carry = p.carry + blockIdx.x * carry_floats(kSoftWarps * 32 * DIMS / D, D);
  float2 *stats = reinterpret_cast<float2 *>(carry) + threadIdx.x;
  float4 *sums = reinterpret_cast<float4 *>(carry + 2 * kSoftWarps * 32) +
                 warp * (DIMS / 4 * 32) + lane;  // [warps][DIMS / 4][32]
  const bool take0 = !(f0 < 0.f), take1 = !(f1 < 0.f);
  bool take = false;  // the segments before
  float f = 0.f;
  if ((w.z & (kMore - 1)) >= kSegments) {
    const float2 y = *stats;
    const float up = fmaxf(ml.x, y.x);
    take = y.x != -INFINITY;
    const float g = ml.x == -INFINITY ? 1.f : fast_exp2((ml.x - up) * c);
    f = take ? fast_exp2((y.x - up) * c) : 0.f;
    ml = make_float2(up, ml.y * g + (take ? y.y * f : y.y));
    f0 *= g;
    f1 *= g;
  }
  if (w.z & kMore) *stats = ml;
#pragma unroll 1
  for (int i = 0; i < DIMS; i += 16) {
    uint32_t v[16];
    float o[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = 0.f;
    if (__any_sync(0xffffffffu, take0)) {
      tmem_load16(own + i, v);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (take0) o[e] = __uint_as_float(v[e]) * f0;
    }
    if (__any_sync(0xffffffffu, take1)) {
      tmem_load16(other + i, v);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (take1) o[e] += __uint_as_float(v[e]) * f1;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (take) {
        const float4 x = sums[(i / 4 + q) * 32];
        o[4 * q] += x.x * f;
        o[4 * q + 1] += x.y * f;
        o[4 * q + 2] += x.z * f;
        o[4 * q + 3] += x.w * f;
      }
      if (w.z & kMore)
        sums[(i / 4 + q) * 32] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
    }
    if (!(w.z & kMore)) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(o[e]);
      tmem_store16(own + i, v);
    }
  }
  tmem_wait_st();
  return ml;
}

// The join of an item's parts, by the softmax warps.  First each row's (m, 1 / l) over the parts
// and its lse: a row by as many neighbouring lanes as there are threads for (1 to 32), 16 parts in
// flight by each; the lanes' sums go together in a fixed tree.
template <int D, Mode MODE>
__device__ __noinline__ void join_stats(const Params &p, const Work &w, float2 *stats) {
  const ChunkArgs &a = p.a;
  const int G = p.group, TQ = p.tq;
  const float c = a.scale * kLog2e;
  constexpr int kRows = Cfg<D, MODE>::kRows;
  constexpr size_t pitch = kRows * (D + 2);
  const float *base = p.part + static_cast<size_t>(w.slot) * pitch;
  const int rows = w.tokens * G, parts = w.parts;
  int lanes = 32;
  while (lanes > 1 && rows * lanes > kSoftWarps * 32) lanes >>= 1;
  const int sub = threadIdx.x & (lanes - 1);
  for (int r0 = 0; r0 < rows; r0 += kSoftWarps * 32 / lanes) {
    const int rr = r0 + static_cast<int>(threadIdx.x) / lanes;
    const bool real = rr < rows;
    const int tok = rr / G, hh = rr % G;
    const int row = (MODE == kPair ? (tok / TQ) * kQ + (tok % TQ) * G : tok * G) + hh;
    float m = -INFINITY, l = 0.f;
    for (int q0 = sub; q0 < parts && real; q0 += 16 * lanes) {
      float2 ml[16];
      float up = m;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        ml[q] = make_float2(-INFINITY, 0.f);
        if (q0 + q * lanes < parts)
          ml[q] = __ldcg(reinterpret_cast<const float2 *>(base + (q0 + q * lanes) * pitch) + row);
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) up = fmaxf(up, ml[q].x);
      if (m != -INFINITY) l *= fast_exp2((m - up) * c);
      m = up;
      // a part that saw nothing has m = -inf, l = 0; one with a NaN score l = NaN
#pragma unroll
      for (int q = 0; q < 16; ++q)
        l += ml[q].x == -INFINITY ? ml[q].y : ml[q].y * fast_exp2((ml[q].x - m) * c);
    }
    for (int off = 1; off < lanes; off *= 2) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, off),
                  l2 = __shfl_xor_sync(0xffffffffu, l, off), up = fmaxf(m, m2);
      l = (m == -INFINITY ? l : l * fast_exp2((m - up) * c)) +
          (m2 == -INFINITY ? l2 : l2 * fast_exp2((m2 - up) * c));
      m = up;
    }
    if (!real || sub != 0) continue;
    stats[rr] = make_float2(m, l == 0.f ? 0.f : 1.f / l);
    if (a.lse != nullptr)
      a.lse[(static_cast<long long>(w.token) + tok) * a.Hq + w.g * G + hh] =
          l == 0.f ? -INFINITY : m * a.scale + logf(l);
  }
}

// ... and the outputs, after the warps have met.  A thread adds up 4 dims of a row at a time, parts
// in order, kParts of kQuads such quads in flight: the parts come out of L2, some 700 cycles away.
// Few rows have no more than a quad for a thread, and then 16 parts in flight (one token over 40000
// keys, 4 heads on 1, cut into 105 parts: 53.7 us with 4 parts in flight, 24.4 with 16).
template <int D, Mode MODE, int kQuads, int kParts>
__device__ __noinline__ void join_outputs(const Params &p, const Work &w, const float2 *stats) {
  const ChunkArgs &a = p.a;
  const int G = p.group, TQ = p.tq;
  const float c = a.scale * kLog2e;
  constexpr int kRows = Cfg<D, MODE>::kRows, kThr = kSoftWarps * 32;
  constexpr size_t pitch = kRows * (D + 2);
  const float *base = p.part + static_cast<size_t>(w.slot) * pitch;
  const int rows = w.tokens * G, work = rows * (D / 4), parts = w.parts;
  for (int e0 = threadIdx.x; e0 < work; e0 += kThr * kQuads) {
    const float *src[kQuads];  // m of the row in the first part, and where its quad begins
    int quad[kQuads];
    float2 st[kQuads];
    float4 o[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const int e = min(e0 + i * kThr, work - 1), rr = e % rows, tok = rr / G, hh = rr % G;
      const int row = (MODE == kPair ? (tok / TQ) * kQ + (tok % TQ) * G : tok * G) + hh;
      src[i] = base + 2 * row;
      quad[i] = 2 * kRows + (e / rows) * 4 * kRows + 4 * row - 2 * row;
      st[i] = stats[rr];
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int q0 = 0; q0 < parts; q0 += kParts) {
      float m[kParts][kQuads];
      float4 x[kParts][kQuads];
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        const size_t off = static_cast<size_t>(min(q0 + q, parts - 1)) * pitch;
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          m[q][i] = __ldcg(src[i] + off);
          x[q][i] = __ldcg(reinterpret_cast<const float4 *>(src[i] + off + quad[i]));
        }
      }
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          if (q0 + q >= parts || m[q][i] == -INFINITY) continue;  // it may hold NaN
          const float f = fast_exp2((m[q][i] - st[i].x) * c) * st[i].y;
          o[i].x += x[q][i].x * f;
          o[i].y += x[q][i].y * f;
          o[i].z += x[q][i].z * f;
          o[i].w += x[q][i].w * f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const int e = e0 + i * kThr;
      if (e >= work) break;
      const int rr = e % rows, tok = rr / G, hh = rr % G;
      const long long at = (static_cast<long long>(w.token) + tok) * a.Hq + w.g * G + hh;
      *reinterpret_cast<uint2 *>(a.out + at * D + (e / rows) * 4) =
          make_uint2(pack_bf16x2(o[i].x, o[i].y), pack_bf16x2(o[i].z, o[i].w));
    }
  }
}

// ---------------------------------------------------------------------------

template <int D, Mode MODE>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map,
                      const __grid_constant__ Params p) {
  using C = Cfg<D, MODE>;
  constexpr bool PAIR = C::kPairs, FEW = C::kFews, APART = C::kApart;
  constexpr int NK = C::kKeyPlaces, NV = C::kValuePlaces;
  constexpr int A = PAIR ? 1 : 2;  // key tiles whose scores are in use
  extern __shared__ __align__(1024) uint8_t tiles[];
  uint8_t *k_ring = tiles + C::kQTiles * C::kQBytes, *v_ring = k_ring + NK * C::kTileBytes;
  float *sums = reinterpret_cast<float *>(v_ring + NV * C::kTileBytes);
  Ctl &ctl = *reinterpret_cast<Ctl *>(v_ring + NV * C::kTileBytes + C::kSumBytes);
  static_assert(C::kWeights + 2 * C::kPitch <= 512, "");
  static_assert(sizeof(Ctl) <= kCtlBytes && NK >= 2 && NV <= 8 && NK < kBadRing, "");
  static_assert(2 * kSoftRegs + kOtherRegs <= 3 * 168 && C::kSmem <= 227 * 1024, "");
  const ChunkArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.group, TQ = p.tq, TT = TQ * C::kQTiles;

  if (warp == kValueWarp) {
    if (lane < 8) {
      mbar_init(&ctl.k_full[lane], 1);
      mbar_init(&ctl.k_empty[lane], 1);
      mbar_init(&ctl.v_full[lane], 1);
      mbar_init(&ctl.v_empty[lane], 1);
    } else if (lane < 10) {
      mbar_init(&ctl.s_full[lane - 8], 1);
      mbar_init(&ctl.s_free[lane - 8], 4);
      mbar_init(&ctl.p_early[lane - 8], 4);
      mbar_init(&ctl.p_full[lane - 8], 4);
      mbar_init(&ctl.o_done[lane - 8], 1);
    } else if (lane < 10 + kWork) {
      mbar_init(&ctl.work_full[lane - 10], 1);
      mbar_init(&ctl.work_empty[lane - 10], kSoftWarps + 3);
    } else if (lane == 31) {
      mbar_init(&ctl.q_full, 1);
      mbar_init(&ctl.q_empty, 1);
      mbar_init(&ctl.soft, kSoftWarps);
      mbar_init(&ctl.drain, 1);
      ctl.abort = ctl.alive = 0;
    }
    fence_mbar_init();
  } else if (warp == kMmaWarp) {
    tmem_alloc(&ctl.tmem, 512);
    tmem_fence_before();
  } else if (warp == kKeyWarp && lane == 0) {
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  Rows rows{};
  if (warp == kWorkWarp)  // one CTA reports the rows' flags
    rows = load_rows(a, 0, TT, blockIdx.x == 0 ? a.status : nullptr);
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = ctl.tmem;

  if (warp == kWorkWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    hand_out_work(p, ctl, TT, rows, costs<MODE>());
  } else if (warp == kKeyWarp || warp == kValueWarp) {
    // ------------------------------------------------------------ loads
    // Two warps, for a page of 16 tokens takes a copy each, and a warp issues one in some 60
    // cycles: with one warp, cross attention of one token over pages of 16 (32 sequences, 16 heads
    // of 64, 200 to 1500 states) took 28% longer.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    const bool keys = warp == kKeyWarp, paged = a.kv.table != nullptr;
    const int log_bs = paged ? __ffs(a.kv.bs) - 1 : 7, bs = 1 << log_bs;
    const int ppt = kKeys >> log_bs;          // boxes of a tile and half
    const int groups = 32 >> (7 - log_bs);    // tiles whose ids 32 lanes hold
    const int box = lane & (ppt - 1), half = lane >> (7 - log_bs);
    const int none = static_cast<int>(  // a row past the pool: the box reads as zeros
        paged ? static_cast<long long>(a.kv.num_pages) * a.Hkv * bs
              : static_cast<long long>(a.B) * a.Hkv * a.T);
    const CUtensorMap *map = keys ? &k_map : &v_map;
    uint8_t *ring = keys ? k_ring : v_ring;
    uint64_t *full = keys ? ctl.k_full : ctl.v_full, *empty = keys ? ctl.k_empty : ctl.v_empty;
    const int places = keys ? NK : NV;
    int stage = 0, puts = 0, mark = 0;
    uint32_t drained = 1, q_turn = 1;  // a place's first filling waits for nothing
    bool ok = true;
    auto load_q = [&](const Work &w) {
      ok = warp_wait(&ctl.q_empty, q_turn, &ctl.abort);
      if (!ok) return;
      q_turn ^= 1u;
      if (lane == 0) {
        const int boxes = FEW ? 4 : PAIR && w.tokens > TQ ? 2 : 1;  // copies, or tiles
        mbar_arrive_expect_tx(&ctl.q_full, static_cast<uint32_t>(boxes * G * TQ * D * 2));
        for (int i = 0; i < boxes; ++i)
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(tiles + i * (FEW ? 32 * 128 : C::kQBytes) + h * (kQ * 128), &q_map, h * 64,
                        w.g * G, w.token + (FEW ? 0 : i * TQ), &ctl.q_full);
      }
      __syncwarp();
    };
    Take take;
    Work w;
    while (ok && take.get(ctl, w) && w.token >= 0) {
      const int32_t *table =
          paged ? a.kv.table + static_cast<size_t>(w.b) * a.kv.max_blocks : nullptr;
      const int kend = a.causal ? max(0, w.seen + w.tokens - 1) : w.len;
      const int blocks = (kend + bs - 1) >> log_bs;
      auto load_ids = [&](int group) {  // the page of block (t0 + group * groups) * ppt + lane
        const int j = (w.t0 + group * groups) * ppt + lane;
        return paged && j < blocks && j < a.kv.max_blocks ? __ldg(table + j) : -1;
      };
      int ids = load_ids(0), next = load_ids(1), in_group = 0, group = 0;
      for (int j = 0; j < w.nt && ok; ++j) {
        int y = none;
        uint32_t bad = 0u;
        if (paged) {
          if (in_group == groups) {
            ids = next;
            next = load_ids(++group + 1);
            in_group = 0;
          }
          const int block = (w.t0 + j) * ppt + box;
          const int id = __shfl_sync(0xffffffffu, ids, in_group++ * ppt + box);
          const bool inside = block < blocks, good = id >= 0 && id < a.kv.num_pages;
          if (inside && good) y = (id * a.Hkv + w.g) * bs;
          bad = __ballot_sync(0xffffffffu, lane < ppt && inside && !good);
        } else {
          y = (w.b * a.Hkv + w.g) * a.T + (w.t0 + j) * kKeys;
        }
        if (keys && lane == 0) {
          ctl.bad[mark] = bad;
          if (bad != 0u) flag_status(a.status, KSA_FLAG_INDEX_SKIPPED);
        }
        mark = (mark + 1) % kBadRing;
        ok = warp_wait(&empty[stage], drained, &ctl.abort);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], C::kTileBytes);
        __syncwarp();
        if (lane < ppt * (D / 64))
          tma_load_2d(ring + stage * C::kTileBytes + half * (kKeys * 128) + box * bs * 128, map,
                      half * 64, y, &full[stage]);
        ++puts;
        if (++stage == places) {
          stage = 0;
          drained ^= 1u;
        }
        if (keys && j == 0) load_q(w);  // the first keys are on their way: now the queries
      }
      take.release(ctl);
    }
    // leave no copy in flight behind (also after an aborted wait)
    for (int i = max(0, puts - places); i < puts; ++i)
      mbar_wait(&full[i % places], (i / places) & 1);
    if (keys) mbar_wait(&ctl.q_full, q_turn);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    constexpr uint32_t idesc_s = mma_idesc_bf16(kQ, kKeys, false);
    constexpr uint32_t idesc_o = mma_idesc_bf16(kQ, D, true);
    const uint64_t q_desc = smem_desc_128b(smem_addr(tiles), 16, 1024);
    const uint64_t k_desc = smem_desc_128b(smem_addr(k_ring), 16, 1024);
    const uint64_t v_desc = smem_desc_128b(smem_addr(v_ring), kKeys * 128, 1024);
    const uint32_t one = elect_one();
    int k_next = 0, v_next = 0;  // next places of the rings, and the parities of their filling
    uint32_t k_turn = 0, v_turn = 0, q_turn = 0;
    uint32_t p_turn = 0;  // bit s: parity of stream s's next weights
    uint32_t f_turn = 0;  // and of the reading of its next scores
    // A vote after each wait would stand between the weights and their products.  So a lane that a
    // wait has failed waits no more, but stays in step to the item's end, where the warp votes: the
    // products until then are of no use, and harm nothing.
    bool ok = true;
    auto next_keys = [&]() {  // waits for the next key tile: its place
      const int st = k_next;
      ok = ok && wait_bar(&ctl.k_full[st], k_turn, &ctl.abort);
      if (++k_next == NK) {
        k_next = 0;
        k_turn ^= 1u;
      }
      return st;
    };
    Take take;
    Work w;
    while (ok && take.get(ctl, w) && w.token >= 0) {
      take.release(ctl);
      if (w.nt == 0) continue;
      const int streams = PAIR ? (w.tokens > TQ ? 2 : 1) : 2;
      // scores of stream s's next tile, its keys in place st
      auto scores = [&](int s, int st) {
        const uint64_t qd = q_desc + static_cast<uint64_t>((PAIR ? s : 0) * C::kQBytes >> 4);
        const uint64_t kd = k_desc + static_cast<uint64_t>(st * C::kTileBytes >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(one, tmem + s * kKeys,
                 qd + static_cast<uint64_t>(((i / 4) * (kQ * 128) + (i % 4) * 32) >> 4),
                 kd + static_cast<uint64_t>(((i / 4) * (kKeys * 128) + (i % 4) * 32) >> 4), idesc_s,
                 i > 0);
        mma_commit(one, &ctl.s_full[s]);
        if (!PAIR || s == streams - 1) mma_commit(one, &ctl.k_empty[st]);
      };
      for (int j = 0; j < min(A, w.nt); ++j) {
        const int st = next_keys();
        if (j == 0) {
          ok = ok && wait_bar(&ctl.q_full, q_turn, &ctl.abort);
          q_turn ^= 1u;
        }
        tmem_fence_after();
        if (PAIR)
          for (int s = 0; s < streams; ++s) scores(s, st);
        else
          scores(j, st);
      }
      if (w.nt <= A) mma_commit(one, &ctl.q_empty);
      for (int j = 0; j < w.nt; ++j) {
        const int sv = v_next;
        int sk = 0;
        if (APART) {  // the stream's next scores, as soon as these are read
          const int s = j & 1;
          if (j + A < w.nt) {
            sk = next_keys();
            ok = ok && wait_bar(&ctl.s_free[s], (f_turn >> s) & 1u, &ctl.abort);
            tmem_fence_after();
            scores(s, sk);
            if (j + A + 1 == w.nt) mma_commit(one, &ctl.q_empty);
          }
          // (scores are read before their weights are ready: a turn not waited for has passed)
          f_turn ^= 1u << s;
        }
        ok = ok && wait_bar(&ctl.v_full[sv], v_turn, &ctl.abort);
        if (++v_next == NV) {
          v_next = 0;
          v_turn ^= 1u;
        }
        if ((w.t0 + j + 1) * kKeys > w.len) {
          // the cache behind the row's last token: P is 0 there, but 0 x NaN is not
          const int r0 = w.len - (w.t0 + j) * kKeys;
          for (int e = r0 * 8 + lane; e < kKeys * 8; e += 32)
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              *reinterpret_cast<uint4 *>(v_ring + sv * C::kTileBytes + h * (kKeys * 128) + e * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t vd = v_desc + static_cast<uint64_t>(sv * C::kTileBytes >> 4);
        const bool first = PAIR ? j == 0 : j < 2;  // of its stream
        for (int i = 0; i < (PAIR ? streams : 1); ++i) {
          const int s = PAIR ? i : j & 1;
          for (int part = 0; part < 2; ++part) {
            ok = ok && wait_bar(part == 0 ? &ctl.p_early[s] : &ctl.p_full[s],
                                (p_turn >> s) & 1u, &ctl.abort);
            tmem_fence_after();
            constexpr int kSplit = kEarly / 16, kAll = kKeys / 16;
            if (part == 0) {
#pragma unroll
              for (int x = 0; x < kSplit; ++x)
                mma_ts(one, tmem + 2 * kKeys + s * D, tmem + C::kWeights + s * C::kPitch + x * 8,
                       vd + static_cast<uint64_t>(x * 16 * 128 >> 4), idesc_o, !first || x > 0);
            } else {
#pragma unroll
              for (int x = kSplit; x < kAll; ++x)
                mma_ts(one, tmem + 2 * kKeys + s * D, tmem + C::kWeights + s * C::kPitch + x * 8,
                       vd + static_cast<uint64_t>(x * 16 * 128 >> 4), idesc_o, true);
            }
          }
          p_turn ^= 1u << s;
          mma_commit(one, &ctl.o_done[s]);
          if (!PAIR || s == streams - 1) mma_commit(one, &ctl.v_empty[sv]);
          if (!APART && j + A < w.nt) {
            if (i == 0) sk = next_keys();
            tmem_fence_after();
            scores(s, sk);
            if (j + A + 1 == w.nt && (!PAIR || s == streams - 1)) mma_commit(one, &ctl.q_empty);
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    // the tensor memory goes back only when no product runs
    mma_commit(one, &ctl.drain);
    const uint64_t since = global_timer_ns();
    while (!mbar_try_wait(&ctl.drain, 0) && global_timer_ns() - since < kWaitTimeoutNs) {
    }
  } else if (warp < kSoftWarps) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // stream, row of the query tile (of the statistics: every copy's), row of the queries
    const int s = warp >> 2, r = (warp & 3) * 32 + lane, qr = FEW ? lane : r;
    constexpr int kCols = FEW ? 32 : kKeys;  // keys that a thread weighs, from col0 on
    const int col0 = FEW ? (warp & 3) * 32 : 0;
    const float c = a.scale * kLog2e;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + s * kKeys, to = tmem + lanes + 2 * kKeys + s * D;
    const uint32_t tp = tmem + lanes + C::kWeights + s * C::kPitch;
    uint32_t turn = 0, soft_turn = 0;  // parities of the stream's next scores, of the sync below
    int mark = 0;                      // page marks of the item's first key tile
    bool ok = true;
    auto soft_sync = [&]() {  // all softmax warps; with a limit, unlike a named barrier
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.soft);
      ok = warp_wait(&ctl.soft, soft_turn, &ctl.abort) && ok;
      soft_turn ^= 1u;
    };
    Take take;
    while (ok) {
      int steps, end;
      bool active;
      {
        Work w;
        ok = take.get(ctl, w);
        if (!ok || w.token < 0) break;
        const int tok = qr / G + (PAIR ? s * TQ : 0);
        const bool valid = qr < G * TQ && tok < w.tokens;
        active = __any_sync(0xffffffffu, valid);
        steps = PAIR ? (s == 0 || w.tokens > TQ ? w.nt : 0) : (w.nt - s + 1) / 2;
        end = (valid ? (a.causal ? w.seen + tok : w.len) : 0) - w.t0 * kKeys;
      }
      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < steps; ++k) {
        const int j = PAIR ? k : 2 * k + s;
        ok = warp_wait(&ctl.s_full[s], turn, &ctl.abort);
        if (!ok) break;
        turn ^= 1u;
        tmem_fence_after();
        if (active) {
          uint32_t v[kCols];
          if constexpr (FEW) {
            tmem_load32(ts + col0, v);
          } else {
#pragma unroll
            for (int i = 0; i < kCols; i += 64) tmem_load64(ts + i, v + i);
          }
          if (APART) {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.s_free[s]);
          }
          const int lim = end - j * kKeys - col0;
          const uint32_t bad = ctl.bad[(mark + j) % kBadRing];
          if (lim < kCols) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if (i >= lim) v[i] = 0xff800000u;
          }
          if (bad != 0u) {
            const int sh = __ffs(a.kv.bs) - 1;
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if ((bad >> ((col0 + i) >> sh)) & 1u) v[i] = 0xff800000u;
          }
          float mx[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mx[i] = -INFINITY;
#pragma unroll
          for (int i = 0; i < kCols; i += 2)
            mx[(i >> 1) & 7] = max3_nan(mx[(i >> 1) & 7], __uint_as_float(v[i]),
                                        __uint_as_float(v[i + 1]));
          const float top = max3_nan(max3_nan(mx[0], mx[1], mx[2]), max3_nan(mx[3], mx[4], mx[5]),
                                     max3_nan(mx[6], mx[7], -INFINITY));
          // a NaN or +inf score: the row's softmax is NaN (-inf weighs nothing)
          if (!(top < INFINITY)) l = NAN;
          if (APART && k > 0) {  // the last product reads the weights and adds to O
            ok = warp_wait(&ctl.o_done[s], turn, &ctl.abort);
            if (!ok) break;
            tmem_fence_after();
          }
          if (k == 0) {
            m = top;
          } else if (__any_sync(0xffffffffu, (top - m) * c > kRescale)) {
            const float up = fmaxf(m, top);
            const float f = up == -INFINITY ? 1.f : fast_exp2((m - up) * c);
            m = up;
            l *= f;
            // (the last product into O is done: see above, or these scores' was issued behind it)
#pragma unroll
            for (int i = 0; i < D; i += 32) {
              uint32_t o[32];
              tmem_load32(to + i, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_store32(to + i, o);
            }
          }
          const float ms = m == -INFINITY ? 0.f : m * c;
          const uint64_t cc = f32x2(c, c), mm = f32x2(-ms, -ms);
          uint64_t sum[2] = {0, 0};
          uint32_t x[16];
          if (FEW) {  // the copy's other weights
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 0u;
#pragma unroll
            for (int i = 16; i < kKeys / 2; i += 16)
              tmem_store16(tp + (col0 / 2 + i) % (kKeys / 2), x);
          }
          // a pair's scale, exponential, and sum and rounding run staggered, so that the
          // exponential unit (8 cycles a warp instruction) does not wait for them
#pragma unroll
          for (int e = 0; e < kCols / 2 + kLag; ++e) {
            if (e < kCols / 2) {
              float x0, x1;
              f32x2_split(fma2(f32x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])),
                               cc, mm), x0, x1);
              v[2 * e] = __float_as_uint(x0);
              v[2 * e + 1] = __float_as_uint(x1);
            }
            if (e >= kLead && e - kLead < kCols / 2) {
              exp2_in_place(v[2 * (e - kLead)]);
              exp2_in_place(v[2 * (e - kLead) + 1]);
            }
            if (e >= kLag) {
              const int d = e - kLag;
              const float p0 = __uint_as_float(v[2 * d]), p1 = __uint_as_float(v[2 * d + 1]);
              sum[d & 1] = add2(sum[d & 1], f32x2(p0, p1));
              x[d & 15] = pack_bf16x2(p0, p1);
              if ((d & 15) == 15) tmem_store16(tp + col0 / 2 + (d & ~15), x);
              if (!FEW && d == kEarly / 2 - 1) {  // these weights' products may start
                tmem_wait_st();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_early[s]);
              }
            }
          }
          float l0, l1;
          f32x2_split(add2(sum[0], sum[1]), l0, l1);
          l += l0 + l1;
          tmem_wait_st();
        } else if (APART && k > 0) {  // nor may a warp without rows be a step ahead of the others
          ok = warp_wait(&ctl.o_done[s], turn, &ctl.abort);
          if (!ok) break;
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (APART && !active) mbar_arrive(&ctl.s_free[s]);
          if (FEW || !active) mbar_arrive(&ctl.p_early[s]);
          mbar_arrive(&ctl.p_full[s]);
        }
      }
      if (!ok) break;
      // -------------------------------------------------------- output
      const Work &w = ctl.work[take.at];
      mark = (mark + w.nt) % kBadRing;
      const int tok = qr / G + (PAIR ? s * TQ : 0), h = w.g * G + qr % G;
      const bool valid = qr < G * TQ && tok < w.tokens;
      const long long at = (static_cast<long long>(w.token) + tok) * a.Hq + h;
      float f0 = 1.f, f1 = 0.f;
      float own = m, other = -INFINITY;  // maxima that the streams' outputs belong to
      bool has0 = steps > 0, has1 = false;
      // every step's product arrives on o_done: the last one's parity is behind `turn`
      if (steps > 0) ok = warp_wait(&ctl.o_done[s], turn ^ 1u, &ctl.abort);
      if (PAIR && !ok) break;  // (otherwise behind the join's sync)
      if (!PAIR) {  // join the streams: each half of the warps writes half of the dims
        ctl.ml[s][r] = make_float2(m, l);
        tmem_fence_before();
        soft_sync();
        if (!ok) break;
      }
      if (FEW) {  // the row's eight maxima and sums
        other = ctl.ml[s ^ 1][r].x;
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, ctl.ml[i >> 2][(i & 3) * 32 + lane].x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 y = ctl.ml[i >> 2][(i & 3) * 32 + lane];
          l += y.x == -INFINITY ? y.y : y.y * fast_exp2((y.x - m) * c);
        }
        has1 = w.nt > (s ^ 1);
        f0 = own == -INFINITY ? 0.f : fast_exp2((own - m) * c);
        f1 = other == -INFINITY ? 0.f : fast_exp2((other - m) * c);
      } else if (!PAIR) {
        const float2 y = ctl.ml[s ^ 1][r];
        has1 = w.nt > (s ^ 1);
        other = y.x;
        const float both = fmaxf(m, y.x);
        f0 = m == -INFINITY ? 0.f : fast_exp2((m - both) * c);
        f1 = y.x == -INFINITY ? 0.f : fast_exp2((y.x - both) * c);
        l = l * f0 + y.y * f1;
        m = both;
      }
      tmem_fence_after();
      constexpr int kDims = PAIR ? D : D / 2;  // of this warp
      const int dim0 = PAIR ? 0 : s * kDims;
      if (w.z >= kSegments) {
        const float2 y = add_segment<D, MODE>(p, ctl, w,
                                              has0 && own != -INFINITY ? f0 : -1.f,
                                              has1 && other != -INFINITY ? f1 : -1.f,
                                              make_float2(m, l));
        if (w.z & kMore) {
          tmem_fence_before();
          if (!PAIR) soft_sync();
          take.release(ctl);
          continue;
        }
        own = m = y.x;
        l = y.y;
        if (!PAIR) {
          f0 = 1.f;
          has0 = true;
          has1 = false;
        }
      }
      const bool split = w.parts > 1;
      float *part =
          p.part + static_cast<size_t>(w.slot + (w.z & (kSegments - 1))) * (C::kRows * (D + 2));
      const int row = (PAIR ? s * kQ : 0) + qr;
      const float inv = split ? 1.f : l == 0.f ? 0.f : 1.f / l;
      f0 *= inv;
      f1 *= inv;
      // A row that sees none of a stream's keys takes nothing of its output, which may be NaN by
      // values that other rows see.  (Where a score was NaN, so is l, and no weight is 0.)
      const bool take0 = FEW || own != -INFINITY || f0 != 0.f,
                 take1 = FEW || other != -INFINITY || f1 != 0.f;
      if (valid && (FEW ? warp == 0 : dim0 == 0)) {
        if (split)
          reinterpret_cast<float2 *>(part)[row] = make_float2(m, l);
        else if (a.lse != nullptr)
          a.lse[at] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
      }
      if (FEW) {
        // A warp adds up both streams for its copy and half of the dims; then the copies go
        // together through shared memory, 2 and 3 to 0 and 1, and these to each other by halves.
        constexpr int kOut = D / 4;  // dims that a thread of copy 0 or 1 writes
        const int copy = warp & 3;
        float o[2 * kOut];
#pragma unroll
        for (int i = 0; i < 2 * kOut; i += 16) {
          uint32_t v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) o[i + e] = 0.f;
          if (has0) {
            tmem_load16(to + dim0 + i, v);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (take0) o[i + e] = __uint_as_float(v[e]) * f0;
          }
          if (has1) {
            tmem_load16(tmem + lanes + 2 * kKeys + (s ^ 1) * D + dim0 + i, v);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (take1) o[i + e] += __uint_as_float(v[e]) * f1;
          }
        }
        float *sum = sums + ((copy & 1) * 2 + s) * (2 * kOut * 32) + lane;  // [2][2][D / 2][32]
        if (copy >= 2)
#pragma unroll
          for (int e = 0; e < 2 * kOut; ++e) sum[e * 32] = o[e];
        soft_sync();
        if (copy < 2) {
#pragma unroll
          for (int e = 0; e < 2 * kOut; ++e) o[e] += sum[e * 32];
#pragma unroll
          for (int e = 0; e < kOut; ++e) sum[e * 32] = copy == 0 ? o[kOut + e] : o[e];
        }
        soft_sync();
        if (!ok) break;
        if (copy < 2) {
          const float *from = sums + ((copy ^ 1) * 2 + s) * (2 * kOut * 32) + lane;
          const int dim = dim0 + copy * kOut;
#pragma unroll
          for (int e = 0; e < kOut; ++e) o[e] = (copy == 0 ? o[e] : o[kOut + e]) + from[e * 32];
          float4 *dst =
              split ? reinterpret_cast<float4 *>(part + 2 * C::kRows) + dim / 4 * C::kRows + row
                    : nullptr;
          uint16_t *to = split ? nullptr : a.out + at * D + dim;
          if (valid && split) {
#pragma unroll
            for (int e = 0; e < kOut / 4; ++e)
              dst[e * C::kRows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          } else if (valid) {
#pragma unroll
            for (int e = 0; e < kOut / 8; ++e)
              reinterpret_cast<uint4 *>(to)[e] = make_uint4(
                  pack_bf16x2(o[8 * e], o[8 * e + 1]), pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                  pack_bf16x2(o[8 * e + 4], o[8 * e + 5]), pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
          }
          float zero[4] = {0.f, 0.f, 0.f, 0.f};  // NaN if an output is not finite
#pragma unroll
          for (int e = 0; e < kOut; ++e) zero[e & 3] = fmaf(o[e], 0.f, zero[e & 3]);
          const bool mine = valid && l == l;
          if (__any_sync(0xffffffffu,
                         mine && (zero[0] + zero[1]) + (zero[2] + zero[3]) != 0.f)) {
            const int keys = w.t0 * kKeys;  // before this segment, and before the part
            const int first = keys - (w.z & (kMore - 1)) / kSegments * kSegment * kKeys;
            settle<D>(a, ctl, w, first, l == 0.f ? first : keys + min(end, w.nt * kKeys), dim,
                      kOut, mine, to, dst, C::kRows);
          }
        }
      } else if (active) {
#pragma unroll
        for (int i = 0; i < kDims; i += 32) {
          uint32_t v[32];
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
          if (has0) {
            tmem_load32(to + dim0 + i, v);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (take0) o[e] = __uint_as_float(v[e]) * f0;
          }
          if (has1) {
            tmem_load32(tmem + lanes + 2 * kKeys + (s ^ 1) * D + dim0 + i, v);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (take1) o[e] += __uint_as_float(v[e]) * f1;
          }
          if (!valid) continue;
          if (split) {
            // [dims / 4][rows][4]: a warp's rows are neighbours
            float4 *dst = reinterpret_cast<float4 *>(part + 2 * C::kRows) +
                          (dim0 + i) / 4 * C::kRows + row;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e * C::kRows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          } else {
            uint16_t *dst = a.out + at * D + dim0 + i;
            uint32_t x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
            if (p.wide_out) {  // a lane's whole sectors: half the store instructions' cycles
              store_32(dst, x);
              store_32(dst + 16, x + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                reinterpret_cast<uint4 *>(dst)[e] =
                    make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
          }
        }
      }
      tmem_fence_before();
      if (split) {
        __threadfence();
        soft_sync();
        if (!ok) break;
        if (tid == 0) {
          ctl.last = atomicAdd(p.sem + w.slot, 1u) == static_cast<uint32_t>(w.parts) - 1u;
          if (ctl.last) p.sem[w.slot] = 0u;
        }
        soft_sync();
        if (!ok) break;
        if (ctl.last) {
          __threadfence();
          join_stats<D, MODE>(p, w, &ctl.ml[0][0]);
          soft_sync();
          if (!ok) break;
          if (w.tokens * G * (D / 4) <= kSoftWarps * 32)
            join_outputs<D, MODE, 1, 16>(p, w, &ctl.ml[0][0]);
          else
            join_outputs<D, MODE, 4, 4>(p, w, &ctl.ml[0][0]);
          soft_sync();  // before the statistics' place is used again
          if (!ok) break;
        }
      }
      if (!PAIR) soft_sync();  // the next item's products may overwrite both streams' O
      take.release(ctl);
    }
    tmem_fence_before();
  }

  __syncthreads();
  if (warp == kMmaWarp) {
    tmem_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && ctl.abort != 0) flag_status(a.status, KSA_FLAG_WAIT_TIMEOUT);
}

// By what the host knows: the rows (tokens times heads of a group) of an average sequence and the
// capacity T; the lengths are on the device.  Every form serves every length, but a batch far from
// its average (one-token rows beside a prompt's chunk, an axis that is mostly padding) or far below
// its capacity is not in the form that would be the fastest for it.  What fits in 32 goes as
// kFew: one token over 200 to 1500 states (32 sequences, 16 heads of 64) 32 us, 43 as kOne;
// 5 tokens over 131000 (32 heads on 8 of 128) 96 and 101.  More than a tile of 128 can go in
// pairs, whose tiles share their keys' loads, or one by one, in items of half the length:
//   - by the rounds that the SMs take, at 1.2 of a pair's time for two items (6000 keys, 32 heads
//     on 8 of 128: 512 tokens 73 us in pairs, 55 one by one; 1216: 130 and 122; 1920: 169 and
//     172; 4800: 381 and 411);
//   - at D = 64, where the loads are half as large and twice as many places hold them, with room
//     for more than 2048 keys always one by one (16384 keys, 2368 tokens: 474 and 437 us; over
//     1024 keys 39 and 40);
//   - with room for one key tile the second stream of a single item has no work, so a round costs
//     the same.
Mode choose_mode(int B, int Hq, int Hkv, int D, int T, int N, int num_sms) {
  const int G = Hq / Hkv;
  const long long rows = static_cast<long long>(N) * G, each = (rows + B - 1) / B;
  if (each <= 32 && G <= 32) return kFew;
  if (each <= kQ) return kOne;
  if (D == 64 && T > 2048) return kOne;
  const auto rounds = [&](int tile) {
    return (static_cast<long long>(B) * Hkv * ((each + tile - 1) / tile) + num_sms - 1) / num_sms;
  };
  const long long pairs = rounds(2 * kQ), ones = rounds(kQ);
  return (T <= kKeys ? ones <= pairs : 6 * ones < 10 * pairs) ? kOne : kPair;
}

template <int D, Mode MODE>
cudaError_t launch(const Params &p, const CUtensorMap *maps, int num_sms, cudaStream_t stream) {
  int occ = 0;
  auto kernel = chunk_attn_kernel<D, MODE>;
  const cudaError_t err = kernel_occupancy(reinterpret_cast<const void *>(kernel), kThreads,
                                           Cfg<D, MODE>::kSmem, &occ);
  if (err != cudaSuccess) return err;
  kernel<<<num_sms, kThreads, Cfg<D, MODE>::kSmem, stream>>>(maps[0], maps[1], maps[2], p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_mode(Mode mode, const Params &p, const CUtensorMap *maps, int num_sms,
                        cudaStream_t stream) {
  return mode == kPair  ? launch<D, kPair>(p, maps, num_sms, stream)
         : mode == kOne ? launch<D, kOne>(p, maps, num_sms, stream)
                        : launch<D, kFew>(p, maps, num_sms, stream);
}

size_t sem_bytes(int max_parts) {
  return (256 + static_cast<size_t>(max_parts) * 4 + 255) / 256 * 256;
}

// Query rows of a CTA, at most, in the forms that such calls take.
size_t part_rows(int B, int G, int N) {
  const long long each = (static_cast<long long>(N) * G + B - 1) / B;
  return each > kQ ? 2 * kQ : each > 32 || G > 32 ? kQ : 32;
}

}  // namespace

// workspace: [0] items handed out, [1] CTAs ended, from byte 256 the parts' semaphores (all zero
// between calls), then the parts, as large as any form of these rows needs (so that fewer tokens
// never need more), and where rows may be longer than a segment the CTAs' sums over segments
size_t chunk_attn_workspace_bytes(int B, int Hq, int Hkv, int D, int T, int N, int num_sms) {
  const int max_parts = kPartsPerSm * num_sms;
  const size_t rows = part_rows(B, Hq / Hkv, N);
  return sem_bytes(max_parts) + static_cast<size_t>(max_parts) * rows * (D + 2) * 4 +
         (T > kSegment * kKeys ? num_sms * carry_floats(max(static_cast<int>(rows), kQ), D) * 4
                               : 0);
}

cudaError_t launch_chunk_attn(const ChunkArgs &a, void *ws, int num_sms, cudaStream_t stream) {
  Params p;
  p.a = a;
  p.max_parts = kPartsPerSm * num_sms;
  p.next = static_cast<uint32_t *>(ws);
  p.done = p.next + 1;
  p.sem = p.next + 64;
  p.part = reinterpret_cast<float *>(static_cast<char *>(ws) + sem_bytes(p.max_parts));
  p.carry = p.part + p.max_parts * part_rows(a.B, a.Hq / a.Hkv, a.N) * (a.D + 2);
  const Mode mode = choose_mode(a.B, a.Hq, a.Hkv, a.D, a.T, a.N, num_sms);
  p.group = a.Hq / a.Hkv;
  p.tq = (mode == kFew ? 32 : kQ) / p.group;
  p.wide_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  const bool paged = a.kv.table != nullptr;
  const uint64_t rows = paged ? static_cast<uint64_t>(a.kv.num_pages) * a.Hkv * a.kv.bs
                              : static_cast<uint64_t>(a.B) * a.Hkv * a.T;
  const int box = paged ? a.kv.bs : kKeys;
  CUtensorMap maps[3];
  if (!encode_q_tensor_map(&maps[0], a.q, a.D, a.Hq, a.N, a.q_stride, p.group, p.tq) ||
      !encode_kv_tensor_map(&maps[1], a.K, rows, a.D, box) ||
      !encode_kv_tensor_map(&maps[2], a.V, rows, a.D, box))
    return cudaErrorInvalidValue;
  return a.D == 128 ? launch_mode<128>(mode, p, maps, num_sms, stream)
                    : launch_mode<64>(mode, p, maps, num_sms, stream);
}

}  // namespace ksa
