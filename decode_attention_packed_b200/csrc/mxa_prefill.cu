// Attention of chunks of new tokens over a paged grouped-query cache, for
// sm_100a (mxa_prefill_fwd).
//
//   O = softmax(scale Q K^T + mask) V,   LSE = ln sum_j exp(scale q . k_j)
//
// Each CTA walks a contiguous share of the work with these roles:
//  - two loading warps, one of which finds the CTA's share, gather K and V
//    pages through the block table with TMA into a ring of shared-memory slots
//    and load the packed query rows;
//  - two issuing warps run S = Q K^T and O += P V on the tensor cores
//    (tcgen05, accumulators and P in tensor memory);
//  - softmax warps, one thread per packed query row, turn S into P with a
//    running maximum and sum, and write the rows out.
//
// Units.  The G query heads of one KV head are packed into the rows of a
// tile, row m = t * G + g, so a KV byte serves all of them: a 128-row tile
// holds floor(128 / G) tokens.  A unit is (batch row, KV head, group of
// tiles): two tiles for head dims 64 and 128 (while one tile's scores are in
// the softmax, the tensor cores work on the other's), one for 256, whose
// accumulator fills half of tensor memory (its queries take the second
// tile's place).
//
// Split.  All units, each a fixed cost plus its visible KV blocks, are laid
// end to end and cut into equal contiguous ranges, one per CTA: ragged
// batches, causal triangles and single long rows all give every CTA the same
// work.  A unit cut by a range's end leaves float32 pieces with their LSEs in
// the workspace, which a second small kernel merges.
//
// What bounds it (B200, per pair of tiles and 128 keys).  D = 128: the tensor
// cores 2048 cycles (four products of 512), the exponentials 2048 (16 a cycle
// and SM, both tiles' 32768), shared memory 2048 (256 KB at 128 bytes a cycle:
// operands and loads).  D = 64: 1024, 2048 and 1024.  Measured: 2600 to 2700 in
// either case, since a tile's loads, maximum, hand-overs and stores are only
// partly hidden behind the other tile's exponentials; 4096 tokens after 12288
// keys (64 query heads, 8 KV heads, D = 128) run at 1400 TFLOP/s for a
// millisecond or two and at about 1200 when the card's power limit holds the
// clock.  D = 256, per tile and 64 keys: the tensor cores 1024, measured 1800,
// one tile's hand-overs with nothing beside them.  Tried and not kept: part of the
// exponentials by a polynomial on the floating-point pipe (an eighth: no change;
// a quarter: slower; measured with two threads a row, at 3000 cycles a block),
// turns of the two tiles at the exponentials, a block's scores on their way
// during the hand-over of the weights before (slower), two groups of softmax
// warps that take the blocks of D = 256 in turn (no change).
#include "mxa_config.h"
#include "mxa_device.cuh"
#include "mxa_launch.h"
#include "mxa_prefill.h"
#include "mxa_tcgen05.cuh"
#include "mxa_tmap.h"

namespace mxa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTileRows = 128;
constexpr int kDescs = 4;  // segments published ahead

template <int D>
struct Cfg {
  static constexpr int NT = D <= 128 ? 2 : 1;       // tiles of a unit
  static constexpr int T = D <= 128 ? 128 : 64;     // keys of a block
  static constexpr int CH = D / 64;                 // 64-column chunks of a row
  // A block of K or V in shared memory: groups of 8 keys, each with its
  // chunks one after the other (8 rows of 128 bytes, swizzled), so that one
  // TMA box brings whole keys.
  static constexpr int kGroupBytes = CH * 1024;
  // One thread a row: two would have to exchange their maxima (a ragged batch
  // of 24 requests took 167 us so, now 154; head dim 256 127 us, now 122).
  static constexpr int kSoftmaxWarps = 4 * NT;
  static constexpr int kScoreWarp = kSoftmaxWarps, kValueWarp = kSoftmaxWarps + 1;
  static constexpr int kKeyWarp = kSoftmaxWarps + 2;  // and the one that loads queries and values
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
  static constexpr int kSlotBytes = T * D * 2;      // one block of K or of V
  static constexpr int kSlots = 128 * 1024 / kSlotBytes;
  static_assert(kSlots % 2 == 0, "keys in the even slots, values in the odd ones");
  static constexpr int kQBytes = kTileRows * D * 2;
  // Tensor memory: T columns of scores, two weight buffers of T / 2 (a column
  // holds two weights of a row), and at the end the tiles' accumulators.  All
  // scores take turns in one buffer, which is free again as soon as they are
  // in registers.  The turns keep two tiles out of step, so that one's
  // exponentials run beside the other's loads and stores: with a buffer each
  // (room for it at D = 64) a ragged batch took 161 us instead of 155.
  static constexpr int kPCol = T, kOCol = 512 - NT * D;
  // Head dim 256 has room for the queries, packed as the weights are: with the
  // queries in shared memory 64-key blocks are bound by its bandwidth (a block
  // moves 192 KB through it, 1536 cycles at 128 bytes each, against 1024 of the
  // tensor cores; 128 KB so).
  static constexpr bool kQTmem = D == 256;
  static constexpr int kQCol = kPCol + T;
  static_assert(kQCol + (kQTmem ? D / 2 : 0) <= kOCol, "tensor memory");
  // shared memory
  static constexpr int kQOff = kSlots * kSlotBytes;
  static constexpr int kDescOff = kQOff + NT * kQBytes;
  static constexpr int kBarOff = kDescOff + kDescs * 64;
  static constexpr int kSmem = kBarOff + 512;
  // barriers
  static constexpr int B_FULL = 0, B_EMPTY = kSlots, B_SFULL = 2 * kSlots, B_SFREE = B_SFULL + 2;
  static constexpr int B_PREADY = B_SFREE + 2;
  static constexpr int B_OFULL = B_PREADY + 2, B_QFULL = B_OFULL + 2, B_QEMPTY = B_QFULL + 1;
  static constexpr int B_DFULL = B_QEMPTY + 1, B_DEMPTY = B_DFULL + kDescs;
  static constexpr int B_QREADY = B_DEMPTY + kDescs;  // the queries are in tensor memory
  static constexpr int B_COUNT = B_QREADY + 1;
  static_assert(B_COUNT * 8 + 16 <= 512 && kSmem <= 227 * 1024, "shared memory");
};

// A contiguous range of one unit's KV blocks, as the key warp publishes it.
struct Segment {
  int b, h, it;      // batch row, KV head, group of tiles
  int q0, qn, L;     // the row's first packed token, its tokens and its keys
  int beg, end;      // blocks [beg, end) of the unit's own numbering
  int kind;          // 0: the whole unit; 1 / 2: piece in the CTA's head / tail slot; -1: no more work
  int x, nb, per_cta;  // position of the unit's first block, its blocks, and the ranges' length
  int pad[4];
};
static_assert(sizeof(Segment) == 64, "descriptor slot");

// What the masks leave of a group of tiles: keys [0, sinks) and [low, hi),
// in blocks numbered without the gap between them.  Never less than one
// block, so that a group that sees no key still has a place in the work.
struct Span {
  int hi, low, ns, skip, nb;
  __device__ __forceinline__ int block(int v) const { return v < ns ? v : v + skip; }
};
template <int T>
__device__ __forceinline__ Span span_of(const PrefillArgs &a, int L, int qn, int t0, int t1) {
  Span s;
  const int p0 = L - qn + t0;  // position of the first token
  s.hi = a.causal ? max(0, min(L, L - qn + t1)) : L;
  const long long low = a.window > 0 ? (long long)p0 + 1 - a.window : 0;
  s.low = low > 0 ? (int)low : 0;
  const int first = s.low / T;
  s.ns = min((min(a.sinks, s.hi) + T - 1) / T, first);
  s.skip = first - s.ns;
  s.nb = max(1, (s.hi + T - 1) / T - s.skip);
  return s;
}

__device__ __forceinline__ void row_of(const PrefillArgs &a, int b, int &q0, int &qn, int &L) {
  const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], l = a.seqlens[b];
  const int s = min(max(c0, 0), a.total_q), e = min(max(c1, s), a.total_q);
  q0 = s;
  qn = min(e - s, a.max_q);
  L = min(max(l, 0), a.max_seqlen_k);
}

// Breaches of the call's contract by row b's inputs (clamped by row_of).
__device__ __forceinline__ void check_row(const PrefillArgs &a, int b) {
  const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], l = a.seqlens[b];
  int bad = 0;
  if (l < 0 || l > a.max_seqlen_k) bad |= kErrBadLen;
  if (c1 < c0 || (long long)c1 - c0 > a.max_q || (b == 0 && c0 != 0) || c1 > a.total_q)
    bad |= kErrBadOffsets;
  if (bad) atomicOr(a.err, bad);
}

// Place in the work: block `blk` of unit (b, h, it) is position x.
struct Walk {
  int b, h, it, tiles;
  int q0, qn, L;
  int blk, nb;
  int x, end, per_cta;
};

template <int D>
__device__ __forceinline__ Span walk_span(const PrefillArgs &a, const Walk &w) {
  constexpr int NT = Cfg<D>::NT;
  const int t0 = w.it * NT * a.TQ;
  return span_of<Cfg<D>::T>(a, w.L, w.qn, t0, min(t0 + NT * a.TQ, w.qn));
}

// The first row from b on that has queries (a.B: none), 32 rows at a time; one warp.
__device__ __forceinline__ int next_row(const PrefillArgs &a, int b, int lane) {
  for (; b < a.B; b += 32) {
    int q0, qn = 0, L;
    if (b + lane < a.B) row_of(a, b + lane, q0, qn, L);
    const unsigned some = __ballot_sync(0xffffffffu, qn > 0);
    if (some != 0) return b + __ffs(some) - 1;
  }
  return a.B;
}

// The segment at the walk, which moves past it and past the fixed cost of
// the unit that follows; one warp.
template <int D>
__device__ Segment walk_take(const PrefillArgs &a, Walk &w, int lane) {
  Segment s;
  const int len = min(w.nb - w.blk, w.end - w.x);
  s.b = w.b; s.h = w.h; s.it = w.it;
  s.q0 = w.q0; s.qn = w.qn; s.L = w.L;
  s.beg = w.blk;
  s.end = w.blk + len;
  s.kind = (s.beg == 0 && s.end == w.nb) ? 0 : s.beg > 0 ? 1 : 2;
  s.x = w.x - w.blk;
  s.nb = w.nb;
  s.per_cta = w.per_cta;
  w.x += len;
  w.blk += len;
  if (w.blk == w.nb && w.x < w.end) {
    w.blk = 0;
    if (++w.it == w.tiles) {
      w.it = 0;
      if (++w.h == a.Hkv) {
        w.h = 0;
        w.b = next_row(a, w.b + 1, lane);
        if (w.b == a.B) {
          w.x = w.end;
          return s;
        }
        row_of(a, w.b, w.q0, w.qn, w.L);
        w.tiles = (w.qn + Cfg<D>::NT * a.TQ - 1) / (Cfg<D>::NT * a.TQ);
      }
    }
    w.nb = walk_span<D>(a, w).nb;
    w.x += a.unit_cost;
  }
  return s;
}

// Positions of the groups of tiles first, first + step, ... of a row's units
// of one KV head.
template <int D>
__device__ __forceinline__ int positions_of(const PrefillArgs &a, int qn, int L, int first, int step) {
  const int tokens = Cfg<D>::NT * a.TQ;
  int sum = 0;
  for (int t0 = first * tokens; t0 < qn; t0 += step * tokens)
    sum += a.unit_cost + span_of<Cfg<D>::T>(a, L, qn, t0, min(t0 + tokens, qn)).nb;
  return sum;
}

// Positions of each of 32 rows, b + lane, of one KV head; one warp.  A lane
// counts its own row, and the warp together the rows of many groups.
template <int D>
__device__ __forceinline__ int row_positions(const PrefillArgs &a, int b, int lane) {
  int q0, qn = 0, L = 0;
  if (b + lane < a.B) row_of(a, b + lane, q0, qn, L);
  const bool many = qn > 8 * Cfg<D>::NT * a.TQ;
  int n = many ? 0 : positions_of<D>(a, qn, L, 0, 1);
  for (unsigned left = __ballot_sync(0xffffffffu, many); left != 0; left &= left - 1) {
    const int r = __ffs(left) - 1;
    int sum = positions_of<D>(a, __shfl_sync(0xffffffffu, qn, r), __shfl_sync(0xffffffffu, L, r), lane, 32);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == r) n = sum;
  }
  return n;
}

// This CTA's range, from the rows' positions (`rows`, of one KV head each, in
// shared memory); one warp.
template <int D>
__device__ Walk walk_start(const PrefillArgs &a, const int *rows, int lane) {
  constexpr int NT = Cfg<D>::NT;
  Walk w;
  w.b = w.h = w.it = w.tiles = w.q0 = w.qn = w.L = w.blk = w.nb = 0;
  w.x = w.end = 0;
  w.per_cta = 1;
  // Sums stop at the bound that total_q tokens cannot pass, so that they stay
  // in 32 bits whatever the offsets say.
  auto scan = [&](int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = min(v + u, a.max_positions + 1);
    }
    return v;
  };
  // each lane's share of the rows, then the lane and the row that hold x0
  const int chunk = (a.B + 31) / 32;
  const int lo = lane * chunk, hi = min(lo + chunk, a.B);
  int sum = 0;
  for (int i = lo; i < hi; ++i) sum = min(sum + rows[i], a.max_positions + 1);
  const int incl = scan(sum);
  const int all = __shfl_sync(0xffffffffu, incl, 31);
  // past the bound: rows overlap (check_row reports their offsets); nothing is run
  if (all == 0 || all > a.max_positions) return w;
  const int total = all * a.Hkv;
  w.per_cta = (total + (int)gridDim.x - 1) / (int)gridDim.x;
  const int x0 = blockIdx.x * w.per_cta;
  if (x0 >= total) return w;
  w.end = min(w.per_cta, total - x0) + x0;
  const int owner = __ffs(__ballot_sync(0xffffffffu, incl * a.Hkv > x0)) - 1;
  int pre = __shfl_sync(0xffffffffu, incl - sum, owner), width = 0;  // positions before the row, and its own
  for (int i = owner * chunk;; i += 32) {
    const int n = i + lane < min((owner + 1) * chunk, a.B) ? rows[i + lane] : 0, upto = pre + scan(n);
    const unsigned past = __ballot_sync(0xffffffffu, upto * a.Hkv > x0);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      w.b = i + l;
      width = __shfl_sync(0xffffffffu, n, l);
      pre = __shfl_sync(0xffffffffu, upto, l) - width;
      break;
    }
    pre = __shfl_sync(0xffffffffu, upto, 31);
  }
  row_of(a, w.b, w.q0, w.qn, w.L);
  w.tiles = (w.qn + NT * a.TQ - 1) / (NT * a.TQ);
  const int off = x0 - pre * a.Hkv;
  w.h = off / width;
  const int in_head = off - w.h * width;
  // the group of tiles that holds position in_head: scan them 32 at a time
  int before = 0;
  for (int i0 = 0;; i0 += 32) {
    const int it = i0 + lane, t0 = it * NT * a.TQ;
    const int c = it < w.tiles ? a.unit_cost + span_of<Cfg<D>::T>(a, w.L, w.qn, t0, min(t0 + NT * a.TQ, w.qn)).nb : 0;
    int upto = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    upto += before;
    const unsigned past = __ballot_sync(0xffffffffu, upto > in_head);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      w.it = i0 + l;
      w.nb = __shfl_sync(0xffffffffu, c, l) - a.unit_cost;
      const int start = __shfl_sync(0xffffffffu, upto - c, l);
      const int pos = in_head - start;
      w.blk = pos > a.unit_cost ? pos - a.unit_cost : 0;
      w.x = x0 - pos + a.unit_cost + w.blk;
      break;
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
    if (i0 + 32 >= w.tiles) break;  // not reached: in_head < width
  }
  if (w.x > w.end) w.x = w.end;  // the range ends inside the unit's fixed cost
  return w;
}

// Bounded wait of every lane of a warp for the phase of `bar` with this
// parity; false when it has run out (the role then ends, and its warp records
// the failure).  Few instructions, since every wait is a copy of them.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
  bool done = mbar_try_wait(bar, parity);
  if (!done) {
    uint32_t t0, t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
    do {
      done = mbar_try_wait(bar, parity);
      asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    } while (!done && t - t0 < (uint32_t)kWaitLimitNs);
  }
  return __all_sync(0xffffffffu, done);
}

// ---------------------------------------------------------------------------
// Loading warps: one finds the CTA's share, publishes its segments and loads
// their keys; the other loads each segment's queries, once the unit before has
// issued its last scores, and its values.  Two, because issuing is what bounds
// them: a box takes a warp 50 to 120 cycles whatever its size, and at 16 tokens
// a page a single warp set the pace of the whole kernel (3200 cycles a block
// at D = 64).
// ---------------------------------------------------------------------------
template <int D>
__device__ bool loader(const PrefillMaps &tm, const PrefillArgs &a, uint8_t *smem, bool values, int lane) {
  using C = Cfg<D>;
  constexpr int T = C::T, NT = C::NT;
  const uint32_t sbase = smem_addr(smem), bars = sbase + C::kBarOff;
  Segment *descs = reinterpret_cast<Segment *>(smem + C::kDescOff);
  Walk w;
  if (!values) {
    w = walk_start<D>(a, reinterpret_cast<int *>(smem), lane);
    fence_proxy_async_smem();  // the scan's accesses precede the ring's loads
    __syncwarp();
  }
  const void *map = values ? (const void *)&tm.kv.v : (const void *)&tm.kv.k;
  const int bt = a.box_tokens, ps = a.page_size;
  const int pages = T / ps, rest = T % ps;  // a block's length in pages
  const bool has_box = lane < T / bt;       // this lane has box `lane` of a block
  int slot = values ? 1 : 0, phase = 1;     // ring slot of the next block, and the phase that frees it
  int loaded = 0, asked = 0, seg_n = 0;     // blocks and units' queries on their way
  bool ok = true, bad_page = false;
  auto page_of = [&](int b, int p) { return has_box && p < a.mpps ? a.block_table[(size_t)b * a.mpps + p] : -1; };
  for (;; ++seg_n) {
    const int d = seg_n % kDescs;
    Segment s;
    if (!values) {
      if (w.x < w.end) s = walk_take<D>(a, w, lane);
      else s.kind = -1;
      if (!(ok = wait_phase(bars + 8 * (C::B_DEMPTY + d), ((seg_n / kDescs) & 1) ^ 1))) break;
      if (lane == 0) {
        descs[d] = s;
        mbar_arrive(bars + 8 * (C::B_DFULL + d));
      }
      __syncwarp();
    } else {
      if (!(ok = wait_phase(bars + 8 * (C::B_DFULL + d), (seg_n / kDescs) & 1))) break;
      s = descs[d];
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (C::B_DEMPTY + d));
    }
    if (s.kind < 0) break;
    const int t0 = s.it * NT * a.TQ;
    const Span span = span_of<T>(a, s.L, s.qn, t0, min(t0 + NT * a.TQ, s.qn));
    // place of this lane's box: entry p of the row's table, token `off` of the page
    int p = 0, off = 0, page = 0;
    auto seek = [&](int blk) {
      const int tok = span.block(blk) * T + lane * bt;
      p = tok / ps;
      off = tok - p * ps;
    };
    if (!a.contiguous) {
      seek(s.beg);
      page = page_of(s.b, p);
    }
    if (values) {
      if (!(ok = wait_phase(bars + 8 * C::B_QEMPTY, (seg_n & 1) ^ 1))) break;
      const int tiles = min(NT, (s.qn - t0 + a.TQ - 1) / a.TQ);
      if (lane == 0) mbar_arrive_expect_tx(bars + 8 * C::B_QFULL, (uint32_t)(tiles * C::CH * a.TQ * a.G * 128));
      __syncwarp();
      if (lane < tiles * C::CH) {
        const int t = lane / C::CH, ch = lane % C::CH;
        tma_load_3d(sbase + C::kQOff + t * C::kQBytes + ch * (kTileRows * 128), &tm.q, ch * 64, s.h * a.G,
                    s.q0 + t0 + t * a.TQ, bars + 8 * C::B_QFULL);
      }
      ++asked;
    }
    for (int blk = s.beg; blk < s.end; ++blk) {
      const int tok0 = span.block(blk) * T, tok = tok0 + lane * bt;
      const int valid = max(0, min(T, span.hi - tok0));
      const int nbox = (valid + bt - 1) / bt;
      int row = s.b * ps + tok;
      if (!a.contiguous) {
        // A box of hidden keys only is never read, whatever its table entry
        // holds; a page outside the pool reads as zeros and is reported.
        // Both are placed at negative rows, which the map fills with zeros.
        const bool hidden = tok >= a.sinks && tok + bt <= span.low;
        const bool there = !hidden && page >= 0 && page < a.num_pages;
        bad_page |= !hidden && !there && lane < nbox;
        row = (there ? page * ps : -ps) + off;
        // the next block's page is on its way while this block is issued; the
        // places step on without a division
        if (blk + 1 < s.end) {
          if (blk + 1 == span.ns) {
            seek(blk + 1);
          } else {
            p += pages;
            off += rest;
            if (off >= ps) {
              off -= ps;
              ++p;
            }
          }
          page = page_of(s.b, p);
        }
      }
      const uint32_t full = bars + 8 * (C::B_FULL + slot);
      if (!(ok = wait_phase(bars + 8 * (C::B_EMPTY + slot), phase))) break;
      if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(nbox * bt * D * 2));
      __syncwarp();
      if (lane < nbox) {
        const uint32_t dst = sbase + slot * C::kSlotBytes + lane * (bt / 8) * C::kGroupBytes;
        if (a.grouped) {
          tma_load_4d(dst, map, 0, 0, s.h * C::CH, row >> 3, full);
        } else {
#pragma unroll 1
          for (int ch = 0; ch < C::CH; ++ch) tma_load_3d(dst + ch * 1024, map, ch * 64, s.h, row, full);
        }
      }
      ++loaded;
      slot += 2;
      if (slot >= C::kSlots) {
        slot -= C::kSlots;
        phase ^= 1;
      }
    }
    if (!ok) break;
  }
  if (__any_sync(0xffffffffu, bad_page) && lane == 0) atomicOr(a.err, kErrBadPage);
  // Leave only when the copies issued here have landed.
  for (int j = max(0, loaded - C::kSlots / 2); j < loaded; ++j)
    ok &= wait_phase(bars + 8 * (C::B_FULL + 2 * (j % (C::kSlots / 2)) + (values ? 1 : 0)), (j / (C::kSlots / 2)) & 1);
  if (asked > 0) ok &= wait_phase(bars + 8 * C::B_QFULL, (asked - 1) & 1);
  return ok;
}

// Keys of the block at tok0 that some query of the unit may see, as the
// 16-key steps [k0, k1) of the product with V; hidden keys inside them, [top,
// ..) and [g0, g1), get zeros for values, so that 0 * V stays 0 whatever the
// cache holds there.
struct Steps {
  int top, g0, g1, k0, k1;
  bool clear;
};
template <int T>
__device__ __forceinline__ Steps steps_of(const PrefillArgs &a, const Span &span, int tok0) {
  Steps s;
  s.top = max(0, min(T, span.hi - tok0));
  s.g0 = max(0, min(T, a.sinks - tok0));
  s.g1 = max(s.g0, min(s.top, span.low - tok0));
  s.k0 = s.g0 == 0 ? s.g1 / 16 : 0;
  s.k1 = (s.top + 15) / 16;
  s.clear = s.g1 > s.g0 || s.top % 16 != 0;
  return s;
}

// ---------------------------------------------------------------------------
// Issuing warps: one for the scores and one for the values, so that one's
// waits and bookkeeping pass while the other's products run (a single warp
// spent as long on them as the tensor cores on its products).  All lanes of a
// warp walk through the work together, on values that the compiler can see
// to be the same in all of them, and one elected lane issues: the operands of
// tcgen05.mma are then in uniform registers already (a lane alone in the role
// moved five operands there for every product, and issued one in 65 cycles
// whatever its size).
// ---------------------------------------------------------------------------

// The next segment, for a whole warp; kind < 0: none.
struct Work {
  int kind, n, tiles, beg;
  Span span;
};
template <int D>
__device__ __forceinline__ bool take_segment(const PrefillArgs &a, uint8_t *smem, int seg_n, int lane, Work &w) {
  using C = Cfg<D>;
  const uint32_t bars = smem_addr(smem) + C::kBarOff;
  const int d = seg_n % kDescs;
  if (!wait_phase(bars + 8 * (C::B_DFULL + d), (seg_n / kDescs) & 1)) return false;
  const Segment *s = reinterpret_cast<const Segment *>(smem + C::kDescOff) + d;
  w.kind = __shfl_sync(0xffffffffu, s->kind, 0);
  const int it = __shfl_sync(0xffffffffu, s->it, 0), qn = __shfl_sync(0xffffffffu, s->qn, 0);
  const int L = __shfl_sync(0xffffffffu, s->L, 0);
  w.beg = __shfl_sync(0xffffffffu, s->beg, 0);
  w.n = __shfl_sync(0xffffffffu, s->end, 0) - w.beg;
  if (lane == 0) mbar_arrive(bars + 8 * (C::B_DEMPTY + d));
  const int t0 = it * C::NT * a.TQ;
  w.tiles = min(C::NT, (qn - t0 + a.TQ - 1) / a.TQ);
  w.span = span_of<C::T>(a, L, qn, t0, min(t0 + C::NT * a.TQ, qn));
  return true;
}

// S = Q_t K^T of every block and tile, once the scores before them in the
// buffer are in registers: a tile's next scores wait in tensor memory while
// its softmax works on a block.
template <int D, bool kBf16>
__device__ bool issue_scores(const PrefillArgs &a, uint8_t *smem, uint32_t tmem, int lane) {
  using C = Cfg<D>;
  constexpr int T = C::T, NT = C::NT;
  constexpr uint32_t kHi = smem_desc_hi(1024), kHiKV = smem_desc_hi(C::kGroupBytes);
  // a negative scale becomes positive with Q negated
  const uint32_t idesc = mma_idesc<kBf16>(kTileRows, T, false) | (a.scale_log2 < 0.f ? kIdescNegateA : 0u);
  const uint32_t sbase = smem_addr(smem), bars = sbase + C::kBarOff;
  const uint32_t q_lo = smem_desc_lo(sbase + C::kQOff, 16);
  int slot = 0, phase = 0;  // ring slot of the next keys, and its phase
  // blocks issued, by barrier: with two tiles those of each tile, with one
  // tile the even and the odd ones
  int s_n[2] = {0, 0};
  int last = 0;  // the tile (or parity) whose scores were issued last
  auto wait = [&](int bar, int n) { return wait_phase(bars + 8 * bar, n & 1); };
  Work w;
  for (int seg_n = 0;; ++seg_n) {
    if (!take_segment<D>(a, smem, seg_n, lane, w)) return false;
    if (w.kind < 0) return true;
    if (!wait(C::kQTmem ? C::B_QREADY : C::B_QFULL, seg_n)) return false;
    if (C::kQTmem) tc_fence_after();
    for (int j = 0; j < w.n; ++j) {
      if (!wait(C::B_FULL + slot, phase)) return false;
      const uint32_t k = smem_desc_lo(sbase + slot * C::kSlotBytes, 16);
      for (int t = 0; t < w.tiles; ++t) {
        const int i = NT == 2 ? t : (s_n[0] + s_n[1]) & 1;
        if (s_n[last] > 0 && !wait(C::B_SFREE + last, s_n[last] - 1)) return false;
        tc_fence_after();
        const uint32_t q = q_lo + t * (C::kQBytes / 16);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t kd = k + (kk / 4) * 64 + (kk % 4) * 2;
            if constexpr (C::kQTmem) mma_ts<kHiKV>(tmem, tmem + C::kQCol + kk * 8, kd, idesc, kk > 0);
            else mma_ss<kHi, kHiKV>(tmem, q + (kk / 4) * (kTileRows * 8) + (kk % 4) * 2, kd, idesc, kk > 0);
          }
          mma_commit(bars + 8 * (C::B_SFULL + i));
          if (t + 1 == w.tiles) {
            mma_commit(bars + 8 * (C::B_EMPTY + slot));
            if (!C::kQTmem && j + 1 == w.n) mma_commit(bars + 8 * C::B_QEMPTY);
          }
        }
        __syncwarp();
        ++s_n[i];
        last = i;
      }
      slot += 2;  // past the block's values
      if (slot >= C::kSlots) {
        slot -= C::kSlots;
        phase ^= 1;
      }
    }
  }
}

// O_t += P V of every block and tile, over the 16-key steps that some query sees.
template <int D, bool kBf16>
__device__ bool issue_values(const PrefillArgs &a, uint8_t *smem, uint32_t tmem, int lane) {
  using C = Cfg<D>;
  constexpr int T = C::T, NT = C::NT;
  constexpr uint32_t kHi = smem_desc_hi(C::kGroupBytes);
  constexpr uint32_t kStep = 2 * C::kGroupBytes / 16;  // 16 keys
  constexpr uint32_t kIdesc = mma_idesc<kBf16>(kTileRows, D, true);
  const uint32_t sbase = smem_addr(smem), bars = sbase + C::kBarOff;
  int slot = 1, phase = 0;  // ring slot of the next values, and its phase
  int p_n[2] = {0, 0};      // blocks issued, by barrier as for the scores
  auto wait = [&](int bar, int n) { return wait_phase(bars + 8 * bar, n & 1); };
  Work w;
  for (int seg_n = 0;; ++seg_n) {
    if (!take_segment<D>(a, smem, seg_n, lane, w)) return false;
    if (w.kind < 0) return true;
    for (int j = 0; j < w.n; ++j) {
      const Steps st = steps_of<T>(a, w.span, w.span.block(w.beg + j) * T);
      if (!wait(C::B_FULL + slot, phase)) return false;
      const uint32_t v = smem_desc_lo(sbase + slot * C::kSlotBytes, 1024);
      for (int t = 0; t < w.tiles; ++t) {
        const int i = NT == 2 ? t : (p_n[0] + p_n[1]) & 1;
        const uint32_t o = tmem + C::kOCol + t * D, p = tmem + C::kPCol + i * (T / 2);
        if (!wait(C::B_PREADY + i, p_n[i])) return false;
        tc_fence_after();
        if (elect_one()) {
          if (st.k0 == 0 && st.k1 == T / 16) {
#pragma unroll
            for (int kk = 0; kk < T / 16; ++kk) mma_ts<kHi>(o, p + kk * 8, v + kk * kStep, kIdesc, kk > 0 || j > 0);
          } else {
            for (int kk = st.k0; kk < st.k1; ++kk) mma_ts<kHi>(o, p + kk * 8, v + kk * kStep, kIdesc, kk > st.k0 || j > 0);
          }
          mma_commit(bars + 8 * (C::B_OFULL + i));
          if (t + 1 == w.tiles) mma_commit(bars + 8 * (C::B_EMPTY + slot));
        }
        __syncwarp();
        ++p_n[i];
      }
      slot += 2;
      if (slot >= C::kSlots) {
        slot -= C::kSlots;
        phase ^= 1;
      }
    }
  }
}

// 32 bytes to global memory: one store where the address allows it.
__device__ __forceinline__ void store_sector(void *p, const uint32_t *w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(__cvta_generic_to_global(p)), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// n ones from bit 0 up, for any n.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// ---------------------------------------------------------------------------
// Softmax warps: a thread has row r of tile t.
// ---------------------------------------------------------------------------
template <int D, bool kBf16>
__device__ bool softmax(const PrefillArgs &a, uint8_t *smem, uint32_t tmem, int t, int warp, int lane) {
  using C = Cfg<D>;
  constexpr int T = C::T, NT = C::NT;
  const uint32_t sbase = smem_addr(smem), bars = sbase + C::kBarOff;
  const Segment *descs = reinterpret_cast<const Segment *>(smem + C::kDescOff);
  const int r = warp * 32 + lane;                        // row of the tile:
  const int r_tok = r / a.G, r_head = r - r_tok * a.G;   // its token and head
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;    // this warp's lanes of tensor memory
  const uint32_t o_addr = tmem + lanes + C::kOCol + t * D;
  // The issuing warp has negated the scores for a negative scale.  A zero scale
  // becomes one that leaves nothing of a score, since -inf marks a masked one.
  const float sl2 = fmaxf(fabsf(a.scale_log2), 1e-30f);
  int seg_n = 0, blk_n = 0;   // segments and score blocks seen
  int slot_n = 1;             // ring slot, of all so far, that holds the current block's values
  auto wait = [&](int bar, int n) { return wait_phase(bars + 8 * bar, n & 1); };
  for (;;) {
    const int d = seg_n % kDescs;
    if (!wait(C::B_DFULL + d, seg_n / kDescs)) return false;
    // The slot is kept until the unit is done: what the loop over the blocks
    // does not need is read again from it, not held in registers.
    const volatile Segment &s = descs[d];
    auto done = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (C::B_DEMPTY + d));
      ++seg_n;
    };
    if (s.kind < 0) {
      done();
      return true;
    }
    const int blk_beg = s.beg, blk_end = s.end, L = s.L, qn = s.qn;
    const int u0 = s.it * NT * a.TQ, tt0 = u0 + t * a.TQ;  // first token of the unit and of this tile
    if (tt0 >= qn) {                                        // the unit's second tile is empty
      slot_n += 2 * (blk_end - blk_beg);
      done();
      continue;
    }
    const Span span = span_of<T>(a, L, qn, u0, min(u0 + NT * a.TQ, qn));
    // keys this row sees: [0, sinks) and [low, lim)
    int lim = a.causal ? min(L, L - qn + tt0 + r_tok + 1) : L;
    if (r_tok >= a.TQ || tt0 + r_tok >= qn) lim = 0;
    const int low = a.window > 0 ? max(lim - a.window, 0) : 0;
    // a block lies at an edge unless every row of the tile sees all of it;
    // one whose values need clearing always does: its hidden keys lie past
    // every row's, or before every row's window
    const int tile_lim = a.causal ? L - qn + tt0 + 1 : L;
    const int tile_low = a.window > 0 ? L - qn + min(tt0 + a.TQ, qn) - a.window : 0;

    if constexpr (C::kQTmem) {
      // This row's queries go to tensor memory; the scores of the unit before
      // have been seen, so its queries are done with.
      if (!wait(C::B_QFULL, seg_n)) return false;
#pragma unroll 1
      for (int ch = 0; ch < C::CH; ++ch) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4 *>(w + 4 * i) =
              *reinterpret_cast<const uint4 *>(smem + C::kQOff + ch * (kTileRows * 128) + r * 128 + ((i ^ (r & 7)) << 4));
        tmem_st16(tmem + lanes + C::kQCol + ch * 32, w);
        tmem_st16(tmem + lanes + C::kQCol + ch * 32 + 16, w + 16);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bars + 8 * C::B_QREADY);
        mbar_arrive(bars + 8 * C::B_QEMPTY);
      }
    }

    float m = -INFINITY, l = 0.f;  // running maximum (base 2, scaled) and sum
    for (int blk = blk_beg; blk < blk_end; ++blk) {
      // barriers: the tile's, or with one tile those of the block's parity
      const int u = NT == 2 ? t : blk_n & 1, un = NT == 2 ? blk_n : blk_n >> 1;
      if (!wait(C::B_SFULL + u, un)) return false;
      tc_fence_after();
      ++blk_n;
      const uint32_t s_addr = tmem + lanes;
      float x[T];
#pragma unroll
      for (int c = 0; c < T; c += 32) tmem_ld32(s_addr + c, reinterpret_cast<uint32_t *>(x + c));
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (C::B_SFREE + u));
      const int j0 = span.block(blk) * T;
      if (j0 + T > tile_lim || (j0 < tile_low && j0 + T > a.sinks)) {
        // one bit a key: seen or not; most groups of 32 are seen whole
#pragma unroll
        for (int c = 0; c < T; c += 32) {
          const int j = j0 + c;
          const uint32_t seen = bits_below(lim - j) & (~bits_below(low - j) | bits_below(a.sinks - j));
          if (__any_sync(0xffffffffu, seen != 0xffffffffu)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[c + i] = (seen >> i) & 1u ? x[c + i] : -INFINITY;
          }
        }
        if (t == 0) {
          const int b0 = s.it * NT * a.TQ;
          const Steps st = steps_of<T>(a, span_of<T>(a, s.L, s.qn, b0, min(b0 + NT * a.TQ, (int)s.qn)), j0);
          if (st.clear) {  // values of hidden keys, [g0, g1) and [top, ..) of the steps, become zeros
            const int sl = slot_n % C::kSlots;
            if (!wait(C::B_FULL + sl, slot_n / C::kSlots)) return false;
            const uint32_t v = sbase + sl * C::kSlotBytes;
            const int from = max(st.g0, st.k0 * 16), gap = max(0, st.g1 - from), keys = gap + st.k1 * 16 - st.top;
#pragma unroll 1
            for (int i = r; i < keys * (D / 8); i += kTileRows) {
              const int n = i / (D / 8), c = i % (D / 8), key = n < gap ? from + n : st.top + n - gap;
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + (key / 8) * C::kGroupBytes + (c / 8) * 1024 + (key % 8) * 128 + (c % 8) * 16),
                           "r"(0u) : "memory");
            }
            fence_proxy_async_smem();  // before the product reads them
            __syncwarp();
          }
        }
      }
      slot_n += 2;
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int i = 4; i < T; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], x[i], x[i + 1]);
      const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sl2;
      // The reference m follows the maximum only once it is 2^8 behind, so
      // the accumulator is hardly ever rescaled; weights stay below 2^8.
      const bool behind = top > m + 8.f || (m == -INFINITY && top > -INFINITY);
      if (__any_sync(0xffffffffu, behind)) {
        const float mn = fmaxf(m, top);
        const float alpha = m == mn ? 1.f : ex2(m - mn);
        m = mn;
        l *= alpha;
        if (blk > blk_beg) {
          // the values of the block before are in the accumulator
          const int pu = NT == 2 ? t : u ^ 1, pn = NT == 2 ? un - 1 : (blk_n - 2) >> 1;
          if (!wait(C::B_OFULL + pu, pn)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tmem_ld16(o_addr + c, reinterpret_cast<uint32_t *>(o));
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tmem_st16(o_addr + c, reinterpret_cast<uint32_t *>(o));
          }
        }
      }
      // Weights 2^(scale x - m), rounded to the input type, two in a word: the
      // tensor core takes them in the type of V.  Two words for a weight, as the
      // decode kernel has, would double the products with V (half as much again
      // for the tensor cores, more cycles than the 2650 that a block of two tiles
      // takes at D = 128).  Their sum is taken before the rounding.
      const float base = m == -INFINITY ? 0.f : -m;
      const float2 sc = make_float2(sl2, sl2), bs = make_float2(base, base);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      // Once the product that read the buffer's weights before is done, they go
      // out 32 at a time, beside the exponentials of the next.
      if (un > 0 && !wait(C::B_OFULL + u, un - 1)) return false;
      tc_fence_after();
      const uint32_t p_addr = tmem + lanes + C::kPCol + u * (T / 2);
      uint32_t p[T / 2];
#pragma unroll
      for (int i = 0; i < T; i += 2) {
        float2 e = fma2(make_float2(x[i], x[i + 1]), sc, bs);
        e.x = ex2(e.x);
        e.y = ex2(e.y);
        sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], e);
        p[i >> 1] = pack2<kBf16>(e.x, e.y);
        if (i % 32 == 30) tmem_st16(p_addr + (i >> 1) - 15, p + (i >> 1) - 15);
      }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (C::B_PREADY + u));
    }

    // ---- the rows: O / l and LSE ----
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int hq = s.h * a.G + r_head, v0 = s.it * NT * a.TQ, tok = v0 + t * a.TQ + r_tok;
    const bool real = r_tok < a.TQ && tok < s.qn;
    // Where the row goes: row `row` of the output, or of the CTA's piece slot.
    const int row0 = s.kind == 0 ? (s.q0 + tok) * a.Hq + hq
                                 : (blockIdx.x * 2 + (s.kind - 1)) * (NT * kTileRows) + t * kTileRows + r;
    if (real) {
      const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      if (s.kind != 0) a.lse_part[row0] = lse;
      else if (a.lse != nullptr) a.lse[(size_t)hq * a.total_q + s.q0 + tok] = lse;
    }
    // the head piece's description, for the merge
    if (s.kind == 1 && t == 0 && r == 0) {
      PieceDesc &pd = a.pieces[blockIdx.x];
      pd.q0 = s.q0;
      pd.h = s.h;
      pd.t0 = v0;
      pd.tokens = min(NT * a.TQ, s.qn - v0);
      pd.c_first = s.x / s.per_cta;
      pd.n_pieces = (s.x + s.nb - 1) / s.per_cta - pd.c_first + 1;
    }
    const int lu = NT == 2 ? t : (blk_n - 1) & 1;  // the last block's values
    if (!wait(C::B_OFULL + lu, NT == 2 ? blk_n - 1 : (blk_n - 1) >> 1)) return false;
    tc_fence_after();
    // A lane writes its row, 32 bytes in a store: whole sectors, without
    // a detour through shared memory.  A short loop: code that runs once a unit
    // is fetched anew.
    const bool piece = s.kind != 0;
    uint8_t *dst = piece ? reinterpret_cast<uint8_t *>(a.o_part + (size_t)row0 * D)
                         : static_cast<uint8_t *>(a.out) + (size_t)row0 * D * 2;
#pragma unroll 1
    for (int col = 0; col < D; col += 32) {
      float o[32];
      tmem_ld32(o_addr + col, reinterpret_cast<uint32_t *>(o));
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : o[i] * inv;  // no key: O holds nothing to read
      if (real) {
        if (piece) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) store_sector(dst + (col + i) * 4, reinterpret_cast<const uint32_t *>(o + i), true);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack2<kBf16>(o[2 * i], o[2 * i + 1]);
#pragma unroll
          for (int i = 0; i < 16; i += 8) store_sector(dst + (col + 2 * i) * 2, w + i, a.wide_out);
        }
      }
      __syncwarp();  // the next load wants the whole warp
    }
    tc_fence_before();  // the accumulator has been read before this thread's next arrival
    done();
  }
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    prefill_kernel(const __grid_constant__ PrefillMaps tm, const __grid_constant__ PrefillArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bars = smem_addr(smem) + C::kBarOff;
  const uint32_t tmem_slot = bars + 8 * C::B_COUNT;
  if ((smem_addr(smem) & 1023u) != 0) {  // the swizzle needs 1024-byte aligned slots
    if (tid == 0) atomicOr(a.err, kErrAlign);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(bars + 8 * (C::B_FULL + i), 1);
      mbar_init(bars + 8 * (C::B_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 8 * (C::B_SFULL + i), 1);
      mbar_init(bars + 8 * (C::B_SFREE + i), 4);  // one arrival a softmax warp of the tile
      mbar_init(bars + 8 * (C::B_PREADY + i), 4);
      mbar_init(bars + 8 * (C::B_OFULL + i), 1);
    }
    mbar_init(bars + 8 * C::B_QFULL, 1);
    mbar_init(bars + 8 * C::B_QEMPTY, C::kQTmem ? 4 : 1);
    mbar_init(bars + 8 * C::B_QREADY, 4);
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(bars + 8 * (C::B_DFULL + i), 1);
      mbar_init(bars + 8 * (C::B_DEMPTY + i), C::kSoftmaxWarps + 3);
    }
    fence_mbar_init();
  }
  if (warp == C::kScoreWarp) tmem_alloc(tmem_slot, 512);
  if (tid == 32 * C::kKeyWarp) {
    prefetch_tmap(&tm.kv.k);
    prefetch_tmap(&tm.kv.v);
    prefetch_tmap(&tm.q);
  }
  grid_launch_dependents();
  // Inputs may be written, and outputs and workspace used, by the kernel
  // this launch depends on.
  grid_dependency_wait();
  // the rows' positions, for the key warp's scan (the ring is still unused)
  int *rows = reinterpret_cast<int *>(smem);
  for (int b = warp * 32; b < a.B; b += C::kThreads) {
    const int n = row_positions<D>(a, b, lane);
    if (b + lane < a.B) {
      rows[b + lane] = n;
      if ((b + lane) % (int)gridDim.x == (int)blockIdx.x) check_row(a, b + lane);
    }
  }
  if (tid == 0) a.pieces[blockIdx.x].n_pieces = 0;  // until a head piece says otherwise
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
  tmem = __shfl_sync(0xffffffffu, tmem, 0);
  bool ok;
  if (warp >= C::kSoftmaxWarps) {
    if constexpr (C::NT == 2) regs_dec<72>();  // 168 a thread at launch: 384 x 168 = 256 x 216 + 128 x 72
    if (warp == C::kScoreWarp) ok = issue_scores<D, kBf16>(a, smem, tmem, lane);
    else if (warp == C::kValueWarp) ok = issue_values<D, kBf16>(a, smem, tmem, lane);
    else ok = loader<D>(tm, a, smem, warp != C::kKeyWarp, lane);
  } else {
    if constexpr (C::NT == 2) regs_inc<216>();
    ok = softmax<D, kBf16>(a, smem, tmem, warp / 4, warp % 4, lane);
  }
  if (!ok && lane == 0) atomicOr(a.err, kErrWaitFull);  // a wait ran out
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kScoreWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Merge of the units that ranges cut: cut i (between CTAs i - 1 and i) of a
// unit with n pieces takes the (i - c_first)-th share of its rows, and
// blockIdx.y a part of that: four rows a warp where a unit has two pieces.  A
// row is a chain of a few dependent loads, and the pieces of a full grid are 38
// MB at D = 128, read from L2: with two rows of up to kFewPieces pieces on
// their way at once two windowed prompts take 104 us, one row after the other
// 110.  Merging in the attention kernel, by the last piece to arrive, was
// slower (114 us: a few warps wait where this kernel has them by the hundred).
//   LSE = ln sum_p exp(lse_p),   O = sum_p exp(lse_p - LSE) O_p
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 128, kMergeParts = 16, kFewPieces = 3;
template <int D, bool kBf16>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ PrefillArgs a) {
  constexpr int NT = Cfg<D>::NT;
  constexpr float kLog2e = 1.4426950408889634f;
  grid_launch_dependents();
  grid_dependency_wait();
  const int cta = blockIdx.x + 1;
  const PieceDesc pd = a.pieces[cta];
  const int n = pd.n_pieces;
  if (n < 2) return;
  const int lane = threadIdx.x & 31;
  const int rows = pd.tokens * a.G;
  constexpr int kWarps = kMergeThreads / 32;
  const int parts = (n - 1) * gridDim.y * kWarps;
  const int part = ((cta - pd.c_first - 1) * gridDim.y + blockIdx.y) * kWarps + (threadIdx.x >> 5);
  const int beg = (int)((long long)rows * part / parts), end = (int)((long long)rows * (part + 1) / parts);
  auto slot_of = [&](int i) -> size_t { return i == 0 ? (size_t)pd.c_first * 2 + 1 : (size_t)(pd.c_first + i) * 2; };
  if (n <= kFewPieces) {
    // two rows at once, every load on its way before the first is used
    for (int m = beg; m < end; m += 2) {
      float lp[2][kFewPieces], lse2[2];
      float4 v[2][kFewPieces][D > 128 ? 2 : 1];
      size_t at[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int mi = min(m + i, end - 1), tok = mi / a.G, g = mi - tok * a.G;
        const int row = (tok / a.TQ) * kTileRows + (tok % a.TQ) * a.G + g;
        at[i] = (size_t)(pd.q0 + pd.t0 + tok) * a.Hq + pd.h * a.G + g;
#pragma unroll
        for (int p = 0; p < kFewPieces; ++p) {
          const size_t pr = slot_of(min(p, n - 1)) * (NT * kTileRows) + row;
          lp[i][p] = p < n ? a.lse_part[pr] * kLog2e : -INFINITY;
#pragma unroll
          for (int k = 0; k < (D > 128 ? 2 : 1); ++k)
            v[i][p][k] = p < n && lane * 4 < D ? *reinterpret_cast<const float4 *>(a.o_part + pr * D + k * 128 + lane * 4)
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (m + i >= end) break;
        float mx = -INFINITY, sum = 0.f;
#pragma unroll
        for (int p = 0; p < kFewPieces; ++p) mx = fmaxf(mx, lp[i][p]);
        if (mx == -INFINITY) mx = 0.f;  // no piece saw a key, or all hold NaN, which stays
#pragma unroll
        for (int p = 0; p < kFewPieces; ++p) sum += ex2(lp[i][p] - mx);
        lse2[i] = sum == 0.f ? -INFINITY : mx + log2f(sum);
        if (lane == 0 && a.lse != nullptr)
          a.lse[(at[i] % a.Hq) * a.total_q + at[i] / a.Hq] = lse2[i] * kLn2;
#pragma unroll
        for (int k = 0; k < (D > 128 ? 2 : 1); ++k) {
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int p = 0; p < kFewPieces; ++p) {
            const float wgt = lp[i][p] == -INFINITY ? 0.f : ex2(lp[i][p] - lse2[i]);
            acc.x += wgt * v[i][p][k].x; acc.y += wgt * v[i][p][k].y;
            acc.z += wgt * v[i][p][k].z; acc.w += wgt * v[i][p][k].w;
          }
          if (lane * 4 < D)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at[i] * D + k * 128 + lane * 4) =
                make_uint2(pack2<kBf16>(acc.x, acc.y), pack2<kBf16>(acc.z, acc.w));
        }
      }
    }
    return;
  }
  for (int m = beg; m < end; ++m) {
    const int tok = m / a.G, g = m % a.G;
    const int row = (tok / a.TQ) * kTileRows + (tok % a.TQ) * a.G + g;  // of the unit's tiles
    float mx = -INFINITY;
    for (int p = lane; p < n; p += 32) mx = fmaxf(mx, a.lse_part[slot_of(p) * (NT * kTileRows) + row] * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float sum = 0.f;
    if (mx == -INFINITY) mx = 0.f;
    for (int p = lane; p < n; p += 32) sum += ex2(a.lse_part[slot_of(p) * (NT * kTileRows) + row] * kLog2e - mx);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float lse2 = sum == 0.f ? -INFINITY : mx + log2f(sum);  // NaN stays
    const int hq = pd.h * a.G + g, token = pd.q0 + pd.t0 + tok;
    if (lane == 0 && a.lse != nullptr) a.lse[(size_t)hq * a.total_q + token] = lse2 * kLn2;
    for (int c = lane * 4; c < D; c += 128) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int p = 0; p < n; ++p) {
        const size_t pr = slot_of(p) * (NT * kTileRows) + row;
        const float lp = a.lse_part[pr];
        const float wgt = lp == -INFINITY ? 0.f : ex2(lp * kLog2e - lse2);
        const float4 v = *reinterpret_cast<const float4 *>(a.o_part + pr * D + c);
        acc.x += wgt * v.x; acc.y += wgt * v.y; acc.z += wgt * v.z; acc.w += wgt * v.w;
      }
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + ((size_t)token * a.Hq + hq) * D + c) =
          make_uint2(pack2<kBf16>(acc.x, acc.y), pack2<kBf16>(acc.z, acc.w));
    }
  }
}

// 4-D map {64 elements, 8 tokens, Hkv * D / 64 chunks, groups of 8 tokens} of a K
// or V pool; box {64, 8, D / 64, box_tokens / 8}: whole keys of one head, in
// the layout of a block in shared memory.  One box a page brings 2 to 4 times
// fewer TMA operations than boxes of one chunk, which small pages are bound
// by.
bool encode_grouped_kv_map(CUtensorMap *m, const void *base, int D, int Hkv, long long pool_tokens, int box_tokens,
                           bool bf16) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t token = (cuuint64_t)Hkv * D * 2;
  cuuint64_t dims[4] = {64, 8, (cuuint64_t)Hkv * (D / 64), (cuuint64_t)(pool_tokens / 8)};
  cuuint64_t strides[3] = {token, 128, 8 * token};
  cuuint32_t box[4] = {64u, 8u, (cuuint32_t)(D / 64), (cuuint32_t)(box_tokens / 8)};
  cuuint32_t estride[4] = {1u, 1u, 1u, 1u};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void *>(base), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B,
             D >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map {D, Hq, tokens} of the packed queries; box {64, G, TQ}: one tile's
// packed rows of one 64-column chunk, 128-byte swizzle.
bool encode_q_map(CUtensorMap *m, const void *q, int D, int Hq, int total_q, int G, int TQ, bool bf16) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)total_q};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)Hq * D * 2};
  cuuint32_t box[3] = {64u, (cuuint32_t)G, (cuuint32_t)TQ};
  cuuint32_t estride[3] = {1u, 1u, 1u};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(q),
             dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kBf16>
mxa_status_t launch_typed(const PrefillLaunch &L, PrefillArgs a, cudaStream_t stream) {
  using C = Cfg<D>;
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return MXA_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    const bool known = device >= 0 && device < kMaxDevices;
    if (!known || !done[device]) {
      if (cudaFuncSetAttribute(prefill_kernel<D, kBf16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
        return MXA_ERR_CUDA;
      if (known) done[device] = true;
    }
  }
  const mxa_decode_params_t &p = L.p;
  // Boxes of whole groups of 8 tokens of one page: the largest common divisor
  // of the page and the block serves every page size that is a multiple of
  // 8.  A contiguous cache whose rows do not start at multiples of 8 takes
  // boxes of one group and one chunk.
  int box = C::T;
  a.grouped = p.page_size % 8 == 0;
  while (box > 8 && (a.contiguous ? !a.grouped : p.page_size % box != 0)) box /= 2;
  a.box_tokens = box;
  PrefillMaps tm;
  const long long pool_tokens = (long long)(a.contiguous ? p.B : p.num_pages) * p.page_size;
  const auto encode_kv = a.grouped ? encode_grouped_kv_map : encode_kv_map;
  if (!encode_kv(&tm.kv.k, L.k_cache, D, p.Hkv, pool_tokens, box, kBf16) ||
      !encode_kv(&tm.kv.v, L.v_cache, D, p.Hkv, pool_tokens, box, kBf16) ||
      !encode_q_map(&tm.q, L.q, D, p.Hq, L.total_q, a.G, a.TQ, kBf16))
    return MXA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)L.plan.grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, prefill_kernel<D, kBf16>, tm, a) != cudaSuccess) return MXA_ERR_CUDA;
  if (L.plan.grid > 1) {
    cfg.gridDim = dim3((unsigned)(L.plan.grid - 1), kMergeParts);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, merge_kernel<D, kBf16>, a) != cudaSuccess) return MXA_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? MXA_OK : MXA_ERR_CUDA;
}

}  // namespace

mxa_status_t launch_prefill(const PrefillLaunch &L, cudaStream_t stream) {
  const mxa_decode_params_t &p = L.p;
  PrefillArgs a{};
  mxa_status_t st = device_error_word(&a.err);
  if (st != MXA_OK) return st;
  a.cu_q = L.cu_q;
  a.seqlens = L.seqlens;
  a.block_table = L.block_table;
  a.out = L.out;
  a.lse = L.lse;
  uint8_t *ws = static_cast<uint8_t *>(L.workspace);
  a.pieces = reinterpret_cast<PieceDesc *>(ws);
  a.lse_part = reinterpret_cast<float *>(ws + L.plan.lse_off);
  a.o_part = reinterpret_cast<float *>(ws + L.plan.o_off);
  a.B = p.B;
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.G = p.Hq / p.Hkv;
  a.TQ = kTileRows / a.G;
  a.total_q = L.total_q;
  a.max_q = p.q_len;
  a.page_size = p.page_size;
  a.num_pages = p.num_pages;
  a.mpps = p.max_pages_per_seq;
  a.contiguous = L.block_table == nullptr;
  a.max_seqlen_k = p.max_seqlen_k;
  a.causal = L.causal;
  a.window = L.window < p.max_seqlen_k ? L.window : p.max_seqlen_k;  // a longer one hides nothing
  a.sinks = L.window > 0 ? L.sinks : 0;
  a.wide_out = reinterpret_cast<uintptr_t>(L.out) % 32 == 0;
  a.unit_cost = L.plan.unit_cost;
  a.max_positions = (int)(prefill_positions(p, L.total_q) / p.Hkv);
  a.scale_log2 = L.scale * 1.4426950408889634f;
  const bool bf16 = p.dtype == MXA_BF16;
  if (p.D == 128) return bf16 ? launch_typed<128, true>(L, a, stream) : launch_typed<128, false>(L, a, stream);
  if (p.D == 64) return bf16 ? launch_typed<64, true>(L, a, stream) : launch_typed<64, false>(L, a, stream);
  return bf16 ? launch_typed<256, true>(L, a, stream) : launch_typed<256, false>(L, a, stream);
}

namespace {
// Rows out and the next unit's start, in blocks of KV (1: 24 ragged requests
// 154 us, two windowed prompts 109 us; 3: 150 and 106; 4: 152 and 106).
constexpr int kUnitCost = 3;
// Upper bound on the units of one KV head: every row's last group of tiles may be partial.
long long max_groups(const mxa_decode_params_t &p, int total_q) {
  const int G = p.Hq / p.Hkv, tokens = (p.D <= 128 ? 2 : 1) * (kTileRows / G);
  return (long long)total_q / tokens + (p.B < total_q ? p.B : total_q);
}
long long max_blocks(const mxa_decode_params_t &p) {
  const int T = p.D <= 128 ? 128 : 64;
  return ((long long)p.max_seqlen_k + T - 1) / T + 1;
}
}  // namespace

long long prefill_positions(const mxa_decode_params_t &p, int total_q) {
  return max_groups(p, total_q) * p.Hkv * (max_blocks(p) + kUnitCost);
}

// One CTA per SM, and no more than the work can feed with two blocks each.
PrefillPlan plan_prefill(const mxa_decode_params_t &p, int total_q, int sm_count) {
  const int NT = p.D <= 128 ? 2 : 1;
  PrefillPlan plan = {};
  plan.unit_cost = kUnitCost;
  const long long cap = max_groups(p, total_q) * p.Hkv * ((max_blocks(p) + 1) / 2);
  plan.grid = (int)(cap < sm_count ? (cap < 1 ? 1 : cap) : sm_count);
  plan.lse_off = align256(sizeof(PieceDesc) * (size_t)plan.grid);
  const size_t rows = plan.grid > 1 ? (size_t)plan.grid * 2 * NT * kTileRows : 0;
  plan.o_off = plan.lse_off + align256(rows * 4);
  plan.workspace_bytes = plan.o_off + align256(rows * p.D * 4);
  return plan;
}

}  // namespace mxa
