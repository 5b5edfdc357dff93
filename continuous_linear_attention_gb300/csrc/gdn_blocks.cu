// Block operations of a state pool: copy lists (forks, beam reorders), free
// and compaction, each from device-side indices over one layer or all of them,
// without a host round trip ("Continuous batching for linear attention
// layers", PR description: a state block is copied on fork and never shared).
//
// A copy list means "every source is read before any block is overwritten",
// so a beam reorder may name a block as a source of one entry and the
// destination of another, in chains and cycles.  No scratch blocks and no
// second pass over the data are needed for it: the blocks are cut into byte
// columns, one warp owns a column of every block, and it moves the column's
// pieces one source at a time in an order in which a block is read before it
// is written.  With W[x] the source of the entry that writes x, source x must
// come before source W[x], whose move overwrites x: a graph with one successor
// per node, i.e. trees whose roots are last moves or cycles.  The planning
// kernel orders the trees by their distance to the root (walked where it is
// short, else by pointer jumping: 2 us more) and lists each cycle from its
// lowest block (one thread: 0.13 us a block, 0.2 above 8192 blocks); a cycle's
// last source is first read into a spare buffer.  Components of that graph are
// independent of each other, so the work is cut into (part of the components,
// column).
//
// What depends on each other is moved one after the other: a chain or cycle of
// all 8,191 blocks of 4 KB takes 0.77 us of moves a block.
//
// Measured (whole calls among others, the blocks out of cache): a reorder of 256
// blocks of 2.1 MB in 3 layers 331 us, 0.95 of the copy bandwidth; 400 blocks of
// 19 KiB in 8 layers 29 us, of which the plan takes 10; clearing 37 blocks in 6
// layers 86 us, 5.5 TB/s of writes.
//
// Traffic: every distinct source is read once, however many destinations it
// has, and every destination written once, the least the call can do.  The
// pieces go global -> shared -> global by bulk copies issued by one lane, so
// registers hold none of the data.
#include "gdn_internal.cuh"
#include "gdn_cta.cuh"
#include "gdn_pool.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

constexpr int kPlanThreads = 1024;
// pools of up to this many blocks keep the planning arrays in shared memory
constexpr int kSmemBlocks = 8192;
constexpr int kPlanArrays = 6;
constexpr int kMaxLevels = 64;  // deeper trees are not divided into components
constexpr int kWalk = 16;       // steps to a root that are walked
// kinds of a move, in bits 30-31 of its source
enum Kind : uint32_t { kCopy = 0, kHold = 1, kStoreHeld = 2 };
constexpr uint32_t kBlockMask = (1u << 30) - 1;

// Orders the moves of a copy list (see above) into bw.
__global__ void __launch_bounds__(kPlanThreads, 1)
plan_copies_kernel(const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n, int nb,
                   BlockWork bw, uint32_t* err) {
  extern __shared__ int32_t plan_smem[];
  __shared__ unsigned s_flags;
  __shared__ int s_ops, s_dsts, s_comps, s_depth;
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  const bool in_smem = nb <= kSmemBlocks;
  int32_t* a = in_smem ? plan_smem : bw.tmp();
  int32_t* W = a;             // source of the entry that writes a block, or -1
  int32_t* cnt = a + nb;      // destinations of a source
  int32_t* P = a + 2 * (size_t)nb;
  int32_t* Q = a + 3 * (size_t)nb;
  int32_t* DP = a + 4 * (size_t)nb;
  int32_t* DQ = a + 5 * (size_t)nb;
  auto init = [&]() {
    for (int x = tid; x < nb; x += kPlanThreads) {
      W[x] = -1;
      cnt[x] = 0;
      P[x] = 0;
    }
  };
  if (tid == 0) {
    s_flags = 0u;
    s_ops = s_dsts = s_comps = s_depth = 0;
  }
  if (in_smem) init();
  pdl_wait_then_release();
  if (!in_smem) init();
  // a thread's first entry is read once
  int src0 = -1, dst0 = -1;
  if (tid < n) {
    src0 = src[tid];
    dst0 = dst[tid];
  }
  __syncthreads();
  // how many entries name each destination
  for (int e = tid; e < n; e += kPlanThreads) {
    const int s = e == tid ? src0 : src[e], d = e == tid ? dst0 : dst[e];
    if (s < 0 || d < 0) continue;  // padding
    if (s >= nb || d >= nb)
      atomicOr(&s_flags, GDN_FLAG_BLOCK_RANGE);
    else if (d == 0)
      atomicOr(&s_flags, GDN_FLAG_TRASH_WRITE);
    else
      atomicAdd(&P[d], 1);
  }
  __syncthreads();
  for (int e = tid; e < n; e += kPlanThreads) {
    const int s = e == tid ? src0 : src[e], d = e == tid ? dst0 : dst[e];
    if (s < 0 || d <= 0 || s >= nb || d >= nb) continue;
    if (P[d] > 1) {
      atomicOr(&s_flags, GDN_FLAG_DUPLICATE);
    } else if (s != d) {
      W[d] = s;
      atomicAdd(&cnt[s], 1);
    }
  }
  __syncthreads();
  int hazard = 0;
  for (int x = tid; x < nb; x += kPlanThreads) hazard |= cnt[x] > 0 && W[x] >= 0;
  int32_t *osrc = bw.src(), *obeg = bw.beg(), *ocnt = bw.cnt();
  // move k is x's; cnt[x] becomes where x's destinations go
  auto emit = [&](int k, int x, uint32_t kind) {
    const int c = kind == kHold ? 0 : cnt[x];
    const int at = atomicAdd(&s_dsts, c);
    osrc[k] = (int32_t)((uint32_t)x | (kind << 30));
    obeg[k] = at;
    ocnt[k] = c;
    if (kind != kHold) cnt[x] = at;
  };
  // a cycle from x, its lowest block: its last source into the spare buffer,
  // the others in order, then the held one
  auto emit_cycle = [&](int k, int x) {
    int last = x;
    while (W[last] != x) last = W[last];
    emit(k++, last, kHold);
    for (int z = x; z != last; z = W[z]) emit(k++, z, kCopy);
    emit(k, last, kStoreHeld);
  };
  // moves of the cycle that x leads, or 0 if a lower block does
  auto cycle_moves = [&](int x) {
    int len = 2, y = W[x];
    for (; y > x; y = W[y]) ++len;
    return y == x ? len : 0;
  };
  int single = 0;
  if (!__syncthreads_or(hazard)) {
    // no source is written (a fork): any order, every move by itself
    for (int x = tid; x < nb; x += kPlanThreads)
      if (cnt[x] > 0) emit(atomicAdd(&s_ops, 1), x, kCopy);
    single = 1;
  } else {
    // Every source's root (a last source, or one on a cycle) and its distance to
    // it: by walking up to kWalk steps, first to an end or back to the start,
    // then to a cycle ...
    int32_t* cyc = Q;
    int32_t* nxt = P;
    int far = 0, on_cycle = 0;
    for (int x = tid; x < nb; x += kPlanThreads) {
      int y = x, next = cnt[x] > 0 ? W[x] : -1, steps = 0;
      while (next >= 0 && next != x && steps < kWalk) {
        y = next;
        next = W[y];
        ++steps;
      }
      cyc[x] = next == x;
      DP[x] = next < 0 ? steps : 0;
      nxt[x] = next < 0 ? y : next == x ? x : -1;
      on_cycle |= next == x;
      far |= nxt[x] < 0;
    }
    bool cycles = __syncthreads_or(on_cycle) != 0;
    if (__syncthreads_or(far)) {
      far = 0;
      for (int x = tid; x < nb; x += kPlanThreads) {
        if (nxt[x] >= 0) continue;
        int y = x, steps = 0;
        while (!cyc[y] && steps < kWalk && W[y] >= 0) {
          y = W[y];
          ++steps;
        }
        if (cyc[y]) {
          DP[x] = steps;
          nxt[x] = y;
        } else {
          far = 1;
        }
      }
      far = __syncthreads_or(far);
    } else {
      far = 0;
    }
    if (far) {
      // ... and, where that does not get everywhere, by pointer jumping.
      int rounds = 1;
      while ((1 << rounds) < nb) ++rounds;
      // cycles: 2^rounds >= nb steps from a source that reaches one end on it,
      // and every source of a cycle is such an end; on the way the lowest block
      // passed, which for a source of a cycle is the cycle's
      for (int x = tid; x < nb; x += kPlanThreads) {
        P[x] = cnt[x] > 0 ? W[x] : -1;
        DP[x] = x;
      }
      __syncthreads();
      cycles = true;
      for (int r = 0; r < rounds && cycles; ++r) {
        int more = 0;
        for (int x = tid; x < nb; x += kPlanThreads) {
          const int z = P[x], y = z < 0 ? -1 : P[z];
          Q[x] = y;
          DQ[x] = z < 0 ? DP[x] : min(DP[x], DP[z]);
          more |= y >= 0;
        }
        cycles = __syncthreads_or(more) != 0;
        int32_t* t = P;
        P = Q;
        Q = t;
        t = DP;
        DP = DQ;
        DQ = t;
      }
      for (int x = tid; x < nb; x += kPlanThreads) Q[x] = 0;
      __syncthreads();
      if (cycles)
        for (int x = tid; x < nb; x += kPlanThreads)
          if (P[x] >= 0) Q[P[x]] = 1;
      __syncthreads();
      // every other source's root (a last source, or the lowest of a cycle) and
      // its distance to it (steps along the cycle count nothing)
      cyc = Q;
      nxt = P;
      for (int x = tid; x < nb; x += kPlanThreads) {
        const bool tree = cnt[x] > 0 && W[x] >= 0 && !cyc[x];
        nxt[x] = tree ? W[x] : cyc[x] ? DP[x] : x;
        DP[x] = tree ? 1 : 0;
      }
      __syncthreads();
      for (int r = 0; r < rounds; ++r) {
        for (int x = tid; x < nb; x += kPlanThreads) DQ[x] = DP[x] + DP[nxt[x]];
        __syncthreads();
        int32_t* t = DP;
        DP = DQ;
        DQ = t;
        // the old distances' array takes the jumped pointers
        int more = 0;
        for (int x = tid; x < nb; x += kPlanThreads) {
          const int y = nxt[nxt[x]];
          more |= y != nxt[x];
          DQ[x] = y;
        }
        t = nxt;
        nxt = DQ;
        DQ = t;
        if (!__syncthreads_or(more)) break;
      }
    }
    for (int x = tid; x < nb; x += kPlanThreads)
      if (cnt[x] > 0) atomicMax(&s_depth, DP[x]);
    // the lowest block of a cycle leads it: the root of its component (found by
    // walking the short cycles, with the pointers on the others)
    if (cycles && !far)
      for (int x = tid; x < nb; x += kPlanThreads)
        if (cyc[x] && cycle_moves(x)) {
          int z = x;
          do {
            nxt[z] = x;
            z = W[z];
          } while (z != x);
        }
    __syncthreads();
    const int depth = s_depth;
    int32_t* place = DQ;
    for (int x = tid; x < nb; x += kPlanThreads) place[x] = 0;
    __syncthreads();
    if (depth <= kMaxLevels) {
      // components one after the other, in each the trees from the leaves
      // down, then the cycle
      auto root = [&](int x) { return nxt[nxt[x]]; };
      for (int x = tid; x < nb; x += kPlanThreads) {
        if (cnt[x] == 0) continue;
        if (!cyc[x]) atomicAdd(&place[root(x)], 1);
        else if (nxt[x] == x) atomicAdd(&place[x], cycle_moves(x));
      }
      __syncthreads();
      int moves = 0, comps = 0;
      for (int x0 = 0; x0 < nb; x0 += kPlanThreads) {
        const int x = x0 + tid, n_x = x < nb ? place[x] : 0;
        int tm, tc;
        const int at = moves + cta_scan(n_x, &tm, warp_sums);
        const int ct = comps + cta_scan(n_x > 0, &tc, warp_sums);
        if (n_x > 0) {
          place[x] = at;
          bw.start()[ct] = at;
        }
        moves += tm;
        comps += tc;
      }
      if (tid == 0) {
        s_ops = moves;
        s_comps = comps;
        bw.start()[comps] = moves;
      }
      for (int level = depth; level >= 0; --level) {
        __syncthreads();
        for (int x = tid; x < nb; x += kPlanThreads)
          if (DP[x] == level && !cyc[x] && cnt[x] > 0)
            emit(atomicAdd(&place[root(x)], 1), x, kCopy);
      }
      __syncthreads();
      if (cycles)
        for (int x = tid; x < nb; x += kPlanThreads)
          if (cyc[x] && nxt[x] == x) emit_cycle(place[x], x);
    } else {
      // long chains: all trees by falling distance (a counting sort), then the
      // cycles, as one run of moves
      for (int x = tid; x < nb; x += kPlanThreads)
        if (cnt[x] > 0 && !cyc[x]) atomicAdd(&place[DP[x]], 1);
      __syncthreads();
      int moves = 0;
      for (int x0 = 0; x0 < nb; x0 += kPlanThreads) {
        const int x = nb - 1 - (x0 + tid);
        int total;
        const int before = cta_scan(x >= 0 ? place[x] : 0, &total, warp_sums);
        if (x >= 0) place[x] = moves + before;
        moves += total;
      }
      if (tid == 0) s_ops = moves;
      __syncthreads();
      for (int x = tid; x < nb; x += kPlanThreads)
        if (cnt[x] > 0 && !cyc[x]) emit(atomicAdd(&place[DP[x]], 1), x, kCopy);
      __syncthreads();
      for (int x = tid; x < nb; x += kPlanThreads)
        if (cyc[x] && nxt[x] == x) emit_cycle(atomicAdd(&s_ops, cycle_moves(x)), x);
      __syncthreads();
      if (tid == 0) {
        s_comps = 1;
        bw.start()[0] = 0;
        bw.start()[1] = s_ops;
      }
    }
  }
  __syncthreads();
  int32_t* odst = bw.dst();
  for (int e = tid; e < n; e += kPlanThreads) {
    const int s = e == tid ? src0 : src[e], d = e == tid ? dst0 : dst[e];
    if (s < 0 || d <= 0 || s >= nb || d >= nb || s == d || W[d] != s) continue;
    odst[atomicAdd(&cnt[s], 1)] = d;
  }
  if (tid == 0) {
    bw.header()[0] = s_ops;
    bw.header()[1] = single ? s_ops : s_comps;
    bw.header()[2] = 0;
    bw.header()[3] = single;
    if (s_flags) atomicOr(err, s_flags);
  }
}

// Plans a compaction: with m live blocks, the i-th live block above m moves to
// the i-th free block of 1..m, both ascending.  The two lists are disjoint.
__global__ void __launch_bounds__(kPlanThreads, 1)
plan_compact_kernel(const int32_t* idx, int32_t* new_idx, int n, int nb, BlockWork bw,
                    uint32_t* err) {
  extern __shared__ int32_t plan_smem[];
  __shared__ unsigned s_flags;
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  const bool in_smem = nb <= kSmemBlocks;
  int32_t* live = in_smem ? plan_smem : bw.tmp();
  int32_t* to = live + nb;
  if (tid == 0) s_flags = 0u;
  if (in_smem)
    for (int x = tid; x < nb; x += kPlanThreads) live[x] = 0;
  pdl_wait_then_release();
  if (!in_smem)
    for (int x = tid; x < nb; x += kPlanThreads) live[x] = 0;
  __syncthreads();
  for (int e = tid; e < n; e += kPlanThreads) {
    const int b = idx[e];
    if (b >= nb)
      atomicOr(&s_flags, GDN_FLAG_BLOCK_RANGE);
    else if (b > 0)
      live[b] = 1;
  }
  __syncthreads();
  int m = 0;
  for (int x0 = 0; x0 < nb; x0 += kPlanThreads)
    m += __syncthreads_count(x0 + tid < nb && live[x0 + tid]);
  int32_t *osrc = bw.src(), *obeg = bw.beg(), *ocnt = bw.cnt(), *odst = bw.dst();
  int holes = 0, highs = 0;
  for (int x0 = 0; x0 < nb; x0 += kPlanThreads) {
    const int x = x0 + tid;
    const int hole = x >= 1 && x <= m && !live[x < nb ? x : 0] ? 1 : 0;
    const int high = x > m && x < nb && live[x < nb ? x : 0] ? 1 : 0;
    int th, tg;
    const int rh = holes + cta_scan(hole, &th, warp_sums);
    const int rg = highs + cta_scan(high, &tg, warp_sums);
    holes += th;
    highs += tg;
    if (hole) odst[rh] = x;
    if (high) {
      osrc[rg] = x;
      obeg[rg] = rg;
      ocnt[rg] = 1;
    }
  }
  __syncthreads();
  for (int r = tid; r < highs; r += kPlanThreads) to[osrc[r]] = odst[r];
  __syncthreads();
  for (int e = tid; e < n; e += kPlanThreads) {
    const int b = idx[e];
    new_idx[e] = b > m && b < nb ? to[b] : b;
  }
  if (tid == 0) {
    bw.header()[0] = bw.header()[1] = highs;
    bw.header()[2] = 0;
    bw.header()[3] = 1;
    if (s_flags) atomicOr(err, s_flags);
  }
}

// --- the moves -------------------------------------------------------------
constexpr int kWarps = 4;
constexpr int kPiece = 8192;     // bytes of a column, at most
constexpr int kMinPiece = 1024;  // and at least
constexpr int kSlots = 5;        // pieces in flight per warp, loads and stores
constexpr int kPending = 2;      // stores that may still read their pieces
constexpr int kCached = 1024;    // moves (and destinations) kept in shared memory
constexpr int kUnits = 8;        // units a warp has begun and not finished
struct Unit {
  unsigned char* at;  // the column in block 0
  uint32_t bytes;
  int k0, k1;         // moves
};
struct MoveSmem {
  unsigned char buf[kWarps][kSlots + 1][kPiece];  // the last one holds a cycle's source
  uint64_t full[kWarps][kSlots + 1];
  Unit unit[kWarps][kUnits];
  int32_t src[kCached], beg[kCached], cnt[kCached], dst[kCached];
};
static_assert(sizeof(MoveSmem) <= 227 * 1024, "shared memory of one CTA");

struct MoveParams {
  unsigned char* base;  // block 0 of the first layer moved
  size_t stride;
  int nb, layers;
  BlockWork bw;
  uint32_t* err;
};

__global__ void __launch_bounds__(kWarps * 32, 1) move_blocks_kernel(MoveParams p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  MoveSmem& sm = *reinterpret_cast<MoveSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5;
  if ((tid & 31) == 0) {
    for (int i = 0; i <= kSlots; ++i) mbar_init(&sm.full[warp][i], 1);
    fence_mbar_init();
  }
  // (in this order: a scheduler behind this kernel may read the list that the
  // plan has rewritten before it waits for this kernel)
  pdl_wait_then_release();
  int32_t* hdr = p.bw.header();
  const int ops = hdr[0], comps = hdr[1];
  const bool single = hdr[3] != 0;
  if (ops == 0) return;
  for (int i = tid; i < kCached; i += kWarps * 32) {
    if (i < ops) {
      sm.src[i] = p.bw.src()[i];
      sm.beg[i] = p.bw.beg()[i];
      sm.cnt[i] = p.bw.cnt()[i];
    }
    if (i < p.nb) sm.dst[i] = p.bw.dst()[i];
  }
  __syncthreads();
  if ((tid & 31) != 0) return;
  const int32_t *gsrc = p.bw.src(), *gbeg = p.bw.beg(), *gcnt = p.bw.cnt(), *gdst = p.bw.dst();
  auto src_of = [&](int k) { return (uint32_t)(k < kCached ? sm.src[k] : gsrc[k]); };
  auto dst_of = [&](int i) { return i < kCached ? sm.dst[i] : gdst[i]; };
  unsigned char(*buf)[kPiece] = sm.buf[warp];
  uint64_t* full = sm.full[warp];

  // The units: columns, narrowed while half of the warps would have nothing to
  // do (six requests' beams of 143 KB blocks, 4 layers: 13 us, 26 with four
  // units per warp wherever possible), by parts of the components: eight units
  // per warp, but eight pieces in each where that leaves two (100 requests'
  // beams of 19 KiB, 8 layers: 29 us, 32 with eight units each; at 64 requests'
  // of 2.1 MB two per warp take 354 us and eight 331).
  const long long warps = (long long)gridDim.x * kWarps;
  int piece = kPiece;
  auto cols_of = [&](int b) { return (long long)((p.stride + b - 1) / b); };
  while (piece > kMinPiece && p.layers * cols_of(piece) * comps < warps / 2) piece /= 2;
  const long long cols = cols_of(piece), ncol = p.layers * cols;
  const long long units = min(max(ncol * ops / 8, 2 * warps), 8 * warps);
  const long long want = (units + ncol - 1) / ncol;
  const int parts = (int)(want < comps ? want : comps);
  // first move of part i: that of the first component at or behind its share
  auto part_begin = [&](int i) {
    const int at = (int)((long long)i * ops / parts);
    if (single || at == ops) return at;
    const int32_t* start = p.bw.start();
    int lo = 0, hi = comps;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] < at) lo = mid + 1; else hi = mid;
    }
    return start[lo];
  };
  const unsigned long long n_units = (unsigned long long)ncol * parts;
  // the next unit that has moves, claimed one ahead
  auto claim = [&]() {
    Unit u = {nullptr, 0, 0, 0};
    for (;;) {
      const unsigned long long i = atomicAdd((unsigned*)&hdr[2], 1u);
      if (i >= n_units) return u;
      const int part = (int)(i % parts);
      const long long col = (long long)(i / parts);
      u.k0 = part_begin(part);
      u.k1 = part_begin(part + 1);
      if (u.k0 == u.k1) continue;
      const size_t off = (size_t)(col % cols) * piece;
      u.bytes = (uint32_t)min((size_t)piece, p.stride - off);
      u.at = p.base + (size_t)(col / cols) * p.nb * p.stride + off;
      return u;
    }
  };
  // the load cursor runs ahead of the store cursor over the units' moves;
  // pieces of the ring: loaded, issued to store, and read by their store
  Unit lu = claim(), next = lu.at ? claim() : lu;
  int lk = lu.k0, lq = 0, sq = 0, sk = lu.k0;
  sm.unit[warp][0] = lu;
  long long loads = 0, stores = 0, holds = 0;
  bool held = false;
  while (sm.unit[warp][sq % kUnits].at) {
    // loads, as far ahead as the ring and the spare buffer allow
    while (lu.at) {
      const uint32_t s = src_of(lk), kind = s >> 30;
      if (kind == kCopy && loads - max(stores - kPending, 0ll) >= kSlots) break;
      if (kind == kHold && held) break;
      if (kind != kStoreHeld) {
        const int slot = kind == kHold ? kSlots : (int)(loads % kSlots);
        mbar_arrive_expect_tx(&full[slot], lu.bytes);
        bulk_g2s(buf[slot], lu.at + (size_t)(s & kBlockMask) * p.stride, lu.bytes, &full[slot]);
        if (kind == kHold) held = true;
        else ++loads;
      }
      if (++lk == lu.k1) {
        lu = next;
        lk = lu.k0;
        sm.unit[warp][++lq % kUnits] = lu;
        if (lu.at) next = claim();
      }
    }
    // one move
    const Unit su = sm.unit[warp][sq % kUnits];
    const uint32_t s = src_of(sk), kind = s >> 30;
    const bool ring = kind == kCopy;
    const int slot = ring ? (int)(stores % kSlots) : kSlots;
    if (kind != kStoreHeld) {
      const uint32_t parity = ring ? (uint32_t)((stores / kSlots) & 1) : (uint32_t)(holds & 1);
      if (!mbar_wait_bounded(&full[slot], parity)) {
        atomicOr(p.err, GDN_FLAG_TIMEOUT);
        // the copies already issued land before the CTA ends
        for (long long i = stores + (ring ? 1 : 0); i < loads; ++i)
          mbar_wait_bounded(&full[i % kSlots], (uint32_t)((i / kSlots) & 1));
        if (held && ring) mbar_wait_bounded(&full[kSlots], (uint32_t)(holds & 1));
        bulk_wait_all();
        return;
      }
      if (kind == kHold) ++holds;
    }
    if (kind != kHold) {
      const int beg = sk < kCached ? sm.beg[sk] : gbeg[sk];
      const int cnt = sk < kCached ? sm.cnt[sk] : gcnt[sk];
      for (int i = 0; i < cnt; ++i)
        bulk_s2g(su.at + (size_t)dst_of(beg + i) * p.stride, buf[slot], su.bytes);
      bulk_commit();
      if (ring) {
        // all pieces but those of the last kPending stores may be loaded over
        asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
        ++stores;
      } else {
        bulk_wait_read_all();
        held = false;
      }
    }
    if (++sk == su.k1) {
      ++sq;
      sk = sm.unit[warp][sq % kUnits].k0;
    }
  }
  bulk_wait_all();
}

// Zeroes the named blocks, a piece at a time from a zeroed shared buffer.
constexpr int kZero = 16384;
__global__ void __launch_bounds__(128)
clear_blocks_kernel(unsigned char* base, size_t stride, int nb, int layers, int cols,
                    const int32_t* __restrict__ idx, int n, uint32_t* err) {
  __shared__ __align__(128) unsigned char zero[kZero];
  pdl_wait_then_release();
  for (int i = threadIdx.x * 16; i < kZero; i += 128 * 16)
    *reinterpret_cast<uint4*>(zero + i) = make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  if (threadIdx.x != 0) return;
  const long long per = (long long)layers * cols;
  for (long long u = blockIdx.x; u < per * n; u += gridDim.x) {
    const int e = (int)(u / per);
    const long long r = u % per;
    const int b = idx[e];
    if (b < 0) continue;  // padding
    if (b == 0 || b >= nb) {
      if (r == 0) atomicOr(err, b == 0 ? GDN_FLAG_TRASH_WRITE : GDN_FLAG_BLOCK_RANGE);
      continue;
    }
    const int layer = (int)(r / cols);
    const size_t off = (size_t)(r % cols) * kZero;
    bulk_s2g(base + ((size_t)layer * nb + b) * stride + off, zero,
             (uint32_t)min((size_t)kZero, stride - off));
    bulk_commit();
  }
  bulk_wait_all();
}

// What every block operation checks on the host.
int check_call(const gdn_pool* p, int layer, int n, bool pointers) {
  if (!p) return GDN_ERR_NULL;
  if (layer < -1 || layer >= p->num_layers || n < 0) return GDN_ERR_RANGE;
  if (n > 0 && !pointers) return GDN_ERR_NULL;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
  return dev == p->device ? GDN_OK : GDN_ERR_DEVICE;
}

uint32_t* error_word(const gdn_pool* p, int layer) {
  return reinterpret_cast<uint32_t*>(p->work + (size_t)(layer < 0 ? 0 : layer) *
                                                   WorkArea::words(p->num_blocks) + kErr);
}
unsigned char* first_layer(const gdn_pool* p, int layer) {
  return p->base + (size_t)(layer < 0 ? 0 : layer) * p->num_blocks * p->stride;
}

size_t plan_smem_bytes(int nb) {
  return nb <= kSmemBlocks ? (size_t)kPlanArrays * nb * sizeof(int32_t) : 0;
}

cudaError_t launch_moves(const gdn_pool* p, int layer, const BlockWork& bw, cudaStream_t s) {
  MoveParams mp;
  mp.base = first_layer(p, layer);
  mp.stride = p->stride;
  mp.nb = p->num_blocks;
  mp.layers = layer < 0 ? p->num_layers : 1;
  mp.bw = bw;
  mp.err = error_word(p, layer);
  cudaError_t e = cudaFuncSetAttribute(move_blocks_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(MoveSmem));
  if (e != cudaSuccess) return e;
  return launch_pdl(move_blocks_kernel, dim3(p->sms), dim3(kWarps * 32), sizeof(MoveSmem), s, mp);
}

template <typename K, typename... Args>
cudaError_t launch_plan(K kernel, int nb, cudaStream_t s, Args... args) {
  const size_t smem = plan_smem_bytes(nb);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)plan_smem_bytes(kSmemBlocks));
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(1), dim3(kPlanThreads), smem, s, args...);
}

}  // namespace
}  // namespace gdn

extern "C" {

int gdn_state_pool_copy_blocks(gdn_pool_t* p, int layer, const int32_t* src, const int32_t* dst,
                               int n, void* stream) {
  const int st = gdn::check_call(p, layer, n, src && dst);
  if (st != GDN_OK || n == 0) return st;
  cudaStream_t s = (cudaStream_t)stream;
  const gdn::BlockWork bw{p->blk_work, p->num_blocks};
  if (gdn::launch_plan(gdn::plan_copies_kernel, p->num_blocks, s, src, dst, n, p->num_blocks, bw,
                       gdn::error_word(p, layer)) != cudaSuccess)
    return GDN_ERR_CUDA;
  return gdn::launch_moves(p, layer, bw, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_state_pool_compact(gdn_pool_t* p, const int32_t* idx, int32_t* new_idx, int n,
                           void* stream) {
  const int st = gdn::check_call(p, -1, n, idx && new_idx);
  if (st != GDN_OK || n == 0) return st;
  cudaStream_t s = (cudaStream_t)stream;
  const gdn::BlockWork bw{p->blk_work, p->num_blocks};
  if (gdn::launch_plan(gdn::plan_compact_kernel, p->num_blocks, s, idx, new_idx, n, p->num_blocks,
                       bw, gdn::error_word(p, -1)) != cudaSuccess)
    return GDN_ERR_CUDA;
  return gdn::launch_moves(p, -1, bw, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_state_pool_clear_blocks(gdn_pool_t* p, int layer, const int32_t* idx, int n,
                                void* stream) {
  const int st = gdn::check_call(p, layer, n, idx != nullptr);
  if (st != GDN_OK || n == 0) return st;
  const int layers = layer < 0 ? p->num_layers : 1;
  const int cols = (int)((p->stride + gdn::kZero - 1) / gdn::kZero);
  const long long units = (long long)layers * cols * n;
  const long long most = 8ll * p->sms;
  if (gdn::launch_pdl(gdn::clear_blocks_kernel, dim3((unsigned)(units < most ? units : most)),
                      dim3(128), 0, (cudaStream_t)stream, gdn::first_layer(p, layer), p->stride,
                      p->num_blocks, layers, cols, idx, n,
                      gdn::error_word(p, layer)) != cudaSuccess)
    return GDN_ERR_CUDA;
  return GDN_OK;
}

}  // extern "C"
