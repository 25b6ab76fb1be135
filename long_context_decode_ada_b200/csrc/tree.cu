// tree.cu -- attention of the drafted tokens of a tree over the paged store:
// every row r = (drafted token i, query head g of a kv head) sees the store's
// resident tokens and the drafted tokens its mask names, with scores
// optionally capped by a tanh or biased by distance.
//
//   S = Q K^T / sqrt d,  O = sum_t 2^(S - m) v_t,  l = sum_t 2^(S - m)
//
// Work split: the page list is cut into runs of about equal cost, one per
// CTA; a run is a list of segments (a unit = (sequence, kv head), or a part
// of one), a segment a list of tiles of 64 tokens (64 / P pages), the
// unit's drafted tokens being one more tile behind its pages.  A unit that
// lies in one run is finished there; the parts of a unit that several runs
// share go to the workspace as (m, l, O) and a second grid joins them.
//
// Roles of a CTA (one per SM):
//   planner (1 warp)   turns the page list into tile descriptors (a ring of 32
//                      in shared memory), checks ids and headers, and asks for
//                      the pages' bytes in L2 (bulk prefetch)
//   copier (1 warp)    brings the pages into shared memory by bulk copies, five
//                      coded tiles (or one dense and two coded) in flight: with
//                      the shared memory that the tiles take the L1 is too
//                      small for as many loads in flight
//   decode (8 warps)   two teams of 4 take the tiles in turn, a warp 16 rows:
//                      codes to fp16 keys by gathers from a replicated table
//                      (one conflict-free wavefront a gather), int8 values to
//                      fp16, both written as swizzled operand tiles (32 KB a
//                      tile, three in flight)
//   mma (2 warps)      S = Q K^T, and O += P V, by tcgen05.mma (fp16, fp32
//                      accumulators), a tile a job; Q and P are read from
//                      tensor memory, so that shared memory feeds K and V only
//   softmax (8 warps)  two groups of 4, one per stream: scores from tensor
//                      memory, running maximum and sum, weights back as fp16
//
// The two streams have accumulators of their own.  With at most 128 rows they
// take the tiles in turn, and with at most 64 rows the rows are entered twice,
// each copy handling half of a job's columns: every lane of tensor memory then
// has work, and the copies' sums meet at the segment's end.  With more than
// 128 rows stream b has the rows 128 b .. 128 b + 127 of every tile.  The
// running maximum is raised (and O rescaled) only when a score passes it by
// more than 2^8, so weights stay within fp16.
//
// What bounds it is neither the products (tensor cores 21% busy) nor HBM nor
// instruction issue (49% busy at 128 rows) but the hand-overs between the roles
// and the ends of segments: from a segment's last tile to the next one's first
// product pass 47,000 to 60,000 cycles, in which the pipe drains, the sums are
// written in eight steps and the next queries are read.  Five roles' loops
// share one instruction cache: a few instructions more in a cold branch have
// moved the prompt batch (265 us) by 2 to 28%.  Measured over the 128K store
// (1.05 M token-heads): 32 tokens (128 rows) 166 us; 171 us before units' take-up
// was weighed as it is, 209 us with waits of 35 instructions at their 25 places
// (instruction cache misses 3.6 M against 0.6 M a launch); pages loaded by the
// decode warps themselves instead of by bulk copies 231 us; tiles of 64 tokens
// with one warp issuing both products 274 us.  Three decode teams instead of
// two change nothing (175 us against 171).  Spills: up to 20 bytes a thread.
//
// Roundings: a coded key is a table entry times its radius (two fp16
// roundings), a value an int8 times its scale (one), a weight one; each is
// 2^-11 of its number at most.  Together they put an output about 0.0004 of
// its size off; bf16 outputs are rounded by 0.0017 anyway, fp16 ones by 0.0002.
// Exact values and split weights, as in the form for few rows, would double
// the second product and need 64 columns of tensor memory: with one block's
// queries in shared memory they would be there, which is not tried.
//
// Tensor memory (512 columns): Q 0-63 (and 64-127 for the second block), P of
// the streams at 64 and 96 (over S with two blocks), S at 128 and 192, O at
// 256 and 384.
#include <algorithm>
#include <cstddef>

#include "tree.cuh"

namespace skv {

namespace {

using namespace tree;

constexpr int kTile = 64;            // tokens of a tile (a job of the products)
constexpr int kStages = 3;           // tiles of keys and values in flight
constexpr int kRing = 32;            // tile descriptors
constexpr int kBatch = 8;            // tiles the planner publishes at once
constexpr int kTeams = 2;            // of decode warps, taking the tiles in turn
constexpr int kTeamWarps = 4;        // 16 rows each
constexpr int kSoftWarps = 8;
constexpr int kDecodeWarps = kTeams * kTeamWarps;
constexpr int kPlanner = kSoftWarps + kDecodeWarps, kCopier = kPlanner + 1;
constexpr int kMmaS = kPlanner + 2;  // (and the warp behind it)
constexpr int kThreads = (kSoftWarps + kDecodeWarps + 4) * 32;
// registers a thread (softmax, decode, the others); their sum over the threads
// is what the block is launched with
constexpr int kRegsLaunch = 96, kRegsSoft = 128, kRegsDecode = 80, kRegsHelp = 64;
static_assert(kSoftWarps * kRegsSoft + kDecodeWarps * kRegsDecode + 4 * kRegsHelp <=
                  kThreads / 32 * kRegsLaunch, "registers");
constexpr int kBufRow = 36;          // floats of a row of the output buffer (32 dims)
// pages as they are stored: slots of one coded tile (a dense tile takes three)
constexpr uint32_t kRawSlot = kTile * 196 + 4 * kHdrBytes;
constexpr int kRawSlots = 5, kRawTiles = 8;
static_assert(kTile * 512 + 4 * kHdrBytes <= 3 * kRawSlot && kRawSlot % 16 == 0, "raw slots");

enum : uint32_t { kFirst = 1, kLast = 2, kDraft = 4, kEnd = 8 };

// columns of tensor memory
constexpr uint32_t kColQ = 0, kColP = 64, kColS = 128, kColO = 256;

struct __align__(16) Part {     // 16 rows of a tile
  unsigned long long page;      // address (tier < 3)
  uint32_t off;                 // of the page's bytes in the tile's raw bytes
  uint8_t at, rows, tier;       // first row within the page, rows in use; tier 3: none
  uint8_t zero;
};

struct __align__(16) Tile {
  Part part[4];
  unsigned long long valid;     // bit c: column c holds a token
  int unit, n;                  // (sequence, kv head) and its drafted tokens
  uint32_t flags;
  int first;                    // index of the first page in the page list
  int slot;                     // partial slot, -1: the unit lies in this run
  int bad;                      // a drafted value lies outside fp16
  uint32_t bytes;               // raw bytes
  int shift;                    // drafted values enter times 2^shift
};

struct __align__(16) Fixed {
  unsigned long long kfull[kStages], vfull[kStages], kempty[kStages], vempty[kStages];
  unsigned long long sfull[2], sfree[2], pfull[2], odone[2];
  unsigned long long qfull, sync, fin[2];
  unsigned long long dfull[kRing / kBatch], rfree[kRing / kBatch];
  unsigned long long rawfull[kRawTiles], rawfree[kRawTiles];
  uint32_t raw[kRawTiles];      // where a tile's raw bytes lie
  unsigned long long scan[kThreads / 32];
  Run run;
  int late;                     // a wait gave up
  uint32_t tmem;
  __align__(16) Tile ring[kRing];
  __align__(16) float pos[kStages][kTile];   // positions (from the unit's first q_pos)
  __align__(16) float cs[kStages][kTile];    // drafted keys: what a score is scaled by
};

// behind the output buffer
struct Sums {
  float m[2][128], l[2][128];
};

// Shared memory: [fixed block][stages][T2 table][T1 table][raw slots][output
// buffer, sums]; the stages start on an 8 KB boundary.  Entry e of a table
// (T1: the code byte; T2: angle | share << 4) is at 128 e, in 32 copies of 4
// bytes (copy L is read by lane L), so that a warp's gathers never conflict.
constexpr uint32_t kOperand = kTile * 256;                // a tile's keys or values
constexpr uint32_t kTbl2 = 64 * 128, kTbl1 = 256 * 128;
constexpr uint32_t kAtTbl2 = kStages * 2 * kOperand, kAtTbl1 = kAtTbl2 + kTbl2;
constexpr uint32_t kAtRaw = kAtTbl1 + kTbl1;
constexpr uint32_t kAtBuf = kAtRaw + kRawSlots * kRawSlot;
constexpr uint32_t kAtSums = kAtBuf + 128 * kBufRow * 4;
constexpr uint32_t kHighBytes = kAtSums + sizeof(Sums);
constexpr uint32_t kSmemBytes = 232448;
static_assert(sizeof(Fixed) + 1024 <= 8192, "the stages start at 8 KB");
static_assert(kHighBytes + 8192 <= kSmemBytes + 1024 && kAtTbl2 % 8192 == 0 && kAtBuf % 16 == 0, "layout");
__device__ __forceinline__ uint32_t keys_at(uint32_t base, uint32_t stage) {
  return base + stage * 2 * kOperand;
}
__device__ __forceinline__ uint32_t values_at(uint32_t base, uint32_t stage) {
  return base + stage * 2 * kOperand + kOperand;
}

// ------------------------------------------------------------ tensor memory
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}

// 16 columns of this warp's 32 lanes
__device__ __forceinline__ void tc_ld16(uint32_t a, float* x) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tc_ld8(uint32_t a, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void tc_st8(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// D (128 lanes x N fp32) (+)= A (tensor memory, 128 x 16 fp16) B (shared, 16 x N)
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, unsigned long long b, uint32_t idesc,
                                       uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}

// fp16 A and B, fp32 D, M = 128; B's values contiguous along k, or along n
constexpr uint32_t kIdescS = (1u << 4) | ((kTile / 8) << 17) | (8u << 24);
constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((kHeadDim / 8) << 17) | (8u << 24);

// Operand tiles in shared memory: rows of 128 bytes, their 16-byte chunks
// permuted by the row's low three bits (128-byte swizzle), groups of 8 rows
// 1024 bytes apart; the second 64 dims follow 8 KB behind.
constexpr uint32_t kHalfDims = kTile * 128;   // from dims 0-63 of a tile to dims 64-127
constexpr uint32_t kDescHigh = (1024 / 16) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescKeys = 1u << 16, kDescValues = (kHalfDims / 16) << 16;
__device__ __forceinline__ unsigned long long operand(uint32_t low) {
  return ((unsigned long long)kDescHigh << 32) | low;
}

// How long a wait may take: tries, and ns that one may sleep.  The default stands in
// the code (the limit in a register of every role costs the prompt batch 3%, read
// from the parameters at every wait 6%), a limit set by the caller has instances
// of its own.
struct DefaultLimit {
  __device__ __forceinline__ DefaultLimit(const TreeParams&) {}
  __device__ __forceinline__ uint32_t tries() const { return 100000u; }
  __device__ __forceinline__ uint32_t ns() const { return 20000u; }
};
struct SetLimit {
  uint32_t lim;
  __device__ __forceinline__ SetLimit(const TreeParams& p) : lim(p.wait_limit) {}
  __device__ __forceinline__ uint32_t tries() const { return lim; }
  __device__ __forceinline__ uint32_t ns() const { return lim; }
};

// A bounded wait of a whole warp: false for all lanes after the limit's tries (a
// wait here is on other warps of the block and takes some microseconds).  Every
// role returns at its first wait that gave up, once what it has in flight
// itself has landed; the error is reported at the end.  Short on purpose: the
// code stands at some 25 places of five loops that share an instruction cache.
template <class Limit>
__device__ __forceinline__ bool warp_wait(unsigned long long& bar, uint32_t parity, Fixed& f,
                                          Limit lim) {
  const uint32_t a = smem_u32(&bar);
#pragma unroll 1
  for (uint32_t n = 0; n < lim.tries(); ++n)
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait_sleep(a, parity, lim.ns()))) return true;
  *(volatile int*)&f.late = 1;
  return false;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void warp_arrive(unsigned long long& bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bar));
}

// More than 128 rows cost half as much again (decoded once, multiplied twice).
// A segment's start and end take 47,000 to 60,000 cycles, a coded tile 1,750
// to 2,000 (fitted over the runs of three batches): 1536 tokens for a unit
// taken up.  8 sequences x 16 tokens, 8 KV heads, 32K tokens: 279 us at 512
// tokens, 276 at 1024, 273 at 1536, 276 at 2048.
struct RowsCost {
  static constexpr int kTile = 64, kBegin = 1536;
  __device__ __forceinline__ int operator()(int rows) const { return rows > 128 ? 3 : 2; }
};
static_assert(RowsCost::kTile == kTile, "tiles");

// ---------------------------------------------------------------- the planner
template <class Limit>
__device__ __forceinline__ void planner(const TreeParams& p, Fixed& f, int c, int lane,
                                        Limit lim) {
  const int U = p.B * p.Hkv, ipp = kTile / p.P, lgP = __ffs(p.P) - 1;
  const int mine = lane >> 2, part = lane & 3;      // the lane's tile of a batch, its 16 rows
  const int pg = 16 * part >> lgP, at = 16 * part & (p.P - 1);
  const Run run = f.run;
  int u = run.unit, k = 0, kend = 0, slot = -1, ends = 0;
  bool open = false, draft = false, fresh = false;
  unsigned long long cc = run.before;
  int2 join = make_int2(-1, 0);
  Unit x = {};
  asm volatile("griddepcontrol.wait;" ::: "memory");   // (the shifts)
  // (an end for each team)
#pragma unroll 1
  for (int batch = 0; ends < kTeams; ++batch) {
    if (batch >= 2 &&
        !warp_wait(f.rfree[(batch - 2) & 3], ((batch - 2) >> 2) & 1, f, lim))
      break;
    int t_unit = 0, t_n = 0, t_np = 0, t_slot = -1;
    long long t_first = 0;
    uint32_t t_flags = kEnd;
#pragma unroll 1
    for (int e = 0; e < kBatch; ++e) {
      // the next unit with a part in this run
#pragma unroll 1
      while (!open && u < U && cc < run.to) {
        x = unit_of(p, u, RowsCost());
        Share y;
        if (share_of(p, x, run, c, cc, ipp, y)) {
          k = y.k;
          kend = y.kend;
          draft = y.draft;
          slot = y.slot;
          if (y.starts) join = make_int2(u, y.last);
          open = fresh = true;
        } else {
          cc += x.cost;
          ++u;
        }
      }
      uint32_t fl = kEnd;
      int np = 0;
      long long first = 0;
      if (open) {
        fl = fresh ? (uint32_t)kFirst : 0u;
        fresh = false;
        if (k < kend) {
          first = x.first + (long long)k * ipp;
          np = min(ipp, x.np - k * ipp);
          ++k;
        } else if (draft) {
          fl |= kDraft;
          draft = false;
        }
        // (a part without tiles gets an empty one)
        if (k >= kend && !draft) fl |= kLast;
      } else {
        ++ends;
      }
      if (mine == e) {
        t_unit = u;
        t_n = x.n;
        t_np = np;
        t_first = first;
        t_flags = fl;
        t_slot = slot;
      }
      if (fl & kLast) {
        open = false;
        cc += x.cost;
        ++u;
      }
    }
    // a lane per 16 rows
    Part o = {};
    o.at = (uint8_t)at;
    o.tier = 3;
    uint32_t bytes = 0;          // of the page, at its first part
    if (pg < t_np) {
      const uint32_t id = p.ids[t_first + pg], sl = id & 0x3FFFFFFFu;
      const int t = (int)(id >> 30);
      if (t > 2 || (long long)sl >= p.slots[t]) {
        report(p.err, SKV_ERR_CORRUPT);
      } else {
        const uint8_t* a = p.pool[t] + (long long)sl * p.stride[t];
        if (at == 0) prefetch_page(a, p.P, t);
        const uint32_t h = *reinterpret_cast<const uint32_t*>(a);
        const int rows = (int)(h & 0xFFFFu);
        if ((h >> 16) != ((uint32_t)t | ((uint32_t)kPageMagic << 8)) || rows > p.P) {
          report(p.err, SKV_ERR_CORRUPT);
        } else if (rows > at) {
          o.page = reinterpret_cast<unsigned long long>(a);
          o.rows = (uint8_t)min(rows - at, 16);
          o.tier = (uint8_t)t;
          if (at == 0) bytes = (uint32_t)(kHdrBytes + p.P * tier_row_bytes(t));
        }
      }
    }
    // where the part's page lies behind the tile's pages before it
    uint32_t sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t x = __shfl_sync(0xFFFFFFFFu, bytes, (lane & ~3) + k);
      if (k < part - (at >> 4)) o.off += x;
      sum += x;
    }
    unsigned long long valid = (unsigned long long)((1u << o.rows) - 1) << (16 * part);
    valid |= __shfl_xor_sync(0xFFFFFFFFu, valid, 1);
    valid |= __shfl_xor_sync(0xFFFFFFFFu, valid, 2);
    Tile& d = f.ring[(batch & 3) * kBatch + mine];
    d.part[part] = o;
    if (part == 0) {
      d.valid = (t_flags & kDraft) ? (t_n >= 64 ? ~0ull : (1ull << t_n) - 1) : valid;
      d.unit = t_unit;
      d.n = t_n;
      d.flags = t_flags;
      d.first = (int)t_first;
      d.slot = t_slot;
      d.bad = 0;
      d.bytes = sum;
      d.shift = (t_flags & kDraft) && p.shift ? p.shift[t_unit] : 0;
    }
    warp_arrive(f.dfull[batch & 3]);
  }
  if (lane == 0) p.join[c] = join;
}

// ----------------------------------------------------------------- the copier
// Brings the tiles' pages into the raw slots by bulk copies, whole pages in
// the order of the tiles.
template <class Limit>
__device__ __forceinline__ void copier(const TreeParams& p, Fixed& f, uint32_t base, int lane,
                                       Limit lim) {
  uint32_t used = 0;                 // slots of the last 8 tiles, 4 bits each
  int head = 0, held = 0, pos = 0;   // first tile not given back, slots in use, next slot
  // the copies in flight end before the block does
  const auto drain = [&](int t) {
    int none = 0;
    for (; head < t; ++head) mbar_wait_bounded(smem_u32(&f.rawfull[head & 7]), (head >> 3) & 1, &none);
  };
  for (int t = 0;; ++t) {
    if ((t & (kBatch - 1)) == 0 && !warp_wait(f.dfull[(t / kBatch) & 3], (t / kRing) & 1, f, lim)) {
      drain(t);
      return;
    }
    const Tile& d = f.ring[t & (kRing - 1)];
    if (d.flags & kEnd) {
      drain(t);   // (a decode warp that gave up has not waited for them)
      return;
    }
    const uint32_t bytes = d.bytes;
    int need = (int)((bytes + kRawSlot - 1) / kRawSlot), skip = 0;
    if (pos + need > kRawSlots) {
      skip = kRawSlots - pos;
      pos = 0;
    }
    while (held + need + skip > kRawSlots || t - head >= kRawTiles) {
      if (!warp_wait(f.rawfree[head & 7], (head >> 3) & 1, f, lim)) {
        drain(t);
        return;
      }
      held -= (int)(used >> (4 * (head & 7))) & 15;
      ++head;
    }
    const int x = t & 7;
    used = (used & ~(15u << (4 * x))) | ((uint32_t)(need + skip) << (4 * x));
    held += need + skip;
    const uint32_t to = base + kAtRaw + pos * kRawSlot, bar = smem_u32(&f.rawfull[x]);
    if (lane == 0) {
      f.raw[x] = to;
      if (bytes)
        mbar_arrive_expect_tx(bar, bytes);
      else
        mbar_arrive(bar);
    }
    __syncwarp();
    if (lane < 4) {
      const Part o = d.part[lane];
      if (o.tier < 3 && o.at == 0)
        bulk_g2s(to + o.off, reinterpret_cast<const void*>(o.page),
                 (uint32_t)(kHdrBytes + p.P * tier_row_bytes(o.tier)), bar);
    }
    __syncwarp();
    pos += need;
    if (pos == kRawSlots) pos = 0;
  }
}

// ----------------------------------------------------------------- the decode
// Lane (t, g) = 4 t + g of a warp: row t of its 8, key dims 32 i + 8 g + 0..7.
// Address of a code's entry in the lane's copy: byte k of w (T1); T2 pair j of
// nibbles nw, crumbs cw (the T2 table's address bits are disjoint from the
// index bits).
__device__ __forceinline__ uint32_t t1_at(uint32_t w, int k, uint32_t tb) {
  return tb + (__byte_perm(w, 0u, 0x4440u | (uint32_t)k) << 7);
}
__device__ __forceinline__ uint32_t t2_at(uint32_t nw, uint32_t cw, int j, uint32_t tb) {
  const int sn = 4 * (j & 7) - 7, sc = 2 * j - 11;
  const uint32_t xn = sn >= 0 ? (nw >> sn) : (nw << -sn);
  const uint32_t xc = sc >= 0 ? (cw >> sc) : (cw << -sc);
  return (xn & 0x780u) | (xc & 0x1800u) | tb;
}

// A part's keys (page: behind the header, in shared memory) -> fp16 rows
// T0 .. T0 + 15 of the tile at kb.
__device__ __forceinline__ void store_keys(uint32_t page, uint32_t tier, int at0, int P, uint32_t kb,
                                           int T0, int lane, uint32_t base) {
  const int t = lane >> 2, g = lane & 3, odd = t & 1;
  // odd rows go through their chunks in the order 1 0 3 2, which spreads a
  // quarter warp's stores over all banks
  const uint32_t row = kb + (uint32_t)(T0 + t) * 128;
  const uint32_t at[2] = {row + (((4 * odd + g) ^ t) << 4), row + (((4 * (odd ^ 1) + g) ^ t) << 4)};
  if (tier == SKV_TIER_T1) {
    const uint32_t tb = base + kAtTbl1 + 4 * lane;
    const uint32_t from = page + 2 * P + 64 * (at0 + t) + 16 * g, rad = page + 2 * (at0 + t);
    uint4 k[2];
    uint32_t r[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      k[h] = lds128(from + 512 * h);
      r[h] = lds16(rad + 16 * h);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t r2 = r[h] | (r[h] << 16);
      const uint32_t w[4] = {odd ? k[h].y : k[h].x, odd ? k[h].x : k[h].y, odd ? k[h].w : k[h].z,
                             odd ? k[h].z : k[h].w};
      uint32_t x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = lds32(t1_at(w[e >> 2], e & 3, tb));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sts128(at[e & 1] + (e >> 1) * kHalfDims + 1024 * h,
               make_uint4(hmul2(x[4 * e], r2), hmul2(x[4 * e + 1], r2), hmul2(x[4 * e + 2], r2),
                          hmul2(x[4 * e + 3], r2)));
    }
  } else if (tier == SKV_TIER_T2) {
    const uint32_t tb = base + kAtTbl2 + 4 * lane;
    const uint32_t from = page + 2 * P + 48 * (at0 + t), rad = page + 2 * (at0 + t);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint2 k = lds64(from + 384 * h + 8 * g);
      const uint32_t z = lds32(from + 384 * h + 32 + 4 * g);
      const uint32_t r = lds16(rad + 16 * h), r2 = r | (r << 16);
      // pairs 4 i .. 4 i + 3: nibbles and crumbs 4 i + b; odd rows swap halves
      const int sw = 16 * odd;
      const uint32_t n[2] = {__funnelshift_r(k.x, k.x, sw), __funnelshift_r(k.y, k.y, sw)};
      const uint32_t cw = odd ? ((z >> 8) & 0x00FF00FFu) | ((z << 8) & 0xFF00FF00u) : z;
      uint32_t x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = lds32(t2_at(n[e >> 3], cw, e, tb));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sts128(at[e & 1] + (e >> 1) * kHalfDims + 1024 * h,
               make_uint4(hmul2(x[4 * e], r2), hmul2(x[4 * e + 1], r2), hmul2(x[4 * e + 2], r2),
                          hmul2(x[4 * e + 3], r2)));
    }
  } else if (tier == SKV_TIER_T0) {
    const uint32_t from = page + 256 * (at0 + t);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = lds128(from + 2048 * h + 16 * ((4 * (e ^ odd) + g) ^ (4 * odd)));
#pragma unroll
      for (int e = 0; e < 4; ++e) sts128(at[e & 1] + (e >> 1) * kHalfDims + 1024 * h, x[e]);
    }
  } else {
#pragma unroll 1
    for (int e = 0; e < 8; ++e)
      sts128((e & 1 ? at[1] : at[0]) + ((e >> 1) & 1) * kHalfDims + 1024 * (e >> 2), make_uint4(0, 0, 0, 0));
  }
}

// A part's values -> fp16.  The tile's columns are a permutation of the
// dims that a lane of the pages' fragment order holds together: column
// 64 h + 8 g + 2 m + hi is dim 64 h + 16 m + 8 hi + g.
__device__ __forceinline__ void store_values(uint32_t page, uint32_t tier, int at0, int rows, int P,
                                             uint32_t vb, int T0, int lane) {
  const int g = lane >> 2, a = 2 * (lane & 3), b = a + 1;
  const uint32_t ra = vb + (uint32_t)(T0 + a) * 128 + ((g ^ a) << 4);
  const uint32_t rb = vb + (uint32_t)(T0 + b) * 128 + ((g ^ b) << 4);
  if (tier == SKV_TIER_T1 || tier == SKV_TIER_T2) {
    // v + 128 as the low byte of 1024 + x in fp16, less 1152 (exact), times
    // the scale (rounded once); rows that are not there get the scale 0
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t sec = page + (tier == SKV_TIER_T1 ? 66 : 50) * P;
    const uint32_t from = sec + 2 * P + 128 * at0 + 16 * lane;
    uint4 z[4];
    uint32_t s[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = lds128(from + 512 * e);
#pragma unroll
    for (int e = 0; e < 2; ++e) s[e] = lds32(sec + 2 * at0 + 2 * a + 16 * e);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t sa = a + 8 * e < rows ? __byte_perm(s[e], 0u, 0x1010) : 0u;
      const uint32_t sb = b + 8 * e < rows ? __byte_perm(s[e], 0u, 0x3232) : 0u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {z[2 * e + h].x, z[2 * e + h].y, z[2 * e + h].z, z[2 * e + h].w};
        uint32_t p[4], q[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t u = w[m] ^ 0x80808080u;
          const uint32_t x = __byte_perm(u, 0x64646464u, 0x4240),
                         y = __byte_perm(u, 0x64646464u, 0x4341);
          const __half2 hx = __hsub2(*reinterpret_cast<const __half2*>(&x), bias);
          const __half2 hy = __hsub2(*reinterpret_cast<const __half2*>(&y), bias);
          p[m] = hmul2(*reinterpret_cast<const uint32_t*>(&hx), sa);
          q[m] = hmul2(*reinterpret_cast<const uint32_t*>(&hy), sb);
        }
        sts128(ra + h * kHalfDims + 1024 * e, make_uint4(p[0], p[1], p[2], p[3]));
        sts128(rb + h * kHalfDims + 1024 * e, make_uint4(q[0], q[1], q[2], q[3]));
      }
    }
  } else if (tier == SKV_TIER_T0) {
    const uint32_t from = page + 256 * (P + at0) + 16 * lane;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool ua = a + 8 * e < rows, ub = b + 8 * e < rows;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 x = lds128(from + 2048 * e + 1024 * h), y = lds128(from + 2048 * e + 1024 * h + 512);
        uint4 p = make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.z, x.w, 0x5410),
                             __byte_perm(y.x, y.y, 0x5410), __byte_perm(y.z, y.w, 0x5410));
        uint4 q = make_uint4(__byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x7632),
                             __byte_perm(y.x, y.y, 0x7632), __byte_perm(y.z, y.w, 0x7632));
        if (!ua) p = make_uint4(0, 0, 0, 0);
        if (!ub) q = make_uint4(0, 0, 0, 0);
        sts128(ra + h * kHalfDims + 1024 * e, p);
        sts128(rb + h * kHalfDims + 1024 * e, q);
      }
    }
  } else {
#pragma unroll 1
    for (int e = 0; e < 4; ++e) {
      sts128(ra + (e & 1) * kHalfDims + 1024 * (e >> 1), make_uint4(0, 0, 0, 0));
      sts128(rb + (e & 1) * kHalfDims + 1024 * (e >> 1), make_uint4(0, 0, 0, 0));
    }
  }
}

// Drafted keys and values of 8 tokens.  A key is scaled by a power of two to
// fp16's range (taken off its scores again), so that bf16 keys enter exactly;
// a value outside fp16's range enters as 0 and is added at the segment's end.
__device__ __forceinline__ void store_draft(const TreeParams& p, const Tile& d, uint32_t kb,
                                         uint32_t vb, float* cs, int* bad, int T0, int lane) {
  const int t = lane >> 2, g = lane & 3, j = T0 + t;
  const int b = d.unit / p.Hkv, h = d.unit - b * p.Hkv;
  const bool live = j < d.n;
  const long long at = ((long long)b * p.N + j) * p.kv_stride + (long long)h * kHeadDim;
  uint4 x[4];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = make_uint4(0, 0, 0, 0);
    if (live)
      x[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.K) + at + 32 * i + 8 * g);
    mx = max_bits(max_bits(max_bits(max_bits(mx, x[i].x), x[i].y), x[i].z), x[i].w);
  }
  mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
  mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
  const int e = scale_exp(mx, p.kv_bf16);
  const float up = pow2i(e);
  const uint32_t row = kb + (uint32_t)j * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 y = from16x2(w[k], p.kv_bf16);
      w[k] = pack_f16x2(y.x * up, y.y * up);
    }
    sts128(row + (i >> 1) * kHalfDims + (((4 * (i & 1) + g) ^ t) << 4), make_uint4(w[0], w[1], w[2], w[3]));
  }
  if (g == 0) cs[j] = pow2i(-e);
  const float vup = pow2i(d.shift);
  bool out = false;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const int hf = c >> 1, gg = g + 4 * (c & 1);
    uint32_t w[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      float y[2] = {0.0f, 0.0f};
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        if (live)
          y[hi] = from16(static_cast<const uint16_t*>(p.V)[at + 64 * hf + 16 * m + 8 * hi + gg],
                         p.kv_bf16);
        if (!(fabsf(y[hi]) <= 65504.0f)) {
          y[hi] = 0.0f;
          out = true;
        }
      }
      w[m] = pack_f16x2(y[0] * vup, y[1] * vup);
    }
    sts128(vb + (uint32_t)j * 128 + hf * kHalfDims + ((gg ^ t) << 4), make_uint4(w[0], w[1], w[2], w[3]));
  }
  if (out) *(volatile int*)bad = 1;
}

template <bool BIAS, class Limit>
__device__ __forceinline__ void decode_role(const TreeParams& p, Fixed& f, uint32_t base, int wd,
                                            int lane, Limit lim) {
  const int w = wd & (kTeamWarps - 1), P = p.P, T0 = 16 * w;
  int t = wd / kTeamWarps;
  uint32_t stage = t, use = 0;   // of tile t: its stage, the stage's tiles before
  if (!warp_wait(f.dfull[0], 0, f, lim)) return;
  for (;;) {
    Tile& d = f.ring[t & (kRing - 1)];
    const uint32_t flags = d.flags;
    if (flags & kEnd) return;
    const Part x = d.part[w];
    const uint32_t kb = keys_at(base, stage), vb = values_at(base, stage);
    const int y = t & (kRawTiles - 1);
    if (!warp_wait(f.rawfull[y], (t / kRawTiles) & 1, f, lim)) return;
    const uint32_t page = f.raw[y] + x.off + kHdrBytes;
    if (use > 0 && !warp_wait(f.kempty[stage], (use - 1) & 1, f, lim)) return;
    const bool draft = (flags & kDraft) != 0;
    if (!draft) store_keys(page, x.tier, x.at, P, kb, T0, lane, base);
    if (BIAS || draft) {
      // (positions and scales are in use until the stage's values are free)
      if (use > 0 && !warp_wait(f.vempty[stage], (use - 1) & 1, f, lim)) return;
      if (BIAS && lane < 16) {
        const long long b = d.unit / p.Hkv;
        const int q0 = p.q_pos[b * p.N];
        int q = q0;
        if (draft) {
          if (T0 + lane < d.n) q = p.q_pos[b * p.N + T0 + lane];
        } else if (lane < x.rows) {
          q = p.row_pos[(long long)d.first * P + T0 + lane];  // (a tile's pages follow each other)
          if (q < 0) {
            // no position names the row: its column holds no token
            report(p.err, SKV_ERR_CORRUPT);
            atomicAnd(&d.valid, ~(1ull << (T0 + lane)));
          }
        }
        f.pos[stage][T0 + lane] = (float)(q - q0);
      }
      if (draft) {
#pragma unroll 1
        for (int e = 0; e < 16; e += 8) store_draft(p, d, kb, vb, f.cs[stage], &d.bad, T0 + e, lane);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    warp_arrive(f.kfull[stage]);
    if (!draft) {
      if (use > 0 && !warp_wait(f.vempty[stage], (use - 1) & 1, f, lim)) return;
      store_values(page, x.tier, x.at, x.rows, P, vb, T0, lane);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    warp_arrive(f.vfull[stage]);
    if (lane == 0) mbar_arrive(smem_u32(&f.rawfree[y]));
    const int t2 = t + kTeams;
    if ((t2 ^ t) & kBatch && !warp_wait(f.dfull[(t2 / kBatch) & 3], (t2 / kRing) & 1, f, lim)) return;
    t = t2;
    stage += kTeams;
    if (stage >= kStages) {
      stage -= kStages;
      ++use;
    }
  }
}

// ------------------------------------------------------------------- the MMAs
// S = Q K^T of every job, as soon as the keys are there and the stream's
// scores are read (two blocks: its weights used).
template <class Limit>
__device__ __forceinline__ void mma_scores(const TreeParams& p, Fixed& f, uint32_t base, uint32_t tm,
                                           Limit lim) {
  const int most = 128 * p.Hkv;       // n * Hq above it: two blocks
  uint32_t turn = 3;                  // bit s: parity of stream s's job before
  uint32_t segs = 0, stage = 0, use = 0, s = 0;
  bool two = false;
  for (int t = 0;; ++t) {
    if ((t & (kBatch - 1)) == 0 && !warp_wait(f.dfull[(t / kBatch) & 3], (t / kRing) & 1, f, lim))
      return;
    const uint32_t flags = f.ring[t & (kRing - 1)].flags;
    if (flags & kEnd) return;
    if (flags & kFirst) {
      if (!warp_wait(f.qfull, segs & 1, f, lim)) return;
      ++segs;
      two = f.ring[t & (kRing - 1)].n * p.Hq > most;
      s = 0;
    }
    if (!warp_wait(f.kfull[stage], use & 1, f, lim)) return;
    const uint32_t low = kDescKeys | (keys_at(base, stage) >> 4);
#pragma unroll 1
    for (int y = two ? 1 : 0; y >= 0; --y) {
      if (!warp_wait(f.sfree[s], (turn >> s) & 1, f, lim)) return;
      if (two && !warp_wait(f.odone[s], (turn >> s) & 1, f, lim)) return;
      turn ^= 1u << s;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t a = tm + kColQ + (two ? 64 * s : 0), o = tm + kColS + 64 * s;
#pragma unroll
        for (int k = 0; k < kHeadDim / 16; ++k)
          tc_mma(o, a + 8 * k, operand(low + (k >> 2) * (kHalfDims / 16) + (k & 3) * 2), kIdescS,
                 k > 0);
        tc_commit(smem_u32(&f.sfull[s]));
        if (y == 0) tc_commit(smem_u32(&f.kempty[stage]));
      }
      __syncwarp();
      s ^= 1;
    }
    if (++stage == kStages) {
      stage = 0;
      ++use;
    }
  }
}

// O += P V of every job, as soon as its weights are there.
template <class Limit>
__device__ __forceinline__ void mma_sums(const TreeParams& p, Fixed& f, uint32_t base, uint32_t tm,
                                         Limit lim) {
  const int most = 128 * p.Hkv;
  uint32_t turn = 0;                  // bit s: parity of stream s's job
  uint32_t add = 0;                   // bit s: stream s has had a job in the segment
  uint32_t stage = 0, use = 0, s = 0;
  bool two = false;
  for (int t = 0;; ++t) {
    if ((t & (kBatch - 1)) == 0 && !warp_wait(f.dfull[(t / kBatch) & 3], (t / kRing) & 1, f, lim))
      return;
    const uint32_t flags = f.ring[t & (kRing - 1)].flags;
    if (flags & kEnd) return;
    if (flags & kFirst) {
      add = s = 0;
      two = f.ring[t & (kRing - 1)].n * p.Hq > most;
    }
    if (!warp_wait(f.vfull[stage], use & 1, f, lim)) return;
    const uint32_t low = kDescValues | (values_at(base, stage) >> 4);
#pragma unroll 1
    for (int y = two ? 1 : 0; y >= 0; --y) {
      if (!warp_wait(f.pfull[s], (turn >> s) & 1, f, lim)) return;
      turn ^= 1u << s;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t a = tm + (two ? kColS + 64 * s : kColP + 32 * s), o = tm + kColO + 128 * s;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          tc_mma(o, a + 8 * k, operand(low + 128 * k), kIdescO, k > 0 ? 1u : (add >> s) & 1);
        tc_commit(smem_u32(&f.odone[s]));
        if (y == 0) {
          tc_commit(smem_u32(&f.vempty[stage]));
          if ((t & (kBatch - 1)) == kBatch - 1) tc_commit(smem_u32(&f.rfree[(t / kBatch) & 3]));
        }
      }
      __syncwarp();
      add |= 1u << s;
      s ^= 1;
    }
    if (++stage == kStages) {
      stage = 0;
      ++use;
    }
  }
}

// ---------------------------------------------------------------- the softmax
struct Row {           // a lane's row in its stream
  float c;             // what a product is scaled by (log2 domain; capped: to x / cap)
  float cap, slope, rel;
  float m, l;
  uint32_t turn;       // parity of the stream's next job
  int mine;            // its jobs in the segment
};

// The maximum of the lanes that need it rises to `top`: their sums, O and the
// weights of the job's columns before `done` (at pa) follow.
template <class Limit>
__device__ __forceinline__ bool raise(Fixed& f, Row& r, float top, uint32_t pa, int done,
                                      uint32_t oa, int wg, float up, Limit lim) {
  const float m = top > r.m + kRaise ? top : r.m;
  const float a = m == r.m ? 1.0f : ex2f(r.m - m);
  r.l *= a;
  r.m = m;
  const uint32_t a2 = pack_f16x2(a, a);
  tc_wait_st();
#pragma unroll 1
  for (int k = 0; k < done; k += 16) {
    uint32_t w[8];
    tc_ld8(pa + k / 2, w);
    tc_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = hmul2(w[e], a2);
    tc_st8(pa + k / 2, w);
  }
  if (r.mine > 0) {
    if (!warp_wait(f.odone[wg], r.turn ^ 1, f, lim)) return false;
    tc_fence_after();
    const float au = a * up;
#pragma unroll 1
    for (int k = 0; k < kHeadDim; k += 16) {
      float o[16];
      tc_ld16(oa + k, o);
      tc_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] *= au;
      tc_st8(oa + k, reinterpret_cast<const uint32_t*>(o));
      tc_st8(oa + k + 8, reinterpret_cast<const uint32_t*>(o) + 8);
    }
  }
  tc_wait_st();
  return true;
}

// s <- cap tanh(s c / cap) (log2 domain): z = s r.c = x / cap.  Where every |z| of
// the warp is at most 1/2 (scores are usually small beside their cap) by the
// series of cap_series: packed products instead of two of the three special
// functions a score takes, which are what bounds a job (16 a cycle and SM).
// Else by 1 - 2 / (1 + e^(2 z)), with a high cap score by score (cap_any).
__device__ __forceinline__ void cap_scores(const Row& r, float (&s)[32]) {
  float big[2] = {fabsf(s[0]), fabsf(s[1])};
#pragma unroll
  for (int k = 2; k < 32; ++k) big[k & 1] = fmaxf(big[k & 1], fabsf(s[k]));
  if (!__any_sync(0xFFFFFFFFu, !(fmaxf(big[0], big[1]) * r.c <= 0.5f))) {
    const auto both = [](float x) { return make_float2(x, x); };
    const float2 c2 = both(r.c), a2 = both(r.cap), none = both(0.0f);
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const float2 z = fma2(make_float2(s[k], s[k + 1]), c2, none), u = fma2(z, z, none);
      float2 y = fma2(both(21844.0f / 6081075.0f), u, both(-1382.0f / 155925.0f));
      y = fma2(y, u, both(62.0f / 2835.0f));
      y = fma2(y, u, both(-17.0f / 315.0f));
      y = fma2(y, u, both(2.0f / 15.0f));
      y = fma2(y, u, both(-1.0f / 3.0f));
      const float2 az = fma2(a2, z, none);
      y = fma2(fma2(y, u, none), az, az);
      s[k] = y.x;
      s[k + 1] = y.y;
    }
  } else if (r.cap <= kLowCap * 1.4426950408889634f) {
    const float c = fminf(r.c * (2.0f * 1.4426950408889634f), 3.0e38f);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float e = ex2f(s[k] * c);
      s[k] = fmaf(-2.0f * r.cap, rcpf(1.0f + e), r.cap);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 32; ++k) s[k] = cap_any(s[k] * r.c, r.cap);
  }
}

// n columns (32 or 64) of a job, 32 at a time: scores (at sa) to weights (at
// pa); bits: the columns this row sees.
template <bool CAP, bool BIAS, class Limit>
__device__ __forceinline__ bool softmax_job(Fixed& f, Row& r, uint32_t sa, uint32_t pa,
                                            uint32_t oa, int wg, int n, unsigned long long bits,
                                            const float* cs, const float* pos, int shift,
                                            Limit lim) {
  float s[32];
  tc_ld16(sa, s);
  tc_ld16(sa + 16, s + 16);
#pragma unroll 1
  for (int c = 0; c < n; c += 32) {
    tc_wait_ld();
    if (c + 32 >= n) {
      tc_fence_before();
      warp_arrive(f.sfree[wg]);
    }
    if (cs) {
#pragma unroll
      for (int k = 0; k < 32; ++k) s[k] *= cs[c + k];
    }
    if (CAP) cap_scores(r, s);
    if (BIAS) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        s[k] = fmaf(r.slope, pos[c + k] - r.rel, CAP ? s[k] : s[k] * r.c);
    }
    const uint32_t see = (uint32_t)(bits >> c);
    if (see != 0xFFFFFFFFu) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (!((see >> k) & 1)) s[k] = -INFINITY;
    }
    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int k = 4; k < 32; ++k) mx[k & 3] = fmaxf(mx[k & 3], s[k]);
    float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    if (!(CAP || BIAS)) top *= r.c;
    if (__any_sync(0xFFFFFFFFu, top > r.m + kRaise || (c == 0 && shift != 0))) {
      if (!raise(f, r, top, pa, c, oa, wg, c == 0 ? pow2i(shift) : 1.0f, lim)) return false;
    }
    const float m = r.m == -INFINITY ? 0.0f : r.m;
    const float2 c2 = make_float2(r.c, r.c), m2 = make_float2(-m, -m);
    float2 l2 = make_float2(r.l, 0.0f);
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float2 x = make_float2(s[2 * e], s[2 * e + 1]);
      x = (CAP || BIAS) ? add2(x, m2) : fma2(x, c2, m2);
      x.x = ex2f(x.x);
      x.y = ex2f(x.y);
      l2 = add2(l2, x);
      w[e] = pack_f16x2(x.x, x.y);
    }
    r.l = l2.x + l2.y;
    if (c + 32 < n) {
      tc_ld16(sa + c + 32, s);
      tc_ld16(sa + c + 48, s + 16);
    }
    // (the product before may still read its weights)
    if (c == 0 && r.mine > 0 && !warp_wait(f.odone[wg], r.turn ^ 1, f, lim)) {
      tc_wait_ld();   // the next columns arrive in their registers first
#pragma unroll
      for (int k = 0; k < 32; ++k) asm volatile("" : "+f"(s[k]));
      return false;
    }
    tc_st8(pa + c / 2, w);
    tc_st8(pa + c / 2 + 8, w + 8);
  }
  tc_wait_st();
  return true;
}

template <bool CAP, bool BIAS, class Limit>
__device__ __forceinline__ void softmax_role(const TreeParams& p, Fixed& f, float* buf, Sums& sum,
                                             uint32_t tm0, int warp, int lane, Limit lim) {
  const int G = p.Hq / p.Hkv;
  const int wg = warp >> 2, part = warp & 3, tl = 32 * part + lane;
  const uint32_t tm = tm0 + ((uint32_t)(32 * part) << 16);
  const uint32_t oa = tm + kColO + 128 * wg;
  Row r = {};
  uint32_t syncs = 0;
  const int lgG = __ffs(G) - 1;
  int nb = 1, rc = 128, copy = 0, R = 0;
  bool busy = true;  // the warp has rows
  int next = 0;      // jobs to the stream's next one
  uint32_t stage = kStages - 1;
  unsigned long long see = 0;
  const auto meet = [&]() {
    warp_arrive(f.sync);
    return warp_wait(f.sync, syncs++ & 1, f, lim);
  };
  for (int t = 0;; ++t) {
    if ((t & (kBatch - 1)) == 0 && !warp_wait(f.dfull[(t / kBatch) & 3], (t / kRing) & 1, f, lim))
      return;
    const Tile& d = f.ring[t & (kRing - 1)];
    const uint32_t flags = d.flags;
    if (flags & kEnd) return;
    if (flags & kFirst) {
      R = d.n * G;
      nb = R > 128 ? 2 : 1;
      rc = R <= 64 ? 64 : 128;
      const int row = nb == 2 ? 128 * wg + tl : (tl & (rc - 1));
      copy = nb == 2 ? 0 : tl / rc;
      const int b = d.unit / p.Hkv, h = d.unit - b * p.Hkv;
      const int i = row >> lgG, hq = h * G + (row & (G - 1));
      const bool live = row < R;
      busy = __any_sync(0xFFFFFFFFu, live);
      const long long tok = (long long)b * p.N + i;
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                      tok * p.q_stride + (long long)hq * kHeadDim);
      // the row as fp16 scaled by a power of two (bf16 converts exactly)
      uint32_t mx = 0;
#pragma unroll 4
      for (int k = 0; k < 16; ++k) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (live) x = q[k];
        mx = max_bits(max_bits(max_bits(max_bits(mx, x.x), x.y), x.z), x.w);
      }
      const int e = scale_exp(mx, p.q_bf16);
      const float up = pow2i(e);
      // one block: both streams use it, each group writes half its dims
#pragma unroll 1
      for (int k = 0; k < 16; k += 2) {
        if (nb == 1 && (k >> 3) != wg) continue;
        uint32_t w[8];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (live) x = q[k + y];
          const uint32_t z[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float2 a = from16x2(z[v], p.q_bf16);
            w[4 * y + v] = pack_f16x2(a.x * up, a.y * up);
          }
        }
        tc_st8(tm + kColQ + (nb == 2 ? 64 * wg : 0) + 4 * k, w);
      }
      if (nb == 1) {
        // the weights of the other copies' columns stay zero
        const uint32_t z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 32; k += 8) tc_st8(tm + kColP + 32 * wg + k, z);
      }
      tc_wait_st();
      tc_fence_before();
      warp_arrive(f.qfull);
      const float log2e = 1.4426950408889634f;
      const float c = p.qk_scale * pow2i(-e);
      if (CAP) {
        r.c = fminf(c / p.softcap, 3.0e38f);   // (0 times it stays 0)
        r.cap = p.softcap * log2e;
      } else {
        r.c = c * log2e;
      }
      if (BIAS) {
        r.slope = live ? p.slopes[hq] * log2e : 0.0f;
        const int q0 = p.q_pos[(long long)b * p.N];
        r.rel = live ? (float)(p.q_pos[tok] - q0) : 0.0f;
      }
      r.m = -INFINITY;
      r.l = 0.0f;
      r.mine = 0;
      next = wg;
      see = 0;
      if (live && p.K)
        see = p.mask ? p.mask[tok] : (i >= 63 ? ~0ull : (2ull << i) - 1);
    }
    if (++stage == kStages) stage = 0;
    // one block: the streams take the tiles in turn; two: every tile
    if (nb == 2 || next == 0) {
      if (!warp_wait(f.sfull[wg], r.turn, f, lim)) return;
      tc_fence_after();
      if (busy) {
        const int n = kTile * rc / 128, c0 = copy * n;
        unsigned long long bits = d.valid;
        const float* cs = nullptr;
        if (flags & kDraft) {
          bits &= see;
          cs = f.cs[stage] + c0;
        }
        const uint32_t sa = tm + kColS + 64 * wg + c0;
        const uint32_t pa = nb == 2 ? sa : tm + kColP + 32 * wg + c0 / 2;
        if (!softmax_job<CAP, BIAS>(f, r, sa, pa, oa, wg, n, bits >> c0, cs, f.pos[stage] + c0,
                                    flags & kDraft ? d.shift : 0, lim))
          return;
      } else {
        warp_arrive(f.sfree[wg]);
        // (not ahead of the warps that have rows: the job's weights are complete
        // when all four have arrived)
        if (r.mine > 0 && !warp_wait(f.odone[wg], r.turn ^ 1, f, lim)) return;
      }
      tc_fence_before();
      warp_arrive(f.pfull[wg]);
      r.turn ^= 1;
      ++r.mine;
    }
    next ^= 1;
    if (!(flags & kLast)) continue;
    // the segment's end: the streams' and copies' sums meet, 32 dims at a time
    if (r.mine > 0) {
      if (!warp_wait(f.odone[wg], r.turn ^ 1, f, lim)) return;
      tc_fence_after();
    }
    sum.m[wg][tl] = r.m;
    sum.l[wg][tl] = r.l;
    if (!meet()) return;
    // (now: only the stream that had the drafted tile has waited for its decode)
    const bool bad = *(const volatile int*)&d.bad != 0;
    float* const mine = buf + tl * kBufRow;
    const int copies = 128 / rc, sub = tl & (rc - 1);
    // (the drafted tile is the segment's last: this stream's?)
    float a = (flags & kDraft) && (nb == 2 || next == 1) ? pow2i(-d.shift) : 1.0f;
    if (nb == 1) {
      float M = -INFINITY;
      for (int k = 0; k < copies; ++k)
        M = fmaxf(M, fmaxf(sum.m[0][sub + rc * k], sum.m[1][sub + rc * k]));
      a *= r.m == -INFINITY ? 0.0f : ex2f(r.m - M);
    }
#pragma unroll 1
    for (int step = 0; step < 8; ++step) {
      // one block: the streams in turn, the second adds to the first's; two
      // blocks: a block's quarters in turn
      const int qt = nb == 1 ? step >> 1 : step & 3, s = nb == 1 ? 1 - (step & 1) : step >> 2;
      if (wg == s && busy) {
#pragma unroll 1
        for (int k = 0; k < 32; k += 16) {
          float o[16];
          if (r.mine > 0) {
            tc_ld16(oa + 32 * qt + k, o);
            tc_wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (a != 0.0f) x = make_float4(o[e] * a, o[e + 1] * a, o[e + 2] * a, o[e + 3] * a);
            float4* to = reinterpret_cast<float4*>(mine + k + e);
            if (nb == 1 && s == 0) {
              const float4 y = *to;
              x.x += y.x;
              x.y += y.y;
              x.z += y.z;
              x.w += y.w;
            }
            *to = x;
          }
        }
        tc_fence_before();
      }
      if (!meet()) return;
      if (nb == 1 && s == 1) continue;
      // a quarter's columns 32 qt .. + 31: dims 64 h + 16 m + 8 hi + g of four
      // g, column 8 (g & 3) + 2 m + hi of the buffer.  Lane l of 8 has the
      // dims of (m, hi)
      const int l = lane & 7, top = nb == 1 ? R : min(128, R - 128 * s);
      for (int x = 4 * warp + (lane >> 3); x < top; x += 4 * kSoftWarps) {
        float Mx = -INFINITY, Lx = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < copies; ++k) {
          const int z = x + rc * k;
          const float* from = buf + z * kBufRow + l;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += from[8 * e];
          Mx = nb == 2 ? sum.m[s][z] : fmaxf(Mx, fmaxf(sum.m[0][z], sum.m[1][z]));
        }
        if (nb == 2) {
          Lx = sum.l[s][x];
          if (Mx == -INFINITY) v[0] = v[1] = v[2] = v[3] = 0.0f;
        } else {
          for (int k = 0; k < copies; ++k) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              // (a sum without a maximum: 0, or NaN where every score is NaN)
              const float mz = sum.m[y][x + rc * k], lz = sum.l[y][x + rc * k];
              if (lz != 0.0f) Lx += mz == -INFINITY ? lz : lz * ex2f(mz - Mx);
            }
          }
        }
        const int d0 = 64 * (qt >> 1) + 16 * (l >> 1) + 8 * (l & 1) + 4 * (qt & 1);
        write_row<CAP, BIAS, 8>(p, d.unit, d.n, d.slot, bad, nb == 1 ? x : 128 * s + x, Mx, Lx, v, d0,
                                lane);
      }
      // (behind the last step too: a stream without a tile in the next segment
      // waits for nothing there before it writes its sums)
      if (!meet()) return;
    }
  }
}

template <bool CAP, bool BIAS, class Limit>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(128) uint8_t raw[];
  Fixed& f = *reinterpret_cast<Fixed*>(raw);
  const uint32_t at = smem_u32(raw), base = (at + (uint32_t)sizeof(Fixed) + 8191u) & ~8191u;
  uint8_t* const mem = raw + (base - at);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (base + kHighBytes > at + kSmemBytes) {
    // (the window starts at 1 KB: it fits)
    if (tid == 0) report(p.err, SKV_ERR_CUDA);
    return;
  }

  if (tid == 0) {
    f.late = 0;
    for (int k = 0; k < kStages; ++k) {
      mbar_init(smem_u32(&f.kfull[k]), kTeamWarps);
      mbar_init(smem_u32(&f.vfull[k]), kTeamWarps);
      mbar_init(smem_u32(&f.kempty[k]), 1);
      mbar_init(smem_u32(&f.vempty[k]), 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(smem_u32(&f.sfull[k]), 1);
      mbar_init(smem_u32(&f.sfree[k]), 4);
      mbar_init(smem_u32(&f.pfull[k]), 4);
      mbar_init(smem_u32(&f.odone[k]), 1);
    }
    mbar_init(smem_u32(&f.qfull), kSoftWarps);
    mbar_init(smem_u32(&f.sync), kSoftWarps);
    mbar_init(smem_u32(&f.fin[0]), 1);
    mbar_init(smem_u32(&f.fin[1]), 1);
    for (int k = 0; k < kRawTiles; ++k) {
      mbar_init(smem_u32(&f.rawfull[k]), 1);
      mbar_init(smem_u32(&f.rawfree[k]), kTeamWarps);
    }
    for (int k = 0; k < kRing / kBatch; ++k) {
      mbar_init(smem_u32(&f.dfull[k]), 1);
      mbar_init(smem_u32(&f.rfree[k]), 1);
    }
    fence_mbar_init();
  }
  if (warp == kMmaS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&f.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  key_tables(p, base + kAtTbl1, 128, base + kAtTbl2, tid, kThreads);
  tc_fence_before();
  find_run<kThreads>(p, blockIdx.x, f.scan, &f.run, RowsCost());  // (block-wide barriers)
  tc_fence_after();
  const uint32_t tm = *(volatile uint32_t*)&f.tmem;
  const Limit lim(p);

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    softmax_role<CAP, BIAS>(p, f, reinterpret_cast<float*>(mem + kAtBuf),
                            *reinterpret_cast<Sums*>(mem + kAtSums), tm, warp, lane, lim);
    tc_wait_st();   // (a role that gave up leaves stores in flight)
  } else if (warp < kPlanner) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDecode));
    decode_role<BIAS>(p, f, base, warp - kSoftWarps, lane, lim);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsHelp));
    if (warp == kPlanner) {
      planner(p, f, blockIdx.x, lane, lim);
    } else if (warp == kCopier) {
      copier(p, f, base, lane, lim);
    } else {
      if (warp == kMmaS)
        mma_scores(p, f, base, tm, lim);
      else
        mma_sums(p, f, base, tm, lim);
      // nothing in flight when tensor memory is given back
      unsigned long long& fin = f.fin[warp - kMmaS];
      if (elect_one()) tc_commit(smem_u32(&fin));
      __syncwarp();
      int none = 0;
      if (!mbar_wait_bounded(smem_u32(&fin), 0, &none) && lane == 0) report(p.err, SKV_ERR_TIMEOUT);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && f.late) report(p.err, SKV_ERR_TIMEOUT);
  if (warp == kMmaS) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm));
  }
}

// The parts of the units that several runs share: a warp per row.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const __grid_constant__ TreeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int2 join = p.join[c];
  if (join.x < 0) return;
  const int G = p.Hq / p.Hkv, b = join.x / p.Hkv, h = join.x - b * p.Hkv;
  const int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  const int n = p.count ? min(max(p.count[b], 0), p.N) : p.N;
  if (r >= n * G) return;
  const int rows = p.N * G, parts = join.y - c + 1;
  // part k: slot 2 c + 1 of the first run, 2 (c + k) of the others
  const auto at = [&](int k) {
    return (long long)(k == 0 ? 2 * c + 1 : 2 * (c + k)) * rows + r;
  };
  // 16 parts' loads at once
  float M = -INFINITY, L = 0.0f;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  constexpr int kAtOnce = 16;
  for (int k0 = 0; k0 < parts; k0 += kAtOnce) {
    float2 ml[kAtOnce];
    float4 x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      ml[k] = make_float2(-INFINITY, 0.0f);
      x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (k0 + k < parts) {
        ml[k] = p.part_ml[at(k0 + k)];
        x[k] = *reinterpret_cast<const float4*>(p.part + at(k0 + k) * kHeadDim + 4 * lane);
      }
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) m = fmaxf(m, ml[k].x);
    const float keep = M == m ? 1.0f : ex2f(M - m);
    M = m;
    L *= keep;
    v = make_float4(v.x * keep, v.y * keep, v.z * keep, v.w * keep);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const float a = ml[k].x == -INFINITY ? 0.0f : ex2f(ml[k].x - M);
      L += ml[k].x == -INFINITY ? ml[k].y : a * ml[k].y;
      v.x += a * x[k].x;
      v.y += a * x[k].y;
      v.z += a * x[k].z;
      v.w += a * x[k].w;
    }
  }
  const int i = r >> (__ffs(G) - 1), hq = h * G + (r & (G - 1));
  const long long tok = (long long)b * p.N + i;
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  uint2 w;
  if (p.q_bf16)
    w = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
  else
    w = make_uint2(pack_f16x2(v.x * inv, v.y * inv), pack_f16x2(v.z * inv, v.w * inv));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (tok * p.Hq + hq) * kHeadDim + 4 * lane) = w;
  if (lane == 0 && p.lse)
    p.lse[tok * p.Hq + hq] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// No positions yet (rows that no position below seq_lens names stay at -1): the
// listed pages only, a capacity may be far larger.
__global__ void __launch_bounds__(256) tree_unplaced_kernel(const __grid_constant__ TreeParams p) {
  const long long pages = min((long long)p.indptr[p.B * p.Hkv], p.page_cap), words = pages * p.P / 4;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < words;
       i += (long long)gridDim.x * blockDim.x)
    reinterpret_cast<int4*>(p.row_pos)[i] = make_int4(-1, -1, -1, -1);
}

// Positions of the store's rows: row_pos[page * P + row] = t, by the row map.
__global__ void __launch_bounds__(256) tree_positions_kernel(const __grid_constant__ TreeParams p) {
  const long long U = (long long)p.B * p.Hkv;
  for (long long u = blockIdx.y; u < U; u += gridDim.y) {
    const long long T = min((long long)p.seq_lens[u / p.Hkv], p.Tmax);
    const long long a = p.indptr[u], rows = ((long long)p.indptr[u + 1] - a) * p.P;
    for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < T;
         t += (long long)gridDim.x * blockDim.x) {
      const long long r = p.row_of[u * p.Tmax + t];
      if (r < 0) continue;
      if (a < 0 || r >= rows || a * p.P + r >= p.page_cap * p.P)
        report(p.err, SKV_ERR_CORRUPT);
      else
        p.row_pos[a * p.P + r] = (int32_t)t;
    }
  }
}

// Drafted bf16 values that are all small enter times a power of two (their
// largest between 1 and 2; the sums before them follow, see raise): fp16 holds
// all bits of those above 2^-14 only.  At 2^-6 and above what is lost lies 2^-19
// below the largest.  A warp per unit; the kernel that reads the shifts starts
// beside this one.  (Inside it, in any role, the few instructions cost 2 to 28%
// of the prompt batch by where they put the others' loops.)
__global__ void __launch_bounds__(256) tree_shift_kernel(const __grid_constant__ TreeParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int u = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (u >= p.B * p.Hkv) return;
  const int b = u / p.Hkv, h = u - b * p.Hkv;
  const int n = p.count ? min(max(p.count[b], 0), p.N) : p.N;
  const uint16_t* V = static_cast<const uint16_t*>(p.V) + (long long)b * p.N * p.kv_stride +
                      (long long)h * kHeadDim + 8 * (lane & 15);
  uint32_t mx = 0;
#pragma unroll 8
  for (int j = lane >> 4; j < n; j += 2) {
    const uint4 x = *reinterpret_cast<const uint4*>(V + j * p.kv_stride);
    mx = held_bits(held_bits(held_bits(held_bits(mx, x.x), x.y), x.z), x.w);
  }
  const int e = scale_exp(__reduce_max_sync(0xFFFFFFFFu, mx), 1) - 14;
  if (lane == 0) p.shift[u] = e > 6 ? min(e, 60) : 0;
}

template <bool CAP, bool BIAS>
cudaError_t launch(const TreeParams& p, cudaStream_t stream) {
  const auto kernel = p.wait_limit ? tree_kernel<CAP, BIAS, SetLimit>
                                   : tree_kernel<CAP, BIAS, DefaultLimit>;
  const cudaError_t e = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  if (p.shift) {
    tree_shift_kernel<<<(unsigned)(((long long)p.B * p.Hkv + 7) / 8), 256, 0, stream>>>(p);
    const cudaError_t s = cudaGetLastError();
    if (s != cudaSuccess) return s;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.S);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.shift ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

// Workspace: the positions, then the joins, the units' shifts, then the parts of
// two slots a run.
size_t tree_workspace_bytes(long long page_cap, int P, int positions, int S, int units, int N,
                            int G, TreeParams* p, void* ws) {
  const size_t pos = positions ? ((size_t)page_cap * P * 4 + 127) / 128 * 128 : 0;
  const size_t join = ((size_t)S * 8 + 127) / 128 * 128;
  const size_t shift = N * G > kTreeRows ? ((size_t)units * 4 + 127) / 128 * 128 : 0;
  const size_t rows = 2ull * S * N * G;
  if (p) {
    uint8_t* w = static_cast<uint8_t*>(ws);
    p->row_pos = reinterpret_cast<int32_t*>(w);
    p->join = reinterpret_cast<int2*>(w + pos);
    p->shift = shift && p->V && p->kv_bf16 ? reinterpret_cast<int32_t*>(w + pos + join) : nullptr;
    p->part = reinterpret_cast<float*>(w + pos + join + shift);
    p->part_ml = reinterpret_cast<float2*>(w + pos + join + shift + rows * kHeadDim * 4);
  }
  return pos + join + shift + rows * (kHeadDim * 4 + 8);
}

cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream) {
  const long long U = (long long)p.B * p.Hkv;
  if (U == 0) return cudaSuccess;
  cudaError_t e;
  if (p.slopes && p.page_cap > 0) {
    const long long words = p.page_cap * p.P / 4;
    tree_unplaced_kernel<<<(unsigned)std::min<long long>((words + 255) / 256, 1184), 256, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (p.slopes && p.Tmax > 0) {
    const long long bx = std::min<long long>((p.Tmax + 255) / 256, std::max<long long>(1, 1184 / U));
    tree_positions_kernel<<<dim3((unsigned)bx, (unsigned)std::min<long long>(U, 65535)), 256, 0,
                            stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (p.N * (p.Hq / p.Hkv) <= kTreeRows)
    e = launch_tree_rows(p, stream);
  else if (p.softcap > 0.0f)
    e = p.slopes ? launch<true, true>(p, stream) : launch<true, false>(p, stream);
  else
    e = p.slopes ? launch<false, true>(p, stream) : launch<false, false>(p, stream);
  if (e != cudaSuccess) return e;
  // the join: its launch overlaps the grid before it, its work waits for it
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.S, (unsigned)((p.N * (p.Hq / p.Hkv) + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel, p);
}

}  // namespace skv
