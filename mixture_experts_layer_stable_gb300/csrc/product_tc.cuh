// product_tc.cuh -- the experts' products on the tensor cores (tcgen05 kind::f16;
// product.cu has the formulas and the calls; each form is compiled in a file of its own).
//
// Warp-specialised and persistent, one CTA per SM: warp 0 issues the copies (or sixteen
// more warps load the operands themselves), one thread of warp 1 the tensor-core
// instructions, warps 2..9 the epilogue.
//
// The MMA's M side are the output's columns (the weights; for the weights' gradient dy's
// columns), 128 a CTA, and its N side the output's rows: up to 256 rows of an expert, or
// 256 columns of x.  So the MMA's time goes with the rows there are, rounded up to 32,
// and an expert with a few rows costs its weight stream and little else; and a TMEM lane
// holds one output column, so a warp stores 32 neighbours of a row with one instruction,
// whatever the row's alignment.
//
// A unit is (expert, 128 or 256 output columns, tile of output rows); a stage of the ring
// holds 64 of the contraction: 16 KB of the M side and 128 bytes for every output row.
// What is contiguous along the contraction lies in rows of 128 bytes (x and transposed
// weights), the rest in blocks of 64 columns x 64 rows of 128 bytes; both 128-byte
// swizzled, so in shared memory every operand is rows of 64 elements that were
// contiguous in memory.  The ring has as many stages as the largest tile there is leaves
// room for.  TMEM: two accumulators of 256 columns, so that a unit's epilogue runs beside
// the next unit's products.
//
// PAIR: two CTAs (a cluster) share each MMA of M = 256 columns, 128 in each, and each
// holds half of the rows: 32 KB a stage and SM instead of 48 for the same products.  The
// even CTA's barriers count both CTAs' copies, its one thread issues for both, and its
// commits arrive in both.
//
// Order.  Units are numbered expert by expert, so that those that share operands run side
// by side.  Where experts' rows differ much they are taken from the front and the back of
// that order in turns: experts with many rows (bound by the tensor cores) then run beside
// experts with few (bound by their weights' way from HBM).  32768 rows skewed over 256
// experts, 7168 x 4096: 1864 us, 2020 in one order; 16384 rows of four experts, where two
// experts' operands at a time do not fit into L2: 557 us in turns, 526 in one order.
//
// Ragged edges.  Rows behind an expert's last are other experts': they fill accumulator
// columns that are not stored.  The contraction over an expert's rows (the weights'
// gradient) may end inside a stage: the instructions past its end are not issued, and the
// up to 15 rows of both operands that the last one still takes are overwritten with zeros
// first (one of them would not do: what lies there may be NaN).
//
// Sums.  The tensor cores add to their fp32 accumulators by truncation, always towards zero:
// 4e-6 of a weight gradient of 4096 rows, 4e-4 of one of 65536 rows whose terms have the same
// sign (half of fp16's last place).  So an accumulator takes 512 of the contraction, 1024 for
// results of 16 bits, and the epilogue adds the accumulators up, rounding to nearest: 5e-7,
// whatever the length.  (16384 rows of four experts into 7168 x 4096, fp32: 570 us, as in one
// accumulator; 256 of the contraction at a time 2.4e-7 and 2 % more.  Their forward, 7168 long
// in 1024s, 518 us, in 512s 521, in one 511.)  The sums are in registers, or, for 16-bit results
// beside loading warps, which leave none for 256 rows, in the other accumulator's place: a
// unit of more than 1024 keeps to one.
//
// fp32 operands.  A value is the sum of three of bf16, x = h + m + l exactly (h nearest to x,
// m to x - h, l the rest: |m| <= 2^-8 |x|, |l| <= 2^-17 |x|), and
//   x w = h h' + (h m' + m h' + m m' + h l' + l h') + r,  |r| <= (2^-24 + 2^-34) |x w|,
// so six products on the tensor cores give fp32's precision.  The loading warps split the
// values into three images of each operand; the first product and the other five have an
// accumulator each, so that the small ones lose nothing to the large one's truncation.  A
// stage takes 24 MMAs of 128 x 128 x 16; 128 rows a tile.
#pragma once

#include "gemm_common.cuh"
#include "product.cuh"
#include "tc_roles.cuh"

namespace moe {

namespace {


constexpr int kAccCols = 256;
constexpr int kEpi = 8;        // warps of the epilogue, two for each quarter of the TMEM lanes
constexpr int kLoadWarps = 16;  // of TC_LOAD
constexpr int kABytes = kBlkM * kBlkK * 2;
constexpr int kBoxBytes = 64 * 128;  // 64 rows of 64 elements
constexpr int kStagesP = 12;         // at most
constexpr int kTablesP = 8704;       // static shared memory: the experts' rows and units, barriers
constexpr int kSmemP = 232448 - kTablesP;
constexpr int kRawRow = 144;         // TC_LOAD: 64 elements from anywhere in a 16-byte block
// Stages that an accumulator takes; longer contractions are added up from several.
constexpr int sum_steps(TcMode mode, bool f32) { return mode == TC_SPLIT ? 4 : f32 ? 8 : 16; }

constexpr int threads_of(TcMode mode) { return 64 + 32 * (kEpi + (loads(mode) ? kLoadWarps : 0)); }
// D (+)= A B, 16-bit operands, K = 16; a and b are descriptors' low words.
template <bool PAIR>
MOE_DEV void tc_mma_f16_on(int on, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescSw128), "r"(on)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescSw128), "r"(on)
        : "memory");
  }
}
// 16 consecutive fp32 columns of this thread's TMEM lane, added to v.
MOE_DEV void tmem_add16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "{\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(r[i]);
}
// The same columns, written (tmem_st_wait before they are read).
MOE_DEV void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
MOE_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// An arrival in the even CTA's barrier behind TMEM reads.  Their values are in registers by
// then and nothing was written that the other side reads, so there is nothing to release;
// a release over the cluster would wait for the SM's stores to memory (16384 rows into 64
// weight gradients of 2048 x 1536: 151 us with it, 129 without).
MOE_DEV void mbar_arrive_even(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(bar, 0)) : "memory");
}
// The same behind the warp's writes to its CTA's shared memory (past their proxy fence and
// the warp's barrier), which the even CTA's instructions read: a release over the cluster of
// shared memory alone, which does not wait for the stores either (111 us; 129 with a release
// of all memory here).  The other side is try_wait_cluster and acquire_smem_cluster.
MOE_DEV void mbar_arrive_even_release(uint32_t bar) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(bar, 0))
      : "memory");
}
MOE_DEV void acquire_smem_cluster() { asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory"); }
// A wait for an arrival from the other CTA that orders what that one wrote.
MOE_DEV bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// 32 results of a column to rows q, q + ld, ..., of which `rows` exist; ADD: their sums with
// what is there.
template <typename T, bool ADD>
MOE_DEV void put_rows(T* q, int64_t ld, int rows, const float (&v)[32]) {
  if (rows >= 32) {
    float old[ADD ? 32 : 1];
    if constexpr (ADD) {
#pragma unroll
      for (int j = 0; j < 32; ++j) old[j] = to_f32(q[j * ld]);
    }
#pragma unroll
    for (int j = 0; j < 32; ++j, q += ld) *q = from_f32<T>(ADD ? v[j] + old[ADD ? j : 0] : v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j, q += ld)
      if (j < rows) *q = from_f32<T>(ADD ? v[j] + to_f32(*q) : v[j]);
  }
}
template <typename T, bool DW>
MOE_DEV void put_tile(const ProdArgs& p, int64_t at, int rows, const float (&v)[32]) {
  T* q = static_cast<T*>(p.out) + at;
  if (DW && p.accumulate) put_rows<T, DW>(q, p.ldo, rows, v);
  else put_rows<T, false>(q, p.ldo, rows, v);
}

struct TcUnit {
  int e, row0, count;  // the expert and its rows
  int n0;              // first output column (of a pair: of both CTAs)
  int r0, nt;          // first output row of the tile, in the expert, and rows
  int part, kb0, steps;  // part of the contraction: its first stage and how many
  bool end;              // whether the contraction ends with it
};

// F32: results of 32 bits.  SUMS: contractions that more than one accumulator takes (always
// with F32 and with loading warps; 32768 rows of 8 experts, 64 x 2048, 35 us without, 39
// with).  PARTS: of parts of the contraction (F32; its own kernel, since what it adds to a
// unit costs the others registers: 4096 fp32 rows of 8 experts, 1024 x 1024, 86 us instead
// of 74).
template <ProdForm FORM, TcMode MODE, bool F32, bool SUMS, bool PARTS>
__global__ void __launch_bounds__(threads_of(MODE), 1)
    tc_product_kernel(const __grid_constant__ CUtensorMap tm_m, const __grid_constant__ CUtensorMap tm_n,
                      const __grid_constant__ CUtensorMap tm_n128, const ProdArgs p, const uint32_t formats) {
  constexpr bool PAIR = MODE == TC_PAIR, DW = FORM == PROD_DW;
  constexpr bool M_MN = FORM != PROD_ROWS_T, N_MN = DW;  // operands whose contraction is not contiguous
  constexpr int kCols = PAIR ? 2 * kBlkM : kBlkM;        // output columns of a unit
  constexpr int kTileRows = tile_most(MODE, F32), kSumSteps = sum_steps(MODE, F32);
  constexpr int kImages = MODE == TC_SPLIT ? 3 : 1;  // of each operand in a stage
  constexpr int kBoxRows = DW ? 64 : 32;                 // output rows of a box of the N side
  constexpr uint32_t kNBox = kBoxRows * 128;
  extern __shared__ uint8_t smem_raw[];
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  __shared__ int s_off[kMaxG + 1], s_unit[kMaxG + 1];
  __shared__ alignas(8) uint64_t full[kStagesP], empty[kStagesP], ready[kStagesP], tfull[2], tempty[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_most, s_turns;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < kStagesP; ++i) {
      mbar_init(&full[i], loads(MODE) ? kLoadWarps : 1);
      mbar_init(&empty[i], 1);
      mbar_init(&ready[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], (PAIR ? 2 : 1) * kEpi);
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    fence_mbar_init();
    if (!loads(MODE)) {
      tma_prefetch_desc(&tm_m);
      tma_prefetch_desc(&tm_n);
      tma_prefetch_desc(&tm_n128);
    }
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(&s_tmem), 512);  // both CTAs, collectively
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&s_tmem), 512);
      tmem_relinquish();
    }
  }
  ops_wait();
  if (blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
  const int col_tiles = (p.N + kCols - 1) / kCols, dw_tiles = (p.K + kTileRows - 1) / kTileRows;
  const int2 most = number_units(p, DW ? 0 : kTileRows, (DW ? dw_tiles * col_tiles : col_tiles) * p.splits, s_off, s_unit);
  // in turns: an expert has four times the average of those that have rows
  if (threadIdx.x == 0) s_most = DW ? p.K : most.x;
  if (threadIdx.x == 0) s_turns = most.x > 4 * most.y;
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the other CTA's barriers exist before their use
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)s_tmem);
  const int total = uniform(s_unit[p.G]);
  const bool turns = uniform(s_turns) != 0;
  volatile int* abort_flag = &s_abort;
  const int rank = PAIR ? uniform((int)cluster_ctarank()) : 0;
  const int unit0 = PAIR ? blockIdx.x / 2 : blockIdx.x, unit_step = PAIR ? gridDim.x / 2 : gridDim.x;

  // An output's c rows in tiles as even as multiples of 32 allow; the longest.
  auto tile_rows = [](int c, int tiles) { return ((c + tiles - 1) / tiles + 31) & ~31; };
  // this CTA's rows of a tile of nt, and its share of shared memory for them
  auto mine_of = [&](int nt) { return PAIR ? ((nt + 31) & ~31) / 2 : nt; };
  // Stage layout for the largest tile there is.
  const int cap = uniform(s_most > kTileRows ? kTileRows : max(32, (s_most + 31) & ~31));
  const int cap_n = (mine_of(cap) + kBoxRows - 1) / kBoxRows * kBoxRows;
  const uint32_t n_image = (uint32_t)cap_n * 128u, n_at = kImages * kABytes, stage_bytes = n_at + kImages * n_image;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  // (loading warps: two stages' rows as they lie in memory, 144 bytes each, behind the ring)
  // (of groups in pairs, 64 rows)
  const int raw_n = (cap_n + 63) & ~63;
  const uint32_t raw_bytes = MODE == TC_LOAD ? 2u * (uint32_t)(kBlkM + raw_n) * kRawRow : 0u;
  const int S = min(kStagesP, (int)((kSmemP - raw_bytes - (base - smem_u32(smem_raw))) / stage_bytes));

  // The L-th unit in the order they are taken; each role keeps its place in the experts.
  int at_e = 0;
  auto unit_at = [&](int L) {
    const int u = !turns ? L : L & 1 ? total - 1 - (L >> 1) : L >> 1;
    at_e = uniform(expert_of(s_unit, p.G, u, at_e));
    TcUnit t;
    t.e = at_e;
    t.row0 = uniform(s_off[at_e]);
    t.count = max(0, uniform(s_off[at_e + 1]) - t.row0);
    int r = u - uniform(s_unit[at_e]);
    const int c = DW ? p.K : t.count, stages = ((DW ? t.count : p.K) + kBlkK - 1) / kBlkK;
    t.part = t.kb0 = 0;
    t.steps = stages;
    if constexpr (PARTS) {
      const int each = (stages + p.splits - 1) / p.splits;
      t.part = r % p.splits;
      r /= p.splits;
      t.kb0 = min(stages, t.part * each);
      t.steps = min(stages - t.kb0, each);
    }
    t.end = t.kb0 + t.steps == stages;
    const int tiles = DW ? dw_tiles : (c + kTileRows - 1) / kTileRows, n = tiles == 1 ? r : r / tiles;
    t.n0 = n * kCols;
    const int sz = tile_rows(c, tiles);
    t.r0 = (r - n * tiles) * sz;
    t.nt = min(sz, c - t.r0);  // (sz <= kTileRows, so every tile has a row)
    return t;
  };
  // what is left of the contraction where the unit begins
  auto left_of = [&](const TcUnit& t) { return (DW ? t.count : p.K) - t.kb0 * kBlkK; };
  // whether a unit of so many stages keeps to one accumulator, the other's place holding its
  // sums (the unit behind it begins with the same one, whose last arrival is behind them)
  auto holds = [](int steps) { return MODE == TC_LOAD && !F32 && steps > kSumSteps; };
  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
  // All lanes wait; the result is the same in each.
  auto wait_all = [&](uint32_t bar, uint32_t parity, int where) {
    if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_on(bar, parity, abort_flag, p.status, where)) != 0;
  };
  // Zeros in rows [from, to) of every block of 64 rows of a stage (neither operand's
  // contraction contiguous), visible to the tensor cores.
  auto zero_rows = [&](uint32_t stage, int from, int to) {
    const int n = (to - from) * 8, blocks = (int)(stage_bytes / kBoxBytes);
    for (int i = lane; i < blocks * n; i += 32) {
      const int b = i / n, r = i - b * n;
      st_shared_v4(stage + (uint32_t)(b * kBoxBytes + (from + (r >> 3)) * 128 + (r & 7) * 16), 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp == 0 && !loads(MODE)) {
    const int leader = elect_one();
    int s = 0;
    uint32_t ph = 0, used = 0, last = 0, apart_used = 0, apart_ph = 0;
    for (int u = unit0; u < total; u += unit_step) {
      const TcUnit t = unit_at(u);
      const int mine = mine_of(t.nt), steps = t.steps;
      // boxes of CTA r's M side (64 columns, or all 128); of its N side
      auto m_boxes = [&](int r) {
        const int left = p.N - t.n0 - r * kBlkM;
        return M_MN ? max(0, min(2, (left + 63) / 64)) : left > 0 ? 1 : 0;
      };
      constexpr uint32_t kMBox = M_MN ? kBoxBytes : kABytes;
      const int mb = m_boxes(rank), nb = (mine + kBoxRows - 1) / kBoxRows;
      const uint32_t n_bytes = (uint32_t)nb * kNBox, bytes = (uint32_t)mb * kMBox + n_bytes;
      const uint32_t others = PAIR ? (uint32_t)m_boxes(1) * kMBox + n_bytes : 0u;
      const int col = t.n0 + rank * kBlkM, row = t.r0 + rank * mine;
      const int big = DW ? 0 : nb / 4;  // boxes of 128 rows
      for (int kb = 0; kb < steps; ++kb) {
        if (!wait_all(empty0 + 8u * s, ph ^ 1u, 2000 + s)) goto produced;
        const uint32_t sa = base + (uint32_t)s * stage_bytes, sb = sa + kABytes;
        const int k0 = (t.kb0 + kb) * kBlkK;
        // of a pair, the odd CTA zeroes the end of the contraction in its own shared memory
        // and waits for its own copies first, on its own barrier of the stage (which has no
        // other use)
        const bool apart = PAIR && DW && kb == steps - 1 && t.end && (t.count & 15) != 0;
        uint32_t fb = full0 + 8u * s;
        if constexpr (PAIR) {
          if (apart && rank == 1) {
            expect_tx_on(leader, fb, bytes);
            fb = mapa_shared(fb, 1);
            apart_used |= 1u << s;
            apart_ph ^= 1u << s;  // the parity of this stage's next use
          } else {
            fb = mapa_shared(fb, 0);
            expect_tx_on(leader && rank == 0, full0 + 8u * s, bytes + (apart ? 0u : others));
          }
        } else {
          expect_tx_on(leader, fb, bytes);
        }
        for (int i = 0; i < mb; ++i) {
          const uint32_t dst = sa + i * kMBox;
          if constexpr (DW) tma_load_2d_on<PAIR>(leader, dst, &tm_m, fb, col + i * 64, t.row0 + k0);
          else if constexpr (M_MN) tma_load_3d_on<PAIR>(leader, dst, &tm_m, fb, col + i * 64, k0, t.e);
          else tma_load_3d_on<PAIR>(leader, dst, &tm_m, fb, k0, col, t.e);
        }
        if constexpr (DW) {
          for (int i = 0; i < nb; ++i)
            tma_load_2d_on<PAIR>(leader, sb + i * kNBox, &tm_n, fb, row + i * 64, t.row0 + k0);
        } else {
          for (int i = 0; i < big; ++i)
            tma_load_2d_on<PAIR>(leader, sb + i * 4 * kNBox, &tm_n128, fb, k0, t.row0 + row + i * 128);
          for (int i = 4 * big; i < nb; ++i)
            tma_load_2d_on<PAIR>(leader, sb + i * kNBox, &tm_n, fb, k0, t.row0 + row + i * 32);
        }
        used |= 1u << s;
        last = (last & ~(1u << s)) | (ph << s);
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  produced:
    // every issued copy has landed before the CTA can exit (of a pair the even CTA's
    // barriers count both CTAs'), and of a pair every commit has arrived
    for (int i = 0; i < kStagesP; ++i) {
      if (((used >> i) & 1u) == 0) continue;
      if (rank == 0 && !mbar_wait_drain(&full[i], (last >> i) & 1u)) break;
      if (PAIR && !mbar_wait_drain(&empty[i], (last >> i) & 1u)) break;
    }
    for (int i = 0; i < kStagesP; ++i)
      if (((apart_used >> i) & 1u) != 0 && !mbar_wait_drain(&full[i], ((apart_ph >> i) & 1u) ^ 1u)) break;
  } else if (warp == 1 && rank == 0) {
    const int leader = elect_one();
    int s = 0, acc = 0;
    uint32_t ph = 0, aph = 0, tph = 0;
    constexpr uint32_t kMN = 512u << 16, kKM = 1u << 16;  // leading offsets: 8 KB between blocks of 64 columns
    const uint32_t da0 = (base >> 4) | (M_MN ? kMN : kKM), db0 = ((base + n_at) >> 4) | (N_MN ? kMN : kKM);
    constexpr uint32_t ka = M_MN ? 128u : 2u, kn = N_MN ? 128u : 2u;  // 16 of the contraction, in units of 16 bytes
    for (int u = unit0; u < total; u += unit_step) {
      const TcUnit t = unit_at(u);
      const int steps = t.steps;
      const int mma_n = PAIR ? (t.nt + 31) & ~31 : (t.nt + 15) & ~15;
      const uint32_t id = (1u << 4) | formats | ((M_MN ? 1u : 0u) << 15) | ((N_MN ? 1u : 0u) << 16) |
                          ((uint32_t)(mma_n >> 3) << 17) | ((uint32_t)((PAIR ? 256 : 128) >> 4) << 24);
      int left = left_of(t);
      uint32_t more = 0;
      for (int kb = 0; kb < steps; ++kb) {
        const uint32_t d = tmem + (uint32_t)(acc * kAccCols);
        if (!more) {
          if (!wait_all(smem_u32(&tempty[acc]), ((aph >> acc) & 1u) ^ 1u, 2100 + acc)) goto issued;
        }
        if (!wait_all(full0 + 8u * s, ph, 2200 + s)) goto issued;
        if constexpr (DW && !loads(MODE)) {
          if (left < kBlkK && (left & 15) != 0) {
            zero_rows(base + (uint32_t)s * stage_bytes, left, (left + 15) & ~15);
            if constexpr (PAIR) {
              const uint32_t bar = smem_u32(&ready[s]), par = (tph >> s) & 1u;
              bool ok = __all_sync(0xffffffffu, try_wait_cluster(bar, par));
              if (!ok) {
                ok = __all_sync(0xffffffffu, wait_on(bar, par, abort_flag, p.status, 2300));
                ok = ok && __all_sync(0xffffffffu, try_wait_cluster(bar, par));
              }
              if (!ok) goto issued;
              acquire_smem_cluster();
              tph ^= 1u << s;
            }
          }
        }
        tc_fence_after();
        const uint32_t da = da0 + (uint32_t)s * (stage_bytes / 16u), db = db0 + (uint32_t)s * (stage_bytes / 16u);
        // 64 of the contraction: image i of the M side by image j of the N side
        auto products = [&](uint32_t to, int i, int j, uint32_t onto) {
          const uint32_t a = da + (uint32_t)(i * (kABytes / 16)), b = db + (uint32_t)j * (n_image / 16u);
          tc_mma_f16_on<PAIR>(leader, to, a, b, id, onto);
          tc_mma_f16_on<PAIR>(leader && left > 16, to, a + ka, b + kn, id, 1u);
          tc_mma_f16_on<PAIR>(leader && left > 32, to, a + 2 * ka, b + 2 * kn, id, 1u);
          tc_mma_f16_on<PAIR>(leader && left > 48, to, a + 3 * ka, b + 3 * kn, id, 1u);
        };
        products(d, 0, 0, more);
        if constexpr (MODE == TC_SPLIT) {
          const uint32_t small = d + kTileRows;
          products(small, 0, 2, more);
          products(small, 2, 0, 1u);
          products(small, 1, 1, 1u);
          products(small, 0, 1, 1u);
          products(small, 1, 0, 1u);
        }
        tc_commit_on<PAIR>(leader, empty0 + 8u * s);
        left -= kBlkK;
        more = 1u;
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
        if (kb == steps - 1 || (SUMS && (kb + 1) % kSumSteps == 0)) {
          tc_commit_on<PAIR>(leader, smem_u32(&tfull[acc]));
          more = 0;
          aph ^= 1u << acc;
          if (!holds(steps)) acc ^= 1;
        }
      }
    }
  issued:
    tc_commit_on<PAIR>(leader, smem_u32(&drain), 1);
    mbar_wait_drain(&drain, 0);
  } else if (PAIR && DW && warp == 1) {
    // the odd CTA's part of the contraction's end.  (Barriers of each stage's own: the copies
    // of several units' ends can be under way, but a stage is not filled again before its
    // products are done.)
    int s = 0;
    uint32_t tph = 0;
    for (int u = unit0; u < total; u += unit_step) {
      const TcUnit t = unit_at(u);
      const int steps = t.steps;
      if (steps == 0) continue;
      s = (s + steps - 1) % S;
      if (t.end && (t.count & 15) != 0) {
        if (!wait_all(full0 + 8u * s, (tph >> s) & 1u, 2400)) break;
        tph ^= 1u << s;
        const int left = left_of(t) - (steps - 1) * kBlkK;
        zero_rows(base + (uint32_t)s * stage_bytes, left, (left + 15) & ~15);
        if (lane == 0) mbar_arrive_even_release(smem_u32(&ready[s]));
      }
      if (++s == S) s = 0;
    }
  } else if (MODE == TC_LOAD && warp >= 2 + kEpi) {
    // The operands lie in rows of 64 elements (128 bytes) that start at any element.  Eight
    // warps load the M side, eight the N side, each every eighth row: all of a warp's rows lie
    // alike to 16 bytes and to the swizzle.  The 16-byte blocks that hold a row are copied to
    // shared memory as they are (cp.async, the next stage's while one is worked on: loads into
    // registers left a stage at the latency of two, 8192 rows of 16 experts, 2047 x 1535, 231
    // us), and from there 16 bytes at a time go to the stage by shifts that are the same in all
    // lanes.  (A stage that is not wholly inside the operand's array in such blocks is loaded
    // element by element.)
    const int w7 = (warp - 2 - kEpi) & 7, chunk = lane & 7;
    auto run_side = [&](auto m_side) {
      constexpr bool MS = decltype(m_side)::value, BLK = MS ? M_MN : N_MN;
      const uint16_t* arr = static_cast<const uint16_t*>(MS ? p.b : p.a);
      const int64_t ld = MS ? p.ldb : p.lda;
      const uintptr_t lo = reinterpret_cast<uintptr_t>(arr);
      const uintptr_t hi = reinterpret_cast<uintptr_t>(MS ? (DW ? arr + (int64_t)(p.rows - 1) * ld + p.N : arr + (int64_t)p.G * p.K * p.N)
                                                          : arr + (int64_t)(p.rows - 1) * ld + p.K);
      const int row = w7 + 8 * (lane >> 3);  // group i has row + 32 (i % 2) of block i / 2, or 64 (i / 2) rows on
      const uint32_t off = (uint32_t)((lane >> 3) * 16 * ld + 16 * chunk), half = (uint32_t)(64 * ld);
      const uint32_t apart = BLK ? 128u : (uint32_t)(128 * ld);
      const uint32_t lane_dst = (MS ? 0u : (uint32_t)kABytes) + (uint32_t)(row * 128 + ((chunk ^ w7) << 4));
      // the warp's rows as they lie in memory: group i's four at 4 i, two buffers
      const uint32_t raw_size = (uint32_t)((MS ? kBlkM : raw_n) / 8 * kRawRow);
      const uint32_t raw = base + (uint32_t)S * stage_bytes + (MS ? 0u : 2u * kBlkM * kRawRow) + 2u * raw_size * (uint32_t)w7;
      const uint32_t raw_lane = (uint32_t)((lane >> 3) * kRawRow + 16 * chunk);
      const bool near = ld < (1 << 22);  // a tile's offsets have 32 bits
      struct Stage {
        const uint16_t* src;      // its row 0
        int left, have, put, sh;  // of the contraction; rows or columns that exist, that are stored
        bool fast;
      };
      // Where the next stage is.  What is the same for all of a unit's whole stages is worked
      // out once: a warp's instructions, one after the other, are what a stage takes.
      int u = unit0, kb = 0, steps = 0, fast0 = 0, fast1 = 0;
      uint32_t copies = 0;           // bit i: the lane's block of group i, bit 8 + i: the row's ninth
      const uint8_t* blk = nullptr;  // the lane's block of the stage's group 0
      Stage at = {};
      bool more = true;
      // which blocks hold some of `rows` rows' (or their first `bytes` bytes')
      auto copies_of = [&](int rows, int bytes) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = row + 32 * (i & 1) + (BLK ? 0 : 64 * (i >> 1)), b = BLK ? 128 * (i >> 1) : 0;
          if (32 * i < at.put && r < rows) {
            if (b + 16 * chunk < bytes) m |= 1u << i;
            if (chunk == 7 && at.sh != 0 && b + 128 < bytes) m |= 256u << i;
          }
        }
        return m;
      };
      // whether a stage of `len` at `src` lies in the array's whole blocks
      auto inside = [&](const uint16_t* src, int len) {
        const int64_t span = BLK ? (len - 1) * ld + at.have : (at.have - 1) * ld + len;
        const uintptr_t f = reinterpret_cast<uintptr_t>(src);
        return near && (f & ~(uintptr_t)15) >= lo && ((f + 2 * span + 15) & ~(uintptr_t)15) <= hi;
      };
      auto find_unit = [&]() {  // from unit u on, the first with a contraction
        for (; u < total; u += unit_step) {
          const TcUnit t = unit_at(u);
          steps = t.steps;
          if (steps == 0) continue;
          at.left = left_of(t);
          at.have = MS ? min(kBlkM, p.N - t.n0) : DW ? min((t.nt + 63) & ~63, p.K - t.r0) : t.nt;
          at.put = MS ? kBlkM : DW ? (t.nt + 63) & ~63 : t.nt;
          at.src = arr + (MS ? (DW ? t.row0 * ld : (int64_t)t.e * p.K * p.N) : t.row0 * ld);
          at.src += (MS ? (BLK ? (int64_t)t.n0 : t.n0 * ld) : BLK ? (int64_t)t.r0 : t.r0 * ld) + t.kb0 * (BLK ? kBlkK * ld : kBlkK);
          at.sh = (int)(reinterpret_cast<uintptr_t>(at.src + w7 * ld) & 15);
          blk = reinterpret_cast<const uint8_t*>(at.src + w7 * ld) - at.sh + off;
          copies = copies_of(BLK ? kBlkK : at.have, 2 * (BLK ? at.have : kBlkK) + at.sh);
          // (only the first stage can begin before the array's first whole block, only the last
          // whole one, and what is left, end behind its last; far rows are all loaded singly)
          const int whole = min(steps, at.left / kBlkK);
          const int64_t next = BLK ? kBlkK * ld : kBlkK;
          fast0 = whole > 0 && inside(at.src, kBlkK) ? 0 : 1;
          fast1 = whole == 0 || !near ? 0 : inside(at.src + (whole - 1) * next, kBlkK) ? whole : whole - 1;
          return;
        }
        more = false;
      };
      auto issue = [&](uint32_t to) {
        at.fast = kb >= fast0 && kb < fast1;
        uint32_t m = copies;
        if (!at.fast) {
          const int len = min(at.left, kBlkK);
          at.fast = inside(at.src, len);
          m = at.fast ? copies_of(BLK ? len : at.have, 2 * (BLK ? at.have : len) + at.sh) : 0u;
        }
        // (loops of two groups: the warps' roles share the instruction caches, and whole
        // unrolling made the rows' gradient of that product 375 us, not 182)
        to += raw_lane;
        uint32_t o = 0;
#pragma unroll 1
        for (int i = 0; 32 * i < at.put; i += 2, m >>= 2, o += apart, to += 8 * kRawRow) {
          const uint8_t *e = blk + o, *e1 = blk + (o + half);
          asm volatile(
              "{\n\t.reg .pred p, q, r, s;\n\t.reg .b32 t;\n\t"
              "and.b32 t, %3, 1;\n\tsetp.ne.b32 p, t, 0;\n\t"
              "and.b32 t, %3, 256;\n\tsetp.ne.b32 q, t, 0;\n\t"
              "and.b32 t, %3, 2;\n\tsetp.ne.b32 r, t, 0;\n\t"
              "and.b32 t, %3, 512;\n\tsetp.ne.b32 s, t, 0;\n\t"
              "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t"
              "@r cp.async.cg.shared.global [%0+576], [%2], 16;\n\t"
              "@q cp.async.cg.shared.global [%0+16], [%1+16], 16;\n\t"
              "@s cp.async.cg.shared.global [%0+592], [%2+16], 16;\n\t}" ::"r"(to),
              "l"(e), "l"(e1), "r"(m)
              : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        const Stage now = at;
        at.src += BLK ? kBlkK * ld : kBlkK;
        blk += BLK ? 2 * kBlkK * ld : 2 * kBlkK;
        at.left -= kBlkK;
        if (++kb == steps) {
          kb = 0;
          u += unit_step;
          find_unit();
        }
        return now;
      };
      // two groups' 16 bytes from word W, and half of one if `sel` says so, of their two blocks
      auto store = [&](const Stage& x, uint32_t from, uint32_t to) {
        from += raw_lane;
        const uint32_t sel = x.sh & 2 ? 0x5432 : 0x3210;
        const bool end = x.left < kBlkK;
        auto by = [&](auto words) {
          constexpr int W = decltype(words)::value;
          int r = row;  // of group i
#pragma unroll 1
          for (int i = 0; 32 * i < x.put; i += 2, from += 8 * kRawRow, to += kBoxBytes) {
            uint32_t v[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t w[8];
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from + j * 4 * kRawRow));
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "r"(from + j * 4 * kRawRow + 16));
#pragma unroll
              for (int k = 0; k < 4; ++k) v[j][k] = __byte_perm(w[W + k], w[W + k + 1], sel);
            }
            if (end) {  // zeros past the end of the contraction
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int n = BLK ? (row + 32 * j < x.left ? 8 : 0) : x.left - 8 * chunk;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[j][k] &= (2 * k < n ? 0xFFFFu : 0u) | (2 * k + 1 < n ? 0xFFFF0000u : 0u);
              }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (MS || BLK || r + 32 * j < x.put) st_shared_v4(to + (uint32_t)(j * 4096), v[j][0], v[j][1], v[j][2], v[j][3]);
            r += 64;
          }
        };
        switch (x.sh >> 2) {
          case 0: by(std::integral_constant<int, 0>()); break;
          case 1: by(std::integral_constant<int, 1>()); break;
          case 2: by(std::integral_constant<int, 2>()); break;
          default: by(std::integral_constant<int, 3>());
        }
      };
      // element by element
      auto store_slow = [&](const Stage& x, uint32_t to) {
#pragma unroll 1
        for (int i = 0; 32 * i < x.put; ++i) {
          const int b = BLK ? i >> 1 : 0, r = row + 32 * (i & 1) + (BLK ? 0 : 64 * (i >> 1));
          const uint16_t* q = x.src + r * ld + 64 * b + 8 * chunk;
          // elements that exist
          const int n = r < (BLK ? x.left : x.have) ? (BLK ? x.have : x.left) - 64 * b - 8 * chunk : 0;
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = (2 * k < n ? gload(q + 2 * k) : 0u) | (2 * k + 1 < n ? gload(q + 2 * k + 1) << 16 : 0u);
          if (BLK || r < x.put) st_shared_v4(to + (uint32_t)((i & 1) * 4096 + (i >> 1) * kBoxBytes), v[0], v[1], v[2], v[3]);
        }
      };
      find_unit();
      if (!more) return;
      int s = 0;
      uint32_t ph = 0, buf = 0;
      Stage now = issue(raw);
      for (;;) {
        Stage next = now;
        const bool go_on = more;
        if (go_on) {
          next = issue(raw + raw_size - buf);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
        if (!wait_all(empty0 + 8u * s, ph ^ 1u, 2000 + s)) break;
        const uint32_t to = base + (uint32_t)s * stage_bytes + lane_dst;
        if (now.fast) store(now, raw + buf, to);
        else store_slow(now, to);
        fence_proxy_async_smem();
        __syncwarp();  // (also: this buffer has been read)
        if (lane == 0) mbar_arrive(&full[s]);
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
        if (!go_on) break;
        now = next;
        buf = raw_size - buf;
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    };
    if (warp < 2 + kEpi + 8) run_side(std::true_type());
    else run_side(std::false_type());
  } else if (MODE == TC_SPLIT && warp >= 2 + kEpi) {
    // Eight warps load and split the M side, eight the N side, each every eighth row of 64
    // values.  Where rows are whole 16-byte vectors eight lanes have a row, four rows are a
    // group (row + 32 (i % 2) of block i / 2, or 64 (i / 2) rows on), and two groups' loads are
    // under way while two are split; else a lane has two values of each of eight rows.
    const int w7 = (warp - 2 - kEpi) & 7, chunk = lane & 7;
    auto run_side = [&](auto m_side, auto vectors) {
      constexpr bool MS = decltype(m_side)::value, VEC = decltype(vectors)::value, BLK = MS ? M_MN : N_MN;
      const float* arr = static_cast<const float*>(MS ? p.b : p.a);
      const int64_t ld = MS ? p.ldb : p.lda;
      const int row = w7 + 8 * (lane >> 3);
      const uint32_t lane_dst = (MS ? 0u : n_at) + (VEC ? (uint32_t)(row * 128 + ((chunk ^ w7) << 4))
                                                        : (uint32_t)(w7 * 128 + (((lane >> 2) ^ w7) << 4) + (lane & 3) * 4));
      const uint32_t image = MS ? (uint32_t)kABytes : n_image;
      // where the next half stage (two groups) is
      int u = unit0, kb = 0, steps = 0, h = 0, left = 0, have = 0, put = 0;
      const float* src = nullptr;  // the half's first value of this lane
      const int64_t ld8 = 8 * ld, ld32 = 32 * ld, to_half = BLK ? 64 : 64 * ld, to_stage = BLK ? kBlkK * ld : kBlkK;
      bool more = true;
      auto find_unit = [&]() {  // from unit u on, the first with a contraction
        for (; u < total; u += unit_step) {
          const TcUnit t = unit_at(u);
          steps = t.steps;
          if (steps == 0) continue;
          left = left_of(t);
          have = MS ? min(kBlkM, p.N - t.n0) : DW ? min((t.nt + 63) & ~63, p.K - t.r0) : t.nt;
          put = MS ? kBlkM : DW ? (t.nt + 63) & ~63 : t.nt;
          src = arr + (MS ? (DW ? t.row0 * ld : (int64_t)t.e * p.K * p.N) : t.row0 * ld);
          src += (MS ? (BLK ? (int64_t)t.n0 : t.n0 * ld) : BLK ? (int64_t)t.r0 : t.r0 * ld) + t.kb0 * to_stage;
          src += VEC ? row * ld + 8 * chunk : w7 * ld + 2 * lane;
          return;
        }
        more = false;
      };
      struct Half {
        uint32_t v[16];
        int h, put;  // of its stage the first (0) or second; rows or columns that are stored
      };
      auto advance = [&]() {  // (in front of the loads: behind them it would wait for them)
        src += to_half;
        if (64 * ++h >= put) {
          src += to_stage - h * to_half;
          h = 0;
          left -= kBlkK;
          if (++kb == steps) {
            kb = 0;
            u += unit_step;
            find_unit();
          }
        }
      };
      auto load = [&](Half& x) {
        x.h = h;
        x.put = put;
        // the half's rows that exist, and of a row's values those that do from this lane's on
        const int rows = BLK ? left : have - 64 * h, values = (BLK ? have - 64 * h : left) - (VEC ? 8 * chunk : 2 * lane);
        const float* q = src;
        if constexpr (VEC) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int n = row + 32 * i < rows ? values : 0;
            uint32_t* v = x.v + 8 * i;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.gt.s32 p, %9, 0;\n\t"
                "setp.gt.s32 q, %9, 4;\n\t"
                "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
                "mov.b32 %4, 0;\n\tmov.b32 %5, 0;\n\tmov.b32 %6, 0;\n\tmov.b32 %7, 0;\n\t"
                "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%8];\n\t"
                "@q ld.global.v4.u32 {%4, %5, %6, %7}, [%8+16];\n\t}"
                : "=&r"(v[0]), "=&r"(v[1]), "=&r"(v[2]), "=&r"(v[3]), "=&r"(v[4]), "=&r"(v[5]), "=&r"(v[6]), "=&r"(v[7])
                : "l"(q), "r"(n));
            q += ld32;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int n = w7 + 8 * j < rows ? values : 0;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.gt.s32 p, %3, 0;\n\t"
                "setp.gt.s32 q, %3, 1;\n\t"
                "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
                "@p ld.global.u32 %0, [%2];\n\t"
                "@q ld.global.u32 %1, [%2+4];\n\t}"
                : "=&r"(x.v[2 * j]), "=&r"(x.v[2 * j + 1])
                : "l"(q), "r"(n));
            q += ld8;
          }
        }
      };
      int s = 0;
      uint32_t ph = 0;
      auto split = [&](const Half& x) {
        if (x.h == 0 && !wait_all(empty0 + 8u * s, ph ^ 1u, 2000 + s)) return false;
        const uint32_t to = base + (uint32_t)s * stage_bytes + lane_dst + (uint32_t)(x.h * kBoxBytes);
        // two values' parts
        auto parts = [](const uint32_t* v, uint32_t& h2, uint32_t& m2, uint32_t& l2) {
          auto top = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
          // (rounded, values over the largest bf16 would be infinities)
          asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(h2) : "f"(__uint_as_float(v[1])), "f"(__uint_as_float(v[0])));
          const float2 r = sub2(F2(__uint_as_float(v[0]), __uint_as_float(v[1])), F2(__uint_as_float(h2 << 16), top(h2))).get();
          m2 = pack_bf16x2(r.x, r.y);
          const float2 t = sub2(F2(r.x, r.y), F2(__uint_as_float(m2 << 16), top(m2))).get();
          l2 = __byte_perm(__float_as_uint(t.x), __float_as_uint(t.y), 0x7632);
        };
        if constexpr (VEC) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t w[3][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) parts(x.v + 8 * i + 2 * k, w[0][k], w[1][k], w[2][k]);
            if (BLK || row + 32 * i + 64 * x.h < x.put) {
#pragma unroll
              for (int j = 0; j < 3; ++j)
                st_shared_v4(to + (uint32_t)(i * 4096) + (uint32_t)j * image, w[j][0], w[j][1], w[j][2], w[j][3]);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t w[3];
            parts(x.v + 2 * j, w[0], w[1], w[2]);
            if (BLK || w7 + 8 * j + 64 * x.h < x.put) {
#pragma unroll
              for (int i = 0; i < 3; ++i)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + (uint32_t)(j * 1024) + (uint32_t)i * image), "r"(w[i]) : "memory");
            }
          }
        }
        if (64 * (x.h + 1) >= x.put) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
          if (++s == S) {
            s = 0;
            ph ^= 1u;
          }
        }
        return true;
      };
      find_unit();
      if (!more) return;
      Half x, y;
      load(x);
      for (;;) {
        advance();
        if (!more) {
          split(x);
          break;
        }
        load(y);
        if (!split(x)) break;
        advance();
        if (!more) {
          split(y);
          break;
        }
        load(x);
        if (!split(y)) break;
      }
    };
    // 16 bytes at a time where every row starts on them and is a whole number of them
    const bool vec = ((reinterpret_cast<uintptr_t>(p.a) | reinterpret_cast<uintptr_t>(p.b) |
                       (uintptr_t)(p.lda | p.ldb | p.K | p.N) * 4) & 15) == 0;
    if (warp < 2 + kEpi + 8) {
      if (vec) run_side(std::true_type(), std::true_type());
      else run_side(std::true_type(), std::false_type());
    } else {
      if (vec) run_side(std::false_type(), std::true_type());
      else run_side(std::false_type(), std::false_type());
    }
  } else if (warp > 1 && warp < 2 + kEpi) {
    // A lane holds an output column; a warp takes 32 rows in kStep of its quarter's 32 columns.
    // (Sixteen warps, half of the sums each, were 9 % slower for 16384 rows of four experts
    // into 7168 x 4096.)
    constexpr int kStep = 8 * kEpi;
    const int q = warp & 3, c_first = 32 * ((warp - 2) >> 2);
    const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
    int acc = 0;
    uint32_t aph = 0;
    auto done = [&](bool hold = false) {  // this accumulator may be filled again
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_even(smem_u32(&tempty[acc]));
        else mbar_arrive(&tempty[acc]);
      }
      aph ^= 1u << acc;
      if (!hold) acc ^= 1;
    };
    auto filled = [&]() { return wait_all(smem_u32(&tfull[acc]), (aph >> acc) & 1u, 2500 + acc); };
    for (int u = unit0; u < total; u += unit_step) {
      const TcUnit t = unit_at(u);
      const int steps = t.steps;
      if (steps == 0 && p.accumulate) continue;
      const int n = t.n0 + rank * kBlkM + q * 32 + lane;
      const bool there = n < p.N;
      // the lane's column of the tile's first row
      const int64_t first = ((DW ? (int64_t)t.e * p.K : (int64_t)t.row0) + t.r0) * p.ldo + n + (PARTS ? t.part * p.split_stride : 0);
      const int nt = t.nt;
      // 32 rows from c0 on
      auto store = [&](int c0, const float (&v)[32]) {
        if (!there) return;
        const int64_t at = first + c0 * p.ldo;
        if constexpr (F32) put_tile<float, DW>(p, at, nt - c0, v);
        else if (p.odt == MOE_DT_BF16) put_tile<__nv_bfloat16, DW>(p, at, nt - c0, v);
        else put_tile<__half, DW>(p, at, nt - c0, v);
      };
      if (!F32 && steps == 0) {
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
        for (int c0 = c_first; c0 < nt; c0 += kStep) store(c0, v);
      } else if (!F32 && (!SUMS || steps <= kSumSteps)) {
        if (!filled()) goto stored;
        tc_fence_after();
        for (int c0 = c_first; c0 < nt; c0 += kStep) {
          float v[32];
          tmem_ld32(tq + (uint32_t)(acc * kAccCols + c0), v);
          store(c0, v);
        }
        done();
      } else if constexpr (!SUMS) {
        // (there is no longer contraction)
      } else if constexpr (MODE == TC_LOAD && !F32) {
        // each time the same thread has the same columns of both places
        for (int k = 0; k < steps; k += kSumSteps) {
          if (!filled()) goto stored;
          tc_fence_after();
          for (int c0 = c_first; c0 < nt; c0 += kStep) {
            const uint32_t from = tq + (uint32_t)(acc * kAccCols + c0), sums = tq + (uint32_t)((acc ^ 1) * kAccCols + c0);
            float v[32];
            tmem_ld32(from, v);
            if (k > 0) {
              tmem_add16(sums, v);
              tmem_add16(sums + 16, v + 16);
            }
            if (k + kSumSteps < steps) {
              tmem_st16(sums, v);
              tmem_st16(sums + 16, v + 16);
            } else {
              store(c0, v);
            }
          }
          tmem_st_wait();
          done(true);
        }
      } else {
        constexpr int kParts = kTileRows / kStep;
        float sum[kParts][32];
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[i][j] = 0.f;
        for (int k = 0; k < steps; k += kSumSteps) {
          if (!filled()) goto stored;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kParts; ++i) {
            if (c_first + kStep * i < nt) {
              // (16 at a time where loading warps leave a thread 72 registers)
              const uint32_t from = tq + (uint32_t)(acc * kAccCols + c_first + kStep * i);
              if constexpr (loads(MODE)) {
                if constexpr (MODE == TC_SPLIT) {
                  tmem_add16(from + kTileRows, sum[i]);
                  tmem_add16(from + kTileRows + 16, sum[i] + 16);
                }
                tmem_add16(from, sum[i]);
                tmem_add16(from + 16, sum[i] + 16);
              } else {
                float v[32];
                tmem_ld32(from, v);
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[i][j] += v[j];
              }
            }
          }
          done();
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          if (c_first + kStep * i < nt) store(c_first + kStep * i, sum[i]);
      }
    }
  stored:;
  }
  ops_let_next();
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the pair's MMAs and remote arrivals are done
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

// Results from their partial sums, added in order: n columns of rows first..last (of experts
// [offsets[0], offsets[G]); NULL: of all).
template <typename T>
__global__ void __launch_bounds__(256)
    sum_parts_kernel(const float* __restrict__ part, int splits, int64_t stride, const int* off, int G, int64_t rows, int n,
                     T* out, int64_t ldo, bool add) {
  ops_begin();
  const int64_t first = off ? min((int64_t)max(gload(off), 0), rows) : 0, last = off ? min((int64_t)max(gload(off + G), 0), rows) : rows;
  // (at most 76 tiles of 256 x 256: 32 bits)
  const int total = last > first ? (int)((last - first) * n) : 0;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < total; i += gridDim.x * blockDim.x) {
    const int64_t r = first + i / n, c = i % n;
    const float* q = part + r * n + c;
    T* o = out + r * ldo + c;
    float s = add ? to_f32(*o) : 0.f;
#pragma unroll 8
    for (int k = 0; k < splits; ++k) s += gload(q + k * stride);
    *o = from_f32<T>(s);
  }
}

// ------------------------------------------------------------------ host side
uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// A map of 16-bit elements: rows of d0 contiguous ones with strides in elements, boxes of
// b0 x b1 (x 1), 128-byte swizzle; what a box reads past the sizes is zeros.
bool tc_map(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t ld1, uint64_t d2, uint64_t ld2,
            uint32_t b0, uint32_t b1) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {ld1 * 2, ld2 * 2};
  const cuuint32_t box[3] = {b0, b1, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d2 ? 3 : 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <ProdForm FORM, TcMode MODE, bool F32, bool SUMS, bool PARTS>
cudaError_t launch_tc(const CUtensorMap* tm, const ProdArgs& p, uint32_t formats, cudaStream_t st) {
  auto kern = tc_product_kernel<FORM, MODE, F32, SUMS, PARTS>;
  static SmemAllowed allowed;
  const cudaError_t e = allow_smem(kern, kSmemP, allowed);
  if (e != cudaSuccess) return e;
  const char* name = FORM == PROD_DW ? "grouped_product_dw" : "grouped_product";
  const int64_t units = units_of(FORM, MODE, F32, p.rows, p.K, p.N, p.G) * p.splits;
  const dim3 block(threads_of(MODE));
  if constexpr (MODE != TC_PAIR) {
    const int grid = units < num_sms() ? (int)units : num_sms();
    return launch_ops(name, kern, dim3(grid), block, kSmemP, st, tm[0], tm[1], tm[2], p, formats);
  } else {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms() & ~1));
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = kSmemP;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static std::atomic<int> resident[64];
    const int most = pair_clusters(kern, cfg, resident);
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(2 * (unsigned)(units < most ? units : most));
    TraceScope ts(name, st);
    return cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], p, formats);
  }
}

// The kernel in mode MODE, with its contraction in parts if that pays.
template <ProdForm FORM, TcMode MODE, bool F32>
cudaError_t launch_parts(const CUtensorMap* tm, const ProdArgs& p, uint32_t formats, cudaStream_t st) {
  const int splits = splits_of(FORM, MODE, p.rows, p.K, p.N, p.G);
  if (splits <= 1) {
    if constexpr (!F32 && MODE != TC_LOAD) {
      if ((FORM == PROD_DW ? p.rows : p.K) <= kBlkK * sum_steps(MODE, false))
        return launch_tc<FORM, MODE, false, false, false>(tm, p, formats, st);
    }
    return launch_tc<FORM, MODE, F32, true, false>(tm, p, formats, st);
  }
  ProdArgs q = p;
  const int64_t n = results_of(FORM, p.rows, p.K, p.N, p.G);
  q.out = p.ws;
  q.ldo = p.N;
  q.odt = MOE_DT_F32;
  q.accumulate = 0;
  q.splits = splits;
  q.split_stride = n;
  cudaError_t e = launch_tc<FORM, MODE, true, true, true>(tm, q, formats, st);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (n + 255) / 256, most = (int64_t)num_sms() * 8;
  return with_dtype(p.odt, [&](auto t) {
    using T = decltype(t);
    const bool dw = FORM == PROD_DW;
    return launch_ops("grouped_product_sum", sum_parts_kernel<T>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0,
                      st, static_cast<const float*>(p.ws), splits, n, dw ? (const int*)nullptr : p.off, p.G,
                      dw ? (int64_t)p.G * p.K : (int64_t)p.rows, p.N, static_cast<T*>(p.out), p.ldo, p.accumulate != 0);
  });
}

template <ProdForm FORM, bool F32>
cudaError_t launch_form(int dtype, const ProdArgs& p, cudaStream_t st) {
  const uint32_t fmt = dtype == MOE_DT_BF16 ? 1u : 0u, formats = (fmt << 7) | (fmt << 10);
  // tensor copies: every row starts on 16 bytes (and there are rows)
  const bool copy = dtype != MOE_DT_F32 && p.rows > 0 && ((bits(p.a) | bits(p.b) | (uintptr_t)p.lda * 2 | (uintptr_t)p.ldb * 2) & 15) == 0;
  CUtensorMap tm[3];
  if (!copy) {
    memset(tm, 0, sizeof(tm));
    if constexpr (F32) {
      if (dtype == MOE_DT_F32) return launch_parts<FORM, TC_SPLIT, true>(tm, p, (1u << 7) | (1u << 10), st);
    }
    return launch_parts<FORM, TC_LOAD, F32>(tm, p, formats, st);
  }
  const bool pair = takes_pairs(p.rows, p.N, p.G);
  const uint64_t R = (uint64_t)p.rows, K = (uint64_t)p.K, N = (uint64_t)p.N, G = (uint64_t)p.G;
  bool ok;
  if (FORM == PROD_DW) {
    ok = tc_map(&tm[0], p.b, N, R, p.ldb, 0, 0, 64, 64) && tc_map(&tm[1], p.a, K, R, p.lda, 0, 0, 64, 64);
    tm[2] = tm[1];
  } else {
    ok = (FORM == PROD_ROWS ? tc_map(&tm[0], p.b, N, K, N, G, K * N, 64, 64) : tc_map(&tm[0], p.b, K, N, K, G, K * N, 64, 128)) &&
         tc_map(&tm[1], p.a, K, R, p.lda, 0, 0, 64, 32);
    // (boxes of 128 rows: of no use to fewer, and a map takes the host a while)
    if (p.rows < 97) tm[2] = tm[1];
    else ok = ok && tc_map(&tm[2], p.a, K, R, p.lda, 0, 0, 64, 128);
  }
  if (!ok) return cudaErrorInvalidValue;
  return pair ? launch_parts<FORM, TC_PAIR, F32>(tm, p, formats, st) : launch_parts<FORM, TC_COPY, F32>(tm, p, formats, st);
}

}  // namespace

}  // namespace moe
