// product_tc.cu -- the experts' products of 16-bit operands on the tensor cores
// (tcgen05 kind::f16; product.cu has the formulas and the calls).
//
// Warp-specialised and persistent, one CTA per SM: warp 0 issues the copies (or eight
// more warps load the operands themselves), one thread of warp 1 the tensor-core
// instructions, warps 2..9 the epilogue.  A unit is (expert, tile of D): A is the M side
// (128 rows of x; for the weights' gradient 128 columns of x), B the N side (256 columns
// of the weights or of dy), and a stage of the ring holds 64 of the contraction:
//   A 128 x 64 (16 KB), B 256 x 64 (32 KB).
// What is contiguous along the contraction lies in rows of 128 bytes (x and transposed
// weights), the rest in blocks of 64 columns x 64 rows of 128 bytes; both 128-byte
// swizzled, so in shared memory every operand is rows of 64 elements that were
// contiguous in memory.
// TMEM: two accumulators of 256 columns, so that a unit's epilogue runs beside the next
// unit's products.
//
// PAIR: two CTAs (a cluster) share each MMA of M = 256 rows, 128 in each, and each holds
// half of B's columns: 32 KB a stage and SM instead of 48 for the same products.  The even
// CTA's barriers count both CTAs' copies, its one thread issues for both, and its commits
// arrive in both.
//
// Ragged edges.  Rows of x behind an expert's last are other experts': they fill rows of D
// that are not stored.  The contraction over an expert's rows (the weights' gradient) may
// end inside a stage: the instructions past its end are not issued, and the up to 15 rows
// of both operands that the last one still takes are overwritten with zeros first (one of
// them would not do: what lies there may be NaN).
#include "gemm_common.cuh"
#include "product.cuh"
#include "tc_roles.cuh"

namespace moe {

namespace {

enum TcMode { TC_COPY, TC_PAIR, TC_LOAD };  // tensor copies, the same by CTA pairs, plain loads

constexpr int kBlkM = 128, kBlkN = 256, kBlkK = 64;
constexpr int kEpiWarpsP = 8;   // two for each quarter of the TMEM lanes
constexpr int kLoadWarps = 8;   // of TC_LOAD
constexpr int kABytes = kBlkM * kBlkK * 2;
constexpr int kBoxBytes = 64 * 128;  // 64 rows of 64 elements
constexpr int kRingBytes = 192 * 1024;
constexpr int kStagesCopy = 4, kStagesPair = 6;
constexpr int kStageRow = 17;        // floats between the rows of an epilogue warp's staging: 32 x 16
constexpr int kStagingP = 32 * kStageRow * 4;
constexpr int kSmemP = 1024 + kRingBytes + kEpiWarpsP * kStagingP;

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

// Two 16-bit elements of a row in one register, the second behind the first; only those
// below n exist.  WORD: the row starts with a 32-bit word.
template <bool WORD>
MOE_DEV void load_two(const uint16_t* p, int i, int n, uint32_t& lo, uint32_t& hi) {
  if constexpr (WORD) {
    asm volatile(
        "{\n\t.reg .pred l, h;\n\t"
        "setp.ne.b32 l, %3, 0;\n\t"
        "setp.ne.b32 h, %4, 0;\n\t"
        "mov.b32 %0, 0;\n\t"
        "mov.b32 %1, 0;\n\t"
        "@h ld.global.u32 %0, [%2];\n\t"
        "@l ld.global.u16 %1, [%2];\n\t}"
        : "=&r"(lo), "=&r"(hi)
        : "l"(p + i), "r"((int)(i + 1 == n)), "r"((int)(i + 1 < n)));
  } else {
    gload_pair(p + i, i < n, i + 1 < n, lo, hi);
  }
}

struct TcUnit {
  int e, row0, count, m0, n0;
};

template <ProdForm FORM, TcMode MODE>
__global__ void __launch_bounds__(64 + 32 * (kEpiWarpsP + (MODE == TC_LOAD ? kLoadWarps : 0)), 1)
    tc_product_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_a128,
                      const __grid_constant__ CUtensorMap tm_b, const ProdArgs p, const uint32_t formats) {
  constexpr bool PAIR = MODE == TC_PAIR, DW = FORM == PROD_DW, B_MN = FORM != PROD_ROWS_T;
  constexpr int S = PAIR ? kStagesPair : kStagesCopy;
  constexpr uint32_t kStage = kRingBytes / S;
  constexpr int kTileM = PAIR ? 2 * kBlkM : kBlkM;
  extern __shared__ uint8_t smem_raw[];
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  __shared__ int s_off[kMaxG + 1], s_unit[kMaxG + 1];
  __shared__ alignas(8) uint64_t full[S], empty[S], tfull[2], tempty[2], drain, tail_full, tail_ready;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], MODE == TC_LOAD ? kLoadWarps : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], (PAIR ? 2 : 1) * kEpiWarpsP);
    }
    mbar_init(&drain, 1);
    mbar_init(&tail_full, 1);
    mbar_init(&tail_ready, 1);
    s_abort = 0;
    fence_mbar_init();
    if (MODE != TC_LOAD) {
      tma_prefetch_desc(&tm_a);
      tma_prefetch_desc(&tm_a128);
      tma_prefetch_desc(&tm_b);
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
  const int nts = (p.N + kBlkN - 1) / kBlkN, mts_dw = (p.K + kTileM - 1) / kTileM;
  number_units(p, DW ? 0 : kTileM, DW ? mts_dw * nts : nts, s_off, s_unit);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the other CTA's barriers exist before their use
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)s_tmem);
  const int total = uniform(s_unit[p.G]);
  volatile int* abort_flag = &s_abort;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int rank = PAIR ? uniform((int)cluster_ctarank()) : 0;
  const int unit0 = PAIR ? blockIdx.x / 2 : blockIdx.x, unit_step = PAIR ? gridDim.x / 2 : gridDim.x;

  // Unit u; each role walks its units upwards and keeps its place in the experts.
  int at_e = 0;
  auto unit_at = [&](int u) {
    while (u >= uniform(s_unit[at_e + 1])) ++at_e;
    TcUnit t;
    t.e = at_e;
    t.row0 = uniform(s_off[at_e]);
    t.count = max(0, uniform(s_off[at_e + 1]) - t.row0);
    const int mts = DW ? mts_dw : (t.count + kTileM - 1) / kTileM, r = u - uniform(s_unit[at_e]);
    const int n = r / mts;
    t.n0 = n * kBlkN;
    t.m0 = (r - n * mts) * kTileM;
    return t;
  };
  // columns of the MMA, and of this CTA's B
  auto mma_n = [&](const TcUnit& t) { return min(kBlkN, (p.N - t.n0 + 31) & ~31); };
  auto steps_of = [&](const TcUnit& t) { return ((DW ? t.count : p.K) + kBlkK - 1) / kBlkK; };
  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
  // All lanes wait; the result is the same in each.
  auto wait_all = [&](uint32_t bar, uint32_t parity, int where) {
    if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_on(bar, parity, abort_flag, p.status, where)) != 0;
  };
  // Zeros in rows [from, to) of every block of 64 rows of a stage (MN-major operands),
  // visible to the tensor cores.
  auto zero_rows = [&](uint32_t stage, int from, int to) {
    constexpr int kBlocks = (int)(kStage / kBoxBytes);
    const int n = (to - from) * 8;
    for (int i = lane; i < kBlocks * n; i += 32) {
      const int b = i / n, r = i - b * n;
      st_shared_v4(stage + (uint32_t)(b * kBoxBytes + (from + (r >> 3)) * 128 + (r & 7) * 16), 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp == 0 && MODE != TC_LOAD) {
    const int leader = elect_one();
    int s = 0;
    uint32_t ph = 0, used = 0, last = 0, apart_n = 0;
    for (int u = unit0; u < total; u += unit_step) {
      const TcUnit t = unit_at(u);
      const int hw = PAIR ? mma_n(t) / 2 : mma_n(t), steps = steps_of(t);
      // boxes of CTA r's A (32 rows, or 64 columns) and B (64)
      auto a_boxes = [&](int r) {
        if (DW) return max(0, min(2, (p.K - t.m0 - r * kBlkM + 63) / 64));
        return max(0, min(4, (t.count - t.m0 - r * kBlkM + 31) / 32));
      };
      const int ab = a_boxes(rank), bb = (hw + 63) / 64;
      const uint32_t bytes = (uint32_t)(ab * (DW ? kBoxBytes : kBoxBytes / 2) + bb * kBoxBytes);
      const uint32_t others = PAIR ? (uint32_t)(a_boxes(1) * (DW ? kBoxBytes : kBoxBytes / 2) + bb * kBoxBytes) : 0u;
      const int am = t.m0 + rank * kBlkM, bn = t.n0 + rank * hw;
      for (int kb = 0; kb < steps; ++kb) {
        if (!wait_all(empty0 + 8u * s, ph ^ 1u, 2000 + s)) goto produced;
        const uint32_t sa = base + (uint32_t)s * kStage, sb = sa + kABytes;
        const int k0 = kb * kBlkK;
        // of a pair, the odd CTA zeroes the end of the contraction in its own shared memory
        // and waits for its own copies first
        const bool apart = PAIR && DW && kb == steps - 1 && (t.count & 15) != 0;
        uint32_t fb = full0 + 8u * s;
        if constexpr (PAIR) {
          if (apart && rank == 1) {
            fb = mapa_shared(smem_u32(&tail_full), 1);
            expect_tx_on(leader, smem_u32(&tail_full), bytes);
            ++apart_n;
          } else {
            fb = mapa_shared(fb, 0);
            expect_tx_on(leader && rank == 0, full0 + 8u * s, bytes + (apart ? 0u : others));
          }
        } else {
          expect_tx_on(leader, fb, bytes);
        }
        if constexpr (DW) {
          for (int i = 0; i < ab; ++i)
            tma_load_2d_on<PAIR>(leader, sa + i * kBoxBytes, &tm_a, fb, am + i * 64, t.row0 + k0);
        } else {
          tma_load_2d_on<PAIR>(leader && ab == 4, sa, &tm_a128, fb, k0, t.row0 + am);
          for (int i = ab == 4 ? 4 : 0; i < ab; ++i)
            tma_load_2d_on<PAIR>(leader, sa + i * (kBoxBytes / 2), &tm_a, fb, k0, t.row0 + am + i * 32);
        }
        for (int i = 0; i < bb; ++i) {
          const uint32_t dst = sb + i * kBoxBytes;
          if constexpr (DW) tma_load_2d_on<PAIR>(leader, dst, &tm_b, fb, bn + i * 64, t.row0 + k0);
          else if constexpr (B_MN) tma_load_3d_on<PAIR>(leader, dst, &tm_b, fb, bn + i * 64, k0, t.e);
          else tma_load_3d_on<PAIR>(leader, dst, &tm_b, fb, k0, bn + i * 64, t.e);
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
    for (int i = 0; i < S; ++i) {
      if (((used >> i) & 1u) == 0) continue;
      if (rank == 0 && !mbar_wait_drain(&full[i], (last >> i) & 1u)) break;
      if (PAIR && !mbar_wait_drain(&empty[i], (last >> i) & 1u)) break;
    }
    if (apart_n > 0) mbar_wait_drain(&tail_full, (apart_n - 1) & 1u);
  } else if (warp == 1 && rank == 0) {
    const int leader = elect_one();
    int s = 0, acc = 0;
    uint32_t ph = 0, aph = 0, tph = 0;
    constexpr uint32_t kMN = 512u << 16, kKM = 1u << 16;  // leading offsets: 8 KB between blocks of 64 columns
    const uint32_t da0 = (base >> 4) | (DW ? kMN : kKM), db0 = ((base + kABytes) >> 4) | (B_MN ? kMN : kKM);
    constexpr uint32_t ka = DW ? 128u : 2u, kb_ = B_MN ? 128u : 2u;  // 16 of the contraction, in units of 16 bytes
    for (int u = unit0; u < total; u += unit_step) {
      const TcUnit t = unit_at(u);
      const int steps = steps_of(t);
      if (steps == 0) continue;
      const uint32_t id = (1u << 4) | formats | ((DW ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) |
                          ((uint32_t)(mma_n(t) >> 3) << 17) | ((uint32_t)((PAIR ? 256 : 128) >> 4) << 24);
      const uint32_t d = tmem + (uint32_t)(acc * kBlkN);
      if (!wait_all(smem_u32(&tempty[acc]), aph ^ 1u, 2100 + acc)) goto issued;
      tc_fence_after();
      int left = DW ? t.count : p.K;
      uint32_t more = 0;
      for (int kb = 0; kb < steps; ++kb) {
        if (!wait_all(full0 + 8u * s, ph, 2200 + s)) goto issued;
        if constexpr (DW && MODE != TC_LOAD) {
          if (left < kBlkK && (left & 15) != 0) {
            zero_rows(base + (uint32_t)s * kStage, left, (left + 15) & ~15);
            if constexpr (PAIR) {
              const uint32_t bar = smem_u32(&tail_ready);
              bool ok = __all_sync(0xffffffffu, try_wait_cluster(bar, tph));
              if (!ok) {
                ok = __all_sync(0xffffffffu, wait_on(bar, tph, abort_flag, p.status, 2300));
                ok = ok && __all_sync(0xffffffffu, try_wait_cluster(bar, tph));
              }
              if (!ok) goto issued;
              tph ^= 1u;
            }
          }
        }
        tc_fence_after();
        const uint32_t da = da0 + (uint32_t)s * (kStage / 16u), db = db0 + (uint32_t)s * (kStage / 16u);
        tc_mma_f16_on<PAIR>(leader, d, da, db, id, more);
        tc_mma_f16_on<PAIR>(leader && left > 16, d, da + ka, db + kb_, id, 1u);
        tc_mma_f16_on<PAIR>(leader && left > 32, d, da + 2 * ka, db + 2 * kb_, id, 1u);
        tc_mma_f16_on<PAIR>(leader && left > 48, d, da + 3 * ka, db + 3 * kb_, id, 1u);
        tc_commit_on<PAIR>(leader, empty0 + 8u * s);
        left -= kBlkK;
        more = 1u;
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
      tc_commit_on<PAIR>(leader, smem_u32(&tfull[acc]));
      if (++acc == 2) {
        acc = 0;
        aph ^= 1u;
      }
    }
  issued:
    tc_commit_on<PAIR>(leader, smem_u32(&drain), 1);
    mbar_wait_drain(&drain, 0);
  } else if (PAIR && DW && warp == 1) {
    // the odd CTA's part of the contraction's end
    int s = 0;
    uint32_t tph = 0;
    for (int u = unit0; u < total; u += unit_step) {
      const TcUnit t = unit_at(u);
      const int steps = steps_of(t);
      if (steps == 0) continue;
      s = (s + steps - 1) % S;
      if ((t.count & 15) != 0) {
        if (!wait_all(smem_u32(&tail_full), tph, 2400)) break;
        tph ^= 1u;
        const int left = t.count - (steps - 1) * kBlkK;
        zero_rows(base + (uint32_t)s * kStage, left, (left + 15) & ~15);
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tail_ready), 0));
      }
      if (++s == S) s = 0;
    }
  } else if (MODE == TC_LOAD && warp >= 2 + kEpiWarpsP) {
    // Rows of 64 elements, a lane two of each.  Eight rows of loads are under way in a warp.
    const int w = warp - 2 - kEpiWarpsP;
    int s = 0;
    uint32_t ph = 0;
    const uint16_t *A = static_cast<const uint16_t*>(p.a), *B = static_cast<const uint16_t*>(p.b);
    // rows [w, n) of shared memory from `to`: row r is row_at(r, pointer) elements of memory
    auto fill = [&](uint32_t to, int n, auto word, auto row_at) {
      constexpr int U = 8;
      for (int r0 = w; r0 < n; r0 += kLoadWarps * U) {
        uint32_t lo[U], hi[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int r = r0 + i * kLoadWarps;
          const uint16_t* src = A;
          const int have = r < n ? row_at(r, src) : 0;
          load_two<decltype(word)::value>(src, 2 * lane, have, lo[i], hi[i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int r = r0 + i * kLoadWarps;
          const uint32_t v = decltype(word)::value ? lo[i] | hi[i] : lo[i] | hi[i] << 16;
          if (r < n)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + (uint32_t)(r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4)),
                         "r"(v)
                         : "memory");
        }
      }
    };
    auto fill_any = [&](uint32_t to, int n, bool words, auto row_at) {
      if (words) fill(to, n, std::true_type(), row_at);
      else fill(to, n, std::false_type(), row_at);
    };
    const bool a_words = ((reinterpret_cast<uintptr_t>(A) | (uintptr_t)p.lda * 2) & 3) == 0;
    const bool b_words = ((reinterpret_cast<uintptr_t>(B) | (uintptr_t)p.ldb * 2 | (DW ? 0 : (uintptr_t)p.K * p.N * 2)) & 3) == 0;
    for (int u = unit0; u < total; u += unit_step) {
      const TcUnit t = unit_at(u);
      const int nn = mma_n(t), steps = steps_of(t), kk = DW ? t.count : p.K;
      const uint16_t* we = DW ? B + (int64_t)t.row0 * p.ldb : B + (int64_t)t.e * p.K * p.N;
      for (int kb = 0; kb < steps; ++kb) {
        if (!wait_all(empty0 + 8u * s, ph ^ 1u, 2000 + s)) goto loaded;
        const uint32_t sa = base + (uint32_t)s * kStage, sb = sa + kABytes;
        const int k0 = kb * kBlkK;
        // contraction along the row (K-major): row c of D's side, `have` elements from k0;
        // else row r % 64 of the contraction, 64 columns from 64 * (r / 64)
        if constexpr (DW)
          fill_any(sa, kBlkM, a_words, [&](int r, const uint16_t*& src) {
            const int k = k0 + (r & 63), c = t.m0 + (r & ~63);
            src = A + (int64_t)(t.row0 + k) * p.lda + c;
            return k < kk ? p.K - c : 0;
          });
        else
          fill_any(sa, min(kBlkM, t.count - t.m0), a_words, [&](int r, const uint16_t*& src) {
            src = A + (int64_t)(t.row0 + t.m0 + r) * p.lda + k0;
            return kk - k0;
          });
        if constexpr (B_MN)
          fill_any(sb, (nn + 63) & ~63, b_words, [&](int r, const uint16_t*& src) {
            const int k = k0 + (r & 63), c = t.n0 + (r & ~63);
            src = we + (int64_t)k * p.ldb + c;
            return k < kk ? p.N - c : 0;
          });
        else
          fill_any(sb, min(nn, p.N - t.n0), b_words, [&](int r, const uint16_t*& src) {
            src = we + (int64_t)(t.n0 + r) * p.ldb + k0;
            return kk - k0;
          });
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  loaded:;
  } else if (warp > 1 && warp < 2 + kEpiWarpsP) {
    // A lane holds a row of D; a warp takes every other 32 columns of its quarter's 32 rows.
    // Rows that are 16-byte aligned are stored from the lanes, others through the warp's
    // staging, 16 columns at a time, so that neighbouring lanes store neighbouring elements.
    const int q = warp & 3;  // TMEM lane quarter of this warp
    const uint32_t stg = base + kRingBytes + (uint32_t)(warp - 2) * kStagingP;
    int acc = 0;
    uint32_t aph = 0;
    const int osz = p.odt == MOE_DT_F32 ? 4 : 2;
    uint8_t* out = static_cast<uint8_t*>(p.out);
    const bool rows16 = ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)p.ldo * osz) & 15) == 0;
    for (int u = unit0; u < total; u += unit_step) {
      const TcUnit t = unit_at(u);
      const bool some = steps_of(t) > 0;
      if (!some && p.accumulate) continue;
      if (some) {
        if (!wait_all(smem_u32(&tfull[acc]), aph, 2500 + acc)) break;
        tc_fence_after();
      }
      const int m0 = t.m0 + rank * kBlkM + q * 32, left = (DW ? p.K : t.count) - m0;  // rows of this warp
      const int64_t row = DW ? (int64_t)t.e * p.K + m0 : (int64_t)t.row0 + m0;
      const int nend = min(kBlkN, p.N - t.n0);
      for (int c0 = 32 * ((warp - 2) >> 2); c0 < nend && left > 0; c0 += 64) {
        float v[32];
        if (some) {
          tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kBlkN + c0), v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        uint8_t* dst = out + ((row + lane) * p.ldo + t.n0 + c0) * osz;
        if (rows16 && c0 + 32 <= nend) {
          if (lane < left) {
            if (osz == 4) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float4* d4 = reinterpret_cast<float4*>(dst) + i;
                float4 w = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                if (DW && p.accumulate) {
                  const float4 o = *d4;
                  w.x += o.x;
                  w.y += o.y;
                  w.z += o.z;
                  w.w += o.w;
                }
                *d4 = w;
              }
            } else {
              const bool bf = p.odt == MOE_DT_BF16;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint4* d4 = reinterpret_cast<uint4*>(dst) + i;
                uint32_t w[4];
                if (DW && p.accumulate) {
                  const uint4 o = *d4;
                  w[0] = o.x;
                  w[1] = o.y;
                  w[2] = o.z;
                  w[3] = o.w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  F2 r(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
                  if (DW && p.accumulate) r = add2(r, bf ? pair_f32<__nv_bfloat16>(w + j) : pair_f32<__half>(w + j));
                  if (bf) pair_to<__nv_bfloat16>(w + j, r);
                  else pair_to<__half>(w + j, r);
                }
                *d4 = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        } else {
#pragma unroll
          for (int h = 0; h < 32; h += 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(stg + (uint32_t)(lane * kStageRow + i) * 4u), "f"(v[h + i]) : "memory");
            __syncwarp();
            const int col = lane & 15;
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
              const int r = 2 * i + (lane >> 4);
              float x;
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(stg + (uint32_t)(r * kStageRow + col) * 4u));
              if (r < left && c0 + h + col < nend) {
                const int64_t at = (row + r) * p.ldo + t.n0 + c0 + h + col;
                if (osz == 4) {
                  float* f = reinterpret_cast<float*>(out) + at;
                  *f = DW && p.accumulate ? x + *f : x;
                } else if (p.odt == MOE_DT_BF16) {
                  __nv_bfloat16* f = reinterpret_cast<__nv_bfloat16*>(out) + at;
                  *f = from_f32<__nv_bfloat16>(DW && p.accumulate ? x + to_f32(*f) : x);
                } else {
                  __half* f = reinterpret_cast<__half*>(out) + at;
                  *f = from_f32<__half>(DW && p.accumulate ? x + to_f32(*f) : x);
                }
              }
            }
            __syncwarp();
          }
        }
      }
      if (!some) continue;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
        else mbar_arrive(&tempty[acc]);
      }
      if (++acc == 2) {
        acc = 0;
        aph ^= 1u;
      }
    }
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

template <ProdForm FORM, TcMode MODE>
cudaError_t launch_tc(const CUtensorMap* tm, const ProdArgs& p, uint32_t formats, cudaStream_t st) {
  auto kern = tc_product_kernel<FORM, MODE>;
  static SmemAllowed allowed;
  const cudaError_t e = allow_smem(kern, kSmemP, allowed);
  if (e != cudaSuccess) return e;
  const char* name = FORM == PROD_DW ? "grouped_product_dw" : "grouped_product";
  const int64_t units = most_units(FORM, p, MODE == TC_PAIR ? 2 * kBlkM : kBlkM, kBlkN);
  const dim3 block(64 + 32 * (kEpiWarpsP + (MODE == TC_LOAD ? kLoadWarps : 0)));
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

template <ProdForm FORM>
cudaError_t launch_form(int dtype, const ProdArgs& p, cudaStream_t st) {
  const uint32_t fmt = dtype == MOE_DT_BF16 ? 1u : 0u, formats = (fmt << 7) | (fmt << 10);
  // tensor copies: every row starts on 16 bytes (and there are rows)
  const bool copy = p.rows > 0 && ((bits(p.a) | bits(p.b) | (uintptr_t)p.lda * 2 | (uintptr_t)p.ldb * 2) & 15) == 0;
  CUtensorMap tm[3];
  if (!copy) {
    memset(tm, 0, sizeof(tm));
    return launch_tc<FORM, TC_LOAD>(tm, p, formats, st);
  }
  const bool pair = FORM != PROD_DW && p.rows >= 128 * (int64_t)p.G;
  const uint64_t R = (uint64_t)p.rows, K = (uint64_t)p.K, N = (uint64_t)p.N, G = (uint64_t)p.G;
  bool ok;
  if (FORM == PROD_DW) {
    ok = tc_map(&tm[0], p.a, K, R, p.lda, 0, 0, 64, 64) && tc_map(&tm[2], p.b, N, R, p.ldb, 0, 0, 64, 64);
    tm[1] = tm[0];
  } else {
    ok = tc_map(&tm[0], p.a, K, R, p.lda, 0, 0, 64, 32) && tc_map(&tm[1], p.a, K, R, p.lda, 0, 0, 64, 128) &&
         (FORM == PROD_ROWS ? tc_map(&tm[2], p.b, N, K, N, G, K * N, 64, 64) : tc_map(&tm[2], p.b, K, N, K, G, K * N, 64, 64));
  }
  if (!ok) return cudaErrorInvalidValue;
  return pair ? launch_tc<FORM, TC_PAIR>(tm, p, formats, st) : launch_tc<FORM, TC_COPY>(tm, p, formats, st);
}

}  // namespace

cudaError_t launch_product_tc(ProdForm form, int dtype, const ProdArgs& p, cudaStream_t st) {
  switch (form) {
    case PROD_ROWS: return launch_form<PROD_ROWS>(dtype, p, st);
    case PROD_ROWS_T: return launch_form<PROD_ROWS_T>(dtype, p, st);
    default: return launch_form<PROD_DW>(dtype, p, st);
  }
}

}  // namespace moe
